"""The decoding operators' cases for measurement: rotary positions, the paged key/value
cache's write and read, and the attention of drafted tokens over that cache.

``run`` computes one pass, in a plain form of elementary torch operations (``own`` false)
or through the package (``own`` true).  Shapes follow the repository's configurations: 16
query heads, 1 to 16 key/value heads, head_dim 256, states of 15,231 / 30,468 / 60,926 tokens.
"""

import math

import torch

own = False

D = 256
E4M3 = torch.float8_e4m3fn
_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}
_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# --------------------------------------------------------------------------- cases


def _rope(name, **kw):
    c = dict(name=name, op="rope", B=1, L=1, Hq=16, Hkv=4, dtype="bf16", layout="half", rot=256, scaling="none",
             factor=1.0, original=8192, far=0, per_row=False, backward=False)
    c.update(kw)
    return c


def _write(name, **kw):
    c = dict(name=name, op="write", B=1, L=1, Hkv=4, src="bf16", cache="e4m3", page=64, start=0, ragged=False,
             rope=True, layout="half", rot=256, scaling="none", factor=1.0, original=8192)
    c.update(kw)
    return c


def _read(name, **kw):
    c = dict(name=name, op="read", B=1, L=1, Hkv=4, cache="e4m3", dst="bf16", page=64, ragged=False)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", B=1, T=1, ctx=1, Hq=16, Hkv=4, cache="bf16", dtype="bf16", page=64, ragged=False,
             tree=False, shared_mask=False, pad=False)
    c.update(kw)
    return c


def listed():
    return [
        # One decoding step of 16 sequences at their own far positions: latency only.
        _rope("rope_step_partial", B=16, L=1, layout="interleaved", rot=64, scaling="linear", factor=8.0, far=900_000,
              per_row=True),
        # A training step's q and k over a 15,231-token document, scaled for long contexts, and their gradients.
        _rope("rope_train_15231", L=15_231, scaling="yarn", factor=8.0, backward=True),
        # One decoding step's keys and values of 32 sequences of different lengths, appended to the cache.
        _write("write_step_e4m3", B=32, L=1, start=4000, ragged=True, page=32),
        # A 30,468-token state's keys and values quantised into the cache as they are written.
        _write("write_state_e4m3", L=30_468),
        # Quantised states of three sequences read back for a dense prefill over them.
        _read("read_states_e4m3", B=3, L=15_231, ragged=True),
        # A short fp32 state read back from small pages.
        _read("read_short_f32", B=2, L=601, cache="f32", dst="f32", page=16),
        # One token against a short context: the smallest decoding call.
        _attend("attend_one_777", ctx=777),
        # One token against the longest document.
        _attend("attend_one_60926", ctx=60_926, page=128),
        # One token of 32 sequences of different lengths over a quantised cache: ordinary serving.
        _attend("attend_batch_e4m3", B=32, ctx=8_192, cache="e4m3", ragged=True, page=32),
        # Trees of 24 drafted tokens, some rows of padding, over quantised states.
        _attend("attend_tree24_e4m3", B=8, T=24, ctx=15_231, cache="e4m3", tree=True, ragged=True, pad=True),
        # Trees of 64 drafted tokens over bf16 states: the largest call, near the matrix units' rate.
        _attend("attend_tree64_bf16", B=4, T=64, ctx=30_468, tree=True, shared_mask=True),
        # A small tree in fp32, the type of the repository's headline path.
        _attend("attend_tree5_f32", B=2, T=5, ctx=15_231, cache="f32", dtype="f32", tree=True, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _scaling(rng):
    s = rng.choice(["none", "linear", "ntk", "yarn"])
    return dict(scaling=s, factor=1.0 if s == "none" else rng.choice([2.0, 4.0, 8.0, 16.0]),
                original=rng.choice([2048, 8192, 32768]))


def _cost(c):
    """Seconds at the card's rates, fp32 products on the CUDA cores."""
    w = work(c)
    return w["bytes"] / 6.5e12 + w["flops"] / (6e13 if "f32" in (c.get("dtype"), c.get("cache")) else 1.6e15)


def _within(c):
    """The case with fewer sequences, then shorter ones, until it costs no more than the operator's largest above."""
    most = max(_cost(x) for x in listed() if x["op"] == c["op"])
    length = "ctx" if c["op"] == "attend" else "L"
    while _cost(c) > most and (c["B"] > 1 or c[length] > 1):
        c["B" if c["B"] > 1 else length] = max(1, c["B" if c["B"] > 1 else length] * 3 // 4)
    return c


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend", "attend"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 64)
    if op == "rope":
        return _within(_rope(
            "", B=B, L=_log(rng, 1, 15_231), Hkv=Hkv, dtype=rng.choice(["bf16", "bf16", "f32"]),
            layout=rng.choice(["half", "interleaved"]), rot=rng.choice([32, 64, 96, 128, 256]),
            far=rng.choice([0, 10_000, 1_000_000]), per_row=rng.random() < 0.5, backward=rng.random() < 0.5,
            **_scaling(rng)))
    if op == "write":
        return _within(_write(
            "", B=B, L=_log(rng, 1, 30_468), Hkv=Hkv, src=rng.choice(["bf16", "bf16", "f32"]),
            cache=rng.choice(["e4m3", "e4m3", "bf16", "f32"]), page=page, start=rng.randint(0, 5000),
            ragged=rng.random() < 0.5, rope=rng.random() < 0.7, layout=rng.choice(["half", "interleaved"]),
            rot=rng.choice([64, 128, 256]), **_scaling(rng)))
    kind = rng.choice(["bf16", "e4m3", "bf16", "e4m3", "f32"])
    if op == "read":
        return _within(_read("", B=B, L=_log(rng, 16, 15_231), Hkv=Hkv, cache=kind, page=page,
                             dst="f32" if kind == "f32" else rng.choice(["bf16", "bf16", "f32"]),
                             ragged=rng.random() < 0.5))
    T = rng.choice([1, 1, 1, 2, 5, 8, 13, 24, 33, 48, 64])
    return _within(_attend(
        "", B=B, T=T, ctx=_log(rng, 1, 60_926), Hkv=Hkv, cache=kind, dtype="f32" if kind == "f32" else "bf16", page=page,
        ragged=rng.random() < 0.5, tree=T > 1 and rng.random() < 0.7, shared_mask=rng.random() < 0.3,
        pad=T > 1 and rng.random() < 0.4))


# --------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _lens(B, top, ragged, g):
    """Lengths of B sequences: all `top`, or from an eighth of it up, the first the longest."""
    if not ragged:
        return torch.full((B,), top, dtype=torch.int32, device="cuda")
    n = torch.randint(max(1, top // 8), top + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = top
    return n


def _frequencies(c):
    """Angle per position of each rotated pair, fp64 on the host, and the magnitude."""
    R, base, s = c["rot"], 10000.0, c["factor"]
    if c["scaling"] == "ntk":
        base *= s ** (R / (R - 2.0))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    m = 1.0
    if c["scaling"] == "linear":
        f = [x / s for x in f]
    if c["scaling"] == "yarn":
        for i, x in enumerate(f):
            g = min(1.0, max(0.0, (c["original"] * x / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
            f[i] = x * (g + (1.0 - g) / s)
        m = 0.1 * math.log(s) + 1.0
    return f, m


def _table(c):
    from long_context_causal_flash_b200 import rotary

    return rotary.Table(rot=c["rot"], base=10000.0, layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                        original_length=c["original"], device="cuda")


def _pages(B, tokens, page, g):
    """A pool a little larger than needed and each sequence's pages in it, in a shuffled order."""
    per = -(-tokens // page)
    n = B * per + 3
    ids = torch.randperm(n, generator=g, device="cuda")[: B * per].to(torch.int32)
    return n, ids.view(B, per).contiguous()


def _power_scale(amax):
    """2^ceil(log2(amax / 448)), 1 for a row of zeros: found from the float's own exponent."""
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e.clamp(-120, 120)), torch.ones_like(amax))


def _quantised(x):
    scale = _power_scale(x.abs().amax(-1))
    return (x / scale[..., None]).clamp(-448, 448).to(E4M3), scale


def _pool(n, Hkv, page, kind, g):
    """Filled key and value pages (and their scales): rows of unit variance, some heads larger."""
    out = []
    gain = 1.0 + torch.arange(Hkv, device="cuda").view(1, Hkv, 1, 1) / 8
    for _ in range(2):
        x = torch.randn((n, Hkv, page, D), generator=g, device="cuda") * gain
        if kind == "e4m3":
            out.append(_quantised(x))
        else:
            out.append((x.to(_DT[kind]), None))
        del x
    return out


def _tree_mask(B, T, g):
    """[B, T, T]: each drafted token sees itself and its ancestors; the parent is an earlier token."""
    near = torch.arange(T, device="cuda").view(1, T).expand(B, T)
    parent = (torch.rand((B, T), generator=g, device="cuda") * near).long()
    mask = torch.zeros((B, T, T), dtype=torch.bool, device="cuda")
    b = torch.arange(B, device="cuda")
    for t in range(T):
        if t:
            mask[:, t] = mask[b, parent[:, t]]
        mask[:, t, t] = True
    return mask


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] in ("rope", "write") and c.get("rope", True):
        f, m = _frequencies(c)
        s["freq"], s["magnitude"] = torch.tensor(f, dtype=torch.float64, device="cuda"), m
        if own:
            s["table"] = _table(c)
    if c["op"] == "rope":
        dt = _DT[c["dtype"]]
        s["q"] = _randn((c["B"], c["Hq"], c["L"], D), g, dt)
        s["k"] = _randn((c["B"], c["Hkv"], c["L"], D), g, dt)
        if c["per_row"]:
            first = torch.randint(0, c["far"] + 1, (c["B"], 1), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(c["L"], device="cuda")).to(torch.int32)
        if c["backward"]:
            s["dq"], s["dk"] = _randn(s["q"].shape, g, dt), _randn(s["k"].shape, g, dt)
            s["q"].requires_grad_(own)
            s["k"].requires_grad_(own)
        return s
    if c["op"] == "write":
        dt, kind = _DT[c["src"]], c["cache"]
        # the projections' output: tokens outside heads, as views
        x = _randn((c["B"], c["L"], 2, c["Hkv"], D), g, dt)
        s["k"], s["v"] = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
        s["start"] = _lens(c["B"], c["start"], c["ragged"], g) if c["start"] else torch.zeros(
            c["B"], dtype=torch.int32, device="cuda")
        n, s["table_of_pages"] = _pages(c["B"], c["start"] + c["L"], c["page"], g)
        shape = (n, c["Hkv"], c["page"], D)
        s["kp"], s["vp"] = (torch.zeros(shape, device="cuda").to(_DT[kind]) for _ in range(2))
        s["ks"] = s["vs"] = None
        if kind == "e4m3":
            s["ks"], s["vs"] = torch.ones(shape[:3], device="cuda"), torch.ones(shape[:3], device="cuda")
        return s
    if c["op"] == "read":
        s["lens"] = _lens(c["B"], c["L"], c["ragged"], g)
        n, s["table_of_pages"] = _pages(c["B"], c["L"], c["page"], g)
    else:
        s["lens"] = _lens(c["B"], c["ctx"], c["ragged"], g)
        n, s["table_of_pages"] = _pages(c["B"], c["ctx"] + c["T"], c["page"], g)
        s["q"] = _randn((c["B"], c["Hq"], c["T"], D), g, _DT[c["dtype"]])
        s["mask"] = s["drafted"] = None
        if c["tree"]:
            s["mask"] = _tree_mask(1 if c["shared_mask"] else c["B"], c["T"], g)
            if c["shared_mask"]:
                s["mask"] = s["mask"][0].contiguous()
        if c["pad"]:
            s["drafted"] = torch.randint(1, c["T"] + 1, (c["B"],), generator=g, device="cuda", dtype=torch.int32)
    (s["kp"], s["ks"]), (s["vp"], s["vs"]) = _pool(n, c["Hkv"], c["page"], c["cache"], g)
    return s


# --------------------------------------------------------------------------- the plain forms


def _positions(s, B, L):
    if s.get("positions") is not None:
        return s["positions"].long()
    if "start" in s:
        return s["start"].long()[:, None] + torch.arange(L, device="cuda")
    return s["case"]["far"] + torch.arange(L, device="cuda").expand(B, L)


def _turn(x, s, sign=1.0):
    """Rotated fp32 values of x [B, H, L, D]; angles in 64 bits, sign -1 turns back."""
    c = s["case"]
    R, m = c["rot"], s["magnitude"]
    a = (_positions(s, x.shape[0], x.shape[2])[..., None].double() * s["freq"])[:, None]
    cos, sin = (torch.cos(a) * m).float(), (torch.sin(a) * (m * sign)).float()
    x = x.float()
    rot, rest = x[..., :R], x[..., R:]
    if c["layout"] == "half":
        x1, x2 = rot[..., : R // 2], rot[..., R // 2:]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    else:
        x1, x2 = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    return torch.cat((y, rest), -1)


def _plain_rope(s):
    dt = _DT[s["case"]["dtype"]]
    got = {"q": _turn(s["q"].detach(), s).to(dt), "k": _turn(s["k"].detach(), s).to(dt)}
    if s["case"]["backward"]:
        got["dq"], got["dk"] = _turn(s["dq"], s, -1.0).to(dt), _turn(s["dk"], s, -1.0).to(dt)
    return got


def _plain_write(s):
    c = s["case"]
    k = _turn(s["k"], s) if c["rope"] else s["k"].float()
    v = s["v"].float()
    at = s["start"].long()[:, None] + torch.arange(c["L"], device="cuda")
    page = torch.gather(s["table_of_pages"].long(), 1, at // c["page"])
    slot = (page, slice(None), at % c["page"])
    for x, pool, scales in ((k, s["kp"], s["ks"]), (v, s["vp"], s["vs"])):
        x = x.transpose(1, 2)  # [B, L, Hkv, D], the order of the indexed pool
        if scales is None:
            pool[slot] = x.to(pool.dtype)
        else:
            codes, scale = _quantised(x)
            pool.view(torch.uint8)[slot] = codes.view(torch.uint8)
            scales[slot] = scale
    return _pool_outputs(s)


def _pool_outputs(s):
    got = {"k": s["kp"], "v": s["vp"]}
    if s["ks"] is not None:
        got.update(k_scale=s["ks"], v_scale=s["vs"])
    return got


def _dense(pool, scales, table):
    """[B, Hkv, capacity, D] in fp32."""
    at = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[at].view(E4M3).float() if scales is not None else pool[at].float()
    if scales is not None:
        x = x * scales[at][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_read(s):
    c = s["case"]
    live = (torch.arange(c["L"], device="cuda") < s["lens"][:, None])[:, None, :, None]
    got = []
    for pool, scales in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        x = _dense(pool, scales, s["table_of_pages"])[:, :, : c["L"]]
        got.append(torch.where(live, x, torch.zeros_like(x)).to(_DT[c["dst"]]))
    return {"k": got[0], "v": got[1]}


def _plain_attend(s):
    c = s["case"]
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    k, v = _dense(s["kp"], s["ks"], s["table_of_pages"]), _dense(s["vp"], s["vs"], s["table_of_pages"])
    n = k.shape[2]
    t, j = torch.arange(T, device="cuda"), torch.arange(n, device="cuda")
    ctx = s["lens"].long()[:, None, None]
    drafted = (s["drafted"].long() if s["drafted"] is not None else torch.full((B,), T, device="cuda"))[:, None, None]
    u = j[None, None, :] - ctx
    mask = s["mask"] if s["mask"] is not None else t[:, None] >= t[None, :]
    mask = mask.expand(B, T, T)
    named = torch.gather(mask, 2, u.clamp(0, T - 1).expand(B, T, n))
    seen = ((u < 0) | ((u < drafted) & named)) & (t[None, :, None] < drafted)
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv * T, D)
    sc = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, T, n) / math.sqrt(D)
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(sc - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, -1, n), v).view(B, Hkv, -1, T, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return {"out": out.reshape(B, Hq, T, D).to(_DT[c["dtype"]]), "lse": (top + torch.log(total)).reshape(B, Hq, T)}


# --------------------------------------------------------------------------- the package's calls


def _own(s):
    from long_context_causal_flash_b200 import cache, rotary

    c = s["case"]
    if c["op"] == "rope":
        kw = dict(positions=s.get("positions"), pos_offset=0 if c["per_row"] else c["far"])
        if not c["backward"]:
            q, k = rotary.rotate(s["q"], s["k"], s["table"], **kw)
            return {"q": q, "k": k}
        q, k = rotary.rotate_autograd(s["q"], s["k"], s["table"], **kw)
        dq, dk = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))
        return {"q": q.detach(), "k": k.detach(), "dq": dq, "dk": dk}
    pool = cache.PagedCache(s["kp"], s["vp"], s["ks"], s["vs"])
    if c["op"] == "write":
        cache.write(pool, s["k"], s["v"], s["table_of_pages"], s["start"], rope=s.get("table"))
        return _pool_outputs(s)
    if c["op"] == "read":
        k, v = cache.read(pool, s["table_of_pages"], s["lens"], c["L"], dtype=_DT[c["dst"]])
        return {"k": k, "v": v}
    out, lse = cache.attend(s["q"], pool, s["table_of_pages"], s["lens"], tree_mask=s["mask"], tree_lens=s["drafted"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read,
            "attend": _plain_attend}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the definitions in 64 bits


def _exact_turn(x, c, f, m, first, sign):
    """One sequence's x [H, L, D] (any float type) turned by sign * (first + l) * f, as complex products."""
    x, R = x.double(), c["rot"]
    f = torch.tensor(f, dtype=torch.float64, device=x.device)
    a = sign * (first.double() + torch.arange(x.shape[1], device=x.device, dtype=torch.float64))[:, None] * f
    w = torch.polar(torch.full_like(a, m), a)
    lo = slice(0, R // 2) if c["layout"] == "half" else slice(0, R, 2)
    hi = slice(R // 2, R) if c["layout"] == "half" else slice(1, R, 2)
    z = torch.complex(x[..., lo], x[..., hi]) * w
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """(values on the e4m3 grid of x / scale, scale) with scale the least power of two that fits 448."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / 448.0) - 1e-12)), torch.ones_like(amax))
    y = x / scale[..., None]
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step, scale


def _rows_of(pool, scales, ids, n):
    """The first n rows [Hkv, n, D] of a sequence whose pages are `ids`, in 64 bits."""
    page = pool.shape[2]
    j = torch.arange(n, device=pool.device)
    raw = pool.view(torch.uint8) if scales is not None else pool
    x = raw[ids.long()[j // page], :, j % page]
    x = x.view(E4M3).double() * scales[ids.long()[j // page], :, j % page].double()[..., None] if scales is not None \
        else x.double()
    return x.transpose(0, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        f, m = _frequencies(c)
        got = {}
        for name, sign in (("q", 1.0), ("k", 1.0)) + ((("dq", -1.0), ("dk", -1.0)) if c["backward"] else ()):
            x = s[name].detach()
            first = [s["positions"][b, 0] if c["per_row"] else torch.tensor(c["far"], device="cuda")
                     for b in range(c["B"])]
            got[name] = torch.stack([_exact_turn(x[b], c, f, m, first[b], sign) for b in range(c["B"])])
        return got
    if c["op"] == "write":
        pools = {"k": s["kp"].double(), "v": s["vp"].double()}
        scales = {"k": None if s["ks"] is None else s["ks"].double(), "v": None if s["vs"] is None else s["vs"].double()}
        f, m = _frequencies(c)
        for b in range(c["B"]):
            at = s["start"][b].long() + torch.arange(c["L"], device="cuda")
            page, slot = s["table_of_pages"][b].long()[at // c["page"]], at % c["page"]
            for name in ("k", "v"):
                x = s[name][b].double()
                if name == "k" and c["rope"]:
                    x = _exact_turn(s["k"][b], c, f, m, s["start"][b], 1.0)
                x = x.transpose(0, 1)
                if scales[name] is not None:
                    x, e = _exact_e4m3(x)
                    scales[name][page, :, slot] = e
                pools[name][page, :, slot] = x
        if s["ks"] is not None:
            pools.update(k_scale=scales["k"], v_scale=scales["v"])
        return pools
    if c["op"] == "read":
        got = {"k": torch.zeros((c["B"], c["Hkv"], c["L"], D), dtype=torch.float64, device="cuda")}
        got["v"] = torch.zeros_like(got["k"])
        for b, n in enumerate(s["lens"].tolist()):
            got["k"][b, :, :n] = _rows_of(s["kp"], s["ks"], s["table_of_pages"][b], n)
            got["v"][b, :, :n] = _rows_of(s["vp"], s["vs"], s["table_of_pages"][b], n)
        return got
    B, T, G = c["B"], c["T"], c["Hq"] // c["Hkv"]
    out = torch.zeros((B, c["Hq"], T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"], T), -math.inf, dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["lens"].tolist()):
        t = T if s["drafted"] is None else int(s["drafted"][b])
        k = _rows_of(s["kp"], s["ks"], s["table_of_pages"][b], ctx + t).repeat_interleave(G, 0)
        v = _rows_of(s["vp"], s["vs"], s["table_of_pages"][b], ctx + t).repeat_interleave(G, 0)
        hidden = torch.ones((t, t), dtype=torch.bool, device="cuda").triu(1)
        if s["mask"] is not None:
            hidden = ~(s["mask"] if c["shared_mask"] else s["mask"][b])[:t, :t]
        x = torch.einsum("htd,hnd->htn", s["q"][b, :, :t].double(), k) * 0.0625
        x[:, :, ctx:][:, hidden] = -math.inf
        lse[b, :, :t] = torch.logsumexp(x, -1)
        out[b, :, :t] = torch.einsum("htn,hnd->htd", torch.softmax(x, -1), v)
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------------- the work


def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["B"] * c["L"] * (c["Hq"] + c["Hkv"]) * (2 if c["backward"] else 1)
        return {"bytes": rows * 2 * D * _BYTES[c["dtype"]] + (c["B"] * c["L"] * 4 if c["per_row"] else 0),
                "flops": rows * 3 * c["rot"]}
    if c["op"] == "write":
        rows = 2 * c["B"] * c["L"] * c["Hkv"]
        per = D * _BYTES[c["src"]] + D * _BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0)
        return {"bytes": rows * per, "flops": rows * D * ((1 if c["rope"] else 0) * 1.5 + 2)}
    part = 0.5625 if c["ragged"] else 1.0  # the mean length, of the longest
    if c["op"] == "read":
        rows = 2 * c["B"] * c["Hkv"] * c["L"]
        live = rows * ((1 + (c["B"] - 1) * part) / c["B"])
        return {"bytes": live * (D * _BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0))
                + rows * D * _BYTES[c["dst"]], "flops": live * D}
    keys = c["ctx"] * (1 + (c["B"] - 1) * part) + c["B"] * c["T"]
    rows = c["B"] * c["Hq"] * c["T"]
    drafted = c["T"] * (0.5 if c["pad"] else 1.0)
    e = 2 * D * _BYTES[c["cache"]] + (8 if c["cache"] == "e4m3" else 0)
    return {"bytes": keys * c["Hkv"] * e + rows * (2 * D * _BYTES[c["dtype"]] + 4),
            "flops": 4 * D * c["Hq"] * drafted * keys}
