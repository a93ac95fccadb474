"""The attention kernels over the cache take their timeout exits without a GPU fault.

As in ``test_faults``: a producer that skips one fill (test hook GQA_ATTN_TEST_SKIP_FILL) leaves
the waits on it without an arrival.  Every form of the three kernels has to give up after its
budget (50 ms here), record GQA_ERR_DEVICE_TIMEOUT in the pool's status word, free its
tensor memory, leave with its pair partner (where it has one), and leave the context
usable: the next call, without the hook, has the bits of the call before.  The second fill is one
of the first tile, the tenth one of a later tile, with products in flight.  In a child process (the
budget is read once per process).
"""

import json
import os
import subprocess
import sys

import pytest

from long_context_causal_flash_b200 import _lib

pytestmark = pytest.mark.gpu

_SCRIPT = r"""
import json, os, sys, time
sys.path.insert(0, sys.argv[1])
import torch
from long_context_causal_flash_b200 import cache

dev = torch.device("cuda:0")
E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
res = {}
for dtype, kind, T in ((BF16, BF16, 1), (BF16, E4M3, 1), (BF16, BF16, 5), (BF16, E4M3, 5), (BF16, BF16, 12),
                       (BF16, E4M3, 12), (BF16, BF16, 24), (BF16, E4M3, 24), (BF16, BF16, 40), (BF16, E4M3, 40),
                       (F32, F32, 1), (F32, F32, 5), (F32, BF16, 4), (F32, E4M3, 5), (BF16, F32, 5)):
    g = torch.Generator().manual_seed(T)
    n, page = 20_000, 64
    per = -(-(n + T) // page)
    pool = cache.PagedCache.empty(per, 4, page, kind, dev)
    table = torch.randperm(per, generator=g).to(torch.int32)[None].to(dev)
    k, v = (torch.randn((1, 4, n + T, 256), generator=g).to(BF16).to(dev) for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    cache.write(pool, k, v, table, zero)
    q = torch.randn((1, 16, T, 256), generator=g).to(dtype).to(dev)
    want = cache.attend(q, pool, table, zero + n)
    before = cache.status(pool)
    got = []
    for fill in (1, 9):
        os.environ["GQA_ATTN_TEST_SKIP_FILL"] = str(fill)
        t0 = time.time()
        cache.attend(q, pool, table, zero + n)
        faulted = cache.status(pool)
        took = time.time() - t0
        del os.environ["GQA_ATTN_TEST_SKIP_FILL"]
        pool.status_word.zero_()
        out, lse = cache.attend(q, pool, table, zero + n)
        same = bool(torch.equal(out, want[0]) and torch.equal(lse, want[1]))
        got.append([faulted, cache.status(pool), same, took])
    res[f"{dtype} over {kind}, {T}"] = [before, got]
print("RESULT " + json.dumps(res))
"""


def test_the_kernels_over_the_cache_take_their_timeout_exit(cuda_device):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, GQA_ATTN_WAIT_BUDGET_NS="50000000")
    env.pop("GQA_ATTN_TEST_SKIP_FILL", None)
    r = subprocess.run([sys.executable, "-c", _SCRIPT, root], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("RESULT ")][-1]
    for name, (before, got) in json.loads(line[len("RESULT "):]).items():
        assert before == _lib.GQA_OK, name
        for faulted, after, same, took in got:
            assert faulted == _lib.GQA_ERR_DEVICE_TIMEOUT, (name, faulted)
            assert after == _lib.GQA_OK and same, (name, after, same)
            assert took < 5.0, (name, took)
