/*
 * gqa_attn.h -- C ABI of libgqa_attn.so: exact causal grouped-query attention
 * forward for NVIDIA B200 (sm_100a).
 *
 *   out[b,h,i,:] = sum_j softmax_j( scale * <q[b,h,i,:], k[b,g,j,:]> + mask(i,j) ) * v[b,g,j,:]
 *   lse[b,h,i]   = ln sum_{visible j} exp( scale * <q[b,h,i,:], k[b,g,j,:]> )
 *
 * with g = h / (Hq / Hkv) and scale = 1/sqrt(d).
 *
 * Sources.  The operation is the attention that PyTorch's SDPA computes for a
 * grouped-query model: 16 query heads sharing 4 key/value heads (kev PR #202,
 * "Why fp32 fell to the L x L kernel"), head_dim 256 (system1-omni issue #27,
 * "The closest planned or implemented model").  The library computes it in memory
 * linear in L: the 16 x L x L score matrix that the L x L "math" kernel
 * materialises (69 GB at 32k, 275 GB at 64k per layer, same section) is never
 * formed, and keys/values are never repeated per query head (the 1 GiB per
 * tensor at 64k of kev PR #202, "The change").  Masks: causal; a shared state
 * followed by per-question branches (system1-omni issue #27, item 3: state once,
 * then one branch per question); and segment ids for block-causal packing
 * (maxtext PR #4929, description).  Like the model-agnostic kernel library of
 * system1-omni issue #27 ("The closest planned or implemented model"), this ABI
 * knows no model; unlike the attention entry point named there, it takes a mask.
 *
 * Conventions shared by every entry point
 * --------------------------------------
 * - Layouts are dense and contiguous, batch-major then head-major (SDPA's
 *   [B, H, L, d]):  q, out: [B, Hq, Lq, d];  k, v: [B, Hkv, Lk, d];
 *   lse: [B, Hq, Lq] fp32.  Element type of q, k, v and out is given by dtype
 *   (GQA_F32 = float, GQA_BF16 = bfloat16 stored as uint16, round-to-nearest-even
 *   on output).  Segment ids are int32 arrays of length Lq and Lk, shared by all
 *   batch entries and heads.
 * - Query row i sits at absolute position p = i + q_pos_offset and sees keys
 *   j <= p (so Lk must equal q_pos_offset + Lq).  With segment ids it also needs
 *   segment_ids_q[i] == segment_ids_kv[j].  With GQA_MASK_PREFIX_BRANCH the first
 *   q_pos_offset keys (the shared state) are visible to every query row whatever
 *   their ids; the remaining keys follow the segment (branch) rule.
 * - A query row with no visible key gets out = 0 and lse = -inf.
 * - Pointers named "device" must point to device memory of the current CUDA
 *   device (or be managed memory).  The caller owns every buffer and the stream;
 *   the library allocates, frees and synchronises nothing, except where an entry
 *   point says so.  Work is enqueued on `stream` (NULL = legacy default stream)
 *   and runs asynchronously; the return value reports host-side validation and
 *   launch errors only.  Errors detected on the device (a bounded wait that ran
 *   out) are recorded in the workspace and read with gqa_attn_status().
 * - Every entry point returns a gqa_status_t (0 on success, negative on error)
 *   unless stated otherwise, and leaves outputs untouched on a validation error.
 */
#ifndef GQA_ATTN_H_
#define GQA_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The caller's cudaStream_t, passed through untouched. */
typedef struct CUstream_st *gqa_stream_t;

/*
 * Element types.  GQA_F32 and GQA_F32_TC both take and return fp32 (float)
 * tensors; they differ in how the two contractions run:
 *   GQA_F32     fp32 FFMA on the CUDA cores.
 *   GQA_F32_TC  the tensor cores (tcgen05, kind::f16) on a two-term fp16 split
 *               of every operand, x = hi + lo with hi = fp16(x'), lo = fp16(x' - hi)
 *               after an exact per-head power-of-two scaling x' = x * 2^e that puts
 *               max |x'| in [2^14, 2^15); each product is summed as
 *               hi*hi + hi*lo + lo*hi in fp32, so an element keeps about 22
 *               significant bits and a product about 21.  The scaled split
 *               operands live in the workspace (4 bytes per element of q, k and v).
 *               Forward entry points gqa_attn_fwd and gqa_attn_fwd_split only.
 *               The scale exponent is clamped to [-60, 60]: a head whose max |x| is
 *               2^75 or more (q and k that large overflow fp32 scores on any path; v
 *               is the case that matters) overflows fp16 -- use GQA_F32 there.
 * kev PR #202 ("Measurements") loads its models in fp32 with TF32 off: GQA_F32_TC
 * uses no TF32; its split operands carry twice TF32's 11 significant bits.
 */
typedef enum {
  GQA_F32 = 0,
  GQA_BF16 = 1,
  GQA_F32_TC = 2,
  GQA_E4M3 = 3 /* cache pages only: float8 e4m3 codes with one fp32 scale per row of d */
} gqa_dtype_t;

typedef enum { GQA_MASK_CAUSAL = 0, GQA_MASK_PREFIX_BRANCH = 1 } gqa_mask_t;

typedef enum {
  GQA_OK = 0,
  GQA_ERR_INVALID_ARG = -1,    /* bad shape, null pointer, Lk != q_pos_offset + Lq, ... */
  GQA_ERR_UNSUPPORTED = -2,    /* d != 256, or Hq / Hkv not in {1, 2, 4, 8, 16}        */
  GQA_ERR_MISALIGNED = -3,     /* q/k/v/out/lse/workspace not 16-byte aligned            */
  GQA_ERR_WORKSPACE = -4,      /* workspace null or smaller than gqa_attn_workspace_bytes */
  GQA_ERR_LAUNCH = -5,         /* a CUDA launch or API call failed                       */
  GQA_ERR_DEVICE_TIMEOUT = -6, /* a bounded device-side wait ran out (see gqa_attn_status) */
  GQA_ERR_DEVICE_BOUNDS = -7   /* checked builds only: a shared- or global-memory index
                                  fell outside its buffer (the access was skipped)      */
} gqa_status_t;

/* Tile classes reported by gqa_attn_tile_plan. */
typedef enum { GQA_TILE_SKIP = 0, GQA_TILE_PARTIAL = 1, GQA_TILE_FULL = 2 } gqa_tile_class_t;

/*
 * Bytes of device workspace that gqa_attn_fwd / gqa_attn_tile_plan need for this
 * problem.  Linear in Lq + Lk: a status word plus, when segment ids are used,
 * the [min, max] segment id of every query tile and key tile and the key-tile
 * range of every query tile (maxtext PR #4929, description: block-pair mask
 * tables of O((L / block)^2) entries are what overflowed splash's scalar memory at
 * 1M tokens; this plan keeps O(L / block)).  GQA_F32_TC adds, after 256-byte
 * aligned sections, one fp32 word per query and key/value head (the per-head
 * maxima |x| that fix the split scales) and the split operands: 2 x 2 bytes per
 * element of q, k and v.  Returns 0 for arguments that gqa_attn_fwd would reject.
 * Host-only; touches no device.
 */
size_t gqa_attn_workspace_bytes(int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d,
                                int dtype, int mask_kind, int has_segments);

/*
 * The attention forward (see the top of this file for the operation).
 *
 *   q, k, v        device, read-only, layouts above, 16-byte aligned.
 *   out            device, written, [B, Hq, Lq, d] of dtype, 16-byte aligned.
 *   lse            device, written, [B, Hq, Lq] fp32 (natural log of the scaled
 *                  scores' exp-sum; -inf for a row with no visible key).
 *   B, Hq, Hkv     batch and head counts; Hq % Hkv == 0, Hq / Hkv in {1,2,4,8,16}.
 *   Lq, Lk         query rows and keys, >= 1, Lk == q_pos_offset + Lq.
 *   d              head dimension; must be 256.
 *   dtype          GQA_F32 (fp32 FFMA kernel), GQA_BF16 (tcgen05 kernel) or
 *                  GQA_F32_TC (fp32 tensors, tcgen05 kernel on split operands).
 *   mask_kind      GQA_MASK_CAUSAL or GQA_MASK_PREFIX_BRANCH (needs segment ids).
 *   q_pos_offset   keys preceding query row 0 (a state before its branch rows).
 *   segment_ids_q, segment_ids_kv
 *                  device int32 [Lq] and [Lk], both NULL (no segments) or both set.
 *                  Arbitrary int32 values; nondecreasing ids skip the most tiles.
 *   workspace      device, >= gqa_attn_workspace_bytes(...), 16-byte aligned;
 *                  overwritten by the call.  Calls that share a workspace must be
 *                  ordered on one stream.
 *   stream         the caller's cudaStream_t.
 *
 * Returns GQA_OK once all kernels are enqueued, or an error code with nothing
 * enqueued (validation) or a partly enqueued call (GQA_ERR_LAUNCH).
 */
int gqa_attn_fwd(const void *q, const void *k, const void *v, void *out, float *lse,
                 int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d, int dtype,
                 int mask_kind, int64_t q_pos_offset,
                 const int32_t *segment_ids_q, const int32_t *segment_ids_kv,
                 void *workspace, size_t workspace_bytes, gqa_stream_t stream);

/*
 * Split-KV forward for short query blocks.  The branch rows after a shared state
 * (system1-omni issue #27, item 3: the state is computed once, then one branch per
 * question) and kev PR #202's re-prefill per question ("End to end") put few query
 * rows against a long key range; their query tiles alone leave most of the GPU's SMs
 * idle.  gqa_attn_fwd_split cuts the key-tile range of every query tile into `splits`
 * consecutive chunks, runs each chunk as its own work unit writing a normalised
 * partial output and its log-sum-exp, and merges them exactly:
 *     lse = ln sum_s exp(lse_s),   out = sum_s exp(lse_s - lse) * O_s.
 * The result equals gqa_attn_fwd's up to fp32 rounding order (it is the same online
 * softmax with one more combination step).
 *
 * gqa_attn_split_hint: a split count for this shape on a B200 (148 SMs): 1 when the
 *   query tiles already keep the SMs busy (last wave of work units >= 90 % full for
 *   GQA_F32, >= 60 % for the tensor-core dtypes GQA_BF16 and GQA_F32_TC, whose fp32
 *   partials cost relatively more) or the key ranges are short, else the smallest
 *   count in [2, 16] whose last wave is at least 90 % (GQA_F32) / 80 % full.
 *   Returns a negative gqa_status_t for a shape gqa_attn_fwd rejects.  Host-only.
 * gqa_attn_split_workspace_bytes: device workspace for gqa_attn_fwd_split with this
 *   split count: gqa_attn_workspace_bytes(...) plus splits * B * Hq * Lq * (d + 1)
 *   fp32 values for the partials, 256-byte aligned sections.  0 for a rejected shape
 *   or splits outside [1, 16].  Host-only.
 * gqa_attn_fwd_split: arguments as gqa_attn_fwd, plus `splits` in [1, 16] (1 is
 *   gqa_attn_fwd itself) and a workspace of at least
 *   gqa_attn_split_workspace_bytes(...).  Enqueues the attention kernel and, for
 *   splits > 1, one merge kernel on `stream`.  Errors as gqa_attn_fwd
 *   (GQA_ERR_INVALID_ARG also for splits outside [1, 16]).
 */
int gqa_attn_split_hint(int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int dtype, int mask_kind,
                        int has_segments);
size_t gqa_attn_split_workspace_bytes(int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d, int dtype,
                                      int mask_kind, int has_segments, int splits);
int gqa_attn_fwd_split(const void *q, const void *k, const void *v, void *out, float *lse,
                       int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d, int dtype,
                       int mask_kind, int64_t q_pos_offset,
                       const int32_t *segment_ids_q, const int32_t *segment_ids_kv, int splits,
                       void *workspace, size_t workspace_bytes, gqa_stream_t stream);

/*
 * Context-parallel blocks.  maxtext PR #4929 trains at 1,048,576 tokens with context
 * parallelism ("Effect"), and its code review names the ring attention path
 * (use_tokamax_ring): the sequence is sharded across devices, each device's query
 * rows attend to every earlier device's key/value block in turn, and the partial
 * results are merged by their log-sum-exps.  These two calls are the per-device
 * compute of such a ring; the transport between devices is the caller's (the Python
 * package's `ring` module uses NCCL send / receive through torch.distributed).
 *
 * gqa_attn_fwd_offset: causal attention of Lq query rows against a block of Lk keys
 *   that starts q_pos_offset >= 0 positions before query row 0: row i sees key j iff
 *   j <= i + q_pos_offset.  Unlike gqa_attn_fwd, Lk is free (Lk <= q_pos_offset covers
 *   a block wholly before the queries, every key visible).  No segment ids, causal
 *   mask only.  Arguments, layouts, dtypes and errors otherwise as gqa_attn_fwd; the
 *   workspace needs 256 bytes (16-byte aligned), which is why dtype GQA_F32_TC (whose
 *   split operands live in the workspace) returns GQA_ERR_UNSUPPORTED here.  Every
 *   row sees key 0, so no row is empty.
 * gqa_attn_merge: exact combination of two partial results over disjoint key sets,
 *       lse = ln(exp(lse_a) + exp(lse_b)),
 *       out = exp(lse_a - lse) * o_a + exp(lse_b - lse) * o_b,
 *   row by row over `rows` rows of d = 256 columns.  o_a: device fp32 [rows][d] with
 *   lse_a [rows], or both NULL (an empty partial, lse = -inf); o_b: device fp32 or
 *   bf16 (dtype_b) with lse_b, or both NULL; o_out: device [rows][d] in dtype_out and
 *   lse_out [rows] fp32, written.  o_out / lse_out may be o_a / lse_a (in place,
 *   dtype_out = GQA_F32), not o_b.  A row empty on both sides gets out = 0, lse = -inf.
 *   All pointers 16-byte aligned.  Enqueues one kernel on `stream`.  Errors:
 *   GQA_ERR_INVALID_ARG (rows < 1, an output NULL, a half-given pair, a bad dtype),
 *   GQA_ERR_UNSUPPORTED (d != 256), GQA_ERR_MISALIGNED, GQA_ERR_LAUNCH.
 */
int gqa_attn_fwd_offset(const void *q, const void *k, const void *v, void *out, float *lse,
                        int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d, int dtype,
                        int64_t q_pos_offset, void *workspace, size_t workspace_bytes,
                        gqa_stream_t stream);
int gqa_attn_merge(const float *o_a, const float *lse_a, const void *o_b, const float *lse_b,
                   void *o_out, float *lse_out, int64_t rows, int d, int dtype_b, int dtype_out,
                   gqa_stream_t stream);

/*
 * Attention backward: the gradients of sum(out * dout) with respect to q, k and v,
 * for training on packed long sequences (maxtext PR #4929, description: the splash
 * kernel runs inside training steps over 1,048,576-token packed batches).  With
 * P = exp(scale * S - lse) recomputed from the forward's saved log-sum-exp,
 * D_i = <dout_i, out_i>, dP = dout V^T and dS = P * (dP - D):
 *     dq = scale * dS K,   dk = scale * sum over the group's query heads of dS^T Q,
 *     dv = sum over the group's query heads of P^T dout.
 *
 *   q, k, v, out, lse   device, the forward's inputs and outputs (out and lse as
 *                       written by gqa_attn_fwd or gqa_attn_fwd_split for the same
 *                       arguments), layouts as for gqa_attn_fwd.
 *   dout                device, [B, Hq, Lq, d] of dtype: the upstream gradient.
 *   dq, dk, dv          device, written, shapes of q, k, v, of dtype (bf16 outputs are
 *                       rounded to nearest even from fp32 accumulation).
 *   dtype               GQA_F32 or GQA_BF16; GQA_F32_TC returns GQA_ERR_UNSUPPORTED
 *                       (the fp32 backward is dtype GQA_F32).
 *   other arguments     as for gqa_attn_fwd; every pointer 16-byte aligned.
 *   workspace           device, >= gqa_attn_bwd_workspace_bytes(...): status word,
 *                       block-skip plan at the backward's tile sizes (fp32: 64 query
 *                       rows x 32 keys; bf16: 128 / G positions x 128 keys), and the
 *                       fp32 row dot products D (bf16: also the log2-domain LSE; rows
 *                       padded to a multiple of 128).
 *
 * Rows with no visible key contribute nothing (their dq is 0).  Enqueues on `stream`:
 * GQA_F32 -- a row-dot kernel, the plan kernels (with segment ids), a dK/dV kernel and a
 * dQ kernel, fp32 arithmetic on the CUDA cores; GQA_BF16 -- a row-state kernel, the
 * plan kernels (with segment ids) and three tensor-core kernels (dV, dK, dQ; bf16
 * operands, fp32 accumulation).  Errors as gqa_attn_fwd.  gqa_attn_bwd_workspace_bytes
 * returns 0 for a shape gqa_attn_fwd rejects and for GQA_F32_TC.  Host-only.
 */
size_t gqa_attn_bwd_workspace_bytes(int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d, int dtype,
                                    int mask_kind, int has_segments);
int gqa_attn_bwd(const void *q, const void *k, const void *v, const void *out, const float *lse,
                 const void *dout, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int64_t Lq,
                 int64_t Lk, int d, int dtype, int mask_kind, int64_t q_pos_offset,
                 const int32_t *segment_ids_q, const int32_t *segment_ids_kv, void *workspace,
                 size_t workspace_bytes, gqa_stream_t stream);

/*
 * gqa_attn_bwd_offset: the backward of one block of gqa_attn_fwd_offset (causal
 * attention of Lq query rows against a block of Lk keys that starts q_pos_offset >= 0
 * positions before query row 0; row i sees key j iff j <= i + q_pos_offset; Lk free),
 * for a sequence sharded into blocks (context-parallel training; maxtext PR #4929,
 * description and code review: 1,048,576-token training with a ring attention path).
 * `out` and `lse` are the WHOLE sequence's (the merged forward's rows), so
 * P = exp(scale * S - lse) is the block's share of each row's softmax and D = <dout,
 * out> is the full row's: the call writes the block's contributions to dq (over this
 * key block only), dk and dv (over these query rows only), which the caller sums over
 * the blocks.  Causal mask only, no segment ids; dtype GQA_F32 or GQA_BF16.  Workspace:
 * gqa_attn_bwd_workspace_bytes(B, Hq, Hkv, Lq, Lq, d, dtype, GQA_MASK_CAUSAL, 0) bytes
 * (it does not depend on Lk or the offset).  Other arguments and errors as gqa_attn_bwd.
 */
int gqa_attn_bwd_offset(const void *q, const void *k, const void *v, const void *out, const float *lse,
                        const void *dout, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int64_t Lq,
                        int64_t Lk, int d, int dtype, int64_t q_pos_offset, void *workspace,
                        size_t workspace_bytes, gqa_stream_t stream);

/*
 * Tile shape used by gqa_attn_fwd for this dtype and group size G = Hq / Hkv:
 * *br = query positions per query tile (each tile holds br positions of all G
 * heads of one key/value head), *bc = keys per key tile.  Host-only.
 */
int gqa_attn_tile_sizes(int dtype, int Hq, int Hkv, int *br, int *bc);

/*
 * Test and debug export of the block-skip plan that gqa_attn_fwd computes on the
 * device for the same arguments (same dtype and group size, hence same tiles).
 *
 *   classes     device, written, [nq, nk] uint8 gqa_tile_class_t, nq = ceil(Lq/br),
 *               nk = ceil(Lk/bc) (this matrix exists only in this export; the
 *               forward never forms it).
 *   kv_ranges   device, written, [nq, 2] int32: [first, last + 1) of the non-SKIP
 *               key tiles of each query tile, (0, 0) if none.
 *
 * The class of a (query tile, key tile) pair follows from the tiles' positions and
 * their [min, max] segment ids only; SKIP tiles hold no visible pair and are never
 * read, FULL tiles hold only visible pairs and skip the per-element mask.
 */
int gqa_attn_tile_plan(int Hq, int Hkv, int64_t Lq, int64_t Lk, int dtype, int mask_kind,
                       int64_t q_pos_offset, const int32_t *segment_ids_q,
                       const int32_t *segment_ids_kv, void *workspace, size_t workspace_bytes,
                       uint8_t *classes, int32_t *kv_ranges, gqa_stream_t stream);

/*
 * Device-side status of the last call that used this workspace: GQA_OK,
 * GQA_ERR_DEVICE_TIMEOUT (a bounded wait on an mbarrier ran out; the kernel
 * stopped, its outputs are undefined) or, in a library built with
 * GQA_DEBUG_BOUNDS, GQA_ERR_DEVICE_BOUNDS (an index check of the FFMA kernels
 * failed; the access was skipped, the outputs are undefined).  Synchronises `stream` (copies one word
 * back).  Returns GQA_ERR_LAUNCH if the copy itself fails.
 */
int gqa_attn_status(const void *workspace, gqa_stream_t stream);

/*
 * Self-test of the bounded-wait machinery: launches one CTA that waits on an
 * mbarrier nothing ever arrives on, with a budget of `budget_ns` nanoseconds
 * (1 ms .. 10 s).  The wait must give up and record GQA_ERR_DEVICE_TIMEOUT in
 * the workspace, which gqa_attn_status() then returns; the context stays usable.
 * `workspace` needs gqa_attn_workspace_bytes(...) >= 256 bytes.
 */
int gqa_attn_selftest_wait(void *workspace, size_t workspace_bytes, int64_t budget_ns,
                           gqa_stream_t stream);

/*
 * Self-test of the index checks of a checked build (compiled with GQA_DEBUG_BOUNDS:
 * the fp32 FFMA kernels then check each shared-memory access against the region it
 * belongs to and each output row against its buffer, skip a failing access and record
 * GQA_ERR_DEVICE_BOUNDS).  One CTA evaluates in-range checks and, with planted = 1,
 * one out-of-range shared address and global index as well; only the comparisons
 * run, no access is made.  Afterwards gqa_attn_status() returns GQA_OK (planted = 0)
 * or GQA_ERR_DEVICE_BOUNDS (planted = 1).  Returns GQA_ERR_UNSUPPORTED, launching
 * nothing, in a normal build (which is how a caller tells the two apart);
 * GQA_ERR_INVALID_ARG for planted other than 0 or 1.  `workspace`: >= 256 bytes,
 * 16-byte aligned.
 */
int gqa_attn_selftest_bounds(void *workspace, size_t workspace_bytes, int planted, gqa_stream_t stream);

/*
 * Measurement aid (no attention work): the throughput ceiling of fp32 FMAs with every
 * operand in registers, by operand form:
 *   form 0: fma.rn.f32x2 in the GQA_F32 kernels' operand form, (s_r, s_r+1) +=
 *           (q_r, q_r+1) * (k, k), consecutive FMAs sharing the duplicated k;
 *   form 1: the same FMAs, consecutive ones sharing the (q_r, q_r+1) pair (the order
 *           the kernels use for most of their packed FMAs);
 *   form 2: packed FMAs with no duplicated operand ((q_r, q_r+1) * (k_m, k_m+1) and
 *           the crossed pair);
 *   form 3: scalar fma.rn.f32.
 * Launches `ctas` CTAs of 256 threads; each thread runs `iters` rounds of 64 FMAs and
 * writes one float to out[cta * 256 + thread] (device, ctas * 256 floats, 16-byte
 * aligned, caller-owned).  Asynchronous on `stream`: time it with events; 2 x ctas x
 * 256 x iters x 64 flop over the time is the attainable FP32 rate of that form.  Form
 * 1 is the denominator the bench reports next to the nominal FP32 peak (kev PR #202,
 * "Measurements": the fp32 path is the one evaluated).  GQA_ERR_INVALID_ARG for a null
 * `out`, ctas outside 1 .. 65535, iters < 1 or form outside 0 .. 3;
 * GQA_ERR_MISALIGNED; GQA_ERR_LAUNCH.
 */
int gqa_attn_probe_ffma2(float *out, int ctas, int iters, int form, gqa_stream_t stream);

/*
 * Size of the device scratch behind gqa_attn_fwd_static_ws (2 MiB).  Calls without
 * segment ids need only the 256-byte status header, at any length.  With segment ids
 * the block-skip tables grow with the number of query tiles, Lq * G / 64 (GQA_F32) or
 * Lq * G / 128 (GQA_BF16) with G = Hq / Hkv: 1,048,576-token calls fit for G <= 4 in
 * GQA_F32 and G <= 8 in GQA_BF16; at G = 16 (and G = 8 in GQA_F32) they need more and
 * return GQA_ERR_WORKSPACE.  GQA_F32_TC keeps split operand planes as large as the
 * fp32 inputs in its workspace, so only tiny shapes fit this scratch.
 */
#define GQA_ATTN_STATIC_WORKSPACE_BYTES ((size_t)2 << 20)

/*
 * gqa_attn_fwd without a workspace argument, for callers that cannot allocate device
 * memory (no counterpart on the pages: this is an integration convenience).  Such
 * callers include plug-ins inside a host framework that owns all device memory and
 * exposes no allocator, services held to a fixed memory budget after start-up, and
 * latency-critical paths that must avoid the device synchronisation an allocation can
 * cause.  The caller still provides q, k, v, out, lse and the segment ids exactly as
 * for gqa_attn_fwd (same arguments, layouts, semantics and return codes).
 *
 * Scratch: a file-scope device array of GQA_ATTN_STATIC_WORKSPACE_BYTES in this
 * library, which every GPU that loads the library holds until the process exits.
 * Calls whose gqa_attn_workspace_bytes(...) exceeds that size return
 * GQA_ERR_WORKSPACE and enqueue nothing.  This call allocates and frees nothing and
 * calls no allocating routine.
 *
 * Set-up: the first call on each device (with that device current) looks up the
 * array's device address once; make that first call before any stream capture.
 * Sharing: every call on a device uses the same array and leaves the last call's
 * contents in it (each call resets what must start at zero), so calls that overlap
 * on the GPU -- on different streams, or from several host threads -- race; order
 * them on one stream.  gqa_attn_status() cannot read this scratch.
 */
int gqa_attn_fwd_static_ws(const void *q, const void *k, const void *v, void *out, float *lse,
                           int B, int Hq, int Hkv, int64_t Lq, int64_t Lk, int d, int dtype,
                           int mask_kind, int64_t q_pos_offset,
                           const int32_t *segment_ids_q, const int32_t *segment_ids_kv,
                           gqa_stream_t stream);

/*
 * Decoding from a cache.  The shared state of system1-omni issue #27 (item 3: the state
 * is computed once, then one branch per question) is what a decoder keeps: its keys and
 * values stay in a cache, the next tokens' rotated keys and their values are appended,
 * and one token, or a tree of drafted ones, attends to all of it.  The entry points
 * below are the four steps: rotary positions, the cache's write and read, and the
 * attention of drafted tokens over it.  They differ from those above in three ways:
 * inputs may be strided, lengths live on the device, and device-side errors go to a
 * status word that belongs to the cache.
 *
 * gqa_rows_t: a [B, H, L, d] tensor (d = 256) whose rows of d elements are contiguous.
 *   The strides count elements; data and every stride of a dimension longer than one
 *   are multiples of 16 bytes.  The output of a projection ([B, L, H, d]) is one such
 *   view.
 */
typedef struct {
  void *data;
  int64_t stride_b, stride_h, stride_l;
  int32_t H;
} gqa_rows_t;

/*
 * gqa_cache_t: a pool of pages that sequences share out through their page tables.
 *   k, v              device, [n_pages][Hkv][page_size][d] of dtype, 16-byte aligned;
 *                     stride_page, stride_head and stride_token (elements, the same for
 *                     k and v, multiples of 16 bytes) allow other orders of the first
 *                     three dimensions.
 *   k_scale, v_scale  device fp32 [n_pages][Hkv][page_size], dense: the value of a
 *                     GQA_E4M3 row is code * scale, of any sign.  NULL for the other dtypes.
 *   status            device, one int32 word that the owner zeroes when it makes the
 *                     pool, or NULL.  The calls record the first device-side error in
 *                     it (GQA_ERR_DEVICE_BOUNDS: a page index outside 0 .. n_pages - 1
 *                     or a length outside the page table; GQA_ERR_DEVICE_TIMEOUT) and
 *                     never clear it; read it with gqa_attn_status(status, stream).
 *                     What a bad index or length names is neither read nor written.
 *   Hkv, page_size    key/value heads; tokens per page, a power of two in 8 .. 1024.
 *   dtype             GQA_F32, GQA_BF16 or GQA_E4M3.
 * A page table is device int32 [B][max_pages], dense: token j of sequence b is slot
 * j % page_size of page page_table[b][j / page_size].  Entries past a sequence's last
 * token are not read.  Sequences may share pages that nothing writes.
 */
typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  int32_t *status;
  int64_t stride_page, stride_head, stride_token, n_pages;
  int32_t Hkv, page_size, dtype;
} gqa_cache_t;

typedef enum { GQA_ROPE_HALF = 0, GQA_ROPE_INTERLEAVED = 1 } gqa_rope_layout_t;
typedef enum {
  GQA_ROPE_PLAIN = 0,
  GQA_ROPE_LINEAR = 1,
  GQA_ROPE_NTK = 2,
  GQA_ROPE_YARN = 3
} gqa_rope_scaling_t;

/*
 * gqa_rope_t: the rotation of a [.., d] row at position p.  Pair i < rot / 2 of the
 * first `rot` columns -- (x[i], x[i + rot / 2]) with GQA_ROPE_HALF, (x[2 i], x[2 i + 1])
 * with GQA_ROPE_INTERLEAVED -- turns by the angle a = p * f_i:
 *     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a);
 * the other columns are left as they are.
 *   turns      device, rot / 2 words from gqa_attn_rope_turns: f_i / (2 pi) as a binary
 *              fraction of 64 bits.  p * turns modulo 2^64 is then the angle's exact
 *              fraction of a turn, so far positions lose nothing.
 *   magnitude  m; rot: a multiple of 16 in 16 .. 256; layout: gqa_rope_layout_t.
 *   positions  device int32 [B][L] with row stride positions_stride_b (0: one row for
 *              all sequences), any values; or NULL: token l of sequence b is at
 *              pos_offset + l (gqa_attn_cache_write: at its own place in the sequence
 *              plus pos_offset).
 */
typedef struct {
  const uint64_t *turns;
  const int32_t *positions;
  int64_t positions_stride_b, pos_offset;
  float magnitude;
  int32_t rot, layout;
} gqa_rope_t;

/*
 * gqa_attn_rope_freqs: writes f_i, i < rot / 2, to inv_freq (host) and m to *magnitude.
 *   GQA_ROPE_PLAIN   f_i = base^(-2 i / rot)
 *   GQA_ROPE_LINEAR  f_i / factor: positions interpolated
 *   GQA_ROPE_NTK     base * factor^(rot / (rot - 2)) in place of base: the slowest pair
 *                    slows by factor, the fastest by nothing
 *   GQA_ROPE_YARN    by parts: f_i g + f_i / factor (1 - g) with g = clamp((r_i -
 *                    beta_slow) / (beta_fast - beta_slow), 0, 1), r_i = original_length
 *                    f_i / (2 pi) the pair's turns over the length trained on, and
 *                    m = 0.1 ln(factor) + 1 (the YaRN paper, Peng et al. 2023, section 3; some
 *                    loaders ramp in i between rounded bounds instead: pass their frequencies to
 *                    gqa_attn_rope_turns)
 *   m = 1 but for GQA_ROPE_YARN.  GQA_ERR_INVALID_ARG: a null pointer, base <= 1, factor
 *   < 1, original_length < 1 or beta_fast <= beta_slow (GQA_ROPE_YARN), rot of 2 with
 *   GQA_ROPE_NTK, or rot not an even number in 2 .. 256.  Host-only.
 * gqa_attn_rope_turns: the n words of `turns` (host) for any finite frequencies inv_freq
 *   (host; computed above or the user's own).  GQA_ERR_INVALID_ARG for a null pointer, n <
 *   1 or a frequency that is not finite.  Host-only; the caller copies them to the device.
 */
int gqa_attn_rope_freqs(int rot, double base, int scaling, double factor, int64_t original_length, double beta_fast,
                        double beta_slow, double *inv_freq, double *magnitude);
int gqa_attn_rope_turns(const double *inv_freq, int n, uint64_t *turns);

/*
 * gqa_attn_rope: rotates the rows of x (and of x2, when it is not NULL: q and k in one
 * launch) into out (and out2), of the same dtype (GQA_F32 or GQA_BF16; fp32 arithmetic,
 * one rounding).  With inverse != 0 it turns by -a with the same m, which is the
 * gradient of the rotation: dx = the inverse rotation of dy.  out may be x itself.
 * Enqueues one kernel on `stream`; B or L of 0 enqueues nothing.  Errors:
 * GQA_ERR_INVALID_ARG (a null pointer, a negative size, H < 1, another dtype or layout,
 * rot out of its range), GQA_ERR_UNSUPPORTED (d != 256), GQA_ERR_MISALIGNED (data or a
 * stride not a multiple of 16 bytes), GQA_ERR_LAUNCH.
 */
int gqa_attn_rope(const gqa_rows_t *x, const gqa_rows_t *out, const gqa_rows_t *x2, const gqa_rows_t *out2, int B,
                  int64_t L, int d, int dtype, const gqa_rope_t *rope, int inverse, gqa_stream_t stream);

/*
 * gqa_attn_cache_write: appends L tokens of each of B sequences to the cache.
 *   k, v        views of H = Hkv heads, dtype GQA_F32 or GQA_BF16.
 *   page_table  [B][max_pages]; start: device int32 [B], the tokens a sequence holds
 *               already: its token i goes to place start[b] + i.
 *   lens        device int32 [B], tokens of each sequence to write (values above L count
 *               as L, below 0 as 0), or NULL: L of each.
 *   rope        the keys are rotated in fp32 before they are rounded; NULL: stored as they
 *               are.  rope->positions NULL: position = start[b] + i + pos_offset.  Drafted
 *               tokens of a tree share positions: give them.
 * GQA_F32 and GQA_BF16 pages get the value rounded once.  GQA_E4M3 pages get, per row, the
 * scale 2^ceil(log2(amax / 448)) with amax the largest finite |x| of the row (scale 1 when
 * amax is 0; the exponent kept in -120 .. 120), and the codes of x / scale, rounded to
 * nearest even; a power of two makes the division exact, and costs a float format no
 * precision.  Infinities become +-448, NaN stays NaN.
 * No two tokens of a call may go to the same slot.  Slots that no token goes to are left as
 * they were.  A token whose place is outside the page table, or whose page index is outside
 * the pool, is skipped and recorded in cache->status.  Enqueues one kernel.  Errors as
 * gqa_attn_rope, and GQA_ERR_INVALID_ARG for scales that do not fit the dtype, k or v with
 * other heads than the cache, a page_size or max_pages out of range.
 *
 * gqa_attn_cache_read: the first lens[b] tokens of each sequence as dense k_out and v_out
 * [B, Hkv, max_len, d] of dtype_out (GQA_F32 or GQA_BF16, one rounding), zeros behind them
 * and for a bad page index (recorded); lens above max_len count as max_len, below 0 as 0.
 * Enqueues one kernel.  Errors as above.
 */
int gqa_attn_cache_write(const gqa_cache_t *cache, const gqa_rows_t *k, const gqa_rows_t *v,
                         const int32_t *page_table, int64_t max_pages, const int32_t *start, const int32_t *lens,
                         int B, int64_t L, int d, int dtype, const gqa_rope_t *rope, gqa_stream_t stream);
int gqa_attn_cache_read(const gqa_cache_t *cache, const int32_t *page_table, int64_t max_pages, const int32_t *lens,
                        void *k_out, void *v_out, int B, int64_t max_len, int d, int dtype_out, gqa_stream_t stream);

/*
 * gqa_attn_fwd_tree: attention of T drafted tokens per sequence over the cache, B and T at least
 * 1 as in gqa_attn_fwd (the rotation, the write and the read take 0 and do nothing).  T = 1 is
 * one decoding step.  Sequence b holds context_lens[b] tokens and, behind them, its first
 * tree_lens[b] drafted ones, whose keys and values are in the cache already.  Drafted token
 * t sees the whole context and the drafted tokens u < tree_lens[b] with tree_mask[t][u]:
 *     out[b,h,t] = sum_j softmax_j(<q[b,h,t], k[b,g,j]> / 16) v[b,g,j],  lse as gqa_attn_fwd.
 *   q             view of Hq heads and T tokens, dtype GQA_F32 or GQA_BF16; Hq / Hkv in
 *                 {1, 2, 4, 8, 16}.
 *   page_table, max_pages, context_lens  as above (context_lens: device int32 [B], 0 or
 *                 more; context and drafted tokens fit the page table).
 *   tree_lens     device int32 [B], or NULL: T of each.  Tokens t >= tree_lens[b] are
 *                 padding: no visible key.
 *   tree_mask     device bytes [T][T], or [B][T][T] with mask_stride_b = T * T (0: one mask
 *                 for all); not 0 = visible, and nothing else is implied: a row's own token
 *                 too has to be named.  NULL: a chain, token t sees u <= t.
 *   out, lse      device, written whole: [B, Hq, T, d] of dtype and [B, Hq, T] fp32.  A row
 *                 with no visible key gets out = 0 and lse = -inf.
 *   workspace     device, >= gqa_attn_tree_workspace_bytes(...), 16-byte aligned,
 *                 overwritten; calls that share one must be ordered on one stream.
 * What a row's mask hides does not reach the row, NaN and infinities among it.  Work is cut
 * evenly over the SMs whatever the lengths; partial results are merged in a fixed order, so
 * equal calls give equal bits.
 * Accuracy.  Sums, maxima and the log-sum-exp are fp32.  GQA_BF16 queries over GQA_BF16 pages:
 * products of the numbers as they are; a probability is off by 2^-15 of itself before it is
 * multiplied with its value, or, with T Hq / Hkv above 32, rounded to bf16 (2^-8), as in
 * gqa_attn_fwd.  Over GQA_E4M3 pages: products of the codes as they are; a query is off by 2^-10
 * after its row is scaled to at most 448, and a probability by 2^-8.8 of itself down to 2^-20 of
 * the largest p x scale that the row sees, and by 2^-28 of that below, so many small ones keep what
 * they hold together (2^18 of them lose 2^-10 of the largest).  That holds for value scales, among the
 * keys of a row, of 2^-100 .. 2^100 in magnitude that lie within 2^100 of one another, beside values of
 * zeros (whose scale does not matter) of 2^-60 .. 2^60; a subnormal scale counts as zero.
 * The other pairs of types are multiplied to fp32 accuracy (two tf32 pieces of each fp32 number):
 * there an infinite key makes the rows that see it NaN, and an infinite value their column.
 * Errors: as gqa_attn_cache_write, GQA_ERR_UNSUPPORTED (d, Hq / Hkv, T > 1024,
 * B Hq above 2^31 - 1), GQA_ERR_WORKSPACE.
 * gqa_attn_tree_workspace_bytes returns 0 for a shape that the call rejects.  Host-only.
 */
size_t gqa_attn_tree_workspace_bytes(int B, int Hq, int Hkv, int64_t T, int64_t max_pages, int page_size, int d,
                                     int dtype, int cache_dtype);
int gqa_attn_fwd_tree(const gqa_rows_t *q, const gqa_cache_t *cache, const int32_t *page_table, int64_t max_pages,
                      const int32_t *context_lens, const int32_t *tree_lens, const uint8_t *tree_mask,
                      int64_t mask_stride_b, void *out, float *lse, int B, int64_t T, int d, int dtype,
                      void *workspace, size_t workspace_bytes, gqa_stream_t stream);

/* Static, human-readable text for a gqa_status_t; never NULL. */
const char *gqa_attn_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ATTN_H_ */
