// Attention of drafted tokens over the paged cache to fp32 accuracy, sm_100a: fp32 queries
// over any pages, and bf16 queries over fp32 ones.
//
// fp32 numbers go through the tensor cores in two pieces: x = hi + lo, hi the nearest number
// of 11 significant bits (tf32), lo the nearest such number to the rest, so the pieces keep
// 22 bits; a product is lo hi + hi lo + hi hi.  bf16 and e4m3 numbers are tf32 numbers, and
// have no lo.  The instruction is mma.sync m16n8k8, keys (in the second product output
// columns) as its M and query rows as its N: a step of decoding has few rows, and they are
// padded to a multiple of 8 only.  The operands' pieces are made in registers on the way;
// tcgen05 would want them written to shared memory, two or three times the bytes of the pages.
// The accumulator drops bits towards zero, so it sums 12 products of a score and 6 of an
// output before they are added in fp32.
//
// A CTA streams its worker's tiles 32 keys at a time.  In a step its 16 warps
//   take 16 keys and 32 columns each of S = K Q^T, the columns' shares added through shared
//     memory (Q's fragments stay in registers: of the registers they take the most);
//   take two rows each of the softmax, 16 lanes to a row, P to shared memory in its pieces;
//   take 32 columns and 16 keys each of the step before's O += V^T P^T, the two key halves
//     added at the end of a segment.
// Two barriers are enough for that: S | softmax and O.  Keys have two slots and values three,
// filled by two warps that have no rows of the softmax, a box per page: a copy of 1 KiB per
// row costs its warp 95 cycles, 3,000 a step.
//
// 5 tokens of 4 heads to a key/value head, 2 x 15,231 fp32 keys, 249 MB: 111 us, of which
// memory alone takes 38.  A step of 24 rows takes 6,300 cycles, 2,300 of them the tensor
// cores' (8 cycles of a scheduler per instruction, 288 of them): S 1,650, softmax 900 and O
// 1,950 come one after another, barriers and waits 900.  Tried: the O before the softmax in
// half of the warps (spills, 132 us); five warps that take keys of their own and 16 rows as M
// (184 us); packed FMAs, eight rows (140 us).
#include "internal.h"
#include "tree_tc.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 16;  // four per scheduler with 128 registers a thread
constexpr int kThreads = 32 * kWarps;
constexpr int kLoadK = 12, kLoadV = 13;  // the warps that load keys, values: 24 rows' softmax takes the first 12
constexpr int kChunk = 1 << kTreeTileShiftF32;   // keys of a step
constexpr int kParts = 8;                        // of the columns, in a score's sum

template <int NT, int kCache, typename QT>
struct F32Cfg {
  static constexpr bool kSplitQ = sizeof(QT) == 4, kSplitKV = kCache == GQA_F32;
  static constexpr int kR = 8 * NT;  // query rows
  static constexpr int kEs = kCache == GQA_F32 ? 4 : kCache == GQA_BF16 ? 2 : 1;
  static constexpr int kRow = kHeadDim * kEs;
  static constexpr int kSlotsK = 8 / kEs, kSlotsV = 12 / kEs;
  static constexpr int kPitchS = 36;   // of a row's partial scores, in floats
  static constexpr int kPitchO = 260;  // of a row's outputs, which take their place
  static constexpr int kPitchP = 320;  // of a row's probabilities, both pieces side by side
  static constexpr int kSlot = kChunk * kRow, kK = 0, kV = kK + kSlotsK * kSlot, kS = kV + kSlotsV * kSlot;
  static constexpr int kSBytes = kParts * kR * kPitchS * 4;
  static constexpr int kP = kS + kSBytes, kPBytes = kR * kPitchP;
  static constexpr int kSmem = kP + 2 * kPBytes + 1024 /* alignment */;
  static_assert(kR * kPitchO * 4 <= kSBytes && kSmem <= 232448 - 4096, "shared memory per block");
};

// (the instruction keeps NaN and infinity; adding half a step to the bits would not)
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
  return y;
}
// The rest of x after its leading piece: NaN for an infinity (and for what rounds to one, from
// 2^128 - 2^116 on), so that the row that sees it becomes NaN.
__device__ __forceinline__ uint32_t rest(float x, uint32_t hi) { return tf32(x - __uint_as_float(hi)); }

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four neighbouring elements of a staged row, as floats.
template <int kCache>
__device__ __forceinline__ void four(const char* at, float (&x)[4]) {
  if constexpr (kCache == GQA_F32) {
    const float4 v = *reinterpret_cast<const float4*>(at);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else if constexpr (kCache == GQA_BF16) {
    const uint2 u = *reinterpret_cast<const uint2*>(at);
    x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
    e4m3_decode4(*reinterpret_cast<const uint32_t*>(at), x);
  }
}

// Four neighbours of a query row (zero for a row that is not there), as floats.
__device__ __forceinline__ void query4(const float* q, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(q);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void query4(const __nv_bfloat16* q, float (&x)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(q);
  x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
}

// What the loading warps tell of a chunk of keys.
template <int kCache>
struct __align__(16) ChunkInfo {
  __align__(16) float scale[kCache == GQA_E4M3 ? 2 * kChunk : 1];  // of key 0's K, V, key 1's K, V, ...
  uint32_t there;                                                  // a bit per key
};

// Where a loading warp is: the next chunk, of all its worker's segments.  In shared memory, for
// registers are what this kernel has none of to spare.
struct FeedState {
  TreeCursor cur;
  TreeSegment g;
  uint32_t j0, n;  // the chunk's first key; chunks so far
  int left;        // chunks of the segment, 0 at the end of all
};

// One warp: the next segment.  Returns the page table's entry of this lane's first key.
__device__ __forceinline__ int feed_segment(const TreeParams& p, TreeCursor cur, uint32_t n, FeedState& st) {
  const int lane = threadIdx.x & 31;
  TreeSegment g;
  const bool live = tree_next(p, cur, &g);
  const uint32_t j0 = live ? uint32_t(g.t0) * kChunk : 0;
  __syncwarp();  // all lanes have read `cur` and `n` from it
  if (lane == 0) {
    st.cur = cur;
    if (live) st.g = g;
    st.j0 = j0;
    st.n = n;
    st.left = live ? g.t1 - g.t0 : 0;
  }
  __syncwarp();
  return live && j0 + lane < g.s.keys ? page_entry(p.c, p.table + int64_t(g.b) * p.max_pages, p.max_pages, j0 + lane) : -1;
}

// One warp: a chunk into its slot of the ring, which is free: a box of all columns for each page
// (or part of a page) of it, rows of 128 bytes, column block by column block, swizzled.  Rows of
// a page past the last key come with it; pages that are not there leave the slot as it was.
template <bool kIsV, int kSlots, int kCache, int kEs>
__device__ __forceinline__ void feed_issue(const TreeParams& p, const CUtensorMap* map, FeedState& st, int& entry,
                                           uint32_t ring, uint32_t full, ChunkInfo<kCache>* info) {
  const int lane = threadIdx.x & 31;
  const uint32_t n = st.n, j = st.j0 + lane, keys = st.g.s.keys;
  const int left = st.left, b = st.g.b, h = st.g.h;
  if (left == 0) return;
  const bool skip = !kIsV && int(n) == p.test_skip_fill;  // test hook: neither armed nor copied
  const uint32_t slot = n % kSlots, slot_mask = (1u << p.c.page_shift) - 1, rows = min(1 << p.c.page_shift, kChunk);
  const int page = j < keys ? page_checked(p.c, entry) : -1;
  const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
  const bool send = page >= 0 && (lane & (rows - 1)) == 0 && !skip;
  const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, send));
  if (lane == 0) {
    if (!kIsV) info[slot].there = there;
    if (!skip) mbar_arrive_expect_tx(full + 8u * slot, boxes * rows * (kHeadDim * kEs));
  }
  __syncwarp();
  if (send)
    tma_load_5d(ring + (slot * kChunk + lane) * uint32_t(kHeadDim * kEs), map, full + 8u * slot, 0, int(j & slot_mask), 0,
                h, page);
  if constexpr (!kIsV && kCache == GQA_E4M3) {
    if (page >= 0 && !skip) {
      const int64_t si = ((int64_t(page) * p.c.Hkv + h) << p.c.page_shift) + (j & slot_mask);
      const uint32_t to = smem_u32(info[slot].scale + 2 * lane);
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p.c.ks + si) : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4), "l"(p.c.vs + si) : "memory");
    }
    // (a key that is not there has no factors; what stands in their place is not used)
    if (!skip) asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(full + 8u * slot) : "memory");
  }
  __syncwarp();
  if (left > 1) {
    entry = j + kChunk < keys ? page_entry(p.c, p.table + int64_t(b) * p.max_pages, p.max_pages, j + kChunk) : -1;
    if (lane == 0) st.n = n + 1, st.j0 += kChunk, st.left = left - 1;
    __syncwarp();
  } else {
    entry = feed_segment(p, st.cur, n + 1, st);
  }
}

// No copy may be in flight when the CTA ends.
template <int kSlots>
__device__ __forceinline__ void feed_drain(const TreeParams& p, const FeedState& st, uint32_t full) {
  for (uint32_t i = st.n < kSlots ? 0 : st.n - kSlots; i < st.n; ++i)
    mbar_wait_inline(full + 8u * (i % kSlots), (i / kSlots) & 1u, p.wait_budget_ns, p.c.status);
}

template <int NT, int kCache, typename QT>
__global__ void __launch_bounds__(kThreads, 1) tree_f32_kernel(const __grid_constant__ TreeParams p,
                                                               const __grid_constant__ CUtensorMap map_k,
                                                               const __grid_constant__ CUtensorMap map_v) {
  using F = F32Cfg<NT, kCache, QT>;
  constexpr int kR = F::kR;
  extern __shared__ __align__(16) char smem_raw[];
  char* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ TreeCursor start;
  __shared__ __align__(16) ChunkInfo<kCache> info[F::kSlotsK];
  __shared__ __align__(8) uint64_t bars[F::kSlotsK + F::kSlotsV];
  __shared__ FeedState feed_k, feed_v;
  __shared__ __align__(8) float sh_alpha[2][kR];   // factors of the outputs so far
  __shared__ uint32_t sh_seen[2][kR];              // keys of a masked chunk that a row sees
  __shared__ float sh_m[kR], sh_l[kR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  const uint32_t full_k = smem_u32(bars), full_v = full_k + 8u * F::kSlotsK;
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kSlotsK; ++i) mbar_init(full_k + 8u * i, kCache == GQA_E4M3 ? 33 : 1);
    for (int i = 0; i < F::kSlotsV; ++i) mbar_init(full_v + 8u * i, 1);
    fence_barrier_init();
  }
  wait_for_grid();  // what comes before in the stream may still have been running
  if (warp == 0) {
    const TreeCursor c = tree_start(p, worker);
    if (lane == 0) start = c;
  }
  __syncthreads();
  launch_dependents();
  int entry = -1;  // of a loading warp's next chunk
  auto issue_k = [&]() {
    feed_issue<false, F::kSlotsK, kCache, F::kEs>(p, &map_k, feed_k, entry, smem_u32(smem + F::kK), full_k, info);
  };
  auto issue_v = [&]() {
    feed_issue<true, F::kSlotsV, kCache, F::kEs>(p, &map_v, feed_v, entry, smem_u32(smem + F::kV), full_v, info);
  };
  if (warp == kLoadK) {
    entry = feed_segment(p, start, 0, feed_k);
#pragma unroll 1
    for (int i = 0; i < F::kSlotsK; ++i) issue_k();
  } else if (warp == kLoadV) {
    entry = feed_segment(p, start, 0, feed_v);
#pragma unroll 1
    for (int i = 0; i < F::kSlotsV; ++i) issue_v();
  }

  const int lq = lane >> 2, lr = lane & 3;        // fragments: lq an outer, lr an inner index
  const int part = warp & 7, half = warp >> 3;    // S: columns 32 part .. + 31, keys 16 half .. + 15 of a chunk;
                                                  // O: the same, as outputs' columns and as summands
  const int srow = threadIdx.x >> 4, pair = threadIdx.x & 15;  // softmax: a row's keys 2 pair, 2 pair + 1
  // A chunk's rows lie in groups of eight keys, [box of min(page, 32) keys][128-byte column block]
  // [key]: this half's two groups, at the block that holds the part's columns.
  constexpr int kPerBlock = 4 / F::kEs;  // parts
  const uint32_t box = min(1 << p.c.page_shift, kChunk);
  uint32_t group[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t key = 16 * half + 8 * i;
    group[i] = key / box * box * F::kRow + part / kPerBlock * (box * 128) + key % box * 128;
  }
  // Row lq of S's fragments is the key of its group that keeps the lanes' loads off each other's banks.
  const uint32_t skey = kCache == GQA_F32 ? (lq >> 1) + 4 * (lq & 1) : kCache == GQA_BF16 ? 2 * (lq & 3) + (lq >> 2) : lq;
  // Byte of a 128-byte row, swizzled, where this part's column `col` of key `key` of a group is.
  auto at = [&](uint32_t key, uint32_t col) {
    const uint32_t byte = (part % kPerBlock * 32 + col) * F::kEs;
    return key * 128 + (byte ^ (key << 4));
  };
  float* const sh_s = reinterpret_cast<float*>(smem + F::kS);
  TreeCursor cur = start;
  uint32_t kn = 0, vn = 0;  // chunks of keys, of values so far
  int v_free = 0;           // slots of values that steps have freed since: two at a segment's end
  bool ok = true;
  TreeSegment g;
  while (tree_next(p, cur, &g)) {
    const int chunks = g.t1 - g.t0;
    // Q's fragments: k = lr of step i of the j-th 16 columns stands for column 4 lr + 2 i of them and
    // k = lr + 4 for the next one, so that a lane has four neighbours of a row in two steps.
    // All loads before their use: one after another they take 9,000 cycles of a cold start.
    float x[2][NT][4];
    bool is[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = rt * kR + 8 * nt + lq, t = n / p.G;
      is[nt] = t < g.s.drafted;  // a row that is not there is loaded as the head's first one, and cleared
      const int64_t row = is[nt] ? int64_t(g.h * p.G + n - t * p.G) * p.q.sh + t * p.q.sl : int64_t(g.h * p.G) * p.q.sh;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        query4(reinterpret_cast<const QT*>(p.q.p) + g.b * p.q.sb + row + 32 * part + 16 * j + 4 * lr, x[j][nt]);
    }
    uint32_t qh[2][NT][4], ql[F::kSplitQ ? 2 : 1][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = is[nt] ? x[j][nt][i] : 0.f;
          qh[j][nt][i] = F::kSplitQ ? tf32(y) : __float_as_uint(y);
          if constexpr (F::kSplitQ) ql[j][nt][i] = rest(y, qh[j][nt][i]);
        }
    float o[2][NT][4];  // columns 32 part + 4 lq + 2 a + (i >> 1), rows 8 nt + 2 lr + (i & 1)
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[a][nt][i] = 0.f;
    float m = -INFINITY, l = 0.f;  // of row srow; l: this lane's keys
    bool masked_before = false;
    const int srow_t = (rt * kR + srow) / p.G;

    for (int c = 0; c <= chunks; ++c) {
      bool masked = false;
      uint32_t there = 0;
      float4 scale = make_float4(1.f, 1.f, 1.f, 1.f);
      const uint32_t j0 = uint32_t(g.t0) * kChunk + uint32_t(c) * kChunk;
      if (c < chunks) {
        const uint32_t slot = kn % F::kSlotsK;
        ok = mbar_wait_inline(full_k + 8u * slot, (kn / F::kSlotsK) & 1u, p.wait_budget_ns, p.c.status);
        __syncwarp();
        there = info[slot].there;
        masked = there != 0xffffffffu || j0 + kChunk > g.s.ctx;
        if constexpr (kCache == GQA_E4M3) scale = *reinterpret_cast<const float4*>(info[slot].scale + 4 * pair);
        // The scores' share of this warp's columns: 16 keys (M) x the rows (N).
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        const char* const k = smem + F::kK + slot * F::kSlot;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x[4], y[4];
          four<kCache>(k + group[0] + at(skey, 16 * j + 4 * lr), x);
          four<kCache>(k + group[1] + at(skey, 16 * j + 4 * lr), y);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float e[4] = {x[2 * i], y[2 * i], x[2 * i + 1], y[2 * i + 1]};
            uint32_t hi[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) hi[u] = F::kSplitKV ? tf32(e[u]) : __float_as_uint(e[u]);
            if constexpr (F::kSplitKV) {
              uint32_t lo[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) lo[u] = rest(e[u], hi[u]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_tf32(s[nt], lo, qh[j][nt][2 * i], qh[j][nt][2 * i + 1]);
            }
            if constexpr (F::kSplitQ) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_tf32(s[nt], hi, ql[j][nt][2 * i], ql[j][nt][2 * i + 1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_tf32(s[nt], hi, qh[j][nt][2 * i], qh[j][nt][2 * i + 1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sh_s[(part * kR + 8 * nt + 2 * lr + (i & 1)) * F::kPitchS + 16 * half + skey + 8 * (i >> 1)] = s[nt][i];
        if (__syncthreads_or(!ok)) {
          ok = false;
          break;
        }
        // All have read the keys, and before that the values of the last step.
        ++kn;
        if (warp == kLoadK) issue_k();
        if (warp == kLoadV) {
#pragma unroll 1
          for (; v_free > 0; --v_free) issue_v();
        }
      }
      if (c < chunks && srow < kR) {
        float x[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kParts; ++u) {
          const float2 y = *reinterpret_cast<const float2*>(sh_s + (u * kR + srow) * F::kPitchS + 2 * pair);
          x[0] += y.x, x[1] += y.y;
        }
        x[0] *= p.scale_log2 * scale.x;
        x[1] *= p.scale_log2 * scale.z;
        bool vis[2] = {true, true};
        if (masked) {
          uint32_t seen = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t key = 2 * pair + i;
            vis[i] = (there >> key) & 1u;
            // (rows past the last drafted token are cleared at the end)
            if (vis[i] && j0 + key >= g.s.ctx && srow_t < g.s.drafted)
              vis[i] = tree_sees(p, g.b, srow_t, int(j0 + key - g.s.ctx));
            if (vis[i]) seen |= 1u << key;
            if (!vis[i]) x[i] = -INFINITY;
          }
#pragma unroll
          for (int u = 1; u < 16; u <<= 1) seen |= __shfl_xor_sync(0xffffffffu, seen, u);
          if (pair == 0) sh_seen[c & 1][srow] = seen;
        }
        float top = fmaxf(x[0], x[1]);
#pragma unroll
        for (int u = 1; u < 16; u <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, u));
        const float m_new = fmaxf(m, top), ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2f(m - ref);  // 0 for the first visible key
        m = m_new;
        const float y0 = vis[0] ? exp2f(x[0] - ref) : 0.f, y1 = vis[1] ? exp2f(x[1] - ref) : 0.f;
        l = fmaf(l, alpha, y0 + y1);
        if (pair == 0) sh_alpha[c & 1][srow] = alpha;
        const float w0 = y0 * scale.y, w1 = y1 * scale.w;
        const uint32_t h0 = tf32(w0), h1 = tf32(w1);
        *reinterpret_cast<uint4*>(smem + F::kP + (c & 1) * F::kPBytes + srow * F::kPitchP + 16 * pair) =
            make_uint4(h0, rest(w0, h0), h1, rest(w1, h1));
      }
      if (c > 0) {
        const int par = (c - 1) & 1;
        const uint32_t slot = vn % F::kSlotsV;
        ok = mbar_wait_inline(full_v + 8u * slot, (vn / F::kSlotsV) & 1u, p.wait_budget_ns, p.c.status);
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 alpha = *reinterpret_cast<const float2*>(&sh_alpha[par][8 * nt + 2 * lr]);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            o[a][nt][0] *= alpha.x, o[a][nt][2] *= alpha.x;
            o[a][nt][1] *= alpha.y, o[a][nt][3] *= alpha.y;
          }
        }
        const char* const v = smem + F::kV + slot * F::kSlot;
        const char* const w = smem + F::kP + par * F::kPBytes + 16 * half * 8;
        if (!masked_before) {
          // O^T: 32 columns (M) x the rows (N) of 16 keys; keys 2 lr and 2 lr + 1 of a step's eight are
          // its k = lr and lr + 4.
          float d[2][NT][4];
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) d[a][nt][0] = d[a][nt][1] = d[a][nt][2] = d[a][nt][3] = 0.f;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float x[4], y[4];
            four<kCache>(v + group[s] + at(2 * lr, 4 * lq), x);
            four<kCache>(v + group[s] + at(2 * lr + 1, 4 * lq), y);
            uint4 pr[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              pr[nt] = *reinterpret_cast<const uint4*>(w + (8 * nt + lq) * F::kPitchP + (8 * s + 2 * lr) * 8);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              const float e[4] = {x[2 * a], x[2 * a + 1], y[2 * a], y[2 * a + 1]};
              uint32_t hi[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) hi[u] = F::kSplitKV ? tf32(e[u]) : __float_as_uint(e[u]);
              if constexpr (F::kSplitKV) {
                uint32_t lo[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) lo[u] = rest(e[u], hi[u]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_tf32(d[a][nt], lo, pr[nt].x, pr[nt].z);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_tf32(d[a][nt], hi, pr[nt].y, pr[nt].w);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_tf32(d[a][nt], hi, pr[nt].x, pr[nt].z);
            }
          }
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[a][nt][i] += d[a][nt][i];
        } else {
          // A chunk with keys that are not there or that some row does not see: on the FP32 pipe, so
          // that a hidden value takes no part at all (0 times an infinity would be NaN).
          uint32_t seen[NT][2], any = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              seen[nt][i] = sh_seen[par][8 * nt + 2 * lr + i] >> (16 * half);
              any |= seen[nt][i];
            }
#pragma unroll 1
          for (int key = 0; key < 16; ++key) {
            if (!((any >> key) & 1u)) continue;
            float x[4];
            four<kCache>(v + (key < 8 ? group[0] : group[1]) + at(key & 7, 4 * lq), x);
            float2 pr[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                pr[nt][i] = *reinterpret_cast<const float2*>(w + (8 * nt + 2 * lr + i) * F::kPitchP + key * 8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if ((seen[nt][i] >> key) & 1u) {
                  const float pp = pr[nt][i].x + pr[nt][i].y;
                  o[0][nt][i] = fmaf(pp, x[0], o[0][nt][i]);
                  o[0][nt][2 + i] = fmaf(pp, x[1], o[0][nt][2 + i]);
                  o[1][nt][i] = fmaf(pp, x[2], o[1][nt][i]);
                  o[1][nt][2 + i] = fmaf(pp, x[3], o[1][nt][2 + i]);
                }
          }
        }
      }
      if (__syncthreads_or(!ok)) {
        ok = false;
        break;
      }
      if (c > 0) {
        ++vn;
        ++v_free;
      }
      masked_before = masked;
    }
    if (!ok) break;

    // The halves' outputs together, then a warp per row.
    float* const outs = reinterpret_cast<float*>(smem + F::kS);
    if (srow < kR) {
#pragma unroll
      for (int u = 1; u < 16; u <<= 1) l += __shfl_xor_sync(0xffffffffu, l, u);
      if (pair == 0) sh_m[srow] = m, sh_l[srow] = l;
    }
#pragma unroll
    for (int h = 1; h >= 0; --h) {
      if (half == h) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float4* const at = reinterpret_cast<float4*>(outs + (8 * nt + 2 * lr + i) * F::kPitchO + 32 * part + 4 * lq);
            float4 y = make_float4(o[0][nt][i], o[0][nt][2 + i], o[1][nt][i], o[1][nt][2 + i]);
            if (h == 0) {
              const float4 other = *at;
              y.x += other.x, y.y += other.y, y.z += other.z, y.w += other.w;
            }
            *at = y;
          }
      }
      __syncthreads();
    }
    const bool whole = g.whole();
    const int64_t piece = (int64_t(worker) * 2 + g.slot()) * p.row_tiles + rt;
    for (int r = warp; r < kR; r += kWarps) {
      const int n = rt * kR + r, t = n / p.G;
      if (t >= p.T) break;
      const float sum = sh_l[r];
      const bool none = t >= g.s.drafted || sum == 0.f;
      const float inv = none ? 0.f : 1.f / sum;  // a NaN sum stays one
      float acc[8];
      load8(outs + r * F::kPitchO + 8 * lane, acc);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = none ? 0.f : acc[i] * inv;
      const float lse = none ? -INFINITY : (sh_m[r] + log2f(sum)) * kLn2;
      if (whole) {
        const int64_t row = (int64_t(g.b) * p.c.Hkv * p.G + g.h * p.G + n % p.G) * p.T + t;
        if (p.out_bf16)
          store8(static_cast<__nv_bfloat16*>(p.out) + row * kHeadDim + 8 * lane, acc);
        else
          store8(static_cast<float*>(p.out) + row * kHeadDim + 8 * lane, acc);
        if (lane == 0) p.lse[row] = lse;
      } else {
        store8(p.o_part + (piece * kR + r) * kHeadDim + 8 * lane, acc);
        if (lane == 0) p.lse_part[piece * kR + r] = lse;
      }
    }
    __syncthreads();  // the next segment's scores take the outputs' place
  }
  if (!ok) {
    if (warp == kLoadK) feed_drain<F::kSlotsK>(p, feed_k, full_k);
    if (warp == kLoadV) feed_drain<F::kSlotsV>(p, feed_v, full_v);
  }
}

template <int NT, int kCache, typename QT>
int launch_one(const TreeParams& p, cudaStream_t stream) {
  constexpr int smem = F32Cfg<NT, kCache, QT>::kSmem;
  if (!allow_smem<tree_f32_kernel<NT, kCache, QT>>(smem)) return GQA_ERR_LAUNCH;
  CUtensorMap map_k, map_v;
  constexpr int blocks = 2 * F32Cfg<NT, kCache, QT>::kEs;
  if (!encode_tokens(&map_k, p.c, p.c.k, kChunk, blocks, blocks) || !encode_tokens(&map_v, p.c, p.c.v, kChunk, blocks, blocks))
    return GQA_ERR_LAUNCH;
  return launch_programmatic(tree_f32_kernel<NT, kCache, QT>, unsigned(p.workers) * unsigned(p.row_tiles), kThreads, smem,
                             stream, p, map_k, map_v);
}

template <int NT>
int launch_rows(const TreeParams& p, bool q_bf16, cudaStream_t stream) {
  if (q_bf16) return launch_one<NT, GQA_F32, __nv_bfloat16>(p, stream);
  if (p.c.dtype == GQA_F32) return launch_one<NT, GQA_F32, float>(p, stream);
  if (p.c.dtype == GQA_BF16) return launch_one<NT, GQA_BF16, float>(p, stream);
  return launch_one<NT, GQA_E4M3, float>(p, stream);
}

}  // namespace

int launch_tree_f32(const TreeParams& p, int rows, bool q_bf16, cudaStream_t stream) {
  return rows == 8 ? launch_rows<1>(p, q_bf16, stream) : rows == 16 ? launch_rows<2>(p, q_bf16, stream)
                                                                    : launch_rows<3>(p, q_bf16, stream);
}

}  // namespace gqa
