// Attention of drafted tokens over the paged cache on the 5th-generation tensor cores
// (tcgen05 / TMEM), sm_100a: bf16 queries, bf16 or e4m3 pages.
//
// Few query rows meet many keys, so the keys take the long side of every product: a tile
// of 128 keys is the M of S^T = K Q^T (N = the query rows, 16 .. 128), and the 256 columns
// of the values, in two halves, are the M of O^T += V^T P^T.  With the rows as M, 4 rows
// would cost what 128 do.  TMEM, per CTA: two S^T buffers of N columns (lane = key) and the
// two halves of O^T (lane = column of the output), 4 N columns in all.
//
// e4m3 pages are multiplied as they are (kind::f8f6f4, exact products in fp32): the query
// is scaled by a power of two so that its largest element lies in [224, 448) and taken
// apart into two e4m3 pieces, q = hi + lo, off by at most 2^-10 of that scale; so is each
// probability.  Both pieces are multiplied into the same accumulator, which costs a second
// instruction at twice the rate.  The scales of a key go into its scores, those of a value
// into its probability, before that is rounded.
//
// Softmax: one thread per key and up to 32 rows; the running maximum m of a row is raised
// only when a score passes it by kSlack (in powers of two), so most tiles need no
// reduction over the keys and no rescaling of O.  P = 2^(x - m) goes to shared memory as
// the B operand; the row sum stays with the threads, in fp32, until the end.  For e4m3, x
// includes log2 of the value's scale, so that m follows the largest product p v rather
// than the largest p, and P is stored as 64 P <= 256: a probability then keeps 8 bits down
// to 2^-10 of the largest, and is off by 2^-15 of it below.
//
// Warps: 4 softmax warps per 32 (or 16) rows, one producer warp per 32 KiB slot of the
// ring (cp.async, 16 bytes at a time, through the page table; two rows to an
// instruction), and one warp whose first lane issues the MMAs.
#include "internal.h"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace gqa {
namespace {

constexpr int kSlotBytes = 32768;  // 128 keys x 256 bytes: half of a bf16 tile, a whole e4m3 one
constexpr int kChunk = 16384;      // 128 keys x 128 bytes, one swizzled column block
constexpr float kNoMax = -1e30f;   // a row's maximum before its first visible key

template <int kN, bool kFp8>
struct Cfg {
  static constexpr int kCols = kN < 32 ? kN : 32;  // rows of a softmax thread
  static constexpr int kParts = kN / kCols;
  static constexpr int kSoftWarps = 4 * kParts;
  static constexpr int kPieces = kFp8 ? 2 : 1;
  static constexpr int kItems = kFp8 ? 2 : 4;  // slots of a tile
  static constexpr int kQBytes = kN * 512;     // bf16, or two e4m3 pieces
  static constexpr int kPBytes = kFp8 || kN > 64 ? 2 * kChunk : kChunk;
  static constexpr int kSlots = kN > 64 ? 4 : kFp8 || kN > 32 ? 5 : 6;  // what shared memory has room for
  static constexpr int kWarps = kSoftWarps + kSlots + 1;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffRing = kOffP + kPBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
  static constexpr int kOffM = kOffBar + 256;     // [kN] maxima
  static constexpr int kOffF = kOffM + kN * 4;    // [kN] factor of a row's scores (e4m3 pages)
  static constexpr int kOffBad = kOffF + kN * 4;  // 32 words: drafted tokens with a value that is not finite
  static constexpr int kSmem = kOffBad + 128;
  static constexpr float kSlack = kFp8 ? 2.f : 8.f;
  static constexpr uint32_t kTmem = 4 * kN;
  static_assert(kSmem <= 232448 - 64, "shared memory per block");
};

// Barriers: S^T, its release, P and O per parity of the tile; the ring's slots.
enum { kBarQ = 0, kBarS = 1, kBarSFree = 3, kBarP = 5, kBarPV = 7, kBarDrain = 9, kBarFull = 10, kBarEmpty = 16 };

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int64_t budget, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, budget, status));
}

// Barriers over `n` threads, and the OR of `pred` over them: all take the same branch.
__device__ __forceinline__ void sync_threads(uint32_t id, uint32_t n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ bool any_thread(uint32_t id, uint32_t n, bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(uint32_t(pred)), "r"(id), "r"(n)
      : "memory");
  return out != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// D[tmem] (+)= A[smem] B[smem]^T in the type of the pages.
template <bool kFp8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)));
  else
    umma::mma_ss(d, a, b, idesc, add);
}

// Instruction descriptor: fp32 accumulator, M = 128; e4m3 is format 0 of kind::f8f6f4, bf16
// format 1 of kind::f16.
template <bool kFp8>
__host__ __device__ constexpr uint32_t idesc(int N, int a_mn, int b_mn) {
  return (1u << 4) | (kFp8 ? 0u : (1u << 7) | (1u << 10)) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         (uint32_t(N >> 3) << 17) | (8u << 24);
}

template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[C]) {
  if constexpr (C == 32)
    umma::tmem_ld32(addr, v);
  else
    umma::tmem_ld16(addr, v);
}

// Sum or maximum over the 32 lanes of each of C values: lane l ends with value l (C = 32)
// or l / 2 (C = 16).  A lane sends the half that it does not keep.
template <int C, bool kMax>
__device__ __forceinline__ float lanes_reduce(float (&v)[C]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = C / 2, off = 16; half >= 1; half >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
      if (i < half) {
        const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
        const float got = __shfl_xor_sync(0xffffffffu, send, off);
        v[i] = kMax ? fmaxf(keep, got) : keep + got;
      }
  }
  if (C == 16) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
    v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

template <int kN, bool kFp8>
__global__ void __launch_bounds__(Cfg<kN, kFp8>::kThreads, 1) tree_tc_kernel(const __grid_constant__ TreeParams p) {
  using F = Cfg<kN, kFp8>;
  constexpr int C = F::kCols;
  extern __shared__ __align__(1024) char smem_raw[];
  __shared__ TreeCursor start;
  __shared__ uint32_t tmem_slot;
  const uint32_t sbase = smem_u32(smem_raw);
  const bool misaligned = (sbase & 1023u) != 0;  // the swizzle needs it; never expected to fail
  const uint32_t sQ = sbase + F::kOffQ, sP = sbase + F::kOffP, sRing = sbase + F::kOffRing;
  auto bar = [&](int i) { return sbase + F::kOffBar + 8u * uint32_t(i); };
  float* sh_m = reinterpret_cast<float*>(smem_raw + F::kOffM);
  float* sh_f = reinterpret_cast<float*>(smem_raw + F::kOffF);
  uint32_t* sh_bad = reinterpret_cast<uint32_t*>(smem_raw + F::kOffBad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  const int64_t budget = p.wait_budget_ns;
  int32_t* status = p.c.status;

  if (warp == 0) {
    const TreeCursor c = tree_start(p, worker);
    if (lane == 0) {
      start = c;
      mbar_init(bar(kBarQ), F::kSoftWarps);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kBarS + i), 1);
        mbar_init(bar(kBarSFree + i), F::kSoftWarps);
        mbar_init(bar(kBarP + i), F::kSoftWarps);
        mbar_init(bar(kBarPV + i), 1);
      }
      mbar_init(bar(kBarDrain), 1);
      for (int i = 0; i < F::kSlots; ++i) {
        mbar_init(bar(kBarFull + i), 1);
        mbar_init(bar(kBarEmpty + i), 1);
      }
      fence_barrier_init();
      if (misaligned) set_status(status, GQA_ERR_LAUNCH);
    }
  }
  if (warp == F::kWarps - 1) umma::tmem_alloc(smem_u32(&tmem_slot), F::kTmem);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  TreeCursor cur = start;
  TreeSegment g;

  if (misaligned) {
    // no role
  } else if (warp >= F::kSoftWarps && warp < F::kWarps - 1) {
    // ---------------------------------------------------------------- producers
    // This warp fills slot `s`: items s, s + kSlots, ... of the tiles' list.  A bf16 tile is
    // four items (key columns 0 - 127, 128 - 255, the same of the values), an e4m3 tile two.
    // Image of an item: two column blocks of 128 bytes, [128 keys][128 bytes] each, 16-byte
    // units at unit ^ (key & 7).  Keys past the end are zeros.
    const int s = warp - F::kSoftWarps;
    const uint32_t slot = sRing + uint32_t(s) * kSlotBytes;
    const int unit = lane & 15, odd = lane >> 4;
    const uint32_t dst0 = slot + uint32_t(unit >> 3) * kChunk;
    constexpr int kEs = kFp8 ? 1 : 2;
    const int64_t slot_mask = (int64_t(1) << p.c.page_shift) - 1;
    int64_t idx = s;
    bool live = tree_next(p, cur, &g);
    // The page of each group of eight keys of this item, in lanes 0 .. 15.
    auto pages = [&]() {
      while (live && idx >= (g.t1 - g.t0) * F::kItems) {
        idx -= (g.t1 - g.t0) * F::kItems;
        live = tree_next(p, cur, &g);
      }
      if (!live) return -1;
      const int64_t j = (g.t0 + idx / F::kItems) * kTreeTile + lane * 8;
      return lane < 16 && j < g.s.keys ? page_of(p.c, p.table + int64_t(g.b) * p.max_pages, p.max_pages, j) : -1;
    };
    int pg = pages();
    for (uint32_t n = 0; live; ++n) {
      if (!warp_wait(bar(kBarEmpty + s), (n & 1u) ^ 1u, budget, status)) break;
      const int item = int(idx % F::kItems);
      const int64_t j0 = (g.t0 + idx / F::kItems) * kTreeTile;
      const char* pool = (item >= F::kItems / 2 ? p.c.v : p.c.k) + int64_t(g.h) * p.c.sh * kEs;
      const int column = kFp8 ? 0 : (item & 1) * 256;
      const int64_t row_bytes = p.c.st * kEs;
#pragma unroll 4
      for (int grp = 0; grp < 16; ++grp) {
        const int page = __shfl_sync(0xffffffffu, pg, grp);
        const int64_t in_page = (j0 + grp * 8) & slot_mask;
        const char* src = pool + (int64_t(page) * p.c.sp + in_page * p.c.st) * kEs + column + unit * 16 + odd * row_bytes;
        const int rows = page < 0 ? 0 : int(min(int64_t(8), g.s.keys - (j0 + grp * 8)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * i + odd;
          const bool there = r < rows;
          cp_async16(dst0 + uint32_t(grp * 8 + r) * 128u + uint32_t(((unit & 7) ^ r) << 4),
                     there ? src + 2 * i * row_bytes : pool, there ? 16u : 0u);
        }
      }
      idx += F::kSlots;
      pg = pages();  // the next item's, while this one's copies are under way
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarFull + s));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == F::kWarps - 1) {
    // ---------------------------------------------------------------- MMA issuer
    // S(t + 1) is issued ahead of O += P(t) V(t), so that the softmax of a tile runs beside
    // the products of its neighbours.
    if (lane == 0) {
      constexpr uint32_t id_s = idesc<kFp8>(kN, 0, 0), id_o = idesc<kFp8>(kN, 1, 1);
      constexpr int kRowSteps = kFp8 ? 4 : 8;  // K steps of O: 32 or 16 keys each
      uint32_t item = 0;   // next item of the ring
      uint32_t ts = 0, tp = 0;  // tiles whose S / whose O has been issued
      bool ok = true;
      uint32_t segs = 0;
      auto full = [&](uint32_t it) {
        return mbar_wait_inline(bar(kBarFull + int(it % F::kSlots)), (it / F::kSlots) & 1u, budget, status);
      };
      auto release = [&](uint32_t it) { umma::commit(bar(kBarEmpty + int(it % F::kSlots))); };
      auto slot_of = [&](uint32_t it) { return sRing + (it % F::kSlots) * uint32_t(kSlotBytes); };
      auto issue_s = [&]() {
        const uint32_t b = ts & 1u;
        if (ts >= 2 && !mbar_wait_inline(bar(kBarSFree + int(b)), ((ts - 2) >> 1) & 1u, budget, status)) return false;
        const uint32_t d = tmem + b * kN;
        const uint64_t dq = umma::smem_desc(sQ, 16, 1024);
        for (int half = 0; half < F::kItems / 2; ++half) {
          if (!full(item + half)) return false;
          umma::fence_after_sync();
          const uint64_t dk = umma::smem_desc(slot_of(item + half), 16, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // column block (kFp8: 128 columns, else 64) and 32-byte step inside it
            const uint32_t a = uint32_t(k >> 2) * kChunk + uint32_t(k & 3) * 32u;
            const uint32_t q = uint32_t((kFp8 ? 0 : 2 * half) + (k >> 2)) * (kN * 128u) + uint32_t(k & 3) * 32u;
#pragma unroll
            for (int piece = 0; piece < F::kPieces; ++piece)
              mma<kFp8>(d, umma::desc_add(dk, a), umma::desc_add(dq, q + uint32_t(piece) * (kN * 256u)), id_s,
                        (half | k | piece) != 0);
          }
          release(item + half);
        }
        umma::commit(bar(kBarS + int(b)));
        item += F::kItems / 2;
        ++ts;
        return true;
      };
      auto issue_o = [&](uint32_t it, bool first) {
        const uint32_t b = tp & 1u;
        if (!mbar_wait_inline(bar(kBarP + int(b)), (tp >> 1) & 1u, budget, status)) return false;
        const uint64_t dp = umma::smem_desc(sP, kChunk, 1024);
        for (int half = 0; half < 2; ++half) {
          const uint32_t vit = kFp8 ? it : it + half;
          if ((!kFp8 || half == 0) && !full(vit)) return false;
          umma::fence_after_sync();
          const uint64_t dv = umma::smem_desc(slot_of(vit) + (kFp8 ? uint32_t(half) * kChunk : 0u), kChunk, 1024);
          const uint32_t d = tmem + (2 + half) * kN;
#pragma unroll
          for (int k = 0; k < kRowSteps; ++k) {
            const uint32_t rows = uint32_t(k) * (kFp8 ? 4096u : 2048u);
#pragma unroll
            for (int piece = 0; piece < F::kPieces; ++piece)
              mma<kFp8>(d, umma::desc_add(dv, rows), umma::desc_add(dp, rows + uint32_t(piece) * kChunk), id_o,
                        !first || (k | piece) != 0);
          }
          if (!kFp8 || half == 1) release(vit);
        }
        umma::commit(bar(kBarPV + int(b)));
        ++tp;
        return true;
      };
      while (ok && tree_next(p, cur, &g)) {
        if (!(ok = mbar_wait_inline(bar(kBarQ), segs & 1u, budget, status))) break;
        ++segs;
        const int64_t n = g.t1 - g.t0;
        // Items run K(0) V(0) K(1) V(1) ...: V(t) lies kItems / 2 behind K(t).
        ok = issue_s();
        for (int64_t t = 0; ok && t < n; ++t) {
          const uint32_t v = item;
          item += F::kItems / 2;
          if (t + 1 < n) ok = issue_s();
          ok = ok && issue_o(v, t == 0);
        }
      }
      if (ts > 0) {  // every product complete before TMEM is released
        umma::commit(bar(kBarDrain));
        mbar_wait_inline(bar(kBarDrain), 0, budget, status);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    constexpr uint32_t kAll = 32 * F::kSoftWarps;  // threads of barrier 15
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t part_bar = 1u + uint32_t(part);
    const int n0 = part * C;              // first row (column of S^T and O^T) of this thread
    const int key = quarter * 32 + lane;  // TMEM lane: key of the tile, column of O's half
    const uint32_t lane_addr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(n0);
    const int g_shift = __ffs(p.G) - 1;
    const int rows_all = p.T * p.G;
    const int row0 = rt * kN;  // this CTA's first row among the T G of a head
    const int64_t slot_mask = (int64_t(1) << p.c.page_shift) - 1;
    // This thread's 16-byte unit `i` of P (its key, eight or sixteen rows from n0 on).
    auto p_unit = [&](int k, int i) {
      const int un = n0 / (kFp8 ? 16 : 8) + i;
      return sP + uint32_t(un >> 3) * kChunk + uint32_t(k) * 128u + uint32_t(((un & 7) ^ (k & 7)) << 4);
    };
    // The quarters' exchange of one value per row lies in the part's own columns of P, which
    // no product reads then: row n's from quarter q is with the thread of lane n % 32 of it.
    static_assert(C == 16 || C == 32, "a row's value fits a lane");
    auto put = [&](float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(p_unit(key, 0)), "f"(v) : "memory"); };
    auto get = [&](int q, int n) {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p_unit(q * 32 + n, 0)) : "memory");
      return v;
    };
    uint32_t tt = 0;  // tiles so far
    bool ok = true;

    while (ok && tree_next(p, cur, &g)) {
      const int32_t* table = p.table + int64_t(g.b) * p.max_pages;
      // Q of this head: all softmax warps, a row each time; every reader of the last one is done.
      for (int r = warp; r < kN; r += F::kSoftWarps) {
        const int n = row0 + r, t = n >> g_shift;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (t < g.s.drafted)
          u = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q.p) + g.b * p.q.sb +
                                              int64_t(g.h * p.G + (n & (p.G - 1))) * p.q.sh + t * p.q.sl + 8 * lane);
        if constexpr (!kFp8) {
          sts16(sQ + uint32_t(lane >> 3) * (kN * 128u) + uint32_t(r) * 128u + uint32_t(((lane & 7) ^ (r & 7)) << 4), u);
        } else {
          float x[8], lo[8];
          unpack8(u, x);
          float amax = 0.f;
          bool finite = true;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            amax = fmaxf(amax, fabsf(x[i]));
            finite = finite && fabsf(x[i]) < INFINITY;
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          finite = __all_sync(0xffffffffu, finite);
          const float scale = e4m3_row_scale(finite ? amax : 0.f);
          const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= inv;
          const uint32_t h0 = e4m3_encode4(x), h1 = e4m3_encode4(x + 4);
          e4m3_decode4(h0, lo);
          e4m3_decode4(h1, lo + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) lo[i] = x[i] - lo[i];
          const uint32_t a = sQ + uint32_t(lane >> 4) * (kN * 128u) + uint32_t(r) * 128u +
                             uint32_t((((lane & 15) >> 1) ^ (r & 7)) << 4) + uint32_t(lane & 1) * 8u;
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(h0), "r"(h1) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a + kN * 256u), "r"(e4m3_encode4(lo)),
                       "r"(e4m3_encode4(lo + 4))
                       : "memory");
          // A row with an infinity or NaN has no finite score.
          if (lane == 0) sh_f[r] = finite ? scale * p.scale_log2 : __uint_as_float(0x7fc00000u);
        }
      }
      if (quarter == 0 && lane < C) sh_m[n0 + lane] = kNoMax;
      if (warp == 0) sh_bad[lane] = 0;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQ));
      sync_threads(15, kAll);  // sh_f and sh_bad are other parts' too

      float l[C];
#pragma unroll
      for (int i = 0; i < C; ++i) l[i] = 0.f;

      for (int64_t tile = g.t0; tile < g.t1; ++tile, ++tt) {
        const uint32_t sb = tt & 1u, ph = (tt >> 1) & 1u;
        const int64_t j = tile * kTreeTile + key;
        // Is the key there, and what are its scales?
        const int page = j < g.s.keys ? page_of(p.c, table, p.max_pages, j) : -1;
        float ks = p.scale_log2, lvs = 0.f, inv_vs = 1.f;
        if constexpr (kFp8) {
          float vs = 1.f;
          ks = 0.f;
          if (page >= 0) {
            const int64_t at = (int64_t(page) * p.c.Hkv + g.h) * (slot_mask + 1) + (j & slot_mask);
            ks = p.c.ks[at];
            vs = p.c.vs[at];
            if (vs == 0.f) vs = 7.8886090522101181e-31f;  // 2^-100: the weight stays, the value is as good as none
          }
          lvs = log2f(vs);
          inv_vs = 1.f / vs;
        }
        const bool ok_s = ok && warp_wait(bar(kBarS + int(sb)), ph, budget, status);
        float x[C];
        if (ok_s) {
          umma::fence_after_sync();
          tmem_ld<C>(lane_addr + sb * kN, x);
          umma::tmem_wait_ld();
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarSFree + int(sb)));
        } else {
#pragma unroll
          for (int i = 0; i < C; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < C; i += 4) {
          if constexpr (kFp8) {
            const float4 f = *reinterpret_cast<const float4*>(sh_f + n0 + i);
            x[i] = fmaf(x[i], ks * f.x, lvs);
            x[i + 1] = fmaf(x[i + 1], ks * f.y, lvs);
            x[i + 2] = fmaf(x[i + 2], ks * f.z, lvs);
            x[i + 3] = fmaf(x[i + 3], ks * f.w, lvs);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] *= ks;
          }
        }
        // Keys that are not there, and drafted tokens that a row does not see.
        const bool drafted = page >= 0 && j >= g.s.ctx;
        if (__any_sync(0xffffffffu, page < 0 || drafted)) {
          const int u = int(j - g.s.ctx);
#pragma unroll
          for (int i = 0; i < C; ++i) {
            const int t = (row0 + n0 + i) >> g_shift;
            if (page < 0 || (drafted && t < g.s.drafted && !tree_sees(p, g.b, t, u))) x[i] = -INFINITY;
          }
        }
        bool raise = false;
#pragma unroll
        for (int i = 0; i < C; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(sh_m + n0 + i);
          raise = raise || x[i] > m.x + F::kSlack || x[i + 1] > m.y + F::kSlack || x[i + 2] > m.z + F::kSlack ||
                  x[i + 3] > m.w + F::kSlack;
        }
        // Values that some row must not see: elements that are not finite would reach it as 0 x
        // infinity.  They are cleared in the tile, and added at the end for the rows that see them.
        const bool scrub = p.T > 1 && (tile + 1) * kTreeTile > g.s.ctx;
        if (any_thread(part_bar, 128, raise || scrub || !ok_s)) {
          // O holds tiles up to the last one: complete before it is rescaled, and before the
          // exchange takes P's place.
          bool fine = ok_s;
          if (tt > 0)
            fine = warp_wait(bar(kBarPV + int((tt - 1) & 1u)), ((tt - 1) >> 1) & 1u, budget, status) && fine;
          bool zero_row = false;
          if (kFp8 || scrub) {  // a look at the tile's values
            const uint32_t v_item = tt * F::kItems + F::kItems / 2;
#pragma unroll
            for (int i = 0; i < F::kItems / 2; ++i)
              fine = warp_wait(bar(kBarFull + int((v_item + i) % F::kSlots)), ((v_item + i) / F::kSlots) & 1u, budget,
                               status) &&
                     fine;
            uint32_t any = 0, bad = 0;
            if (fine) {
#pragma unroll 1
              for (int c = 0; c < 8 * F::kItems; ++c) {  // 16-byte units of the row, in any order
                const uint32_t a = sRing + ((v_item + uint32_t(c >> 4)) % F::kSlots) * uint32_t(kSlotBytes) +
                                   uint32_t((c >> 3) & 1) * kChunk + uint32_t(key) * 128u + uint32_t(((c ^ key) & 7) << 4);
                const uint4 v = lds16(a);
                uint32_t w[4] = {v.x, v.y, v.z, v.w}, hit = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  any |= w[k] & (kFp8 ? 0x7f7f7f7fu : 0u);
                  const uint32_t m = kFp8 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu)  // e4m3 has NaN alone
                                          : __vcmpeq2(w[k] & 0x7f807f80u, 0x7f807f80u);
                  hit |= m;
                  w[k] &= ~m;
                }
                if (scrub && drafted && hit) {
                  bad = 1;
                  if (part == 0) sts16(a, make_uint4(w[0], w[1], w[2], w[3]));  // for all parts
                }
              }
            }
            // A row of zeros puts nothing into O: its scale must not set the maximum.
            zero_row = kFp8 && any == 0;
            if (part == 0 && bad) {
              const int u = int(j - g.s.ctx);
              atomicOr(&sh_bad[u >> 5], 1u << (u & 31));
            }
            fence_proxy_async_smem();
          }
#pragma unroll
          for (int c0 = 0; c0 < C; c0 += 16) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = zero_row ? -INFINITY : x[c0 + i];
            const float mx = lanes_reduce<16, true>(y);  // lane l: row c0 + l / 2
            const float v = __shfl_sync(0xffffffffu, mx, (2 * lane) & 31);
            if ((lane & 16) == c0) put(v);  // lane n of the quarter: row n (only lanes below C have one)
          }
          if (any_thread(part_bar, 128, !fine)) {
            ok = false;
            break;
          }
          umma::fence_after_sync();
#pragma unroll
          for (int c0 = 0; c0 < C; c0 += 16) {
            float alpha[16];
            bool any = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int n = c0 + i;
              const float top = fmaxf(fmaxf(get(0, n), get(1, n)), fmaxf(get(2, n), get(3, n)));
              const float m = sh_m[n0 + n];
              const bool up = top > m + F::kSlack;
              alpha[i] = up ? ex2(m - top) : 1.f;
              any = any || up;
              l[n] *= alpha[i];
            }
            if (any && tile > g.t0) {  // the same in all threads of the part
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                float o[16];
                const uint32_t a = lane_addr + uint32_t((2 + half) * kN + c0);
                umma::tmem_ld16(a, o);
                umma::tmem_wait_ld();
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * alpha[i]);
                umma::tmem_st16u(a, w);
              }
              umma::tmem_wait_st();
            }
          }
          float top = 0.f;
          if (lane < C) top = fmaxf(fmaxf(get(0, lane), get(1, lane)), fmaxf(get(2, lane), get(3, lane)));
          sync_threads(part_bar, 128);  // all have read the old maxima and the exchange
          if (quarter == 0 && lane < C && top > sh_m[n0 + lane] + F::kSlack) sh_m[n0 + lane] = top;
          sync_threads(part_bar, 128);
        }
        // P and the row sums.
        uint32_t hi[kFp8 ? C / 4 : C / 2];
        uint32_t lo[kFp8 ? C / 4 : 1];
        (void)lo;
#pragma unroll
        for (int i = 0; i < C; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(sh_m + n0 + i);
          float e[4] = {ex2(x[i] - m.x), ex2(x[i + 1] - m.y), ex2(x[i + 2] - m.z), ex2(x[i + 3] - m.w)};
          if constexpr (kFp8) {
            float h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              l[i + k] = fmaf(e[k], inv_vs, l[i + k]);
              e[k] *= 64.f;
              h[k] = __uint_as_float(__float_as_uint(e[k]) & 0xfff00000u);  // three mantissa bits
              e[k] -= h[k];
            }
            hi[i / 4] = e4m3_encode4(h);
            lo[i / 4] = e4m3_encode4(e);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) l[i + k] += e[k];
            hi[i / 2] = pack_bf16x2(e[0], e[1]);
            hi[i / 2 + 1] = pack_bf16x2(e[2], e[3]);
          }
        }
        // P's last reader is the product of the tile before.
        if (tt > 0) ok = warp_wait(bar(kBarPV + int((tt - 1) & 1u)), ((tt - 1) >> 1) & 1u, budget, status) && ok;
#pragma unroll
        for (int i = 0; i < (kFp8 ? C / 16 : C / 8); ++i) {
          const uint32_t a = p_unit(key, i);
          sts16(a, make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]));
          if constexpr (kFp8) sts16(a + kChunk, make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]));
        }
        fence_proxy_async_smem();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(bar(kBarP + int(sb)));
      }
      // ------------------------------------------------------------ the segment's result
      const uint32_t last = tt - 1;
      if (ok) ok = warp_wait(bar(kBarPV + int(last & 1u)), (last >> 1) & 1u, budget, status);
      umma::fence_after_sync();
      ok = !any_thread(15, kAll, !ok);
      if (ok) {
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += 16) {
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = l[c0 + i];
          const float sum = lanes_reduce<16, false>(y);
          const float v = __shfl_sync(0xffffffffu, sum, (2 * lane) & 31);
          if ((lane & 16) == c0) put(v);
        }
        sync_threads(part_bar, 128);
        const bool whole = g.whole();
        const int64_t part_at = ((int64_t(worker) * 2 + g.slot()) * p.row_tiles + rt) * kN;
        const int64_t head_row = (int64_t(g.b) * p.c.Hkv + g.h) * p.G;
        uint32_t bad = 0;
        for (int i = 0; i < 32; ++i) bad |= sh_bad[i];
#pragma unroll 1
        for (int n = 0; n < C; ++n) {
          const int row = row0 + n0 + n, t = row >> g_shift;
          if (row >= rows_all) break;
          const float sum = (get(0, n) + get(1, n)) + (get(2, n) + get(3, n));
          const bool none = t >= g.s.drafted || sum == 0.f;
          const float inv = none ? 0.f : (kFp8 ? 0.015625f : 1.f) / sum;
          const int64_t out_row = (head_row + (row & (p.G - 1))) * p.T + t;
          if (key == 0) {
            const float lse = none ? -INFINITY : (sh_m[n0 + n] + log2f(sum)) * kLn2;
            if (whole)
              p.lse[out_row] = lse;
            else
              p.lse_part[part_at + n0 + n] = lse;
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                         : "=r"(w)
                         : "r"(lane_addr + uint32_t((2 + half) * kN + n)));
            umma::tmem_wait_ld();
            float v = none ? 0.f : __uint_as_float(w) * inv;
            const int d = half * 128 + key;
            if (bad && !none) {  // values that were cleared, for the rows that see them
#pragma unroll 1
              for (int u = 0; u < g.s.drafted; ++u) {
                if (!((sh_bad[u >> 5] >> (u & 31)) & 1u) || !tree_sees(p, g.b, t, u)) continue;
                const int64_t jb = g.s.ctx + u;
                const int64_t at = table[jb >> p.c.page_shift] * p.c.sp + g.h * p.c.sh + (jb & slot_mask) * p.c.st + d;
                if constexpr (kFp8) {
                  if ((uint8_t(p.c.v[at]) & 0x7f) == 0x7f) v = __uint_as_float(0x7fc00000u);
                } else {
                  const float y = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.c.v)[at]);
                  if (!(fabsf(y) < INFINITY)) v += y;
                }
              }
            }
            if (!whole)
              p.o_part[(part_at + n0 + n) * kHeadDim + d] = v;
            else if (p.out_bf16)
              static_cast<__nv_bfloat16*>(p.out)[out_row * kHeadDim + d] = __float2bfloat16_rn(v);
            else
              static_cast<float*>(p.out)[out_row * kHeadDim + d] = v;
          }
        }
        umma::fence_before_sync();
      }
      // The next segment's Q, factors and maxima take this one's place: all parts are done.
      ok = !any_thread(15, kAll, !ok);
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  if (warp == F::kWarps - 1) {
    umma::fence_after_sync();
    umma::tmem_dealloc(tmem, F::kTmem);
  }
}

template <int kN, bool kFp8>
int launch_n(const TreeParams& p, cudaStream_t stream) {
  using F = Cfg<kN, kFp8>;
  if (cudaFuncSetAttribute(tree_tc_kernel<kN, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem) !=
      cudaSuccess)
    return GQA_ERR_LAUNCH;
  tree_tc_kernel<kN, kFp8><<<unsigned(p.workers) * unsigned(p.row_tiles), F::kThreads, F::kSmem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

template <bool kFp8>
int launch_type(const TreeParams& p, int rows, cudaStream_t stream) {
  switch (rows) {
    case 16: return launch_n<16, kFp8>(p, stream);
    case 32: return launch_n<32, kFp8>(p, stream);
    case 64: return launch_n<64, kFp8>(p, stream);
    default: return launch_n<128, kFp8>(p, stream);
  }
}

}  // namespace

int launch_tree_tc(const TreeParams& p, int rows, cudaStream_t stream) {
  return p.c.dtype == GQA_E4M3 ? launch_type<true>(p, rows, stream) : launch_type<false>(p, rows, stream);
}

}  // namespace gqa
