// Attention of drafted tokens over the paged cache on the 5th-generation tensor cores
// (tcgen05 / TMEM), sm_100a: bf16 queries, bf16 or e4m3 pages.
//
// Few query rows meet many keys, so the keys take the long side of every product: a tile
// of 128 keys is the M of S^T = K Q^T (N = the query rows, 16 .. 64), and the 256 columns
// of the values, in two halves, are the M of O^T += V^T P^T.  With the rows as M, 4 rows
// would cost what 128 do (tree_rows.cu, for more rows).  TMEM, per CTA: two S^T buffers (lane = key) and the
// two halves of O^T (lane = column of the output), N columns each, or as many times that as there are
// pieces side by side.
//
// e4m3 pages are multiplied as they are (kind::f8f6f4, exact products in fp32): the query
// is scaled by a power of two so that its largest element lies in (224, 448] and taken
// apart into two e4m3 pieces, q = hi + lo, off by at most 2^-10 of that scale; a probability into
// three e5m2 pieces (tree_tc.cuh), which keep the bits of a bf16 one over 20 powers of two.  The
// pieces lie side by side in N and their products are added afterwards; of 64 rows there is room
// for two beside one another, and the third is multiplied by itself into the first one's place.
// The scales of a key go into its scores, those of a value into its probability, before
// that is rounded.
//
// Softmax: one thread per key and up to 32 rows; the running maximum m of a row is raised
// only when a score passes it by kSlack (in powers of two), so most tiles need no
// reduction over the keys and no rescaling of O.  P = 2^(x - m) goes to shared memory as
// the B operand; the row sum stays with the threads, in fp32, until the end.  Over bf16 pages P is
// two bf16 pieces up to 32 rows, off by 2^-15 of itself, which memory hides (one token, 60,926
// keys: 48.4 us with two, 48.0 with one); of more rows it is rounded to one, off by 2^-8 (with two,
// 64 rows took 3 % longer, and 128 would double the product that bounds them).  For e4m3, x
// includes log2 of the value's scale, so that m follows the largest product p v rather
// than the largest p, and P is stored as 2^11 P <= 2^15.
//
// Warps: 4 softmax warps per 32 (or 16) rows, a producer each for keys and values (TMA,
// through the page table, into rings of 16 KiB slots), and two warps that issue the products.
//
// One token of 4 heads, 60,926 bf16 keys (249 MB): 48 us, 38 for the bytes alone; the kernel
// itself 47 of which 4.5 pass before the first scores and 3.5 behind the last.  32 sequences of up
// to 8,192 e4m3 keys (313 MB): 70 us against 48; a tile takes 2,100 cycles where memory allows it
// (the softmax's 128 threads), and each head begun costs 4 us (Q, an empty pipeline, the output).
#include "tree_tc.cuh"

namespace gqa {
namespace {

template <int kN, bool kFp8>
struct Cfg {
  static constexpr int kCols = kN < 32 ? kN : 32;  // rows of a softmax thread
  static constexpr int kParts = kN / kCols;
  static constexpr int kSoftWarps = 4 * kParts;
  static constexpr int kNN = kFp8 ? 2 * kN : kN;  // N of S's products: the query's pieces lie side by side
  static constexpr int kPieces = kFp8 ? 3 : kN > 32 ? 1 : 2;   // of a probability,
  static constexpr int kSide = kFp8 && kN > 32 ? 2 : kPieces;  // of them side by side: a row of P has 128 bytes,
  static constexpr int kNO = kSide * kN;                       // tensor memory 512 columns.  N of O's products
  static constexpr int kQBytes = kN * 512;                     // bf16, or two e4m3 pieces
  static constexpr int kPBytes = kSide < kPieces ? 32768 : 16384;  // [128 keys][128 bytes], a third piece behind them
  static constexpr int kKSlots = kN > 32 ? 5 : 6, kVSlots = kSide < kPieces ? 5 : 6;  // what shared memory has room for
  static constexpr int kIssuer = kSoftWarps + 2;  // the S issuer's warp, after the producers; then the O issuer's
  static constexpr int kWarps = kIssuer + 2;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffK = kOffP + kPBytes;
  static constexpr int kOffV = kOffK + kKSlots * kSlotBytes;
  static constexpr int kOffBar = kOffV + kVSlots * kSlotBytes;
  static constexpr int kOffM = kOffBar + 288;     // [kN] maxima
  static constexpr int kOffF = kOffM + kN * 4;    // [kN] factor of a row's scores (e4m3 pages)
  static constexpr int kOffBad = kOffF + kN * 4;  // 32 words: drafted tokens with a value that is not finite
  static constexpr int kSmem = kOffBad + 128;
  static constexpr float kSlack = kFp8 ? 4.f : 8.f;
  static constexpr uint32_t kOffO = 2 * kNN;  // O's columns, behind two buffers of S
  static constexpr uint32_t kTmemCols = kOffO + 2 * kNO;
  static constexpr uint32_t kTmem = kTmemCols <= 64 ? 64 : kTmemCols <= 128 ? 128 : kTmemCols <= 256 ? 256 : 512;
  static_assert(kTmemCols <= 512, "tensor memory");
  static_assert(kSmem <= 232448 - 1024, "shared memory per block");
};

// Barriers: S^T, its release, P and O per parity of the tile; the rings' slots.
enum {
  kBarQ = 0,
  kBarS = 1,
  kBarSFree = 3,
  kBarP = 5,
  kBarPV = 7,
  kBarDrain = 9,
  kBarKFull = 10,
  kBarKEmpty = 16,
  kBarVFull = 22,
  kBarVEmpty = 28
};

// Sum or maximum over the 32 lanes of each of 16 values: lane l ends with value l / 2.  A
// lane sends the half that it does not keep.
template <bool kMax>
__device__ __forceinline__ float lanes_reduce(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 8, off = 16; half >= 1; half >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < half) {
        const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
        const float got = __shfl_xor_sync(0xffffffffu, send, off);
        v[i] = kMax ? fmaxf(keep, got) : keep + got;
      }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
  return kMax ? fmaxf(v[0], got) : v[0] + got;
}

// Four consecutive fp32 columns of this thread's TMEM lane (warp-collective).
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}

template <int kN, bool kFp8>
__global__ void __launch_bounds__(Cfg<kN, kFp8>::kThreads, 1) tree_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ TreeParams p) {
  using F = Cfg<kN, kFp8>;
  using I = Items<kFp8>;
  constexpr int C = F::kCols;
  extern __shared__ __align__(1024) char smem_raw[];
  __shared__ TreeCursor start;
  __shared__ uint32_t tmem_slot;
  const uint32_t sbase = smem_u32(smem_raw);
  const bool misaligned = (sbase & 1023u) != 0;  // the swizzle needs it; never expected to fail
  const uint32_t sQ = sbase + F::kOffQ, sP = sbase + F::kOffP, sK = sbase + F::kOffK, sV = sbase + F::kOffV;
  auto bar = [&](int i) { return sbase + F::kOffBar + 8u * uint32_t(i); };
  float* sh_m = reinterpret_cast<float*>(smem_raw + F::kOffM);
  float* sh_f = reinterpret_cast<float*>(smem_raw + F::kOffF);
  uint32_t* sh_bad = reinterpret_cast<uint32_t*>(smem_raw + F::kOffBad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  const int64_t budget = p.wait_budget_ns;
  int32_t* status = p.c.status;

  wait_for_grid();  // what comes before in the stream may still have been running
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
      mbar_init(bar(kBarDrain), 2);
      for (int i = 0; i < F::kKSlots; ++i) {
        mbar_init(bar(kBarKFull + i), 1);
        mbar_init(bar(kBarKEmpty + i), 1);
      }
      for (int i = 0; i < F::kVSlots; ++i) {
        mbar_init(bar(kBarVFull + i), 1);
        mbar_init(bar(kBarVEmpty + i), 1);
      }
      fence_barrier_init();
      if (misaligned) set_status(status, GQA_ERR_LAUNCH);
    }
  }
  if (warp == F::kIssuer) umma::tmem_alloc(smem_u32(&tmem_slot), F::kTmem);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  launch_dependents();
  TreeCursor cur = start;
  TreeSegment g;

  if (misaligned) {
    // no role
  } else if (warp == F::kSoftWarps) {
    Feed<kFp8, false, F::kKSlots> feed;
    NoFeed none;
    feed.begin(p, cur, &map_k, sK, bar(kBarKFull), bar(kBarKEmpty));
    produce(p, feed, none);
  } else if (warp == F::kSoftWarps + 1) {
    Feed<kFp8, true, F::kVSlots> feed;
    NoFeed none;
    feed.begin(p, cur, &map_v, sV, bar(kBarVFull), bar(kBarVEmpty));
    produce(p, feed, none);
  } else if (warp >= F::kIssuer) {
    // ---------------------------------------------------------------- MMA issuers
    // One warp issues every S^T = K Q^T, another every O^T += V^T P^T, so that neither
    // waits for the other's tiles to arrive.
    {
      const bool is_s = warp == F::kIssuer;
      constexpr uint32_t id_s = idesc<kFp8>(F::kNN, 0, 0), id_o = idesc<kFp8>(F::kNO, 1, 1, false, kFp8),
                         id_third = idesc<kFp8>(kN, 1, 1, false, kFp8);
      (void)id_third;
      const uint64_t dq = umma::smem_desc(sQ, 16, 1024), dp = umma::smem_desc(sP, 16384, 1024);
      const uint32_t high = uint32_t(dq >> 32);
      uint32_t tt = 0, segs = 0;  // tiles issued
      bool ok = true;
      while (ok && tree_next(p, cur, &g)) {
        if (is_s && !(ok = warp_wait(bar(kBarQ), segs & 1u, budget, status))) break;
        ++segs;
        for (int tile = g.t0; ok && tile < g.t1; ++tile, ++tt) {
          const uint32_t b = tt & 1u, ph = (tt >> 1) & 1u;
          const uint32_t slots = is_s ? F::kKSlots : F::kVSlots;
          const uint32_t full = bar(is_s ? kBarKFull : kBarVFull), empty = bar(is_s ? kBarKEmpty : kBarVEmpty);
          // What has been loaded is waited for first: P, or the last reader of S, comes after it, and
          // from then on only the products stand between it and the next one.
#pragma unroll 1
          for (uint32_t i = 0; ok && i < I::kTile; ++i) {
            const uint32_t item = I::kTile * tt + i;
            ok = warp_wait(full + 8u * (item % slots), (item / slots) & 1u, budget, status);
          }
          // The softmax has read S(t - 2), or written P(t).
          if (is_s)
            ok = ok && (tt < 2 || warp_wait(bar(kBarSFree + int(b)), ph ^ 1u, budget, status));
          else
            ok = ok && warp_wait(bar(kBarP + int(b)), ph, budget, status);
          if (!ok) break;
          umma::fence_after_sync();
          if (elect_lane()) {
#pragma unroll
            for (uint32_t i = 0; i < I::kTile; ++i) {
              const uint32_t item = I::kTile * tt + i, slot = item % slots;
              const uint32_t base = (is_s ? sK : sV) + slot * uint32_t(kSlotBytes);
              if (is_s) {
                // column block i of the keys against that of Q: four steps of 32 bytes
                const uint64_t dk = umma::smem_desc(base, 16, 1024);
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
                  mma<kFp8>(tmem + b * F::kNN, desc_low(dk, k * 32u), desc_low(dq, i * (F::kNN * 128u) + k * 32u), high, id_s,
                            (i | k) != 0);
              } else {
                // the slot's keys, in two steps, for both halves of the values' columns
#pragma unroll
                for (uint32_t half = 0; half < 2; ++half) {
                  const uint64_t dv = umma::smem_desc(base + half * (kSlotBytes / 2), I::kVBlock, 1024);
#pragma unroll
                  for (uint32_t k = 0; k < 2; ++k) {
                    const uint32_t o = tmem + F::kOffO + half * F::kNO, v = desc_low(dv, k * I::kStep);
                    mma<kFp8>(o, v, desc_low(dp, (2 * i + k) * I::kStep), high, id_o, tile > g.t0 || (i | k) != 0);
                    if constexpr (F::kSide < F::kPieces)
                      mma<kFp8>(o, v, desc_low(dp, 16384u + (2 * i + k) * I::kStep), high, id_third, true);
                  }
                }
              }
              umma::commit(empty + 8u * slot);
            }
            umma::commit(bar((is_s ? kBarS : kBarPV) + int(b)));
          }
          __syncwarp();
        }
      }
      // Every product complete before TMEM is released.
      if (elect_lane()) {
        if (tt > 0)
          umma::commit(bar(kBarDrain));
        else
          mbar_arrive(bar(kBarDrain));
      }
      __syncwarp();
      warp_wait(bar(kBarDrain), 0, budget, status);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    constexpr uint32_t kAll = 32 * F::kSoftWarps;  // threads of barrier 15
    constexpr float kLogSum = kFp8 ? kLogSumScale : 0.f, kOut = kFp8 ? kSumScale / kPScale : 1.f;
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t part_bar = 1u + uint32_t(part);
    const int n0 = part * C;              // first row (column of S^T and O^T) of this thread
    const int key = quarter * 32 + lane;  // TMEM lane: key of the tile, column of O's half
    const uint32_t lane_addr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(n0);
    const int g_shift = __ffs(p.G) - 1;
    const int rows_all = p.T * p.G;
    const int row0 = rt * kN;  // this CTA's first row among the T G of a head
    const uint32_t slot_mask = (1u << p.c.page_shift) - 1;
    const bool hides = p.T > 1 || p.mask;  // a drafted token from some row: one token without a mask sees itself
    // The 16-byte unit `i` of key k's P: eight or sixteen rows from n0 on, of a piece.
    auto p_unit = [&](int k, int i, int piece) {
      const bool behind = piece >= F::kSide;
      const int un = (n0 + (behind ? 0 : piece) * kN) / (kFp8 ? 16 : 8) + i;
      return sP + (behind ? 16384u : 0u) + uint32_t(k) * 128u + uint32_t((un ^ (k & 7)) << 4);
    };
    // The quarters' exchange of one value for each of sixteen rows lies in the thread's own
    // columns of P, which no product reads then: row c0 + n's from quarter q is with lane n.
    auto put = [&](int c0, float v) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(p_unit(key, c0 / (kFp8 ? 16 : 8), 0)), "f"(v) : "memory");
    };
    auto get = [&](int c0, int q, int n) {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p_unit(q * 32 + n, c0 / (kFp8 ? 16 : 8), 0)) : "memory");
      return v;
    };
    uint32_t tt = 0;  // tiles so far
    bool ok = true;

    // Q's rows of this warp, loaded ahead of their segment.
    constexpr int kQRows = kN / F::kSoftWarps;
    uint4 u[kQRows];
    auto load_q = [&]() {
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        const int n = row0 + warp + i * F::kSoftWarps, t = n >> g_shift;
        u[i] = make_uint4(0, 0, 0, 0);
        if (t < g.s.drafted)
          u[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q.p) + g.b * p.q.sb +
                                                 int64_t(g.h * p.G + (n & (p.G - 1))) * p.q.sh + t * p.q.sl + 8 * lane);
      }
    };
    bool more = tree_next(p, cur, &g);
    if (more) load_q();

    while (ok && more) {
      const int32_t* table = p.table + int64_t(g.b) * p.max_pages;
      // (The code of one row: it is run from a cold instruction cache.)
#pragma unroll 1
      for (int r = warp; r < kN; r += F::kSoftWarps) {
        if constexpr (!kFp8) {
          sts16(sQ + uint32_t(lane >> 3) * (kN * 128u) + uint32_t(r) * 128u + uint32_t(((lane & 7) ^ (r & 7)) << 4), u[0]);
        } else {
          const float f = put_query<kN, true>(u[0], sQ, r);
          if (lane == 0) sh_f[r] = f * p.scale_log2;
        }
#pragma unroll
        for (int i = 1; i < kQRows; ++i) u[i - 1] = u[i];
      }
      if (quarter == 0 && lane < C) sh_m[n0 + lane] = 0.f;
      if (warp == 0) sh_bad[lane] = 0;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQ));
      sync_threads(15, kAll);  // sh_f and sh_bad are other parts' too

      float l[C];
#pragma unroll
      for (int i = 0; i < C; ++i) l[i] = 0.f;

      // The key's page table entry two tiles ahead and its scales one tile ahead of their use:
      // neither load, the second through the first, is waited for.
      auto entry_at = [&](int tile) {
        const uint32_t j = uint32_t(tile) * kTreeTile + key;
        return tile < g.t1 && j < g.s.keys ? page_entry(p.c, table, p.max_pages, j) : -1;
      };
      auto checked = [&](int tile, int entry) {
        return tile < g.t1 && uint32_t(tile) * kTreeTile + key < g.s.keys ? page_checked(p.c, entry) : -1;
      };
      auto scales_at = [&](int tile, int page, float* ks, float* vs) {
        if (kFp8 && page >= 0) {
          const int64_t at =
              (int64_t(page) * p.c.Hkv + g.h) * (slot_mask + 1) + ((uint32_t(tile) * kTreeTile + key) & slot_mask);
          *ks = p.c.ks[at];
          *vs = p.c.vs[at];
        }
      };
      int page = checked(g.t0, entry_at(g.t0)), entry_next = entry_at(g.t0 + 1);
      float ks_next = 0.f, vs_next = 1.f;
      scales_at(g.t0, page, &ks_next, &vs_next);
      uint32_t fresh = (1u << (C / 16)) - 1;  // sixteens of rows, some of which have seen no key yet
      uint32_t has = 0;                       // lane n: whether row 16 i + n has, bit i

#pragma unroll 1
      for (int tile = g.t0; tile < g.t1; ++tile, ++tt) {
        const uint32_t sb = tt & 1u, ph = (tt >> 1) & 1u;
        const uint32_t j = uint32_t(tile) * kTreeTile + key;
        // The product of the tile before: P's last reader, and what O holds.
        auto last_product = [&]() {
          return tt == 0 || warp_wait(bar(kBarPV + int((tt - 1) & 1u)), ((tt - 1) >> 1) & 1u, budget, status);
        };
        // The values of this warp's keys are in their slot.  The product before is over first, so
        // that the barrier stands at no earlier use of the slot.
        const uint32_t v_item = I::kTile * tt + uint32_t(quarter * 32 / I::kVKeys);
        auto values_there = [&]() {
          return last_product() &&
                 warp_wait(bar(kBarVFull + int(v_item % F::kVSlots)), (v_item / F::kVSlots) & 1u, budget, status);
        };
        auto value_unit = [&](int c) {  // 16-byte unit c of the key's values, in any order
          return sV + (v_item % F::kVSlots) * uint32_t(kSlotBytes) + uint32_t(c >> 3) * I::kVBlock +
                 uint32_t(key % I::kVKeys) * 128u + uint32_t(((c ^ key) & 7) << 4);
        };
        const float ks = kFp8 ? (page < 0 ? 0.f : ks_next) : p.scale_log2;
        const float vs = kFp8 && page >= 0 ? vs_next : 1.f;
        float lvs = 0.f, inv_vs = 1.f, store = 1.f;
        (void)store;
        const int page_now = page;
        page = checked(tile + 1, entry_next);
        scales_at(tile + 1, page, &ks_next, &vs_next);
        entry_next = entry_at(tile + 2);
        // Which of this thread's rows see the key: all, unless it is not there or is drafted.
        const bool drafted = page_now >= 0 && j >= g.s.ctx;
        uint32_t vis = page_now >= 0 ? 0xffffffffu : 0u;
        if (drafted) {
          vis = 0;
          const int t0 = (row0 + n0) >> g_shift;
#pragma unroll 4
          for (int i = 0; i < C >> g_shift; ++i)
            // (rows past the last drafted token are cleared at the end)
            if (t0 + i >= g.s.drafted || tree_sees(p, g.b, t0 + i, int(j - g.s.ctx)))
              vis |= ((1u << p.G) - 1u) << (i * p.G);
        }
        const bool masked = __any_sync(0xffffffffu, vis != 0xffffffffu && (C == 32 || (vis & 0xffffu) != 0xffffu));
        bool fine = ok;
        if constexpr (kFp8) {
          // A row of zeros is written with scale 1.
          bool zeros = false;
          if (__any_sync(0xffffffffu, page_now >= 0 && vs == 1.f)) {
            fine = values_there() && fine;
            uint32_t any = 0;
            if (fine && vs == 1.f)
#pragma unroll 4
              for (int c = 0; c < 16; ++c) {
                const uint4 v = lds16(value_unit(c));
                any |= (v.x | v.y | v.z | v.w) & 0x7f7f7f7fu;
              }
            zeros = vs == 1.f && any == 0;
            __syncwarp();
          }
          const ValueScale s(vs, zeros);
          lvs = s.log2, inv_vs = s.inv, store = s.store;
        }
        // Values that take no part reach a row as 0 x what they are, NaN if that is not finite: those
        // of keys that are not there (a page's rest) are cleared in the tile, and those elements of
        // drafted tokens, which some row may not see; they are added at the end for the rows that do.
        if (part == 0 && __any_sync(0xffffffffu, page_now < 0 || (drafted && hides))) {
          fine = values_there() && fine;
          if (fine && (page_now < 0 || (drafted && hides))) {
            uint32_t bad = 0;
#pragma unroll 1
            for (int c = 0; c < (kFp8 ? 16 : 32); ++c) bad |= mend_unit<kFp8>(value_unit(c), page_now < 0);
            const int u = int(j - g.s.ctx);
            if (bad) atomicOr(&sh_bad[u >> 5], 1u << (u & 31));
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        fine = warp_wait(bar(kBarS + int(sb)), ph, budget, status) && fine;
        umma::fence_after_sync();
        bool stop = false;
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += 16) {
          // Scores of the rows n0 + c0 .. + 15 less their maxima so far, in powers of two.  The code is
          // written to be short: a CTA runs it first from a cold instruction cache.
          float x[16];
          umma::tmem_ld16(lane_addr + sb * F::kNN + uint32_t(c0), x);
          if constexpr (kFp8) {
            float y[16];
            umma::tmem_ld16(lane_addr + sb * F::kNN + kN + uint32_t(c0), y);
            umma::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] += y[i];
          } else {
            umma::tmem_wait_ld();
          }
          float top[4];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(sh_m + n0 + c0 + i);
            const float m4[4] = {m.x, m.y, m.z, m.w};
            if constexpr (kFp8) {
              const float4 f = *reinterpret_cast<const float4*>(sh_f + n0 + c0 + i);
              const float f4[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) x[i + k] = fmaf(x[i + k], ks * f4[k], lvs - m4[k]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) x[i + k] = fmaf(x[i + k], ks, -m4[k]);
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!((vis >> (c0 + i + k)) & 1u)) x[i + k] = -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = i == 0 ? x[k] : fmaxf(top[k], x[i + k]);
          }
          const bool raise = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > F::kSlack;
          if (any_thread(part_bar, 128, raise || !fine || ((fresh >> (c0 / 16)) & 1u))) {
            fine = last_product() && fine;
            if (any_thread(part_bar, 128, !fine)) {
              stop = true;
              break;
            }
            umma::fence_after_sync();
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = x[i];
            const float mx = lanes_reduce<true>(y);  // lane l: row c0 + l / 2
            const float v = __shfl_sync(0xffffffffu, mx, (2 * lane) & 31);
            if (lane < 16) put(c0, v);  // lane n of the quarter: row c0 + n
            sync_threads(part_bar, 128);
            float up = -INFINITY;  // the row's largest score, above its maximum so far
            if (lane < 16) up = fmaxf(fmaxf(get(c0, 0, lane), get(c0, 1, lane)), fmaxf(get(c0, 2, lane), get(c0, 3, lane)));
            // The first score a row sees sets its maximum, later ones raise it.
            const bool first = !((has >> (c0 / 16)) & 1u), rise = first ? up > -INFINITY : up > F::kSlack;
            const float delta = rise ? up : 0.f, alpha = rise && !first ? ex2(-up) : 1.f;
            if (rise) has |= 1u << (c0 / 16);
            fresh &= ~(1u << (c0 / 16));
            if (__any_sync(0xffffffffu, lane < 16 && !((has >> (c0 / 16)) & 1u))) fresh |= 1u << (c0 / 16);
            sync_threads(part_bar, 128);  // all have read the old maxima and the exchange
            if (quarter == 0 && rise) sh_m[n0 + c0 + lane] += delta;
            if (__any_sync(0xffffffffu, rise)) {  // the same in the part's four warps
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                x[i] -= __shfl_sync(0xffffffffu, delta, i);
                l[c0 + i] *= __shfl_sync(0xffffffffu, alpha, i);
              }
              if (tile > g.t0) {
#pragma unroll 1
                for (int block = 0; block < 2 * F::kSide; ++block) {  // halves of O, and pieces
                  float o[16];
                  const uint32_t a = lane_addr + F::kOffO + uint32_t((block & 1) * F::kNO + (block >> 1) * kN + c0);
                  umma::tmem_ld16(a, o);
                  umma::tmem_wait_ld();
                  uint32_t w[16];
#pragma unroll
                  for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * __shfl_sync(0xffffffffu, alpha, i));
                  umma::tmem_st16u(a, w);
                }
                umma::tmem_wait_st();
              }
            }
            sync_threads(part_bar, 128);  // the new maxima are there
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = ex2(x[i]);
          if (c0 + 16 == C) {  // the last read of S
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarSFree + int(sb)));
          }
          // The row sums, and P.  A wait that ran out here is agreed upon with the next tile.
          if (c0 == 0) ok = last_product() && ok;
          uint32_t hi[kFp8 ? 4 : 8], mid[4], lo[kFp8 ? 4 : 8];
          (void)mid, (void)lo;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            if constexpr (kFp8) {
              float e[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                l[c0 + i + k] = fmaf(x[i + k], inv_vs, l[c0 + i + k]);
                e[k] = x[i + k] * store;
              }
              e5m2_pieces4(e, hi[i / 4], mid[i / 4], lo[i / 4]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) l[c0 + i + k] += x[i + k];
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                if constexpr (F::kPieces == 1) {
                  hi[(i + k) / 2] = pack_bf16x2(x[i + k], x[i + k + 1]);
                } else {
                  const uint32_t u = __float_as_uint(x[i + k]), v = __float_as_uint(x[i + k + 1]);
                  hi[(i + k) / 2] = __byte_perm(u, v, 0x7632);  // the upper halves: cut to bf16
                  lo[(i + k) / 2] = pack_bf16x2(x[i + k] - __uint_as_float(u & 0xffff0000u),
                                                x[i + k + 1] - __uint_as_float(v & 0xffff0000u));
                }
              }
            }
          }
          if constexpr (kFp8) {
            sts16(p_unit(key, c0 / 16, 0), make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts16(p_unit(key, c0 / 16, 1), make_uint4(mid[0], mid[1], mid[2], mid[3]));
            sts16(p_unit(key, c0 / 16, 2), make_uint4(lo[0], lo[1], lo[2], lo[3]));
          } else {
            sts16(p_unit(key, c0 / 8, 0), make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts16(p_unit(key, c0 / 8 + 1, 0), make_uint4(hi[4], hi[5], hi[6], hi[7]));
            if constexpr (F::kPieces > 1) {
              sts16(p_unit(key, c0 / 8, 1), make_uint4(lo[0], lo[1], lo[2], lo[3]));
              sts16(p_unit(key, c0 / 8 + 1, 1), make_uint4(lo[4], lo[5], lo[6], lo[7]));
            }
          }
        }
        if (stop) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(bar(kBarP + int(sb)));
      }
      // ------------------------------------------------------------ the segment's result
      const uint32_t last = tt - 1;
      const TreeSegment d = g;  // the one that is done; the next one's Q is loaded meanwhile
      more = tree_next(p, cur, &g);
      if (more) load_q();
      if (ok) ok = warp_wait(bar(kBarPV + int(last & 1u)), (last >> 1) & 1u, budget, status);
      umma::fence_after_sync();
      ok = !any_thread(15, kAll, !ok);
      if (ok) {
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += 16) {
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = l[c0 + i];
          const float sum = lanes_reduce<false>(y);
          const float v = __shfl_sync(0xffffffffu, sum, (2 * lane) & 31);
          if (lane < 16) put(c0, v);
        }
        sync_threads(part_bar, 128);
        const bool whole = d.whole();
        const int64_t part_at = ((int64_t(worker) * 2 + d.slot()) * p.row_tiles + rt) * kN;
        const int64_t head_row = (int64_t(d.b) * p.c.Hkv + d.h) * p.G;
        const bool bad = __any_sync(0xffffffffu, sh_bad[lane] != 0);
        // Lane n of every warp: row n's factor.
        const int my_row = row0 + n0 + lane, my_t = my_row >> g_shift;
        float inv = 0.f;
        if (lane < C && my_row < rows_all) {
          const int c0 = lane & 16, n = lane & 15;
          const float sum = (get(c0, 0, n) + get(c0, 1, n)) + (get(c0, 2, n) + get(c0, 3, n));
          const bool none = my_t >= d.s.drafted || sum == 0.f;
          inv = none ? 0.f : 1.f / sum;
          if (quarter == 0) {
            const float lse = none ? -INFINITY : (sh_m[n0 + lane] + log2f(sum) - kLogSum) * kLn2;
            if (whole)
              p.lse[(head_row + (my_row & (p.G - 1))) * p.T + my_t] = lse;
            else
              p.lse_part[part_at + n0 + lane] = lse;
          }
        }
#pragma unroll 1
        for (int c0 = 0; c0 < C; c0 += 4) {
          if (row0 + n0 + c0 >= rows_all) break;
          float o[2][4];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t a = lane_addr + F::kOffO + uint32_t(half * F::kNO + c0);
            tmem_ld4(a, o[half]);
            if constexpr (F::kSide > 1) {  // the pieces worth least first
              float y[F::kSide - 1][4];
#pragma unroll
              for (int piece = 1; piece < F::kSide; ++piece) tmem_ld4(a + piece * kN, y[piece - 1]);
              umma::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[half][i] += F::kSide > 2 ? y[0][i] + y[F::kSide - 2][i] : y[0][i];
            }
          }
          umma::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = row0 + n0 + c0 + i, t = row >> g_shift;
            const float f = __shfl_sync(0xffffffffu, inv, c0 + i);
            const int64_t at = (whole ? (head_row + (row & (p.G - 1))) * p.T + t : part_at + n0 + c0 + i) * kHeadDim + key;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float v = f == 0.f ? 0.f : o[half][i] * kOut * f;  // in this order: a sum may be near either end of fp32
              if (bad && f != 0.f) v += hidden_values<kFp8>(p, d, table, sh_bad, t, half * 128 + key);
              if (row >= rows_all) continue;
              if (whole)
                static_cast<__nv_bfloat16*>(p.out)[at + half * 128] = __float2bfloat16_rn(v);
              else
                p.o_part[at + half * 128] = v;
            }
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
  if (warp == F::kIssuer) {
    umma::fence_after_sync();
    umma::tmem_dealloc(tmem, F::kTmem);
  }
}

template <int kN, bool kFp8>
int launch_n(const TreeParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  using F = Cfg<kN, kFp8>;
  if (!allow_smem<tree_tc_kernel<kN, kFp8>>(F::kSmem)) return GQA_ERR_LAUNCH;
  return launch_programmatic(tree_tc_kernel<kN, kFp8>, unsigned(p.workers) * unsigned(p.row_tiles), F::kThreads, F::kSmem,
                             stream, mk, mv, p);
}

template <bool kFp8>
int launch_type(const TreeParams& p, int rows, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!encode_pages(&mk, p.c, false) || !encode_pages(&mv, p.c, true)) return GQA_ERR_LAUNCH;
  switch (rows) {
    case 16: return launch_n<16, kFp8>(p, mk, mv, stream);
    case 32: return launch_n<32, kFp8>(p, mk, mv, stream);
    default: return launch_n<64, kFp8>(p, mk, mv, stream);
  }
}

}  // namespace

int launch_tree_tc(const TreeParams& p, int rows, cudaStream_t stream) {
  if (rows > 64) return launch_tree_rows(p, stream);
  return p.c.dtype == GQA_E4M3 ? launch_type<true>(p, rows, stream) : launch_type<false>(p, rows, stream);
}

}  // namespace gqa
