// Attention of drafted tokens over the paged cache on the tensor cores with the query rows
// as M, sm_100a: tiles of 128 rows (T G rows of a key/value head, above 64), bf16 queries,
// bf16 or e4m3 pages.  With this many rows the keys as M (tree_tc.cu) would cost more: its
// products take both operands from shared memory, one of them transposed (a 128 x 128 x 16
// step measured 140 cycles against 97 for S and 136 for twice the work of O here).
//
// S = Q K^T (M = rows, N = 128 keys) and O += P V (P in TMEM, N = 256 columns).  TMEM: O in
// columns 0 .. 255, two S buffers of 128; P(t) takes the place of the first columns of
// S(t): 64 of bf16 pairs, or 32 for each of three e5m2 pieces.  Softmax: one thread per row and
// 32 keys, so that maxima and sums are the thread's own, joined over four warps through
// shared memory only when a maximum rises.  e4m3 pages, their scales, the pieces of queries
// and probabilities, lazy maxima and values that a mask hides: as in tree_tc.cu.
//
// Warps: 16 for the softmax (lane quarter x 32 keys), two producers (bf16: keys and values; e4m3,
// with half the bytes: one for both, and one that fetches the keys' scales), two issuers.
//
// Pairs (bf16 pages, an even number of row tiles): the CTAs of two row tiles, which sweep the
// same keys, issue products of M = 256 together (cta_group::2), and each loads 64 of a tile's keys
// and half of its values' columns.  A CTA by itself has room for 1.25 tiles of keys and of
// values, and a tile comes 3,500 cycles after its slot is free, so it takes 3,800 cycles a tile;
// the pair takes 2,850.  64 tokens of 4 heads, 4 sequences of
// 30,468 bf16 keys (500 MB, 128 GFLOP): 132 us in short runs, 155 - 160 in long ones, whose
// clock falls (unpaired: 176); 77 for the bytes, as much for the flops.  e4m3 stays
// single: there the softmax is the bound within a tile, 3,700 cycles with two pieces (128 x 128
// exponentials and their conversions; the third costs 2 - 3 %, 77.7 us for 75.3), not the loads.  24
// tokens of 4 heads over 8 e4m3 sequences of up
// to 15,231 keys (159 MB): 72 - 81 us against 24.5; 11 pass before the first softmax, 5 per head begun
// and 4.5 per head written (128 rows of fp32 from every SM at once), 10 in the merge.
#include <cfloat>

#include "tree_tc.cuh"

namespace gqa {
namespace {

constexpr int kRows = 128;
constexpr int kSoftWarps = 16;

template <bool kFp8>
struct RowsCfg {
  static constexpr int kKSlots = kFp8 ? 4 : 5, kVSlots = 5;  // what shared memory has room for
  static constexpr int kIssuer = kSoftWarps + 2;  // 20 warps leave 96 registers a thread, 21 only 80
  static constexpr int kThreads = 32 * (kIssuer + 2);
  static constexpr int kOffQ = 0;  // bf16 [4][128 rows][128 bytes], or e4m3 [2 pieces][2][128 rows][128 bytes]
  static constexpr int kOffK = kRows * 512;
  static constexpr int kOffV = kOffK + kKSlots * kSlotBytes;
  static constexpr int kOffBar = kOffV + kVSlots * kSlotBytes;
  static constexpr int kOffStart = kOffBar + 8 * 34;  // the worker's cursor, the TMEM address
  static constexpr int kOffBad = kOffStart + 48;      // 32 words: drafted tokens with a value that is not finite
  static constexpr int kOffThere = kOffBad + 128;     // [2][4] words: which keys of the tile are there
  static constexpr int kOffRed = kOffThere + 32;      // [4 parts][128 rows] exchange
  static constexpr int kOffF = kOffRed + 4 * kRows * 4;       // [128] factors of the rows' scores (e4m3)
  static constexpr int kOffScale = kOffF + (kFp8 ? 512 : 0);  // [2][4][128]: ks, what vs does (ValueScale) (e4m3)
  static constexpr int kSmem = kOffScale + (kFp8 ? 2 * 4 * 128 * 4 : 0);
  static constexpr float kSlack = kFp8 ? 4.f : 8.f;
  static_assert(kSmem <= 232448 && kOffRed % 16 == 0 && sizeof(TreeCursor) <= 40, "shared memory per block");
};

// Barriers: Q; S, P, O and the keys' scales per parity of the tile; the rings' slots.
enum {
  kRBarQ = 0,
  kRBarS = 1,
  kRBarP = 3,
  kRBarPV = 5,
  kRBarKeys = 7,
  kRBarDrain = 9,
  kRBarKFull = 10,
  kRBarKEmpty = 15,
  kRBarVFull = 20,
  kRBarVEmpty = 25,
  kRBarRelay = 30  // to the odd CTA of a pair, per part: its values are there
};

// Four consecutive 32-bit columns of raw words into this thread's TMEM lane.
__device__ __forceinline__ void tmem_st4u(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// The pair's products, issued by the even CTA: A's rows 0 .. 127 are its own, 128 .. 255 the odd
// one's; B's N lies half in one, half in the other.
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(uint32_t(add)));
}
__device__ __forceinline__ void mma_ts_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(uint32_t(add)));
}

// An arrival in the other CTA (or this one) that publishes shared memory, not only tensor memory.
__device__ __forceinline__ void arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

template <bool kFp8, bool kPair>
__global__ void __launch_bounds__(RowsCfg<kFp8>::kThreads, 1) tree_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ TreeParams p) {
  using F = RowsCfg<kFp8>;
  using I = Items<kFp8>;
  extern __shared__ __align__(1024) char smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  const bool misaligned = (sbase & 1023u) != 0;  // the swizzle needs it; never expected to fail
  const uint32_t sQ = sbase + F::kOffQ, sK = sbase + F::kOffK, sV = sbase + F::kOffV;
  auto bar = [&](int i) { return sbase + F::kOffBar + 8u * uint32_t(i); };
  TreeCursor& start = *reinterpret_cast<TreeCursor*>(smem_raw + F::kOffStart);
  volatile uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem_raw + F::kOffStart + 40);
  uint32_t* sh_bad = reinterpret_cast<uint32_t*>(smem_raw + F::kOffBad);
  uint32_t* sh_there = reinterpret_cast<uint32_t*>(smem_raw + F::kOffThere);
  float* sh_scale = reinterpret_cast<float*>(smem_raw + F::kOffScale);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  const int64_t budget = p.wait_budget_ns;
  static_assert(!kPair || !kFp8);
  constexpr int kTile = kPair ? 2 : I::kTile;      // items of a tile's keys, and of its values
  constexpr int kVKeys = 128 / kTile;              // keys of a value item
  constexpr uint32_t kVBlock = kVKeys * 128u;      // bytes from one of its column blocks to the next
  constexpr int kUnits = kFp8 || kPair ? 16 : 32;  // 16-byte units of a key's values here
  const uint32_t rank = kPair ? cluster_ctarank() : 0;  // 0: the even CTA, which issues the products
  const uint32_t lead_bar = kPair ? mapa_shared(sbase + F::kOffBar, 0) : 0;
  auto lead = [&](int i) { return lead_bar + 8u * uint32_t(i); };
  int32_t* status = p.c.status;

  wait_for_grid();  // what comes before in the stream may still have been running
  if (warp == 0) {
    const TreeCursor c = tree_start(p, worker);
    if (lane == 0) {
      start = c;
      mbar_init(bar(kRBarQ), kPair ? 2 : kSoftWarps);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kRBarS + i), 1);
        mbar_init(bar(kRBarP + i), kPair ? 2 * kSoftWarps : kSoftWarps);
        mbar_init(bar(kRBarPV + i), 1);
        mbar_init(bar(kRBarKeys + i), 1);
      }
      mbar_init(bar(kRBarDrain), 2);
      for (int i = 0; i < 4; ++i) mbar_init(bar(kRBarRelay + i), 1);
      for (int i = 0; i < F::kKSlots; ++i) {
        mbar_init(bar(kRBarKFull + i), 1);
        mbar_init(bar(kRBarKEmpty + i), 1);
      }
      for (int i = 0; i < F::kVSlots; ++i) {
        mbar_init(bar(kRBarVFull + i), 1);
        mbar_init(bar(kRBarVEmpty + i), 1);
      }
      fence_barrier_init();
      if (misaligned) set_status(status, GQA_ERR_LAUNCH);
    }
  }
  if (warp == F::kIssuer) {
    if constexpr (kPair)
      umma::tmem_alloc_2sm(sbase + F::kOffStart + 40, 512);
    else
      umma::tmem_alloc(sbase + F::kOffStart + 40, 512);
  }
  umma::fence_before_sync();
  if constexpr (kPair)
    cluster_sync();
  else
    __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  launch_dependents();
  TreeCursor cur = start;
  TreeSegment g;

  if (misaligned) {
    // no role
  } else if (warp == kSoftWarps) {
    Feed<kFp8, false, F::kKSlots, kPair> k;
    k.rank = int(rank);
    k.begin(p, cur, &map_k, sK, bar(kRBarKFull), bar(kRBarKEmpty));
    if constexpr (kFp8) {
      Feed<kFp8, true, F::kVSlots> v;
      if (k.ready()) k.issue(p);
      v.begin(p, cur, &map_v, sV, bar(kRBarVFull), bar(kRBarVEmpty));
      produce(p, k, v);
    } else {
      NoFeed none;
      produce(p, k, none);
    }
  } else if (!kFp8 && warp == kSoftWarps + 1) {
    Feed<kFp8, true, F::kVSlots, kPair> v;
    NoFeed none;
    v.rank = int(rank);
    v.begin(p, cur, &map_v, sV, bar(kRBarVFull), bar(kRBarVEmpty));
    produce(p, v, none);
  } else if (warp == kSoftWarps + 1) {
    // ---------------------------------------------------------------- keys (e4m3)
    // Lane i looks after keys i, 32 + i, 64 + i and 96 + i of each tile: which are there, and
    // their scales, in two buffers.  Page table entries are loaded two tiles ahead, scales one.
    const uint32_t slot_mask = (1u << p.c.page_shift) - 1;
    uint32_t tt = 0;
    bool ok = true;
    while (ok && tree_next(p, cur, &g)) {
      const int32_t* table = p.table + int64_t(g.b) * p.max_pages;
      int page[4], entry_next[4];
      float ks[4], vs[4];
      auto entries_at = [&](int tile, int (&e)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t j = uint32_t(tile) * kTreeTile + i * 32 + lane;
          e[i] = tile < g.t1 && j < g.s.keys ? page_entry(p.c, table, p.max_pages, j) : -1;
        }
      };
      auto checked = [&](int tile, const int (&e)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          page[i] =
              tile < g.t1 && uint32_t(tile) * kTreeTile + i * 32 + lane < g.s.keys ? page_checked(p.c, e[i]) : -1;
      };
      auto scales_at = [&](int tile) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[i] = 0.f, vs[i] = 1.f;
          if (page[i] >= 0) {
            const int64_t at = (int64_t(page[i]) * p.c.Hkv + g.h) * (slot_mask + 1) +
                               ((uint32_t(tile) * kTreeTile + i * 32 + lane) & slot_mask);
            ks[i] = p.c.ks[at];
            vs[i] = p.c.vs[at];
          }
        }
      };
      entries_at(g.t0, entry_next);
      checked(g.t0, entry_next);
      entries_at(g.t0 + 1, entry_next);
      scales_at(g.t0);
      for (int tile = g.t0; tile < g.t1; ++tile, ++tt) {
        const uint32_t b = tt & 1u;
        float k_now[4], v_now[4];
        uint32_t there[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          k_now[i] = ks[i], v_now[i] = vs[i];
          there[i] = __ballot_sync(0xffffffffu, page[i] >= 0);
        }
        const bool one = ((page[0] >= 0 && vs[0] == 1.f) || (page[1] >= 0 && vs[1] == 1.f) ||
                                  (page[2] >= 0 && vs[2] == 1.f) || (page[3] >= 0 && vs[3] == 1.f));
        checked(tile + 1, entry_next);
        scales_at(tile + 1);
        entries_at(tile + 2, entry_next);
        // Product t - 2 is over, so the softmax has read what the buffer held for that tile.  This is
        // waited for with every tile, before its scales are given: the product barrier's next phase
        // needs them, so no phase can pass that this warp has not seen (a wait for the phase before
        // last would last until the phase after next, which waits for this warp).  S(t) waits for the
        // same product, so it costs the softmax nothing.
        if (tt >= 2) ok = warp_wait(bar(kRBarPV + int(b)), ((tt - 2) >> 1) & 1u, budget, status);
        {
          uint32_t zeros = 0;  // a bit for each of this lane's keys
          // A row of zeros is written with scale 1.
          if (__any_sync(0xffffffffu, one)) {
            // The product before is over first, so that the slot's barrier stands at no earlier use.
            if (tt > 0) ok = warp_wait(bar(kRBarPV + int((tt - 1) & 1u)), ((tt - 1) >> 1) & 1u, budget, status) && ok;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t it = I::kTile * tt + uint32_t(i * 32 / I::kVKeys), slot = it % F::kVSlots;
              ok = ok && warp_wait(bar(kRBarVFull + int(slot)), (it / F::kVSlots) & 1u, budget, status);
              if (ok && v_now[i] == 1.f && ((there[i] >> lane) & 1u)) {
                uint32_t any = 0;
                for (int c = 0; c < 16; ++c) {
                  const uint4 v = lds16(sV + slot * uint32_t(kSlotBytes) + uint32_t(c >> 3) * I::kVBlock +
                                        uint32_t((i * 32 + lane) % I::kVKeys) * 128u + uint32_t((c & 7) << 4));
                  any |= (v.x | v.y | v.z | v.w) & 0x7f7f7f7fu;
                }
                if (any == 0) zeros |= 1u << i;
              }
            }
            __syncwarp();
          }
          float* sc = sh_scale + b * 512 + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[i * 32] = k_now[i];
            sc[128 + i * 32] = v_now[i];
          }
#pragma unroll 1
          for (int i = 0; i < 4; ++i, sc += 32) {  // one key's code, as with Q
            const ValueScale s(sc[128], (zeros >> i) & 1u);
            sc[128] = s.log2;
            sc[256] = s.inv;
            sc[384] = s.store;
          }
        }
        if (lane < 4) sh_there[b * 4 + lane] = lane == 0 ? there[0] : lane == 1 ? there[1] : lane == 2 ? there[2] : there[3];
        __syncwarp();
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(kRBarKeys + int(b)));
      }
    }
  } else if (warp >= F::kIssuer) {
    // ---------------------------------------------------------------- MMA issuers
    // (of a pair, the even CTA's)
    if (!kPair || rank == 0) {
      const bool is_s = warp == F::kIssuer;
      constexpr uint32_t kM = kPair ? 8u << 24 : 0;  // M = 256 instead of 128
      constexpr uint32_t id_s = idesc<kFp8>(128, 0, 0) + kM, id_o = idesc<kFp8>(256, 0, 1, kFp8) + kM;
      const uint64_t dq = umma::smem_desc(sQ, 16, 1024);
      const uint32_t high = uint32_t(dq >> 32);
      uint32_t tt = 0, segs = 0;  // tiles issued
      bool ok = true;
      while (ok && tree_next(p, cur, &g)) {
        if (is_s && !(ok = warp_wait(bar(kRBarQ), segs & 1u, budget, status))) break;
        ++segs;
        for (int tile = g.t0; ok && tile < g.t1; ++tile, ++tt) {
          const uint32_t b = tt & 1u, ph = (tt >> 1) & 1u;
          const uint32_t slots = is_s ? F::kKSlots : F::kVSlots;
          const uint32_t full = bar(is_s ? kRBarKFull : kRBarVFull), empty = bar(is_s ? kRBarKEmpty : kRBarVEmpty);
          const uint32_t sbuf = tmem + 256u + b * 128u;
          // What has been loaded is waited for first: P, or the last reader of S, comes after it, and
          // from then on only the products stand between it and the next one.
#pragma unroll 1
          for (uint32_t i = 0; ok && i < kTile; ++i) {
            const uint32_t item = kTile * tt + i;
            ok = warp_wait(full + 8u * (item % slots), (item / slots) & 1u, budget, status);
          }
          // O += P(t - 2) V has read what S(t) overwrites; P(t) is there.
          if (is_s)
            ok = ok && (tt < 2 || warp_wait(bar(kRBarPV + int(b)), ph ^ 1u, budget, status));
          else
            ok = ok && warp_wait(bar(kRBarP + int(b)), ph, budget, status);
          if (!ok) break;
          umma::fence_after_sync();
          if (elect_lane()) {
#pragma unroll
            for (uint32_t i = 0; i < kTile; ++i) {
              const uint32_t item = kTile * tt + i, slot = item % slots;
              const uint32_t base = (is_s ? sK : sV) + slot * uint32_t(kSlotBytes);
              if constexpr (kPair) {
                // two column blocks of Q against those of the keys, or four steps of 16 values
                if (is_s) {
                  const uint64_t dk = umma::smem_desc(base, 16, 1024);
#pragma unroll
                  for (uint32_t k = 0; k < 8; ++k)
                    mma_pair(sbuf, desc_low(dq, (2 * i + k / 4) * (kRows * 128u) + k % 4 * 32u),
                             desc_low(dk, k / 4 * 8192u + k % 4 * 32u), high, id_s, (i | k) != 0);
                } else {
                  const uint64_t dv = umma::smem_desc(base, kVBlock, 1024);
#pragma unroll
                  for (uint32_t k = 0; k < 4; ++k)
                    mma_ts_pair(tmem, sbuf + 8u * (4 * i + k), desc_low(dv, k * I::kStep), high, id_o,
                                tile > g.t0 || (i | k) != 0);
                }
                umma::commit_2sm_mc(empty + 8u * slot, 3);
                continue;
              }
              if (is_s) {
                // column block i of Q against that of the keys: four steps of 32 bytes
                const uint64_t dk = umma::smem_desc(base, 16, 1024);
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
#pragma unroll
                  for (uint32_t piece = 0; piece < (kFp8 ? 2 : 1); ++piece)
                    mma<kFp8>(sbuf, desc_low(dq, (i + 2 * piece) * (kRows * 128u) + k * 32u), desc_low(dk, k * 32u), high,
                              id_s, (i | k | piece) != 0);
              } else {
                // the slot's keys in two steps, all columns of the values
                const uint64_t dv = umma::smem_desc(base, kVBlock, 1024);
#pragma unroll
                for (uint32_t k = 0; k < 2; ++k)
#pragma unroll
                  for (uint32_t piece = 0; piece < (kFp8 ? 3 : 1); ++piece)
                    mma_ts<kFp8>(tmem, sbuf + 32u * piece + 8u * (2 * i + k), desc_low(dv, k * I::kStep), high, id_o,
                                 tile > g.t0 || (i | k | piece) != 0);
              }
              umma::commit(empty + 8u * slot);
            }
            const uint32_t done = bar((is_s ? kRBarS : kRBarPV) + int(b));
            if constexpr (kPair)
              umma::commit_2sm_mc(done, 3);
            else
              umma::commit(done);
          }
          __syncwarp();
        }
      }
      // Every product complete before TMEM is released.
      if (elect_lane()) {
        if (tt == 0)
          mbar_arrive(bar(kRBarDrain));
        else if constexpr (kPair)
          umma::commit_2sm(bar(kRBarDrain));
        else
          umma::commit(bar(kRBarDrain));
      }
      __syncwarp();
      warp_wait(bar(kRBarDrain), 0, budget, status);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    constexpr uint32_t kAll = 32 * kSoftWarps;  // threads of barrier 15
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t quarter_bar = 1u + uint32_t(quarter);  // the four parts of a lane quarter
    const int r = quarter * 32 + lane;                    // row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (uint32_t(quarter * 32) << 16);
    const int g_shift = __ffs(p.G) - 1;
    const int row = rt * kRows + r, t = row >> g_shift;
    const bool mine = row < p.T * p.G;
    const bool idle = rt * kRows + quarter * 32 >= p.T * p.G;  // no row in the whole quarter
    float* sh_f = reinterpret_cast<float*>(smem_raw + F::kOffF);
    // One value per part and row.
    float* sh_red = reinterpret_cast<float*>(smem_raw + F::kOffRed);
    auto red = [&](int q) -> float& { return sh_red[q * kRows + r]; };
    uint32_t tt = 0, relays = 0;  // tiles so far; values told of by the even CTA
    (void)relays;
    bool ok = true;

    while (ok && tree_next(p, cur, &g)) {
      const int32_t* table = p.table + int64_t(g.b) * p.max_pages;
      // Q of this head, eight rows per warp, all loads in flight.
      constexpr int kQRows = kRows / kSoftWarps;
      uint4 u[kQRows];
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        const int n = rt * kRows + warp + i * kSoftWarps, tq = n >> g_shift;
        u[i] = make_uint4(0, 0, 0, 0);
        if (tq < g.s.drafted)
          u[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q.p) + g.b * p.q.sb +
                                                 int64_t(g.h * p.G + (n & (p.G - 1))) * p.q.sh + tq * p.q.sl + 8 * lane);
      }
      // (The code of one row: it is run from a cold instruction cache, eight rows' in 10,000 cycles.)
#pragma unroll 1
      for (int rq = warp; rq < kRows; rq += kSoftWarps) {
        if constexpr (!kFp8) {
          sts16(sQ + uint32_t(lane >> 3) * (kRows * 128u) + uint32_t(rq) * 128u + uint32_t(((lane & 7) ^ (rq & 7)) << 4), u[0]);
        } else {
          const float f = put_query<kRows, false>(u[0], sQ, rq);
          if (lane == 0) sh_f[rq] = f * p.scale_log2;
        }
#pragma unroll
        for (int i = 1; i < kQRows; ++i) u[i - 1] = u[i];
      }
      if (warp == 0) sh_bad[lane] = 0;
      fence_proxy_async_smem();
      __syncwarp();
      if (!kPair && lane == 0) mbar_arrive(bar(kRBarQ));
      sync_threads(15, kAll);  // sh_f and sh_bad are other warps' too
      // The odd CTA's Q is read by its own tensor core: its writes are over (the barrier) and visible
      // there (the proxy fence of each writer).  The word to the even CTA is a plain arrival, as
      // with P; a release at cluster scope takes 5,000 cycles.
      if (kPair && threadIdx.x == 0) mbar_arrive_remote(lead(kRBarQ));
      const float factor = kFp8 ? sh_f[r] : p.scale_log2;
      const bool live = t < g.s.drafted;

      const int key = part * 32 + lane;  // the key whose values this thread mends (quarter 0)
      // (bf16) The page table's entry of this lane's key, a tile ahead of its use.
      auto entry_at = [&](int tile) {
        const uint32_t j = uint32_t(tile) * kTreeTile + key;
        return tile < g.t1 && j < g.s.keys ? page_entry(p.c, table, p.max_pages, j) : -1;
      };
      int entry = !kFp8 ? entry_at(g.t0) : -1;
      // This row's maximum (the same in all parts), this part's share of its sum.  It starts at the lowest
      // number rather than -infinity, from which differences would be NaN: any score is above it.
      float m = -FLT_MAX, l = 0.f;
      for (int tile = g.t0; tile < g.t1; ++tile, ++tt) {
        const uint32_t sb = tt & 1u, ph = (tt >> 1) & 1u;
        const uint32_t j0 = uint32_t(tile) * kTreeTile + part * 32;
        bool fine = ok;
        // The values of keys 32 part .. + 31 are in their slot.  The product of the tile before is over
        // first, so that the barrier stands at no earlier use of the slot.
        const uint32_t v_item = kTile * tt + uint32_t(part * 32 / kVKeys);
        auto values_there = [&]() {
          if (tt > 0 && !warp_wait(bar(kRBarPV + int((tt - 1) & 1u)), ((tt - 1) >> 1) & 1u, budget, status)) return false;
          if (!kPair || rank == 0) {
            if (!warp_wait(bar(kRBarVFull + int(v_item % F::kVSlots)), (v_item / F::kVSlots) & 1u, budget, status)) return false;
            // The odd CTA's values are counted here too: its warp of the same part waits for the word.
            if (kPair && lane == 0) arrive_release_cluster(mapa_shared(bar(kRBarRelay + part), 1));
            return true;
          }
          const bool there = warp_wait(bar(kRBarRelay + part), relays & 1u, budget, status);
          fence_cluster();
          ++relays;
          return there;
        };
        auto value_unit = [&](int c) {  // 16-byte unit c of this thread's key's values, in any order
          return sV + (v_item % F::kVSlots) * uint32_t(kSlotBytes) + uint32_t(c >> 3) * kVBlock +
                 uint32_t(key % kVKeys) * 128u + uint32_t(((c ^ key) & 7) << 4);
        };
        auto give_p = [&](bool cleared) {  // one lane
          if constexpr (!kPair)
            mbar_arrive(bar(kRBarP + int(sb)));
          else if (cleared)
            arrive_release_cluster(lead(kRBarP + int(sb)));
          else
            mbar_arrive_remote(lead(kRBarP + int(sb)));
        };
        if (idle) {  // its rows of S and O are nobody's; the tiles are counted
          ok = warp_wait(bar(kRBarS + int(sb)), ph, budget, status);
          if (!ok) break;
          if (lane == 0) give_p(false);
          continue;
        }
        // Which of the 32 keys are there, and which this row sees.
        uint32_t there;
        if constexpr (kFp8) {
          fine = warp_wait(bar(kRBarKeys + int(sb)), ph, budget, status) && fine;
          there = sh_there[sb * 4 + part];
        } else {
          const int page = j0 + lane < g.s.keys ? page_checked(p.c, entry) : -1;
          there = __ballot_sync(0xffffffffu, page >= 0);
          entry = entry_at(tile + 1);
        }
        const float* scale = sh_scale + sb * 512 + part * 32;
        uint32_t vis = there;
        const bool drafted_tile = j0 + 32 > g.s.ctx && vis != 0;
        if (drafted_tile) {
          // A lane looks at one key for each token of the quarter's rows in turn: loads of whole
          // lines, eight in flight.
          const int u = int(j0 + lane - g.s.ctx), t0 = (rt * kRows + quarter * 32) >> g_shift;
          uint32_t mine_sees = 0;
#pragma unroll 8
          for (int i = 0; i < 32 >> g_shift; ++i) {
            const bool sees = u < 0 || (u < g.s.drafted && t0 + i < g.s.drafted && tree_sees(p, g.b, t0 + i, u));
            const uint32_t word = __ballot_sync(0xffffffffu, sees);
            if (t == t0 + i) mine_sees = word;
          }
          if (live) vis &= mine_sees;
        }
        const bool masked = __any_sync(0xffffffffu, vis != 0xffffffffu);
        fine = warp_wait(bar(kRBarS + int(sb)), ph, budget, status) && fine;
        umma::fence_after_sync();
        // Values that take no part, as in tree_tc.cu.  Quarter 0's warps look after the 128 keys.
        // (After S: both CTAs of a pair have then begun this segment.)
        const bool gone = !((there >> lane) & 1u), drafted = !gone && j0 + lane >= g.s.ctx;
        const bool cleared = quarter == 0 && __any_sync(0xffffffffu, gone || drafted);
        if (cleared) {
          fine = values_there() && fine;
          if (fine && (gone || drafted)) {
            uint32_t bad = 0;
#pragma unroll 1
            for (int c = 0; c < kUnits; ++c) bad |= mend_unit<kFp8>(value_unit(c), gone);
            const int u = int(j0 + lane - g.s.ctx);
            if (bad) {
              atomicOr(&sh_bad[u >> 5], 1u << (u & 31));
              if constexpr (kPair) {  // each has half of the columns
                const uint32_t to = mapa_shared(smem_u32(&sh_bad[u >> 5]), rank ^ 1u);
                asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(to), "r"(1u << (u & 31)) : "memory");
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        float x[32];
        umma::tmem_ld32(lane_addr + 256u + sb * 128u + uint32_t(part * 32), x);
        umma::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          if constexpr (kFp8) {
            const float4 k4 = *reinterpret_cast<const float4*>(scale + i);
            const float4 l4 = *reinterpret_cast<const float4*>(scale + 128 + i);
            x[i] = fmaf(x[i] * factor, k4.x, l4.x);
            x[i + 1] = fmaf(x[i + 1] * factor, k4.y, l4.y);
            x[i + 2] = fmaf(x[i + 2] * factor, k4.z, l4.z);
            x[i + 3] = fmaf(x[i + 3] * factor, k4.w, l4.w);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] *= factor;
          }
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((vis >> i) & 1u)) x[i] = -INFINITY;
        }
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // The barrier also tells that all four parts have read S, whose place P takes.
        if (any_thread(quarter_bar, 128, mx > m + F::kSlack || !fine)) {
          red(part) = mx;
          if (any_thread(quarter_bar, 128, !fine)) {
            ok = false;
            break;
          }
          const float all = fmaxf(fmaxf(red(0), red(1)), fmaxf(red(2), red(3)));
          const bool up = all > m + F::kSlack;
          const float alpha = up ? ex2(m - all) : 1.f;
          if (up) m = all;
          l *= alpha;
          if (tile > g.t0 && __any_sync(0xffffffffu, up)) {
            // O holds tiles up to the last one: complete before it is rescaled.
            ok = warp_wait(bar(kRBarPV + int((tt - 1) & 1u)), ((tt - 1) >> 1) & 1u, budget, status) && ok;
            umma::fence_after_sync();
            if (ok) {
#pragma unroll 1
              for (int c0 = part * 64; c0 < part * 64 + 64; c0 += 16) {
                float o[16];
                umma::tmem_ld16(lane_addr + uint32_t(c0), o);
                umma::tmem_wait_ld();
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * alpha);
                umma::tmem_st16u(lane_addr + uint32_t(c0), w);
              }
            }
          }
          sync_threads(quarter_bar, 128);  // the exchange is read
        }
        // P and the row's sum.
        if constexpr (kFp8) {
#pragma unroll
          for (int i0 = 0; i0 < 32; i0 += 16) {
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int i = i0; i < i0 + 16; i += 4) {
              const float4 inv = *reinterpret_cast<const float4*>(scale + 256 + i);
              float e[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) e[k] = ex2(x[i + k] - m);
              l = fmaf(e[0], inv.x, fmaf(e[1], inv.y, fmaf(e[2], inv.z, fmaf(e[3], inv.w, l))));
              const float4 store = *reinterpret_cast<const float4*>(scale + 384 + i);
              e[0] *= store.x, e[1] *= store.y, e[2] *= store.z, e[3] *= store.w;
              e5m2_pieces4(e, hi[(i - i0) / 4], mid[(i - i0) / 4], lo[(i - i0) / 4]);
            }
            const uint32_t to = lane_addr + 256u + sb * 128u + uint32_t(part * 8 + i0 / 4);
            tmem_st4u(to, hi);
            tmem_st4u(to + 32u, mid);
            tmem_st4u(to + 64u, lo);
          }
        } else {
          uint32_t pk[16];
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float a = ex2(x[i] - m), b = ex2(x[i + 1] - m);
            sum[(i >> 1) & 3] += a + b;
            pk[i / 2] = pack_bf16x2(a, b);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          umma::tmem_st16u(lane_addr + 256u + sb * 128u + uint32_t(part * 16), pk);
        }
        umma::tmem_wait_st();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0 && ok) give_p(cleared);
      }
      // ------------------------------------------------------------ the segment's result
      const uint32_t last = tt - 1;
      if (ok) ok = warp_wait(bar(kRBarPV + int(last & 1u)), (last >> 1) & 1u, budget, status);
      umma::fence_after_sync();
      ok = !any_thread(15, kAll, !ok);
      if (ok) {
        red(part) = l;
        sync_threads(quarter_bar, 128);
        const float sum = (red(0) + red(1)) + (red(2) + red(3));
        const bool none = !live || sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        const float lse = none ? -INFINITY : (m + log2f(sum) - (kFp8 ? kLogSumScale : 0.f)) * kLn2;
        const bool whole = g.whole();
        const int64_t part_row = ((int64_t(worker) * 2 + g.slot()) * p.row_tiles + rt) * kRows;
        const int64_t head = (int64_t(g.b) * p.c.Hkv + g.h) * p.G;
        if (mine && part == 0) {
          if (whole)
            p.lse[(head + (row & (p.G - 1))) * p.T + t] = lse;
          else
            p.lse_part[part_row + r] = lse;
        }
        const bool bad = __any_sync(0xffffffffu, sh_bad[lane] != 0);
        // 32 rows x 32 columns at a time through Q's place, so that eight lanes write 128 (64)
        // bytes of a row; a lane that writes its own row takes 8 us for a tile of 128.
        const uint32_t stage = sQ + uint32_t(warp) * 4096u;
#pragma unroll 1
        for (int c0 = part * 64; c0 < part * 64 + 64; c0 += 32) {
          float o[32];
          umma::tmem_ld32(lane_addr + uint32_t(c0), o);
          umma::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i] * (kFp8 ? kSumScale / kPScale : 1.f) * inv;  // (as in tree_tc.cu)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sts16(stage + uint32_t(lane) * 128u + uint32_t((i ^ (lane & 7)) << 4),
                  make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]), __float_as_uint(o[4 * i + 2]),
                             __float_as_uint(o[4 * i + 3])));
          if (bad && !none)
#pragma unroll 1
            for (int i = 0; i < 32; ++i) {
              const uint32_t a = stage + uint32_t(lane) * 128u + uint32_t((((i >> 2) ^ lane) & 7) << 4) + uint32_t(i & 3) * 4u;
              float y;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y) : "r"(a) : "memory");
              y += hidden_values<kFp8>(p, g, table, sh_bad, t, c0 + i);
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(y) : "memory");
            }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), n = rt * kRows + quarter * 32 + rr;
            const uint4 y = lds16(stage + uint32_t(rr) * 128u + uint32_t(((lane ^ rr) & 7) << 4));
            if (n >= p.T * p.G) continue;
            const int col = c0 + 4 * (lane & 7);
            if (whole)
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                        ((head + (n & (p.G - 1))) * p.T + (n >> g_shift)) * kHeadDim + col) =
                  make_uint2(pack_bf16x2(__uint_as_float(y.x), __uint_as_float(y.y)),
                             pack_bf16x2(__uint_as_float(y.z), __uint_as_float(y.w)));
            else
              *reinterpret_cast<uint4*>(p.o_part + (part_row + quarter * 32 + rr) * kHeadDim + col) = y;
          }
          __syncwarp();
        }
        umma::fence_before_sync();
      }
      // The next segment's Q and factors take this one's place: all warps are done.
      ok = !any_thread(15, kAll, !ok);
    }
  }
  umma::fence_before_sync();
  if constexpr (kPair)  // neither leaves while products or copies may touch its memory
    cluster_sync();
  else
    __syncthreads();
  if (warp == F::kIssuer) {
    umma::fence_after_sync();
    if constexpr (kPair)
      umma::tmem_dealloc_2sm(tmem, 512);
    else
      umma::tmem_dealloc(tmem, 512);
  }
}

template <bool kFp8, bool kPair>
int launch(const TreeParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  using F = RowsCfg<kFp8>;
  if (!allow_smem<tree_rows_kernel<kFp8, kPair>>(F::kSmem)) return GQA_ERR_LAUNCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.workers) * unsigned(p.row_tiles));
  cfg.blockDim = dim3(F::kThreads);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, tree_rows_kernel<kFp8, kPair>, mk, mv, p) == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

}  // namespace

int launch_tree_rows(const TreeParams& p, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (p.c.dtype == GQA_BF16 && p.row_tiles % 2 == 0) {
    if (!encode_tokens(&mk, p.c, p.c.k, 64, 2, 1) || !encode_tokens(&mv, p.c, p.c.v, 64, 2, 1)) return GQA_ERR_LAUNCH;
    return launch<false, true>(p, mk, mv, stream);
  }
  if (!encode_pages(&mk, p.c, false) || !encode_pages(&mv, p.c, true)) return GQA_ERR_LAUNCH;
  return p.c.dtype == GQA_E4M3 ? launch<true, false>(p, mk, mv, stream) : launch<false, false>(p, mk, mv, stream);
}

}  // namespace gqa
