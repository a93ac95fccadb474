// What the two tensor-core kernels of the drafted-token attention share: barriers, copies,
// products in the type of the pages, the pieces of queries and probabilities and the values
// that a mask hides.
#pragma once

#include "internal.h"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace gqa {
namespace {

// Slots of the rings, and what lies in them.  Keys: one column block of 128 bytes of a tile's
// 128 keys, [128 keys][128 bytes].  Values: all column blocks of 32 (bf16) or 64 (e4m3) keys,
// [4 or 2 blocks][keys][128 bytes].  Small slots refill the rings evenly: with 32 KiB, a tile's
// keys were two slots of a ring that held no more, and each product waited for a load that
// could start only when the one before it was over (128 rows, bf16: 5,900 cycles a tile).
constexpr int kSlotBytes = 16384;
constexpr float kPScale = 2048.f;  // over e4m3 pages probabilities are stored times this: 2^4 above the maximum is 2^15
template <bool kFp8>
struct Items {
  static constexpr int kTile = kFp8 ? 2 : 4;              // slots of a tile's keys, and of its values
  static constexpr int kVKeys = 128 / kTile;              // keys of a value slot
  static constexpr int kVBlock = kVKeys * 128;            // bytes from one of its column blocks to the next
  static constexpr uint32_t kStep = kFp8 ? 4096u : 2048u;  // bytes of a product's 32 or 16 keys
};

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

__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// One lane of a whole warp, always the same.  The products are issued under this predicate: the
// compiler then keeps their operands in uniform registers, where under `lane == 0` it moves
// every word of them there first.  With softmax warps that fill the scheduler an issue takes 75
// cycles, under `lane == 0` 230 (and the product itself 65 - 130).
__device__ __forceinline__ bool elect_lane() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

// Shared-memory descriptors by their low words: the high words, of strides and layout, are the
// same for all operands of a kernel but for the stride between column blocks in the low ones.
__device__ __forceinline__ uint32_t desc_low(uint64_t d, uint32_t bytes) { return uint32_t(d) + (bytes >> 4); }

// D[tmem] (+)= A[smem] B[smem]^T in the type of the pages.
template <bool kFp8>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, bool add) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(uint32_t(add)));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(uint32_t(add)));
}

// The same with A in TMEM: row m in lane m, a step's 32 bytes in eight columns.
template <bool kFp8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, bool add) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(uint32_t(add)));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(uint32_t(add)));
}

// Instruction descriptor: fp32 accumulator, M = 128; e4m3 and e5m2 are formats 0 and 1 of
// kind::f8f6f4, whose operands may differ in theirs, bf16 is format 1 of kind::f16.
template <bool kFp8>
__host__ __device__ constexpr uint32_t idesc(int N, int a_mn, int b_mn, bool a_e5m2 = false, bool b_e5m2 = false) {
  return (1u << 4) | (!kFp8 || a_e5m2 ? 1u << 7 : 0u) | (!kFp8 || b_e5m2 ? 1u << 10 : 0u) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (8u << 24);
}

// Four probabilities (times kPScale, at most 2^15) in three e5m2 pieces each, the piece that is
// worth most first.  The upper byte of an fp16 number is an e5m2 one: the number cut to three
// bits.  Two cuts, whose rests are exact, and a rounding keep nine of fp16's eleven bits, off by
// 2^-8.8 of the number at most down to 2^-9, and by 2^-17 below it: 2^-20 and 2^-28 of the
// largest probability.  So what many small ones hold beside a large one is kept.  (Two e4m3
// pieces have as many bits, but a smallest step of 2^-9: with room for 2^4 above the largest they
// lost all below 2^-14 of it, a fifth of the output where one of 32,768 keys had half of the weight.)
__device__ __forceinline__ void e5m2_pieces4(const float* e, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  __half2 a = __floats2half2_rn(e[0], e[1]), b = __floats2half2_rn(e[2], e[3]);
  auto cut = [&]() {  // the upper bytes, which a and b lose
    const uint32_t u = *reinterpret_cast<uint32_t*>(&a), v = *reinterpret_cast<uint32_t*>(&b);
    const uint32_t x = u & 0xff00ff00u, y = v & 0xff00ff00u;
    a = __hsub2(a, *reinterpret_cast<const __half2*>(&x));
    b = __hsub2(b, *reinterpret_cast<const __half2*>(&y));
    return __byte_perm(u, v, 0x7531);
  };
  hi = cut();
  mid = cut();
  lo = uint32_t(__nv_cvt_halfraw2_to_fp8x2(__half2_raw(a), __NV_SATFINITE, __NV_E5M2)) |
       uint32_t(__nv_cvt_halfraw2_to_fp8x2(__half2_raw(b), __NV_SATFINITE, __NV_E5M2)) << 16;
}

// What the cleared elements of column d (drafted values that are not finite) add to a row of
// token t: an infinity or NaN for each that the row sees.
template <bool kFp8>
__device__ __noinline__ float hidden_values(const TreeParams& p, const TreeSegment& g, const int32_t* table,
                                            const uint32_t* bad, int t, int d) {
  float sum = 0.f;
  for (int u = 0; u < g.s.drafted; ++u) {
    if (!((bad[u >> 5] >> (u & 31)) & 1u) || !tree_sees(p, g.b, t, u)) continue;
    const uint32_t j = g.s.ctx + u, slot = j & ((1u << p.c.page_shift) - 1);
    const int64_t at = table[j >> p.c.page_shift] * p.c.sp + g.h * p.c.sh + slot * p.c.st + d;
    if constexpr (kFp8) {
      if ((uint8_t(p.c.v[at]) & 0x7f) == 0x7f) sum = __uint_as_float(0x7fc00000u);
    } else {
      const float y = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.c.v)[at]);
      if (!(fabsf(y) < INFINITY)) sum += y;
    }
  }
  return sum;
}

// 5-D tiled TMA load global -> shared, completion counted on `bar` in bytes.  No multicast.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// The same, counted on a barrier of either CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// mbarrier phase `parity` is over; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The keys' or the values' way into shared memory, kept by one whole warp.  They have a ring
// of slots each: their readers wait on a slot's barrier by the parity of its uses, so a
// reader has to wait for every use of the slot, and in a ring that both share one could take
// the use before last for its own.
// TMA boxes of one column block and page (or part of a page): on B200 32 KiB take 435 - 450
// cycles in boxes of 32 keys or more and 530 in boxes of 16, all 148 SMs loading from L2 at
// once.  cp.async by a warp per slot has the same rate, but takes about 2,000 cycles of a warp
// and their latency before the slot is full.  What bounds this warp is its own path per item,
// so that path is short: about 90 cycles for each box and as much around them.
// Whole boxes are loaded: rows of a page past the last key hold what the page holds, pages
// that are not there leave the slot as it was.  The softmax warps hide those keys' scores
// and clear their values.
// A CTA of a pair loads its half of a tile, 64 keys or half of the values' columns, in items
// of 64 keys and two column blocks; the even CTA's barriers count both halves' bytes.
template <bool kFp8, bool kIsV, int kSlots, bool kPair = false>
struct Feed {
  using I = Items<kFp8>;
  static constexpr int kKeys = kPair ? 64 : kIsV ? I::kVKeys : 128;
  static constexpr int kBlocks = kPair ? 2 : kIsV ? (kFp8 ? 2 : 4) : 1;
  static constexpr int kMostShift = kPair ? 6 : kIsV ? (kFp8 ? 6 : 5) : 7;  // log2 kKeys
  static constexpr int kTile = kPair ? 2 : I::kTile;                       // items of a tile
  static_assert(!kPair || !kFp8);
  const CUtensorMap* map;
  uint32_t ring, bar_full, bar_empty;
  TreeCursor cur;
  TreeSegment g;
  int rank = 0;                   // in the pair
  uint32_t slot = 0, parity = 1;  // of the next item; parity: of the wait for the slot to be empty
  int issued = 0;                 // items so far, kSlots at most
  int fill = 0;                   // items so far (keys: the test hook's count)
  int tile = 0, index = 0, page = -1, page_next = -1;
  bool live = false, whole = false;  // whole: all keys of the tile are there
  // This lane's box: `rows` keys from key `k` of the item on, column block `block`, at `offset` of
  // the slot.  Boxes hold one column block, or all of an item's where a page holds its keys.
  int rows, k, block;
  uint32_t offset, bytes;
  bool mine;

  // The page table's entry for each group of eight keys of a tile, in lanes 0 .. 15.
  __device__ __forceinline__ int entries(const TreeParams& p, int t) const {
    const int lane = threadIdx.x & 31;
    const uint32_t j = uint32_t(t) * kTreeTile + lane * 8;
    return t < g.t1 && lane < 16 && j < g.s.keys
               ? page_entry(p.c, p.table + int64_t(g.b) * p.max_pages, p.max_pages, j)
               : -1;
  }
  __device__ __forceinline__ void check(const TreeParams& p, int entry) {
    const int lane = threadIdx.x & 31;
    page = lane < 16 && uint32_t(tile) * kTreeTile + lane * 8 < g.s.keys ? page_checked(p.c, entry) : -1;
    whole = __all_sync(0xffffffffu, page >= 0 || lane >= 16);
  }
  __device__ __forceinline__ void segment(const TreeParams& p) {
    live = tree_next(p, cur, &g);
    if (!live) return;
    tile = g.t0;
    index = 0;
    check(p, entries(p, tile));
    page_next = entries(p, tile + 1);
  }
  __device__ __forceinline__ void begin(const TreeParams& p, const TreeCursor& start, const CUtensorMap* m, uint32_t r,
                                        uint32_t full, uint32_t empty) {
    map = m, ring = r, bar_full = full, bar_empty = empty, cur = start;
    const int lane = threadIdx.x & 31;
    if (lane == 0) tma_prefetch_desc(map);
    const int shift = min(p.c.page_shift, kMostShift), per = kKeys >> shift;
    rows = 1 << shift;
    k = (lane & (per - 1)) * rows;
    block = lane >> (kMostShift - shift);
    mine = lane < (per == 1 ? 1 : per * kBlocks);
    offset = uint32_t(block * kKeys + k) * 128u;
    bytes = uint32_t(per == 1 ? kBlocks : 1) * uint32_t(rows) * 128u;
    segment(p);
  }
  // The next item's slot is free (lanes may differ in the moment they see it).
  __device__ __forceinline__ bool ready() const {
    return live && __all_sync(0xffffffffu, mbar_test(bar_empty + 8u * slot, parity));
  }
  __device__ __forceinline__ void issue(const TreeParams& p) {
    const int lane = threadIdx.x & 31;
    const uint32_t full = bar_full + 8u * slot;
    const int at = (kIsV ? index * kKeys : kPair ? rank * kKeys : 0) + k;  // key of the tile
    const int pg = __shfl_sync(0xffffffffu, page, (at >> 3) & 15);
    const bool skip = !kIsV && fill++ == p.test_skip_fill;  // test hook: neither armed nor copied
    const bool send = mine && pg >= 0 && !skip;
    uint32_t total = kPair ? 2 * kSlotBytes : kSlotBytes;
    if (!whole) {
      uint32_t boxes = __popc(__ballot_sync(0xffffffffu, send));
      if constexpr (kPair) {  // and the other CTA's, whose keys are others
        const int other = kIsV ? at : at ^ kKeys;
        const int its = __shfl_sync(0xffffffffu, page, (other >> 3) & 15);  // by all lanes
        boxes += __popc(__ballot_sync(0xffffffffu, mine && its >= 0));
      }
      total = bytes * boxes;
    }
    if (lane == 0 && (!kPair || rank == 0) && !skip) mbar_arrive_expect_tx(full, total);
    __syncwarp();
    if (send) {
      const uint32_t j = uint32_t(tile) * kTreeTile + uint32_t(at), dst = ring + slot * uint32_t(kSlotBytes) + offset;
      const int in_page = int(j & ((1u << p.c.page_shift) - 1));
      if constexpr (kPair)
        tma_load_5d_pair(dst, map, mapa_shared(full, 0), 0, in_page, (kIsV ? rank * kBlocks : index * kBlocks) + block, g.h, pg);
      else
        tma_load_5d(dst, map, full, 0, in_page, kIsV ? block : index, g.h, pg);
    }
    __syncwarp();
    if (issued < kSlots) ++issued;
    if (++slot == kSlots) slot = 0, parity ^= 1u;
    if (++index == kTile) {
      index = 0;
      if (++tile < g.t1) {
        check(p, page_next);
        page_next = entries(p, tile + 1);
      } else {
        segment(p);
      }
    }
  }
  // No copy may be in flight when the CTA ends: the last use of each slot is complete.
  __device__ __forceinline__ void drain(const TreeParams& p) const {
    if (kPair && rank != 0) return;  // the even CTA's barriers count this one's too; it is waited for at the end
    for (int i = 0; i < issued; ++i) {
      const uint32_t s = slot + kSlots - 1 - i, at = s % kSlots;
      // slots below `slot` have been used in this round (parity ^ 1 of the wait before), others in the last
      warp_wait(bar_full + 8u * at, s >= kSlots ? parity ^ 1u : parity, p.wait_budget_ns, p.c.status);
    }
  }
};

// A producer warp for two rings (fills whichever has a free slot, the first one's first) or,
// with NoFeed, for one.
struct NoFeed {
  bool live = false;
  __device__ __forceinline__ bool ready() const { return false; }
  __device__ __forceinline__ void issue(const TreeParams&) {}
  __device__ __forceinline__ void drain(const TreeParams&) const {}
};
template <class A, class B>
__device__ __forceinline__ void produce(const TreeParams& p, A& a, B& b) {
  uint64_t since = 0;
  int idle = 0;
  while (a.live || b.live) {
    bool moved = false;
    if (a.ready()) {
      a.issue(p);
      moved = true;
    }
    if (b.ready()) {
      b.issue(p);
      moved = true;
    }
    // The clock is read only when nothing has moved for a while.
    idle = moved ? 0 : idle + 1;
    if (idle == 256) since = global_timer_ns();
    if (idle > 256 && (idle & 255) == 0 &&
        __any_sync(0xffffffffu, int64_t(global_timer_ns() - since) > p.wait_budget_ns)) {
      set_status(p.c.status, GQA_ERR_DEVICE_TIMEOUT);
      break;
    }
  }
  a.drain(p);
  b.drain(p);
}

// The tensor map of a pool's keys or values: (columns of a 128-byte block, token of the page,
// block, head, page); boxes of `keys` tokens and `blocks` column blocks, or
// of a page of fewer and `fewer` blocks.
inline bool encode_tokens(CUtensorMap* m, const CacheView& c, const void* data, int keys, int blocks, int fewer) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t es = c.dtype == GQA_F32 ? 4 : c.dtype == GQA_BF16 ? 2 : 1, page = cuuint64_t(1) << c.page_shift;
  const cuuint64_t dims[5] = {128 / es, page, 2 * es, cuuint64_t(c.Hkv), cuuint64_t(c.n_pages)};
  // A dimension of one has no stride of its own (views may carry any number there).
  const cuuint64_t strides[4] = {cuuint64_t(c.st) * es, 128, c.Hkv > 1 ? cuuint64_t(c.sh) * es : 16,
                                 c.n_pages > 1 ? cuuint64_t(c.sp) * es : 16};
  const cuuint32_t box[5] = {cuuint32_t(128 / es), cuuint32_t(page < cuuint64_t(keys) ? page : keys),
                             cuuint32_t(page < cuuint64_t(keys) ? fewer : blocks), 1, 1},
                   estr[5] = {1, 1, 1, 1, 1};
  return enc(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                   : CU_TENSOR_MAP_DATA_TYPE_UINT8,
             5, const_cast<void*>(data), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same as Feed takes them.
inline bool encode_pages(CUtensorMap* m, const CacheView& c, bool values) {
  const bool fp8 = c.dtype == GQA_E4M3;
  return values ? encode_tokens(m, c, c.v, fp8 ? 64 : 32, fp8 ? 2 : 4, 1) : encode_tokens(m, c, c.k, 128, 1, 1);
}

// What the scale of a quantised value does to its key: scores get log2 of its magnitude, P
// is stored times `store`, and a row's sum takes P times `inv`.  A row that puts nothing into O (its
// scale is zero or subnormal, or `zeros`: so are its codes) is stored as 0, and its score
// gets kNoValue, so that it does not set the maximum, on which P's bits hang.  kSumScale
// keeps the sums of values that are tiny throughout within range.  A scale that is not a
// number reaches the rows that see the key through its score alone.
constexpr float kNoValue = -60.f;
constexpr float kLogSumScale = -24.f, kSumScale = 5.9604644775390625e-8f;  // 2^-24
struct ValueScale {
  float log2, inv, store;
  __device__ __forceinline__ ValueScale(float vs, bool zeros) {
    const float a = fabsf(vs);
    const bool none = zeros || a < 1.1754943508222875e-38f;  // 2^-126
    log2 = none ? kNoValue : log2f(a);
    inv = none ? kSumScale * 1152921504606846976.f /* 2^60 */ : a < INFINITY ? kSumScale / a : 1.f;
    store = none ? 0.f : copysignf(kPScale, vs);
  }
};

// One 16-byte unit of a value in shared memory: cleared whole, or its elements that are not
// finite (e4m3 has NaN alone); returns whether it had any of the latter.
template <bool kFp8>
__device__ __forceinline__ uint32_t mend_unit(uint32_t a, bool whole) {
  if (whole) {
    sts16(a, make_uint4(0, 0, 0, 0));
    return 0;
  }
  const uint4 v = lds16(a);
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, hit = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t m = kFp8 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpeq2(w[k] & 0x7f807f80u, 0x7f807f80u);
    hit |= m;
    w[k] &= ~m;
  }
  if (hit) sts16(a, make_uint4(w[0], w[1], w[2], w[3]));
  return hit;
}

// One warp: row r of an e4m3 Q operand, both pieces of the row's eight columns per lane.
// Returns the row's scale, NaN for a row with an infinity or a NaN: it has no finite score.
template <int kN, bool kWide>
__device__ __forceinline__ float put_query(uint4 u, uint32_t sQ, int r) {
  const int lane = threadIdx.x & 31;
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
  constexpr uint32_t kBlock = (kWide ? 2 * kN : kN) * 128u;
  const uint32_t a = sQ + uint32_t(lane >> 4) * kBlock + uint32_t(r) * 128u +
                     uint32_t((((lane & 15) >> 1) ^ (r & 7)) << 4) + uint32_t(lane & 1) * 8u;
  constexpr uint32_t kLo = kWide ? kN * 128u : kN * 256u;  // kN is a multiple of 8: the same swizzle
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(h0), "r"(h1) : "memory");
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a + kLo), "r"(e4m3_encode4(lo)), "r"(e4m3_encode4(lo + 4))
               : "memory");
  return finite ? scale : __uint_as_float(0x7fc00000u);
}

}  // namespace
}  // namespace gqa
