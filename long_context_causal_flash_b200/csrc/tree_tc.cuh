// What the two tensor-core kernels of the drafted-token attention share: barriers, copies,
// products in the type of the pages, the query's two e4m3 pieces and the values that a
// mask hides.
#pragma once

#include "internal.h"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace gqa {
namespace {

constexpr int kSlotBytes = 32768;  // 128 keys x 256 bytes: half of a bf16 tile, a whole e4m3 one
constexpr int kChunk = 16384;      // 128 keys x 128 bytes, one swizzled column block
constexpr float kNoMax = -1e30f;   // a row's maximum before its first visible key
constexpr float kPScale = 16.f;  // e4m3 probabilities are stored times this: 2^4 above the maximum is 256

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

// The same with A in TMEM: row m in lane m, a step's 32 bytes in eight columns.
template <bool kFp8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)));
  else
    umma::mma_ts(d, a, b, idesc, add);
}

// Instruction descriptor: fp32 accumulator, M = 128; e4m3 is format 0 of kind::f8f6f4, bf16
// format 1 of kind::f16.
template <bool kFp8>
__host__ __device__ constexpr uint32_t idesc(int N, int a_mn, int b_mn) {
  return (1u << 4) | (kFp8 ? 0u : (1u << 7) | (1u << 10)) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         (uint32_t(N >> 3) << 17) | (8u << 24);
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
