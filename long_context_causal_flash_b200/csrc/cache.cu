// The paged key/value cache, sm_100a: rows written (keys rotated, both rounded or
// quantised on the way) and read back.
//
// A row of 256 columns belongs to 16 threads (half a warp).  GQA_E4M3 rows need their
// largest |x| first, which those threads find by four shuffles; the row never leaves the
// registers between the read, the rotation and the store of its codes, so both kernels
// move each byte once and are bound by memory (for a few tokens, by the launch).
#include "decode.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = kThreads / 16;

// Writes the 16 columns x of a row (groups of eight at c0 and c1) to the pages.
__device__ __forceinline__ void put_unit(const CacheView& c, char* pool, float* scales, int page, int h, int slot, int c0,
                                         int c1, float* x, int unit) {
  const int64_t at = page * c.sp + h * c.sh + slot * c.st;
  if (c.dtype == GQA_F32) {
    store8(reinterpret_cast<float*>(pool) + at + c0, x);
    store8(reinterpret_cast<float*>(pool) + at + c1, x + 8);
  } else if (c.dtype == GQA_BF16) {
    store8(reinterpret_cast<__nv_bfloat16*>(pool) + at + c0, x);
    store8(reinterpret_cast<__nv_bfloat16*>(pool) + at + c1, x + 8);
  } else {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(x[i]);
      amax = a < INFINITY ? fmaxf(amax, a) : amax;  // NaN fails the comparison too
    }
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
    const float scale = e4m3_row_scale(amax);
    // The reciprocal of a power of two: exponent e -> -e, within -120 .. 120.
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= inv;
    if (page >= 0) {
      uint8_t* dst = reinterpret_cast<uint8_t*>(pool) + at;
      const uint2 a = make_uint2(e4m3_encode4(x), e4m3_encode4(x + 4));
      const uint2 b = make_uint2(e4m3_encode4(x + 8), e4m3_encode4(x + 12));
      *reinterpret_cast<uint2*>(dst + c0) = a;
      *reinterpret_cast<uint2*>(dst + c1) = b;
      if (unit == 0) scales[(int64_t(page) * c.Hkv + h) * (int64_t(1) << c.page_shift) + slot] = scale;
    }
  }
}

// One half-warp per token, its keys (blockIdx.z = 0) or its values (1), for
// heads_per_thread heads from blockIdx.y on.
template <typename T>
__global__ void __launch_bounds__(kThreads)
cache_write_kernel(CacheView c, RowsView k, RowsView v, const int32_t* __restrict__ table, int64_t max_pages,
                   const int32_t* __restrict__ start, const int32_t* __restrict__ lens, int64_t tokens, int64_t L,
                   RopeView r, int heads_per_thread) {
  const int unit = threadIdx.x & 15;
  const bool is_v = blockIdx.z != 0;
  const int64_t token = int64_t(blockIdx.x) * kRowsPerCta + (threadIdx.x >> 4);
  int64_t b = 0, l = 0, place = 0;
  int page = -1;
  if (token < tokens) {
    b = token / L;
    l = token - b * L;
    if (!lens || l < lens[b]) {
      place = int64_t(start[b]) + l;
      page = page_of(c, table + b * max_pages, max_pages, place);
    }
  }
  // Half-warps without a token to write stay for the other half's shuffles.
  if (__all_sync(0xffffffffu, page < 0)) return;
  const bool live = page >= 0;
  const int slot = int(place & ((int64_t(1) << c.page_shift) - 1));
  const bool turned = !is_v && r.turns && unit < r.rot / 16;
  int c0, c1;
  unit_columns(unit, !is_v && r.turns ? r.rot : 0, r.interleaved, &c0, &c1);
  float co[8], si[8];
  if (turned && live) {
    const int64_t p = r.positions ? int64_t(r.positions[b * r.pos_sb + l]) : place + r.pos_offset;
    unit_angles(r.turns, unit, p, r.magnitude, 1.f, co, si);
  }
  const RowsView& s = is_v ? v : k;
  char* pool = is_v ? c.v : c.k;
  float* scales = is_v ? c.vs : c.ks;
  const int h_end = min(c.Hkv, (int(blockIdx.y) + 1) * heads_per_thread);
  for (int h = int(blockIdx.y) * heads_per_thread; h < h_end; ++h) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    if (live) {
      const T* src = reinterpret_cast<const T*>(s.p) + b * s.sb + h * s.sh + l * s.sl;
      load8(src + c0, x);
      load8(src + c1, x + 8);
      if (turned) turn_unit(x, r.interleaved, co, si);
    }
    if (live || c.dtype == GQA_E4M3) put_unit(c, pool, scales, page, h, slot, c0, c1, x, unit);
  }
}

// One half-warp per row of k_out (blockIdx.z = 0) or v_out (1): [B, Hkv, max_len, 256].
template <typename T>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(CacheView c, const int32_t* __restrict__ table, int64_t max_pages, const int32_t* __restrict__ lens,
                  T* k_out, T* v_out, int64_t rows, int64_t max_len) {
  const int unit = threadIdx.x & 15;
  const int64_t row = int64_t(blockIdx.x) * kRowsPerCta + (threadIdx.x >> 4);
  if (row >= rows) return;
  const int64_t bh = row / max_len, j = row - bh * max_len;
  const int64_t b = bh / c.Hkv;
  const int h = int(bh - b * c.Hkv);
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (j < lens[b]) {
    const int page = page_of(c, table + b * max_pages, max_pages, j);
    if (page >= 0) {
      const int slot = int(j & ((int64_t(1) << c.page_shift) - 1));
      const int64_t at = page * c.sp + h * c.sh + slot * c.st + 16 * unit;
      const char* pool = blockIdx.z ? c.v : c.k;
      if (c.dtype == GQA_F32) {
        load8(reinterpret_cast<const float*>(pool) + at, x);
        load8(reinterpret_cast<const float*>(pool) + at + 8, x + 8);
      } else if (c.dtype == GQA_BF16) {
        load8(reinterpret_cast<const __nv_bfloat16*>(pool) + at, x);
        load8(reinterpret_cast<const __nv_bfloat16*>(pool) + at + 8, x + 8);
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(pool + at);
        const float scale = (blockIdx.z ? c.vs : c.ks)[(int64_t(page) * c.Hkv + h) * (int64_t(1) << c.page_shift) + slot];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3_decode4(w[i], x + 4 * i);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= scale;
      }
    }
  }
  T* dst = (blockIdx.z ? v_out : k_out) + row * kHeadDim + 16 * unit;
  store8(dst, x);
  store8(dst + 8, x + 8);
}

}  // namespace

int launch_cache_write(const CacheView& c, const RowsView& k, const RowsView& v, const int32_t* table, int64_t max_pages,
                       const int32_t* start, const int32_t* lens, int B, int64_t L, bool bf16, const RopeView& r,
                       cudaStream_t stream) {
  const int64_t tokens = int64_t(B) * L;
  if (tokens == 0) return GQA_OK;
  const int64_t blocks = (tokens + kRowsPerCta - 1) / kRowsPerCta;
  const int hpt = 4;
  const int64_t groups = (c.Hkv + hpt - 1) / hpt;
  if (blocks > 0x7fffffff || groups > 65535) return GQA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups), 2);
  if (bf16)
    cache_write_kernel<__nv_bfloat16>
        <<<grid, kThreads, 0, stream>>>(c, k, v, table, max_pages, start, lens, tokens, L, r, hpt);
  else
    cache_write_kernel<float><<<grid, kThreads, 0, stream>>>(c, k, v, table, max_pages, start, lens, tokens, L, r, hpt);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

int launch_cache_read(const CacheView& c, const int32_t* table, int64_t max_pages, const int32_t* lens, void* k_out,
                      void* v_out, int B, int64_t max_len, bool bf16, cudaStream_t stream) {
  const int64_t rows = int64_t(B) * c.Hkv * max_len;
  if (rows == 0) return GQA_OK;
  const int64_t blocks = (rows + kRowsPerCta - 1) / kRowsPerCta;
  if (blocks > 0x7fffffff) return GQA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), 1, 2);
  if (bf16)
    cache_read_kernel<<<grid, kThreads, 0, stream>>>(c, table, max_pages, lens, static_cast<__nv_bfloat16*>(k_out),
                                                     static_cast<__nv_bfloat16*>(v_out), rows, max_len);
  else
    cache_read_kernel<<<grid, kThreads, 0, stream>>>(c, table, max_pages, lens, static_cast<float*>(k_out),
                                                     static_cast<float*>(v_out), rows, max_len);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

}  // namespace gqa
