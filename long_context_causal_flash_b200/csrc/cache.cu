// The paged key/value cache, sm_100a: rows written (keys rotated, both rounded or
// quantised on the way) and read back.
//
// A row of 256 columns belongs to 16 threads (half a warp).  GQA_E4M3 rows need their
// largest |x| first, which those threads find by four shuffles; the row never leaves the
// registers between the read, the rotation and the store of its codes, so both kernels
// move each byte once and are bound by memory (for a few tokens, by the launch).
// 30,468 tokens of 4 heads written as e4m3, keys rotated (187 MB): 45 us, 29 for the bytes; a
// row's conversions and shuffles keep the writer's warps busier than the reader's, for which
// 45,000 tokens read back to bf16 (254 MB) take 44 us, 39 for the bytes.  Loads stay raw until
// they are used, so that four rows of a half-warp are in flight in 80 registers (55 and 49 us
// with one row; 47 in 64 registers, which spill, with four CTAs on an SM instead of three).
#include <type_traits>

#include "decode.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = kThreads / 16;
constexpr int kBatch = 4;  // rows of a half-warp whose loads are in flight together

// Writes the 16 columns x of a row (groups of eight at c0 and c1) to its place in the pages, and
// its scale; `there`: it has one (half-warps without stay for the other half's shuffles).
template <int kCache>
__device__ __forceinline__ void put_unit(char* row, float* scale_at, bool there, int c0, int c1, float* x, int unit) {
  if constexpr (kCache == GQA_F32) {
    if (!there) return;
    store8(reinterpret_cast<float*>(row) + c0, x);
    store8(reinterpret_cast<float*>(row) + c1, x + 8);
  } else if constexpr (kCache == GQA_BF16) {
    if (!there) return;
    store8(reinterpret_cast<__nv_bfloat16*>(row) + c0, x);
    store8(reinterpret_cast<__nv_bfloat16*>(row) + c1, x + 8);
  } else {
    float amax = 0.f;  // fmaxf passes NaN over
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    if (__any_sync(0xffffffffu, amax == INFINITY)) {  // infinities do not count
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fabsf(x[i]) < INFINITY ? fmaxf(amax, fabsf(x[i])) : amax;
    }
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
    const float scale = e4m3_row_scale(amax);
    // The reciprocal of a power of two: exponent e -> -e, within -120 .. 120.
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= inv;
    if (there) {
      *reinterpret_cast<uint2*>(row + c0) = make_uint2(e4m3_encode4(x), e4m3_encode4(x + 4));
      *reinterpret_cast<uint2*>(row + c1) = make_uint2(e4m3_encode4(x + 8), e4m3_encode4(x + 12));
      if (unit == 0) *scale_at = scale;
    }
  }
}

// One half-warp per token, its keys (blockIdx.z = 0) or its values (1), for kBatch heads.  What
// bounds it is the instructions per element and the loads that wait for one another (length,
// page, row).
template <typename T, int kCache>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
cache_write_kernel(CacheView c, RowsView k, RowsView v, const int32_t* __restrict__ table, int64_t max_pages,
                   const int32_t* __restrict__ start, const int32_t* __restrict__ lens, int64_t tokens, int64_t L,
                   RopeView r) {
  const int unit = threadIdx.x & 15;
  const bool is_v = blockIdx.z != 0;
  const int64_t token = int64_t(blockIdx.x) * kRowsPerCta + (threadIdx.x >> 4);
  const RowsView& s = is_v ? v : k;
  const bool rotates = !is_v && r.turns;
  const int h0 = int(blockIdx.y) * kBatch;
  int c0, c1;
  unit_columns(unit, rotates ? r.rot : 0, r.interleaved, &c0, &c1);
  int64_t b = 0, l = 0, place = 0;
  int page = -1;
  Raw16<T> raw[kBatch];
  if (token < tokens) {
    b = token / L;
    l = token - b * L;
    if (!lens || l < lens[b]) {
      // The rows' loads, all heads in flight together, go out before the page is known.
      const T* src = reinterpret_cast<const T*>(s.p) + b * s.sb + h0 * s.sh + l * s.sl;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h0 + i < c.Hkv) raw[i].load(src + i * s.sh + c0, src + i * s.sh + c1);
      place = int64_t(start[b]) + l;
      page = page_of(c, table + b * max_pages, max_pages, place);
    }
  }
  // Half-warps without a token to write stay for the other half's shuffles.
  if (__all_sync(0xffffffffu, page < 0)) return;
  const bool live = page >= 0;
  const int slot = int(place & ((int64_t(1) << c.page_shift) - 1));
  const bool turned = rotates && unit < r.rot / 16;
  float co[8], si[8];
  if (turned && live) {
    const int64_t p = r.positions ? int64_t(r.positions[b * r.pos_sb + l]) : place + r.pos_offset;
    unit_angles(r.turns, unit, p, r.magnitude, 1.f, co, si);
  }
  constexpr int kEs = kCache == GQA_F32 ? 4 : kCache == GQA_BF16 ? 2 : 1;
  char* row = (is_v ? c.v : c.k) + (page * c.sp + h0 * c.sh + slot * c.st) * kEs;
  float* scale_at = (is_v ? c.vs : c.ks) + (((int64_t(page) * c.Hkv + h0) << c.page_shift) + slot);
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    if (h0 + i >= c.Hkv) break;
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
    if (live) raw[i].values(x);
    if (turned && live) turn_unit(x, r.interleaved, co, si);
    put_unit<kCache>(row + i * c.sh * kEs, scale_at + (int64_t(i) << c.page_shift), live, c0, c1, x, unit);
  }
}

// One half-warp per kBatch tokens in a row of k_out (blockIdx.z = 0) or v_out (1), [B, Hkv,
// max_len, 256].  They start at a multiple of kBatch, so they lie in one page, which is looked
// up once.
template <typename T>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(CacheView c, const int32_t* __restrict__ table, int64_t max_pages, const int32_t* __restrict__ lens,
                  T* k_out, T* v_out, int64_t batches, int64_t max_len) {
  const int unit = threadIdx.x & 15;
  const int64_t batch = int64_t(blockIdx.x) * kRowsPerCta + (threadIdx.x >> 4);
  if (batch >= batches) return;
  const int64_t per_head = (max_len + kBatch - 1) / kBatch;
  const int64_t bh = batch / per_head, j = (batch - bh * per_head) * kBatch;
  const int64_t b = bh / c.Hkv;
  const int h = int(bh - b * c.Hkv);
  const int64_t len = lens[b];
  const int page = j < len ? page_of(c, table + b * max_pages, max_pages, j) : -1;
  const int live = page < 0 ? 0 : int(min(int64_t(kBatch), len - j));
  const int slot = int(j & ((int64_t(1) << c.page_shift) - 1));
  const char* pool = blockIdx.z ? c.v : c.k;
  const int64_t at = page * c.sp + h * c.sh + slot * c.st;
  // The thread's columns 8 unit + (0..7) and 128 + 8 unit + (0..7): contiguous over the half-warp.
  const int c0 = 8 * unit, c1 = 128 + 8 * unit;
  T* dst = (blockIdx.z ? v_out : k_out) + (bh * max_len + j) * kHeadDim;
  auto put = [&](int i, const float* x) {
    if (j + i < max_len) {
      store8(dst + i * kHeadDim + c0, x);
      store8(dst + i * kHeadDim + c1, x + 8);
    }
  };
  auto copy = [&](auto* rows) {
    using S = typename std::remove_const<typename std::remove_pointer<decltype(rows)>::type>::type;
    Raw16<S> raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < live) raw[i].load(rows + at + i * c.st + c0, rows + at + i * c.st + c1);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = 0.f;
      if (i < live) raw[i].values(x);
      put(i, x);
    }
  };
  if (c.dtype == GQA_F32) {
    copy(reinterpret_cast<const float*>(pool));
  } else if (c.dtype == GQA_BF16) {
    copy(reinterpret_cast<const __nv_bfloat16*>(pool));
  } else {
    uint2 u[kBatch][2];
    float scale[kBatch];
    const float* scales = (blockIdx.z ? c.vs : c.ks) + (int64_t(page) * c.Hkv + h) * (int64_t(1) << c.page_shift) + slot;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < live) {
        u[i][0] = *reinterpret_cast<const uint2*>(pool + at + i * c.st + c0);
        u[i][1] = *reinterpret_cast<const uint2*>(pool + at + i * c.st + c1);
        scale[i] = scales[i];
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = 0.f;
      if (i < live) {
        e4m3_decode4(u[i][0].x, x);
        e4m3_decode4(u[i][0].y, x + 4);
        e4m3_decode4(u[i][1].x, x + 8);
        e4m3_decode4(u[i][1].y, x + 12);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= scale[i];
      }
      put(i, x);
    }
  }
}

}  // namespace

int launch_cache_write(const CacheView& c, const RowsView& k, const RowsView& v, const int32_t* table, int64_t max_pages,
                       const int32_t* start, const int32_t* lens, int B, int64_t L, bool bf16, const RopeView& r,
                       cudaStream_t stream) {
  const int64_t tokens = int64_t(B) * L;
  if (tokens == 0) return GQA_OK;
  const int64_t blocks = (tokens + kRowsPerCta - 1) / kRowsPerCta;
  const int64_t groups = (c.Hkv + kBatch - 1) / kBatch;
  if (blocks > 0x7fffffff || groups > 65535) return GQA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups), 2);
  auto launch = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, stream>>>(c, k, v, table, max_pages, start, lens, tokens, L, r);
  };
  if (c.dtype == GQA_F32)
    bf16 ? launch(cache_write_kernel<__nv_bfloat16, GQA_F32>) : launch(cache_write_kernel<float, GQA_F32>);
  else if (c.dtype == GQA_BF16)
    bf16 ? launch(cache_write_kernel<__nv_bfloat16, GQA_BF16>) : launch(cache_write_kernel<float, GQA_BF16>);
  else
    bf16 ? launch(cache_write_kernel<__nv_bfloat16, GQA_E4M3>) : launch(cache_write_kernel<float, GQA_E4M3>);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

int launch_cache_read(const CacheView& c, const int32_t* table, int64_t max_pages, const int32_t* lens, void* k_out,
                      void* v_out, int B, int64_t max_len, bool bf16, cudaStream_t stream) {
  const int64_t rows = int64_t(B) * c.Hkv * ((max_len + kBatch - 1) / kBatch);  // batches of rows
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
