// Device helpers shared by the decoding kernels (rotary positions, the paged cache, the
// attention over it): 16-column loads and stores, e4m3 rows and page lookups.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace gqa {

// Element strides of a [B, H, L, d] view (gqa_rows_t).
struct RowsView {
  char* p;
  int64_t sb, sh, sl;
  int H;
};

// gqa_cache_t as the kernels take it; page_shift = log2(page_size).
struct CacheView {
  char *k, *v;
  float *ks, *vs;
  int32_t* status;
  int64_t sp, sh, st, n_pages;
  int Hkv, page_shift, dtype;
};

// gqa_rope_t without the frequencies' host part; turns == null: no rotation.
struct RopeView {
  const uint64_t* turns;
  const int32_t* positions;
  int64_t pos_sb, pos_offset;
  float magnitude;
  int rot, interleaved;
};

#if defined(__CUDACC__)

// A row of 256 columns is the work of 16 threads, `unit` 0 .. 15, each with 16 columns.
// A rotated unit (unit < rot / 16) holds pairs 8 unit .. 8 unit + 7: with the half layout
// columns 8 unit + (0..7) and rot / 2 + 8 unit + (0..7), else columns 16 unit + (0..15).
// Rows that are not rotated at all (rot = 0) go like those of rot = 256 in the half layout,
// whose loads and stores are contiguous over the threads.  c0 / c1 are the first columns of
// the unit's two groups of eight.
__device__ __forceinline__ void unit_columns(int unit, int rot, int interleaved, int* c0, int* c1) {
  if (rot == 0) {
    *c0 = 8 * unit;
    *c1 = 128 + 8 * unit;
  } else if (!interleaved && unit < rot / 16) {
    *c0 = 8 * unit;
    *c1 = rot / 2 + 8 * unit;
  } else {
    *c0 = 16 * unit;
    *c1 = 16 * unit + 8;
  }
}

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  unpack8(*reinterpret_cast<const uint4*>(p), x);
}
// Sixteen columns as they were loaded: bf16 in half the registers of their values, so that more
// loads are in flight at the same occupancy.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(q);
  }
  __device__ __forceinline__ void values(float* x) const {
    unpack8(a, x);
    unpack8(b, x + 8);
  }
};
template <>
struct Raw16<float> {
  float x[16];
  __device__ __forceinline__ void load(const float* p, const float* q) {
    load8(p, x);
    load8(q, x + 8);
  }
  __device__ __forceinline__ void values(float* y) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = x[i];
  }
};

__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}

// Four e4m3 codes of a word as floats (exact), and the codes of four floats (nearest
// even, saturating; NaN stays NaN).
__device__ __forceinline__ void e4m3_decode4(uint32_t w, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t((w >> (16 * i)) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t e4m3_encode4(const float* x) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return a | (b << 16);
}

// The scale of a quantised row: the least power of two s with amax / s <= 448 = 1.75 * 2^8,
// found in the bits of amax = f * 2^e, f in [1, 2): e - 8, and one more when f > 1.75.  The
// exponent stays in -120 .. 120, so the scale and its reciprocal are normal numbers; a row
// of zeros gets 1.
__device__ __forceinline__ float e4m3_row_scale(float amax) {
  if (!(amax > 0.f)) return 1.f;
  const uint32_t bits = __float_as_uint(amax);
  int e = int(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(-120, min(120, e));
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// Page index of token `j`: the table's entry (-1 outside the table), which page_checked turns
// into -1 when the pool does not hold it (recorded).  In two steps, so that the entry can be
// loaded ahead of its use.
__device__ __forceinline__ int page_entry(const CacheView& c, const int32_t* table, int64_t max_pages, int64_t j) {
  const int64_t slot = j >> c.page_shift;
  return j >= 0 && slot < max_pages ? __ldg(table + slot) : -1;
}
__device__ __forceinline__ int page_checked(const CacheView& c, int page) {
  if (page < 0 || page >= c.n_pages) {
    set_status(c.status, GQA_ERR_DEVICE_BOUNDS);
    return -1;
  }
  return page;
}
__device__ __forceinline__ int page_of(const CacheView& c, const int32_t* table, int64_t max_pages, int64_t j) {
  return page_checked(c, page_entry(c, table, max_pages, j));
}

// cos and sin of a fraction of a turn, `frac` 2^-64 turns, times m.  The angle is taken to the
// nearest quarter turn and an eighth around it, |a| <= pi / 4, in whole numbers; there the
// Taylor series of sine and cosine to a^9 and a^10 leave less than 2e-9, so the results are
// off by the fp32 roundings of a (half a step) and of the sums.
__device__ __forceinline__ void turn_angle(uint64_t frac, float m, float* co, float* si) {
  const uint32_t top = uint32_t(frac >> 32);                   // 2^-32 turns
  const uint32_t quarter = (top + 0x20000000u) >> 30;          // nearest quarter turn
  const float a = float(int32_t(top - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float z = a * a;
  float s = fmaf(z, 2.7557319224e-6f, -1.9841269841e-4f);  // 1 / 9!, -1 / 7!
  s = fmaf(s, z, 8.3333333333e-3f);
  s = fmaf(s, z, -1.6666666667e-1f);
  s = fmaf(s * z, a, a);
  float c = fmaf(z, -2.7557319224e-7f, 2.4801587302e-5f);  // -1 / 10!, 1 / 8!
  c = fmaf(c, z, -1.3888888889e-3f);
  c = fmaf(c, z, 4.1666666667e-2f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.f);
  const float x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;
  *co = (((quarter + 1u) & 2u) ? -x : x) * m;
  *si = ((quarter & 2u) ? -y : y) * m;
}

// cos and sin of the eight pairs of a rotated unit at position p, times m: p * turns modulo
// 2^64 is the angle as a fraction of a turn, exact.
__device__ __forceinline__ void unit_angles(const uint64_t* turns, int unit, int64_t p, float m, float sign, float* co,
                                            float* si) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    turn_angle(uint64_t(p) * __ldg(reinterpret_cast<const unsigned long long*>(turns) + 8 * unit + i), m, &co[i], &si[i]);
    si[i] *= sign;
  }
}

// Turns the 16 columns of a rotated unit (x[0..7], x[8..15] as loaded from c0 and c1).
// Two branches of fixed indexes: one loop with computed ones would put x in local memory.
__device__ __forceinline__ void turn_pair(float& x1, float& x2, float co, float si) {
  const float a = x1, b = x2;
  x1 = a * co - b * si;
  x2 = b * co + a * si;
}
__device__ __forceinline__ void turn_unit(float* x, int interleaved, const float* co, const float* si) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], co[i], si[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], co[i], si[i]);
  }
}

#endif  // __CUDACC__

}  // namespace gqa
