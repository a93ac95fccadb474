// Rotary positions, sm_100a: pair (x1, x2) of a row at position p turns by a = p f_i,
//     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a);
// turning by -a with the same m is the gradient.  The host part computes the frequencies.
//
// Bound: memory (each element is read and written once; 3 flops per element).  16 threads
// share a row, 16 columns each, so that a half-warp reads and writes whole 256-byte
// pieces; a thread computes the sines and cosines of its eight pairs once and keeps them
// for all the heads of its token that it visits, four heads' loads in flight at a time.
// 15,231 tokens of 20 heads, forward and gradient (621 MB): two launches of 49 us, 6.3 TB/s
// (75 us each with sincospi and one head's loads in flight).
#include <cmath>

#include "decode.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 16;  // tokens per CTA
constexpr int kBatch = 4;               // heads whose loads are in flight together

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) rope_kernel(RowsView x, RowsView y, RowsView x2, RowsView y2, int64_t tokens,
                                                        int64_t L, RopeView r, float sign, int heads_per_thread) {
  const int unit = threadIdx.x & 15;
  const int64_t token = int64_t(blockIdx.x) * kTokens + (threadIdx.x >> 4);
  if (token >= tokens) return;
  const int64_t b = token / L, l = token - b * L;
  const bool turned = unit < r.rot / 16;
  int c0, c1;
  unit_columns(unit, r.rot, r.interleaved, &c0, &c1);
  float co[8], si[8];
  if (turned) {
    const int64_t p = r.positions ? int64_t(r.positions[b * r.pos_sb + l]) : r.pos_offset + l;
    unit_angles(r.turns, unit, p, r.magnitude, sign, co, si);
  }
  const int H = x.H + x2.H;
  const int h_end = min(H, (int(blockIdx.y) + 1) * heads_per_thread);
  for (int h0 = int(blockIdx.y) * heads_per_thread; h0 < h_end; h0 += kBatch) {
    Raw16<T> raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i;
      if (h >= h_end) break;
      const RowsView& s = h < x.H ? x : x2;
      const T* src = reinterpret_cast<const T*>(s.p) + b * s.sb + int64_t(h < x.H ? h : h - x.H) * s.sh + l * s.sl;
      raw[i].load(src + c0, src + c1);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i;
      if (h >= h_end) break;
      float v[16];
      raw[i].values(v);
      if (turned) turn_unit(v, r.interleaved, co, si);
      const RowsView& d = h < x.H ? y : y2;
      T* dst = reinterpret_cast<T*>(d.p) + b * d.sb + int64_t(h < x.H ? h : h - x.H) * d.sh + l * d.sl;
      store8(dst + c0, v);
      store8(dst + c1, v + 8);
    }
  }
}

}  // namespace

int launch_rope(const RowsView& x, const RowsView& y, const RowsView& x2, const RowsView& y2, int B, int64_t L,
                bool bf16, const RopeView& r, bool inverse, cudaStream_t stream) {
  const int64_t tokens = int64_t(B) * L;
  if (tokens == 0) return GQA_OK;
  const int64_t blocks = (tokens + kTokens - 1) / kTokens;
  const int H = x.H + x2.H;
  // Heads of a token per thread.  Its sines and cosines cost about as much as turning four heads,
  // so all heads share them where the tokens alone fill the GPU twice (8 CTAs to an SM), and
  // few tokens are spread over more threads, down to one batch of heads each.
  const int batches = (H + kBatch - 1) / kBatch;
  int64_t groups = (8 * 148 + blocks - 1) / blocks;
  groups = groups < batches ? groups : batches;
  const int hpt = int((batches + groups - 1) / groups) * kBatch;
  groups = (H + hpt - 1) / hpt;
  if (blocks > 0x7fffffff || groups > 65535) return GQA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  const float sign = inverse ? -1.f : 1.f;
  if (bf16)
    rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(x, y, x2, y2, tokens, L, r, sign, hpt);
  else
    rope_kernel<float><<<grid, kThreads, 0, stream>>>(x, y, x2, y2, tokens, L, r, sign, hpt);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

}  // namespace gqa

extern "C" {

int gqa_attn_rope_freqs(int rot, double base, int scaling, double factor, int64_t original_length, double beta_fast,
                        double beta_slow, double* inv_freq, double* magnitude) {
  if (!inv_freq || !magnitude || rot < 2 || rot > gqa::kHeadDim || rot % 2) return GQA_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor)) return GQA_ERR_INVALID_ARG;
  if (scaling < GQA_ROPE_PLAIN || scaling > GQA_ROPE_YARN) return GQA_ERR_INVALID_ARG;
  if (scaling == GQA_ROPE_NTK && rot == 2) return GQA_ERR_INVALID_ARG;
  if (scaling == GQA_ROPE_YARN && (original_length < 1 || !(beta_fast > beta_slow))) return GQA_ERR_INVALID_ARG;
  const double kTwoPi = 6.283185307179586476925;
  *magnitude = scaling == GQA_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  if (scaling == GQA_ROPE_NTK) base *= std::pow(factor, double(rot) / double(rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == GQA_ROPE_LINEAR) f /= factor;
    if (scaling == GQA_ROPE_YARN) {
      const double turns = double(original_length) * f / kTwoPi;
      const double g = std::fmin(1.0, std::fmax(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
      f = f * g + f / factor * (1.0 - g);
    }
    inv_freq[i] = f;
  }
  return GQA_OK;
}

int gqa_attn_rope_turns(const double* inv_freq, int n, uint64_t* turns) {
  if (!inv_freq || !turns || n < 1) return GQA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(inv_freq[i])) return GQA_ERR_INVALID_ARG;
    // Positions are whole numbers, so only the fraction of a turn per position counts.
    const long double t = (long double)inv_freq[i] / 6.283185307179586476925286766559L;
    const long double frac = t - std::floor(t);  // [0, 1]
    const long double scaled = std::rint(std::ldexp(frac, 64));
    turns[i] = scaled >= 18446744073709551616.0L ? 0 : uint64_t(scaled);
  }
  return GQA_OK;
}

}  // extern "C"
