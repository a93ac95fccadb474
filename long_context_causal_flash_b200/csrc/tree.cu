// The merge of the drafted-token attention's partial results, and the shape of its calls.
#include "internal.h"
#include "tree.cuh"

namespace gqa {
namespace {

constexpr int kB200Sms = 148;

// kPerRow warps per output row: heads that one worker holds whole are written already; others
// are merged from their workers' partial results, and rows of sequences without tiles are
// cleared.  With kPerRow = 8 (few rows, and then many partial results to each) warp i takes
// every eighth of them and the warps' sums are added in their order, so the order of the
// additions is fixed.  The kernel may start while the one before it still runs
// (programmatic launch) and waits for it before it reads what that wrote.
template <int kPerRow>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p, int rows_per_tile) {
  __shared__ float sh_sum[8], sh_max[8];
  __shared__ float sh_acc[kPerRow == 8 ? 8 : 1][kHeadDim];
  launch_dependents();
  const int64_t rows_per_seq = int64_t(p.c.Hkv) * p.G * p.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = kPerRow == 8 ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + warp;
  if (row >= rows_per_seq * p.B) {
    wait_for_grid();
    return;
  }
  const int first = kPerRow == 8 ? warp : 0;  // this warp's first partial result
  const int b = int(row / rows_per_seq);
  const int64_t in_seq = row - b * rows_per_seq;
  const int hq = int(in_seq / p.T), t = int(in_seq - int64_t(hq) * p.T);
  const int h = hq / p.G, n = t * p.G + hq % p.G;
  int64_t before;
  const int64_t W = tree_total(p, b, &before) * p.c.Hkv;
  const int64_t tiles = tree_seq(p, b).tiles;
  const int64_t workers = tree_workers(p, W);
  const int64_t s0 = before * p.c.Hkv + h * tiles, e0 = s0 + tiles;
  const int64_t w0 = tiles > 0 ? ((s0 + 1) * workers - 1) / W : 0, w1 = tiles > 0 ? (e0 * workers - 1) / W : -1;
  wait_for_grid();
  if (tiles > 0 && w0 == w1) return;
  const int rt = n / rows_per_tile, r = n % rows_per_tile;
  auto at = [&](int64_t w) {
    return ((w * 2 + (w == w0 ? 1 : 0)) * p.row_tiles + rt) * rows_per_tile + r;
  };
  // Lane i takes the log-sum-exp of this warp's partial result i of each 32: their weights
  // first, then the outputs, four loads in flight.
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float mx = -INFINITY, sum = 0.f;
  for (int64_t w = w0 + first + lane * kPerRow; w <= w1; w += 32 * kPerRow) mx = fmaxf(mx, p.lse_part[at(w)]);
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
  if constexpr (kPerRow == 8) {
    if (lane == 0) sh_max[warp] = mx;
    __syncthreads();
    for (int w = 0; w < 8; ++w) mx = fmaxf(mx, sh_max[w]);
  }
  const float ref = mx == -INFINITY ? 0.f : mx;
  for (int64_t wb = w0 + first; wb <= w1; wb += 32 * kPerRow) {
    const float mine = wb + lane * kPerRow <= w1 ? expf(p.lse_part[at(wb + lane * kPerRow)] - ref) : 0.f;
    const int count = int(min(int64_t(32), (w1 - wb) / kPerRow + 1));
    for (int i = 0; i < count; i += 4) {
      float y[4][8];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        load8(p.o_part + at(wb + min(i + k, count - 1) * kPerRow) * kHeadDim + 8 * lane, y[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __shfl_sync(0xffffffffu, mine, (i + k) & 31);
        if (i + k >= count || a == 0.f) continue;  // a partial result without a visible key is not used
        sum += a;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = fmaf(a, y[k][c], acc[c]);
      }
    }
  }
  if constexpr (kPerRow == 8) {
    store8(&sh_acc[warp][8 * lane], acc);
    if (lane == 0) sh_sum[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < 8; ++w) {
      float y[8];
      load8(&sh_acc[w][8 * lane], y);
      sum += sh_sum[w];
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += y[c];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] *= inv;
  if (p.out_bf16)
    store8(static_cast<__nv_bfloat16*>(p.out) + row * kHeadDim + 8 * lane, acc);
  else
    store8(static_cast<float*>(p.out) + row * kHeadDim + 8 * lane, acc);
  if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

}  // namespace

TreeShape tree_shape(int B, int Hkv, int G, int64_t T, int64_t max_pages, int page_size, bool q_bf16, int cache_dtype) {
  TreeShape s;
  const int64_t rows = T * G;
  s.tensor = q_bf16 && cache_dtype != GQA_F32;
  s.tile_shift = s.tensor ? kTreeTileShift : kTreeTileShiftF32;
  if (s.tensor) {
    s.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  } else {
    // Up to 24 in multiples of eight, in tiles as even as they can be.
    const int64_t tiles = (rows + 23) / 24;
    s.rows = int((rows + 8 * tiles - 1) / (8 * tiles)) * 8;
  }
  s.row_tiles = int((rows + s.rows - 1) / s.rows);
  const int slots = kB200Sms;
  s.workers = slots / s.row_tiles > 1 ? slots / s.row_tiles : 1;
  // No more workers than tiles that the page tables could hold.
  const int64_t per_head = ((max_pages * page_size - 1) >> s.tile_shift) + 1, heads = int64_t(B) * Hkv;
  if (per_head < s.workers && heads * per_head < s.workers) s.workers = int(heads * per_head);
  return s;
}

int launch_tree_merge(const TreeParams& p, int rows_per_tile, cudaStream_t stream) {
  const int64_t rows = int64_t(p.B) * p.c.Hkv * p.G * p.T;
  const bool few = rows <= 2 * kB200Sms;  // a CTA per row then fills the SMs about once
  const int64_t blocks = few ? rows : (rows + 7) / 8;
  if (blocks > 0x7fffffff) return GQA_ERR_UNSUPPORTED;
  return few ? launch_programmatic(tree_merge_kernel<8>, unsigned(blocks), 256, 0, stream, p, rows_per_tile)
             : launch_programmatic(tree_merge_kernel<1>, unsigned(blocks), 256, 0, stream, p, rows_per_tile);
}

}  // namespace gqa
