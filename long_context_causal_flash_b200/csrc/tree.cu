// Attention of drafted tokens over the paged cache on the FP32 pipe, and the merge of
// partial results, sm_100a: fp32 queries over any pages, and bf16 queries over fp32 ones.
//
// A CTA holds R query rows (R / G tokens of the G heads of one key/value head) and
// streams its worker's tiles; 8 warps take 16 of a tile's 128 keys each, four keys at a
// time.  Lane l owns columns 8 l .. 8 l + 7 of q, k, v and of the output.  The 4 R partial
// dot products of a lane are summed over the lanes by halving exchanges (a lane sends the
// half it does not keep), which leaves one score per lane, or per pair of lanes at R = 4,
// where the online softmax runs: the running maximum and sum of a row live in the lanes
// that hold its scores, and the output is rescaled only when some row's maximum rose.
#include "internal.h"
#include "tree.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 4;  // keys a warp takes at a time (a divisor of every page size)
constexpr int kKeysPerWarp = kTreeTile / kWarps;
constexpr int kB200Sms = 148;

// Eight columns of a cache row; e4m3 codes still want their row's scale.
template <int kCache>
__device__ __forceinline__ void load_row(const char* pool, int64_t at, float* x) {
  if constexpr (kCache == GQA_F32) {
    load8(reinterpret_cast<const float*>(pool) + at, x);
  } else if constexpr (kCache == GQA_BF16) {
    load8(reinterpret_cast<const __nv_bfloat16*>(pool) + at, x);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(pool + at);
    e4m3_decode4(u.x, x);
    e4m3_decode4(u.y, x + 4);
  }
}

template <int R, int kCache, typename QT>
__global__ void __launch_bounds__(kThreads, R == 4 ? 2 : 1) tree_ffma_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(16) float smem[];  // [warp][R][256] outputs, then [warp][R] maxima and sums
  __shared__ TreeCursor start;
  float* sh_m = smem + kWarps * R * kHeadDim;
  float* sh_l = sh_m + kWarps * R;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  if (warp == 0) {
    const TreeCursor c = tree_start(p, worker);
    if (lane == 0) start = c;
  }
  __syncthreads();
  TreeCursor cur = start;

  constexpr int kScores = R * kKeys;  // 32 or 16
  const int idx = kScores == 32 ? lane : lane >> 1;
  const int my_key = idx / R, my_row = idx % R;
  const int n_mine = rt * R + my_row;  // this lane's query row among the T G of the head
  const int t_mine = n_mine / p.G;

  TreeSegment g;
  while (tree_next(p, cur, &g)) {
    const int32_t* table = p.table + int64_t(g.b) * p.max_pages;
    float q[R][8], o[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int n = rt * R + r, t = n / p.G;
#pragma unroll
      for (int i = 0; i < 8; ++i) q[r][i] = 0.f, o[r][i] = 0.f;
      if (t < g.s.drafted)
        load8(reinterpret_cast<const QT*>(p.q.p) + g.b * p.q.sb + int64_t(g.h * p.G + n % p.G) * p.q.sh + t * p.q.sl +
                  8 * lane,
              q[r]);
    }
    float m = -INFINITY, l = 0.f;  // of my_row; l: the share of this lane's keys
    for (int tile = g.t0; tile < g.t1; ++tile) {
      for (int k0 = 0; k0 < kKeysPerWarp; k0 += kKeys) {
        const uint32_t j0 = uint32_t(tile) * kTreeTile + warp * kKeysPerWarp + k0;
        if (j0 >= g.s.keys) break;
        const int page = page_of(p.c, table, p.max_pages, j0);
        if (page < 0) continue;  // recorded; its keys are absent
        const int slot = int(j0 & ((1u << p.c.page_shift) - 1));
        const int live = int(min(uint32_t(kKeys), g.s.keys - j0));
        const int64_t at = page * p.c.sp + g.h * p.c.sh + slot * p.c.st + 8 * lane;
        float k[kKeys][8], v[kKeys][8];
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (i < live) {
            load_row<kCache>(p.c.k, at + i * p.c.st, k[i]);
            load_row<kCache>(p.c.v, at + i * p.c.st, v[i]);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) k[i][c] = 0.f, v[i][c] = 0.f;
          }
        float k_scale = 1.f, v_scale = 1.f;
        if constexpr (kCache == GQA_E4M3) {
          const int64_t sat = (int64_t(page) * p.c.Hkv + g.h) * (int64_t(1) << p.c.page_shift) + slot;
          if (my_key < live) k_scale = p.c.ks[sat + my_key], v_scale = p.c.vs[sat + my_key];
        }
        float s[kScores];
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float a = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) a = fmaf(q[r][c], k[i][c], a);
            s[i * R + r] = a;
          }
#pragma unroll
        for (int half = kScores / 2, off = 16; half >= 1; half >>= 1, off >>= 1) {
          const bool up = (lane & off) != 0;
#pragma unroll
          for (int i = 0; i < kScores / 2; ++i)
            if (i < half) {
              const float keep = up ? s[i + half] : s[i], send = up ? s[i] : s[i + half];
              s[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
        }
        if (kScores == 16) s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
        // Visible: any key of the context; a drafted one by the mask.  Rows past the tile's
        // last (t >= T) are nobody's and see all, so that they ask for no masked path.
        const uint32_t j = j0 + my_key;
        bool vis = my_key < live && (t_mine < g.s.drafted || t_mine >= p.T);
        if (vis && j >= g.s.ctx && t_mine < p.T) vis = tree_sees(p, g.b, t_mine, int(j - g.s.ctx));
        const float x = vis ? s[0] * k_scale * p.scale_log2 : -INFINITY;
        const unsigned seen = __ballot_sync(0xffffffffu, vis);
        float mx = x;
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float m_new = fmaxf(m, mx);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        if (__any_sync(0xffffffffu, m_new > m)) {
          const float alpha = exp2f(m - ref);  // 0 for the first visible key
          l *= alpha;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float a = __shfl_sync(0xffffffffu, alpha, kScores == 32 ? r : 2 * r);
#pragma unroll
            for (int c = 0; c < 8; ++c) o[r][c] *= a;
          }
          m = m_new;
        }
        float w = vis ? exp2f(x - ref) : 0.f;
        l += w;
        w *= v_scale;
        if (seen == 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float a = __shfl_sync(0xffffffffu, w, kScores == 32 ? i * R + r : 2 * (i * R + r));
#pragma unroll
              for (int c = 0; c < 8; ++c) o[r][c] = fmaf(a, v[i][c], o[r][c]);
            }
        } else {
          // A hidden value takes no part at all: 0 times an infinity would be NaN.
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const int src = kScores == 32 ? i * R + r : 2 * (i * R + r);
              const float a = __shfl_sync(0xffffffffu, w, src);
              if ((seen >> src) & 1u) {
#pragma unroll
                for (int c = 0; c < 8; ++c) o[r][c] = fmaf(a, v[i][c], o[r][c]);
              }
            }
        }
      }
    }
    // The warps' results: maxima and sums per row, outputs, then one sum over the warps.
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (my_key == 0 && (kScores == 32 || (lane & 1) == 0)) sh_m[warp * R + my_row] = m, sh_l[warp * R + my_row] = l;
#pragma unroll
    for (int r = 0; r < R; ++r) store8(smem + (warp * R + r) * kHeadDim + 8 * lane, o[r]);
    __syncthreads();
    const int slot = g.slot();
    const bool whole = g.whole();
    const int64_t part = (int64_t(worker) * 2 + slot) * p.row_tiles + rt;
    for (int r = warp; r < R; r += kWarps) {
      const int n = rt * R + r, t = n / p.G;
      if (t >= p.T) break;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh_m[w * R + r]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = exp2f(sh_m[w * R + r] - ref);
        const float lw = sh_l[w * R + r];
        if (a == 0.f && lw == lw) continue;  // a warp that saw none of the row's keys (NaN scores go on)
        sum = fmaf(a, lw, sum);
        float y[8];
        load8(smem + (w * R + r) * kHeadDim + 8 * lane, y);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = fmaf(a, y[c], acc[c]);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a NaN sum stays one
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] *= inv;
      const float lse = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      if (whole) {
        const int64_t row = (int64_t(g.b) * p.c.Hkv * p.G + g.h * p.G + n % p.G) * p.T + t;
        if (p.out_bf16)
          store8(static_cast<__nv_bfloat16*>(p.out) + row * kHeadDim + 8 * lane, acc);
        else
          store8(static_cast<float*>(p.out) + row * kHeadDim + 8 * lane, acc);
        if (lane == 0) p.lse[row] = lse;
      } else {
        store8(p.o_part + (part * R + r) * kHeadDim + 8 * lane, acc);
        if (lane == 0) p.lse_part[part * R + r] = lse;
      }
    }
    __syncthreads();
  }
}

// One warp per output row: heads that one worker holds whole are written already; others
// are merged from their workers' partial results in worker order, and rows of sequences
// without tiles are cleared.
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p, int rows_per_tile) {
  const int64_t rows_per_seq = int64_t(p.c.Hkv) * p.G * p.T;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows_per_seq * p.B) return;
  const int lane = threadIdx.x & 31;
  const int b = int(row / rows_per_seq);
  const int64_t in_seq = row - b * rows_per_seq;
  const int hq = int(in_seq / p.T), t = int(in_seq - int64_t(hq) * p.T);
  const int h = hq / p.G, n = t * p.G + hq % p.G;
  int64_t before;
  const int64_t W = tree_total(p, b, &before) * p.c.Hkv;
  const int64_t tiles = tree_seq(p, b).tiles;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float mx = -INFINITY, sum = 0.f;
  if (tiles > 0) {
    const int64_t workers = tree_workers(p, W);
    const int64_t s0 = before * p.c.Hkv + h * tiles, e0 = s0 + tiles;
    const int64_t w0 = ((s0 + 1) * workers - 1) / W, w1 = (e0 * workers - 1) / W;
    if (w0 == w1) return;
    const int rt = n / rows_per_tile, r = n % rows_per_tile;
    auto at = [&](int64_t w) {
      return ((w * 2 + (w == w0 ? 1 : 0)) * p.row_tiles + rt) * rows_per_tile + r;
    };
    // Lane i takes the log-sum-exp of partial result i of each 32: their weights first, then
    // the outputs, eight loads in flight.
    for (int64_t w = w0 + lane; w <= w1; w += 32) mx = fmaxf(mx, p.lse_part[at(w)]);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float ref = mx == -INFINITY ? 0.f : mx;
    for (int64_t wb = w0; wb <= w1; wb += 32) {
      const float mine = wb + lane <= w1 ? expf(p.lse_part[at(wb + lane)] - ref) : 0.f;
      const int n = int(min(int64_t(32), w1 - wb + 1));
      for (int i = 0; i < n; i += 4) {
        float y[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) load8(p.o_part + at(min(wb + i + k, w1)) * kHeadDim + 8 * lane, y[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = __shfl_sync(0xffffffffu, mine, (i + k) & 31);
          if (i + k >= n || a == 0.f) continue;  // a partial result without a visible key is not used
          sum += a;
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[c] = fmaf(a, y[k][c], acc[c]);
        }
      }
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

template <int R, int kCache, typename QT>
int launch_one(const TreeParams& p, cudaStream_t stream) {
  constexpr int smem = (kWarps * R * kHeadDim + 2 * kWarps * R) * 4;
  if (cudaFuncSetAttribute(tree_ffma_kernel<R, kCache, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return GQA_ERR_LAUNCH;
  tree_ffma_kernel<R, kCache, QT><<<unsigned(p.workers) * unsigned(p.row_tiles), kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

template <int R>
int launch_types(const TreeParams& p, bool q_bf16, cudaStream_t stream) {
  if (q_bf16) return launch_one<R, GQA_F32, __nv_bfloat16>(p, stream);
  if (p.c.dtype == GQA_F32) return launch_one<R, GQA_F32, float>(p, stream);
  if (p.c.dtype == GQA_BF16) return launch_one<R, GQA_BF16, float>(p, stream);
  return launch_one<R, GQA_E4M3, float>(p, stream);
}

}  // namespace

TreeShape tree_shape(int B, int Hkv, int G, int64_t T, int64_t max_pages, int page_size, bool q_bf16, int cache_dtype) {
  TreeShape s;
  const int64_t rows = T * G;
  s.tensor = q_bf16 && cache_dtype != GQA_F32;
  if (s.tensor)
    s.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  else
    s.rows = rows <= 4 ? 4 : 8;
  s.row_tiles = int((rows + s.rows - 1) / s.rows);
  const int slots = kB200Sms * (s.rows == 4 ? 2 : 1);
  s.workers = slots / s.row_tiles > 1 ? slots / s.row_tiles : 1;
  // No more workers than tiles that the page tables could hold.
  const int64_t tiles = (max_pages * page_size + kTreeTile - 1) / kTreeTile * B * Hkv;
  if (tiles < s.workers) s.workers = int(tiles);
  return s;
}

int launch_tree_ffma(const TreeParams& p, bool q_bf16, int rows, cudaStream_t stream) {
  return rows == 4 ? launch_types<4>(p, q_bf16, stream) : launch_types<8>(p, q_bf16, stream);
}

int launch_tree_merge(const TreeParams& p, int rows_per_tile, cudaStream_t stream) {
  const int64_t rows = int64_t(p.B) * p.c.Hkv * p.G * p.T;
  const int64_t blocks = (rows + 7) / 8;
  if (blocks > 0x7fffffff) return GQA_ERR_UNSUPPORTED;
  tree_merge_kernel<<<unsigned(blocks), 256, 0, stream>>>(p, rows_per_tile);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

}  // namespace gqa
