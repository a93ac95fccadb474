// Attention of drafted tokens over the paged cache on the FP32 pipe, and the merge of
// partial results, sm_100a: fp32 queries over any pages, and bf16 queries over fp32 ones.
//
// A CTA holds R query rows (R / G tokens of the G heads of one key/value head) and
// streams its worker's tiles; 8 warps take 16 of a tile's 128 keys each, four keys at a
// time, through a ring of three groups of its own in shared memory (a bulk copy per row), so
// that no warp waits for another and two groups per warp are under way.  A lane owns eight columns
// of q, k, v and of the output.  The 4 R partial dot products of a lane (packed FMAs, two
// columns each) are summed over the lanes by halving exchanges (a lane sends the half it
// does not keep), which leaves one score per lane, or per pair of lanes at R = 4, where the
// online softmax runs: the running maximum and sum of a row live in the lanes that hold its
// scores, and the output is rescaled only when some row's maximum rose.  With R = 8 a group
// is 256 packed FMAs, 512 cycles of the FMA pipe, and about as many issue slots; with 4 rows
// fp32 pages are bound by memory, with 8 and more by the FMA pipe.
#include <type_traits>

#include "internal.h"
#include "tree.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 4;    // keys of a group (a divisor of every page size)
constexpr int kStages = 3;  // groups of a warp's ring
constexpr int kKeysPerWarp = kTreeTile / kWarps;
constexpr int kGroups = kKeysPerWarp / kKeys;  // of a tile, per warp
constexpr int kB200Sms = 148;

// Two floats as the operand of a packed FMA: d += a b.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ void ffma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A lane's columns: eight in a row, but two fours 128 apart of fp32 rows, so that a warp's
// 16-byte loads are contiguous.
template <int kCache>
__device__ __forceinline__ int column(int lane, int four) {  // of the lane's columns 4 four .. + 3
  return kCache == GQA_F32 ? 128 * four + 4 * lane : 8 * lane + 4 * four;
}

template <int kCache>
struct RowBytes {
  static constexpr int value = kHeadDim * (kCache == GQA_F32 ? 4 : kCache == GQA_BF16 ? 2 : 1);
};

// The lane's eight columns of a staged row, as four pairs; e4m3 codes want their scale still.
template <int kCache>
__device__ __forceinline__ void staged(const char* row, int lane, uint64_t (&x)[4]) {
  if constexpr (kCache == GQA_F32) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(row + 16 * lane);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(row + 512 + 16 * lane);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
    float f[8];
    if constexpr (kCache == GQA_BF16) {
      unpack8(*reinterpret_cast<const uint4*>(row + 16 * lane), f);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(row + 8 * lane);
      e4m3_decode4(u.x, f);
      e4m3_decode4(u.y, f + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
}

__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

template <int R, int kCache, typename QT>
__global__ void __launch_bounds__(kThreads, 1) tree_ffma_kernel(const __grid_constant__ TreeParams p) {
  // [warp][stage][k, v][4 keys] rows; at the end of a segment [warp][R][256] outputs in their place.
  extern __shared__ __align__(16) char smem[];
  __shared__ TreeCursor start;
  __shared__ float sh_m[kWarps * R], sh_l[kWarps * R];
  __shared__ __align__(16) float sh_w[kWarps][R * kKeys];        // a group's weights
  __shared__ __align__(8) uint64_t sh_bar[kWarps * kStages];  // a ring's slots: their copies are complete
  constexpr int kRow = RowBytes<kCache>::value, kStage = 2 * kKeys * kRow;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  char* ring = smem + warp * kStages * kStage;
  const uint32_t bars = smem_u32(sh_bar) + uint32_t(warp * kStages) * 8u;
  if (lane < kStages) mbar_init(bars + 8u * lane, 1);
  fence_barrier_init();
  if (warp == 0) {
    const TreeCursor c = tree_start(p, worker);
    if (lane == 0) start = c;
  }
  __syncthreads();
  launch_dependents();
  TreeCursor cur = start;
  uint32_t used = 0;  // groups whose copies this warp has asked for
  bool ok = true;

  constexpr int kScores = R * kKeys;  // 32 or 16
  const int idx = kScores == 32 ? lane : lane >> 1;
  const int my_key = idx / R, my_row = idx % R;
  const int t_mine = (rt * R + my_row) / p.G;  // this lane's query row among the T G of the head
  const uint32_t slot_mask = (1u << p.c.page_shift) - 1;
  constexpr int kEs = kRow / kHeadDim;

  TreeSegment g;
  while (ok && tree_next(p, cur, &g)) {
    const int32_t* table = p.table + int64_t(g.b) * p.max_pages;
    uint64_t q[R][4], o[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int n = rt * R + r, t = n / p.G;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (t < g.s.drafted) {
        const QT* src = reinterpret_cast<const QT*>(p.q.p) + g.b * p.q.sb + int64_t(g.h * p.G + n % p.G) * p.q.sh + t * p.q.sl;
        load4(src + column<kCache>(lane, 0), x);
        load4(src + column<kCache>(lane, 1), x + 4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) q[r][i] = pack2(x[2 * i], x[2 * i + 1]), o[r][i] = 0;
    }
    float m = -INFINITY, l = 0.f;  // of my_row; l: the share of this lane's keys

    // Group n of this warp: keys 4 (n % kGroups) .. + 3 of its 16 of tile t0 + n / kGroups.
    const int groups = (g.t1 - g.t0) * kGroups;
    auto first_key = [&](int n) {
      return uint32_t(g.t0 + n / kGroups) * kTreeTile + uint32_t(warp * kKeysPerWarp + n % kGroups * kKeys);
    };
    // The page table's entry of a group, loaded a group ahead of its use.
    auto entry_at = [&](int n) {
      return n < groups && first_key(n) < g.s.keys ? page_entry(p.c, table, p.max_pages, first_key(n)) : -1;
    };
    int entry = entry_at(0);
    // The next group's copies: lanes 0 .. 3 the rows of k, 4 .. 7 those of v.  Rows that are not
    // there are left as they were, and hidden below.  Returns how many keys are.
    auto fetch = [&](int n) {
      const uint32_t stage = used % kStages;
      int live = 0;
      if (n < groups) {
        const uint32_t j0 = first_key(n);
        const int page = j0 < g.s.keys ? page_checked(p.c, entry) : -1;
        entry = entry_at(n + 1);
        live = page < 0 ? 0 : int(min(uint32_t(kKeys), g.s.keys - j0));
        if (lane == 0) mbar_arrive_expect_tx(bars + 8u * stage, uint32_t(2 * live * kRow));
        __syncwarp();
        const int row = lane & (kKeys - 1);
        if (lane < 2 * kKeys && row < live) {
          const int64_t at = (int64_t(page) * p.c.sp + g.h * p.c.sh + ((j0 & slot_mask) + row) * p.c.st) * kEs;
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  smem_u32(ring) + stage * uint32_t(kStage) + uint32_t(lane * kRow)),
              "l"((lane < kKeys ? p.c.k : p.c.v) + at), "r"(uint32_t(kRow)), "r"(bars + 8u * stage)
              : "memory");
        }
        ++used;
      }
      return live;
    };
    const uint32_t base = used;  // the segment's first group in the ring
    int live_at[kStages];        // of the groups in the ring, the next one first
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) live_at[i] = fetch(i);
    for (int n = 0; n < groups; ++n) {
      __syncwarp();  // the stage to be filled has been read by all lanes
      live_at[kStages - 1] = fetch(n + kStages - 1);
      const uint32_t turn = base + uint32_t(n);
      if (!__all_sync(0xffffffffu, mbar_wait_inline(bars + 8u * (turn % kStages), (turn / kStages) & 1u, p.wait_budget_ns,
                                                    p.c.status)))
        ok = false;
      if (!ok) break;
      const int live = live_at[0];
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) live_at[i] = live_at[i + 1];
      if (live == 0) continue;
      const uint32_t j0 = first_key(n);
      const char* stage = ring + turn % kStages * kStage;
      float k_scale = 1.f, v_scale = 1.f;
      if constexpr (kCache == GQA_E4M3) {
        const int page = page_of(p.c, table, p.max_pages, j0);
        const int64_t sat = (int64_t(page) * p.c.Hkv + g.h) * (slot_mask + 1) + (j0 & slot_mask);
        if (my_key < live) k_scale = p.c.ks[sat + my_key], v_scale = p.c.vs[sat + my_key];
      }
      float s[kScores];
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        uint64_t k[4];
        staged<kCache>(stage + i * kRow, lane, k);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          uint64_t a = mul2(q[r][0], k[0]);
          ffma2(a, q[r][1], k[1]);
          ffma2(a, q[r][2], k[2]);
          ffma2(a, q[r][3], k[3]);
          const float2 f = unpack2(a);
          s[i * R + r] = f.x + f.y;
        }
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
          const uint64_t a2 = pack2(a, a);
#pragma unroll
          for (int c = 0; c < 4; ++c) o[r][c] = mul2(o[r][c], a2);
        }
        m = m_new;
      }
      float w = vis ? exp2f(x - ref) : 0.f;
      l += w;
      sh_w[warp][idx] = w * v_scale;
      __syncwarp();
      // A hidden value takes no part at all: 0 times an infinity would be NaN.
      auto add_values = [&](auto all) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          uint64_t v[4];
          staged<kCache>(stage + (kKeys + i) * kRow, lane, v);
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 a = *reinterpret_cast<const float4*>(&sh_w[warp][i * R + r]);
            const float a4[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int src = kScores == 32 ? i * R + r + k : 2 * (i * R + r + k);
              if (decltype(all)::value || ((seen >> src) & 1u)) {
                const uint64_t a2 = pack2(a4[k], a4[k]);
#pragma unroll
                for (int c = 0; c < 4; ++c) ffma2(o[r + k][c], a2, v[c]);
              }
            }
          }
        }
      };
      if (seen == 0xffffffffu)
        add_values(std::true_type{});
      else
        add_values(std::false_type{});
    }
    // Every warp is done with its ring.  After a wait that ran out the others are given one more
    // chance each, so that no copy is left under way, and the call ends.
    if (!__syncthreads_and(ok)) {
      for (uint32_t i = used > kStages ? used - kStages : 0; i < used; ++i)
        mbar_wait_inline(bars + 8u * (i % kStages), (i / kStages) & 1u, p.wait_budget_ns, p.c.status);
      break;
    }
    // The warps' results: maxima and sums per row, outputs, then one sum over the warps.
    float* outs = reinterpret_cast<float*>(smem);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (my_key == 0 && (kScores == 32 || (lane & 1) == 0)) sh_m[warp * R + my_row] = m, sh_l[warp * R + my_row] = l;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const float2 a = unpack2(o[r][2 * f]), b = unpack2(o[r][2 * f + 1]);
        const float y[4] = {a.x, a.y, b.x, b.y};
        store4(outs + (warp * R + r) * kHeadDim + column<kCache>(lane, f), y);
      }
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
        load8(outs + (w * R + r) * kHeadDim + 8 * lane, y);
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
    fence_proxy_async_smem();  // the next segment's copies take the outputs' place
    __syncthreads();
  }
}

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

template <int R, int kCache, typename QT>
int launch_one(const TreeParams& p, cudaStream_t stream) {
  constexpr int ring = kWarps * kStages * 2 * kKeys * RowBytes<kCache>::value, outs = kWarps * R * kHeadDim * 4;
  constexpr int smem = ring > outs ? ring : outs;
  if (!allow_smem<tree_ffma_kernel<R, kCache, QT>>(smem)) return GQA_ERR_LAUNCH;
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
  const int slots = kB200Sms;
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
  const bool few = rows <= 2 * kB200Sms;  // a CTA per row then fills the SMs about once
  const int64_t blocks = few ? rows : (rows + 7) / 8;
  if (blocks > 0x7fffffff) return GQA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<8>, p, rows_per_tile)
                            : cudaLaunchKernelEx(&cfg, tree_merge_kernel<1>, p, rows_per_tile);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

}  // namespace gqa
