// The work split of the drafted-token attention: which tiles of which sequence and
// key/value head a worker takes, and where its partial results go.
//
// Lengths are known to the device only, and differ between sequences.  All tiles of 128 (for
// fp32 accuracy 32) keys are therefore put into one list, ordered by (sequence, key/value head, tile), and
// worker w of n takes the items [w W / n, (w + 1) W / n): every worker streams the same
// number of keys, to one tile.  A worker's range falls into segments, one per (sequence,
// head) it touches.  A segment that holds all of a head's tiles writes the output; any
// other leaves a partial result in one of the worker's two slots (0: the head began in an
// earlier worker; 1: it goes on in a later one), which a second kernel merges in order.
// A worker is as many CTAs as the T G query rows of a head need; they sweep the same
// tiles side by side, so a tile comes from HBM once and from L2 for the others.
#pragma once

#include <atomic>

#include "decode.cuh"

namespace gqa {

constexpr int kTreeTileShift = 7, kTreeTile = 1 << kTreeTileShift;
constexpr int kTreeTileShiftF32 = 5;  // its kernel's step: a worker then has a chunk more than another, not four

struct TreeParams {
  RowsView q;
  CacheView c;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* tree_lens;  // or null
  const uint8_t* mask;       // or null: a chain
  int64_t max_pages, mask_sb;
  void* out;
  float* lse;
  float* o_part;    // [workers][2][row tiles][rows of a tile][256]
  float* lse_part;  // [workers][2][row tiles][rows of a tile]
  int B, T, G, workers, row_tiles;
  int tile_shift;  // log2 of a tile's keys
  bool out_bf16;
  float scale_log2;
  int64_t wait_budget_ns;
  int test_skip_fill;  // test hook (see FwdParams): the keys' producer of every CTA skips this fill of its ring
};

#if defined(__CUDACC__)

// Context, drafted tokens and tiles of sequence b; what lies past the page table is left out.
struct TreeSeq {
  uint32_t ctx, keys;  // below 2^31 + 2^10
  int drafted, tiles;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  const int64_t cap = p.max_pages << p.c.page_shift;
  const int ctx = p.ctx[b];
  s.drafted = p.tree_lens ? min(max(p.tree_lens[b], 0), p.T) : p.T;
  s.ctx = uint32_t(max(ctx, 0));
  if (ctx < 0 || int64_t(s.ctx) + s.drafted > cap) set_status(p.c.status, GQA_ERR_DEVICE_BOUNDS);
  s.keys = uint32_t(min(int64_t(s.ctx) + s.drafted, cap));
  s.tiles = s.drafted > 0 ? int((s.keys + (1u << p.tile_shift) - 1) >> p.tile_shift) : 0;
  return s;
}

// Where a worker starts and how many items it has.
struct TreeCursor {
  int b, h, tile;
  int64_t left;
};

// One warp: sum of the sequences' tiles, and of those before sequence b_end.
__device__ __forceinline__ int64_t tree_total(const TreeParams& p, int b_end, int64_t* before) {
  const int lane = threadIdx.x & 31;
  int64_t all = 0, pre = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int64_t t = tree_seq(p, b).tiles;
    all += t;
    if (b < b_end) pre += t;
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, s);
    pre += __shfl_xor_sync(0xffffffffu, pre, s);
  }
  if (before) *before = pre;
  return all;
}

// Item list of W items over n workers: fewer workers than items leaves none empty.
__device__ __forceinline__ int64_t tree_workers(const TreeParams& p, int64_t W) {
  return W < p.workers ? W : p.workers;
}

// One warp: the cursor of worker w (left = 0 if it has no work).
__device__ __forceinline__ TreeCursor tree_start(const TreeParams& p, int w) {
  const int lane = threadIdx.x & 31;
  const int first = lane < p.B ? tree_seq(p, lane).tiles : 0;  // all there is of up to 32 sequences
  int64_t all = first;
  if (p.B > 32) {
    all = tree_total(p, 0, nullptr);
  } else {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) all += __shfl_xor_sync(0xffffffffu, all, s);
  }
  const int64_t W = all * p.c.Hkv;
  const int64_t n = tree_workers(p, W);
  TreeCursor c{0, 0, 0, 0};
  if (w >= n) return c;
  int64_t at = w * W / n;
  c.left = (w + 1) * W / n - at;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int64_t mine = int64_t(b0 == 0 ? first : b < p.B ? tree_seq(p, b).tiles : 0) * p.c.Hkv;
    int64_t upto = mine;  // inclusive scan
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, upto, s);
      if (lane >= s) upto += o;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int64_t in = at - __shfl_sync(0xffffffffu, upto - mine, src);
      const int64_t tiles = __shfl_sync(0xffffffffu, mine, src) / p.c.Hkv;
      c.b = b0 + src;
      c.h = int(in / tiles);
      c.tile = int(in - c.h * tiles);
      return c;
    }
    at -= __shfl_sync(0xffffffffu, upto, 31);
  }
  c.left = 0;  // not reached
  return c;
}

// A segment: tiles [t0, t1) of (b, h).
struct TreeSegment {
  TreeSeq s;
  int b, h, t0, t1;
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.tiles; }
  __device__ __forceinline__ int slot() const { return t0 > 0 ? 0 : 1; }
};

// The cursor's next segment; false when the worker is done.
__device__ __forceinline__ bool tree_next(const TreeParams& p, TreeCursor& c, TreeSegment* g) {
  if (c.left <= 0) return false;
  g->s = tree_seq(p, c.b);
  while (g->s.tiles == 0) g->s = tree_seq(p, ++c.b);  // items remain, so a later sequence has tiles
  g->b = c.b;
  g->h = c.h;
  g->t0 = c.tile;
  g->t1 = int(min(int64_t(g->s.tiles), c.tile + c.left));
  c.left -= g->t1 - g->t0;
  c.tile = 0;
  if (++c.h == p.c.Hkv) {
    c.h = 0;
    ++c.b;
  }
  return true;
}

// Programmatic launch: the kernel behind may start, and wait for the one before to end.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether drafted token t sees drafted token u (both below s.drafted).
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int u) {
  return p.mask ? p.mask[b * p.mask_sb + int64_t(t) * p.T + u] != 0 : u <= t;
}

#endif  // __CUDACC__

// Lets a kernel use `bytes` of dynamic shared memory on the current device; asked of the driver
// once per kernel and device (about 1 us of a decoding step's 20 on the host).
template <auto kKernel>
bool allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Launches a kernel that may start while the one before it in the stream still runs, and
// itself waits for that one's end (wait_for_grid).
template <typename... Params, typename... Args>
int launch_programmatic(void (*kernel)(Params...), unsigned blocks, int threads, int smem, cudaStream_t stream,
                        const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH;
}

// fp32 accuracy: q of either type, any pages but bf16 q over bf16 or e4m3 ones; rows 8, 16
// or 24.
int launch_tree_f32(const TreeParams& p, int rows, bool q_bf16, cudaStream_t stream);
// Tensor cores: bf16 q over bf16 or e4m3 pages; rows 16, 32, 64 (the keys as M) or 128.
int launch_tree_tc(const TreeParams& p, int rows, cudaStream_t stream);
int launch_tree_rows(const TreeParams& p, cudaStream_t stream);
int launch_tree_merge(const TreeParams& p, int rows_per_tile, cudaStream_t stream);

// Rows per CTA and worker count of a call, by types and shape (host).
struct TreeShape {
  int rows, row_tiles, workers;
  int tile_shift;
  bool tensor;
};
TreeShape tree_shape(int B, int Hkv, int G, int64_t T, int64_t max_pages, int page_size, bool q_bf16, int cache_dtype);

}  // namespace gqa
