// Shared by the attention kernels over the 4-bit cache: the axis of work that
// their CTAs divide, and shared-memory loads.
#pragma once

#include <atomic>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {

constexpr int kUnitTokens = 128;   // keys of a unit of work
constexpr int kMinShare = 2;       // units of a CTA at least
constexpr float kLn2 = 0.69314718055994531f;

// Words of shared memory that find_share and Piece use: [0] abort flag, [2..7]
// the block of the next piece: number, new tokens, length, visible keys, begin
// (64 bits), [8..31] scan.
constexpr int kWorkBytes = 128;

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t &x, uint32_t &y) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t &x, uint32_t &y, uint32_t &z,
                                       uint32_t &w) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
               : "r"(a)
               : "memory");
}
// kN consecutive words; the address is aligned to the widest load that fits.
template <int kN>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *w) {
  if constexpr (kN == 2) {
    lds64(a, w[0], w[1]);
  } else if constexpr (kN == 3) {
    w[0] = lds32(a);
    w[1] = lds32(a + 4);
    w[2] = lds32(a + 8);
  } else {
    lds128(a, w[0], w[1], w[2], w[3]);
    if constexpr (kN == 8) lds128(a + 16, w[4], w[5], w[6], w[7]);
  }
}

// Query blocks on the work axis: block x = (sequence b, row block rb) has
// `heads` segments of tiles(x) units each.
struct Blocks {
  const CacheFwdParams &p;
  int row_blocks, rows;  // rows: query rows of a block

  // New tokens, length and visible keys of block x. A length or count out of
  // range is clamped (and recorded by `note`).
  __device__ __forceinline__ void shape(int x, int &n, int &len, int &vis, bool note) const {
    const int b = p.by_row_blocks.div(x), rb = x - b * row_blocks;
    len = p.lengths[b];
    n = p.counts ? p.counts[b] : p.nq;
    const int cap = p.pool.table_cells * kCellTokens;
    if (note && (len < 0 || len > cap || n < 0 || n > p.nq))
      atomicCAS(p.status, 0u, index_code(kKernCacheFwd, 3));
    len = min(max(len, 0), cap);
    n = min(max(n, 0), p.nq);
    const int first = p.by_group.div(rb * rows);  // first new token of the block
    const int last = min(p.by_group.div(rb * rows + rows - 1), n - 1);
    vis = first >= n ? 0 : p.causal ? min(len, max(len - n + last + 1, 0)) : len;
  }
  // Its segments' weight on the work axis: their units, or one for a segment
  // that stays whole.
  __device__ __forceinline__ int weight(int vis) const { return p.whole ? 1 : tiles(vis); }
  // A segment without visible keys has one unit too: its rows are written.
  __device__ __forceinline__ int tiles(int vis) const {
    return max(1, (vis + kUnitTokens - 1) / kUnitTokens);
  }
};

// A CTA's share [f, f_end) of the axis.
struct Share {
  long long f, f_end;
  bool found;
};

// The total, then the block in which this CTA's share begins, by block-wide
// scans over the blocks' sizes (one scan where the threads hold all blocks).
// Everything that decides which piece comes next is read once and handed to
// all threads through shared memory: they agree even on values that change
// under the kernel.
template <int kThreads>
__device__ __forceinline__ Share find_share(const CacheFwdParams &p, const Blocks &blocks,
                                            int *misc) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 24, "scan words");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_blocks = p.B * blocks.row_blocks;
  long long total = 0;
  Share mine;
  mine.found = false;
  int x = threadIdx.x, n = 0, len = 0, vis = 0, size = 0;
  long long at = 0;  // where block x begins
  auto scan = [&](int x0, bool note) {
    x = x0 + threadIdx.x;
    size = 0;
    if (x < n_blocks) {
      blocks.shape(x, n, len, vis, note);
      size = blocks.weight(vis);
    }
    int incl = size;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) misc[8 + warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int v = misc[8 + w];
      before += w < warp ? v : 0;
      all += v;
    }
    at = total + (long long)(before + incl - size) * p.pool.heads;
    total += (long long)all * p.pool.heads;
  };
  auto find = [&] {
    if (size > 0 && mine.f >= at && mine.f < at + (long long)size * p.pool.heads) {
      misc[2] = x;
      misc[3] = n;
      misc[4] = len;
      misc[5] = vis;
      *reinterpret_cast<long long *>(misc + 6) = at;
    }
    __syncthreads();
  };
  for (int x0 = 0; x0 < n_blocks; x0 += kThreads) {
    if (x0 > 0) __syncthreads();  // the scan words have been read
    scan(x0, blockIdx.x == 0);
  }
  long long share = total < (1ll << 31)
                        ? (long long)(((uint32_t)total + gridDim.x - 1) / gridDim.x)
                        : (total + gridDim.x - 1) / gridDim.x;
  share = max(share, (long long)(p.whole ? 1 : kMinShare));
  mine.f = share * blockIdx.x;
  mine.f_end = min(mine.f + share, total);
  if (n_blocks <= kThreads) {
    mine.found = mine.f < mine.f_end;
    find();
  } else {
    const long long all = total;
    total = 0;
    for (int x0 = 0; x0 < n_blocks && mine.f < all && !mine.found; x0 += kThreads) {
      __syncthreads();
      scan(x0, false);
      find();
      mine.found = mine.f < total;
    }
  }
  return mine;
}

// Units [t0, t1) of the segment (block blk, head h) at the position f of the axis.
struct Piece {
  int blk, n, len, vis;  // block, new tokens, length and visible keys
  int tiles, h, b, row0, t0, t1, cells;
  long long seg_at;

  __device__ __forceinline__ Piece(const CacheFwdParams &p, const Blocks &blocks, const int *misc,
                                   long long f, long long f_end) {
    blk = misc[2];
    n = misc[3];
    len = misc[4];
    vis = misc[5];
    const long long blk_at = *reinterpret_cast<const long long *>(misc + 6);
    tiles = blocks.tiles(vis);
    const int weight = blocks.weight(vis);
    const long long into = f - blk_at;
    h = into < (1ll << 31) ? int((uint32_t)into / (uint32_t)weight) : int(into / weight);
    seg_at = blk_at + (long long)h * weight;
    t0 = int(f - seg_at);
    t1 = p.whole ? tiles : int(min((long long)tiles, f_end - seg_at));
    b = p.by_row_blocks.div(blk);
    row0 = (blk - b * blocks.row_blocks) * blocks.rows;
    cells = (vis + kCellTokens - 1) / kCellTokens;
  }
  __device__ __forceinline__ long long next(const CacheFwdParams &p) const {
    return seg_at + (p.whole ? 1 : t1);
  }
  // chain: the segment that begins here and ends in a later CTA (x: block,
  // y: head, z: its slot here), and w: whether the segment that an earlier
  // CTA began and that continues here ends here (1) or goes on (0).
  __device__ __forceinline__ void link(int4 &chain, bool first) const {
    if (t0 == 0 && t1 < tiles) chain = make_int4(blk, h, first ? 0 : 1, chain.w);
    if (first && t0 > 0) chain.w = t1 == tiles;
  }
  // Hands the next piece's block over (a barrier must follow); false: no more.
  __device__ __forceinline__ bool advance(const CacheFwdParams &p, const Blocks &blocks, int *misc,
                                          long long f) const {
    if (t1 < tiles || h < p.pool.heads - 1) return true;
    if (blk + 1 == p.B * blocks.row_blocks) return false;
    if (threadIdx.x == 0) {
      int n2, len2, vis2;
      blocks.shape(blk + 1, n2, len2, vis2, false);
      misc[2] = blk + 1;
      misc[3] = n2;
      misc[4] = len2;
      misc[5] = vis2;
      *reinterpret_cast<long long *>(misc + 6) = f;
    }
    return true;
  }
};

// Lets a kernel use its dynamic shared memory, once per device.
template <typename Kernel>
inline cudaError_t allow_shared_memory(Kernel kernel, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace fa
