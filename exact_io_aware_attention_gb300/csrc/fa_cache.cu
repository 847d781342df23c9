// Writing keys and values into the 4-bit cache, and reading them back.
//
// A row (one token, one head, K or V) is cut into groups of 32 channels; a
// group x is stored as
//     lo = min x,  s = rn16((max x - lo) / 15),  u_c = min(15, rn((x_c - lo) / s))
// and stands for lo + s u_c. lo is an element of the row, so it is exact in
// the row's 16-bit type; s is rounded to it, which moves the largest element
// by at most 15 s 2^-9 (bf16), a thirtieth of a step. A group with a
// non-finite element, or whose range overflows, is stored as s = 0, lo = NaN.
//
// Both kernels move each byte once: a thread owns 8 channels (16 bytes of a
// row), four threads a group, and K and V of a row go together so that two
// loads are in flight per thread. They are bound by HBM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRowsPerBlock = 16;

struct Place {
  uint8_t *cell;  // null: nothing to access
  int token;      // within the cell
};

// Where row i of (b, h) lies, recording a bad position or page once.
template <int D>
__device__ __forceinline__ Place find(const CacheRowsParams &p, int b, int h, int i,
                                      uint32_t kernel) {
  const long long pos = (long long)p.start[b] + i;
  if (pos < 0 || pos >= (long long)p.pool.table_cells * kCellTokens) {
    atomicCAS(p.status, 0u, index_code(kernel, 1));
    return {nullptr, 0};
  }
  const int c = (int)(pos / kCellTokens);
  const int pi = c / p.pool.page_cells;
  const int page = p.pool.table[(size_t)((long long)b * p.pool.table_stride + pi)];
  if (!p.pool.page_ok(page)) {
    atomicCAS(p.status, 0u, index_code(kernel, 2));
    return {nullptr, 0};
  }
  return {p.pool.template cell_ptr<D>(page, h, c - pi * p.pool.page_cells),
          (int)(pos % kCellTokens)};
}

__device__ __forceinline__ int row_count(const CacheRowsParams &p, int b, uint32_t kernel) {
  if (!p.counts) return p.n;
  const int c = p.counts[b];
  if (c < 0 || c > p.n) {
    atomicCAS(p.status, 0u, index_code(kernel, 3));
    return c < 0 ? 0 : p.n;
  }
  return c;
}

template <bool kF16>
__device__ __forceinline__ uint32_t round16(float x) {
  return pack2<kF16>(x, 0.f) & 0xffffu;
}
template <bool kF16>
__device__ __forceinline__ float widen16(uint32_t w) {
  float lo, hi;
  unpack2<kF16>(w, lo, hi);
  return lo;
}

// Codes of this thread's 8 channels (a quad of threads holds a group): u[i],
// and the group word.
template <bool kF16>
__device__ __forceinline__ uint32_t quantise(const uint4 w, uint32_t (&u)[8]) {
  float x[8];
  unpack2<kF16>(w.x, x[0], x[1]);
  unpack2<kF16>(w.y, x[2], x[3]);
  unpack2<kF16>(w.z, x[4], x[5]);
  unpack2<kF16>(w.w, x[6], x[7]);
  float lo = x[0], hi = x[0], z = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    z = fmaf(x[i], 0.f, z);  // NaN if any element is not finite
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  const uint32_t s16 = round16<kF16>(__fdiv_rn(hi - lo, 15.f));
  const float s = widen16<kF16>(s16);
  const bool bad = !(z == 0.f) || !(s < INFINITY);
  const bool flat = bad || !(s > 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = flat ? 0.f : fminf(rintf(__fdiv_rn(x[i] - lo, s)), 15.f);
    u[i] = (uint32_t)(int)q;
  }
  return bad ? 0x7fff0000u : (s16 | (round16<kF16>(lo) << 16));
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kRowsPerBlock *(D / 8))
    fa_cache_write_kernel(const __grid_constant__ CacheRowsParams p) {
  constexpr int kLanes = D / 8;
  const int lr = threadIdx.x / kLanes, part = threadIdx.x % kLanes;
  const int g = part >> 2, t = part & 3;
  const uint32_t row = blockIdx.x * kRowsPerBlock + lr;  // (b * heads + h) * n + i
  const uint32_t rows = (uint32_t)p.B * p.pool.heads * p.n;
  const bool in = row < rows;
  const uint32_t bh = in ? row / p.n : 0, i = in ? row - bh * p.n : 0;
  const int b = bh / p.pool.heads, h = bh - b * p.pool.heads;
  const bool live = in && (int)i < row_count(p, b, kKernCacheWrite);
  Place at = {nullptr, 0};
  if (live) at = find<D>(p, b, h, i, kKernCacheWrite);
  uint4 wk = make_uint4(0, 0, 0, 0), wv = wk;
  if (at.cell) {
    const uint16_t *k = static_cast<const uint16_t *>(p.k), *v = static_cast<const uint16_t *>(p.v);
    wk = *reinterpret_cast<const uint4 *>(k + p.sk.row(b, h, i) + part * 8);
    wv = *reinterpret_cast<const uint4 *>(v + p.sv.row(b, h, i) + part * 8);
  }
  uint32_t uk[8], uv[8];
  const uint32_t gk = quantise<kF16>(wk, uk);  // (whole warps: the quads shuffle)
  const uint32_t gv = quantise<kF16>(wv, uv);
  uint32_t kw = 0, v0 = 0, v1 = 0;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    kw |= (uk[2 * x] << (4 * x)) | (uk[2 * x + 1] << (16 + 4 * x));
    v0 |= uv[x] << (4 * x);      // halfword r = 2t
    v1 |= uv[4 + x] << (4 * x);  // halfword r = 2t + 1
  }
  const int slot = cell_slot(at.token);
  if (!at.cell) return;
  *reinterpret_cast<uint16_t *>(at.cell + v_half<D>(at.token, 2 * t, g)) = (uint16_t)v0;
  *reinterpret_cast<uint16_t *>(at.cell + v_half<D>(at.token, 2 * t + 1, g)) = (uint16_t)v1;
  *reinterpret_cast<uint32_t *>(at.cell + k_word<D>(slot, t, g)) = kw;
  if (t == 0) *reinterpret_cast<uint32_t *>(at.cell + k_group<D>(slot, g)) = gk;
  if (t == 1) *reinterpret_cast<uint32_t *>(at.cell + v_group<D>(slot, g)) = gv;
}

// lo + s u rounded once to the 16-bit type (s u is exact in fp32).
template <bool kF16>
__device__ __forceinline__ uint32_t value2(uint32_t ua, uint32_t ub, float s, float lo) {
  return pack2<kF16>(fmaf((float)ua, s, lo), fmaf((float)ub, s, lo));
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kRowsPerBlock *(D / 8))
    fa_cache_read_kernel(const __grid_constant__ CacheRowsParams p) {
  constexpr int kLanes = D / 8;
  const int lr = threadIdx.x / kLanes, part = threadIdx.x % kLanes;
  const int g = part >> 2, t = part & 3;
  const uint32_t row = blockIdx.x * kRowsPerBlock + lr;
  const uint32_t rows = (uint32_t)p.B * p.pool.heads * p.n;
  if (row >= rows) return;
  const uint32_t bh = row / p.n, i = row - bh * p.n;
  const int b = bh / p.pool.heads, h = bh - b * p.pool.heads;
  Place at = {nullptr, 0};
  if ((int)i < row_count(p, b, kKernCacheRead)) at = find<D>(p, b, h, i, kKernCacheRead);
  uint4 wk = make_uint4(0, 0, 0, 0), wv = wk;  // rows without a token read zero
  if (at.cell) {
    const int slot = cell_slot(at.token);
    const uint32_t kw = *reinterpret_cast<const uint32_t *>(at.cell + k_word<D>(slot, t, g));
    const uint32_t gk = *reinterpret_cast<const uint32_t *>(at.cell + k_group<D>(slot, g));
    const uint32_t gv = *reinterpret_cast<const uint32_t *>(at.cell + v_group<D>(slot, g));
    const uint32_t v0 = *reinterpret_cast<const uint16_t *>(at.cell + v_half<D>(at.token, 2 * t, g));
    const uint32_t v1 =
        *reinterpret_cast<const uint16_t *>(at.cell + v_half<D>(at.token, 2 * t + 1, g));
    float s, lo;
    unpack2<kF16>(gk, s, lo);
    wk.x = value2<kF16>(kw & 15, (kw >> 16) & 15, s, lo);
    wk.y = value2<kF16>((kw >> 4) & 15, (kw >> 20) & 15, s, lo);
    wk.z = value2<kF16>((kw >> 8) & 15, (kw >> 24) & 15, s, lo);
    wk.w = value2<kF16>((kw >> 12) & 15, (kw >> 28) & 15, s, lo);
    unpack2<kF16>(gv, s, lo);
    wv.x = value2<kF16>(v0 & 15, (v0 >> 4) & 15, s, lo);
    wv.y = value2<kF16>((v0 >> 8) & 15, (v0 >> 12) & 15, s, lo);
    wv.z = value2<kF16>(v1 & 15, (v1 >> 4) & 15, s, lo);
    wv.w = value2<kF16>((v1 >> 8) & 15, (v1 >> 12) & 15, s, lo);
  }
  uint16_t *k = static_cast<uint16_t *>(p.k), *v = static_cast<uint16_t *>(p.v);
  *reinterpret_cast<uint4 *>(k + p.sk.row(b, h, i) + part * 8) = wk;
  *reinterpret_cast<uint4 *>(v + p.sv.row(b, h, i) + part * 8) = wv;
}

template <int D, bool kF16>
cudaError_t launch_rows(const CacheRowsParams &p, bool write, cudaStream_t stream) {
  const uint32_t rows = (uint32_t)p.B * p.pool.heads * p.n;
  const unsigned grid = rows / kRowsPerBlock + (rows % kRowsPerBlock != 0);
  const unsigned block = kRowsPerBlock * (D / 8);
  LaunchProbe probe(write ? kKindCacheWrite : kKindCacheRead, stream);
  if (write)
    fa_cache_write_kernel<D, kF16><<<grid, block, 0, stream>>>(p);
  else
    fa_cache_read_kernel<D, kF16><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rows_any(const CacheRowsParams &p, bool write, cudaStream_t stream) {
  const bool f16 = p.pool.f16 != 0;
  switch (p.pool.d) {
    case 64: return f16 ? launch_rows<64, true>(p, write, stream) : launch_rows<64, false>(p, write, stream);
    case 96: return f16 ? launch_rows<96, true>(p, write, stream) : launch_rows<96, false>(p, write, stream);
    case 128: return f16 ? launch_rows<128, true>(p, write, stream) : launch_rows<128, false>(p, write, stream);
    case 256: return f16 ? launch_rows<256, true>(p, write, stream) : launch_rows<256, false>(p, write, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsParams &p, cudaStream_t stream) {
  return launch_rows_any(p, true, stream);
}
cudaError_t launch_cache_read(const CacheRowsParams &p, cudaStream_t stream) {
  return launch_rows_any(p, false, stream);
}

}  // namespace fa
