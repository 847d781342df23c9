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
// Both kernels move each byte once and are meant to be bound by HBM. D / 2
// threads share a cell (16 tokens of one head): a thread owns 8 channels of
// the tokens t, t + 4, t + 8 and t + 12, K and V, so that eight 16-byte loads
// (or stores) are in flight per thread, the look-up of the cell is shared by
// 64 elements, and V's words, which hold two tokens, are written whole. Four
// neighbouring threads hold a group.
//
// Measured (GB300, one launch, ncu): 4 x 16 x 4096 rows of d = 128, K and V:
// write 42 us (178 MB: 4.2 TB/s; instruction issue 0.71 a cycle and the integer
// pipe 56 %: the rounding of 134 million elements is what is left above the 26 us
// of its bytes), read 32 us (5.5 TB/s). 16 x 65536 rows of d = 256: 280 us
// (5.0 TB/s) and 229 us (6.2 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

template <int D>
constexpr int kCellsPerBlock = D <= 96 ? 4 : D == 128 ? 2 : 1;
template <int D>
constexpr int kBlock = kCellsPerBlock<D> * (D / 2);

// Cells that n rows from any start can touch.
__host__ __device__ constexpr int cells_touched(int n) {
  return int((n + 2ll * (kCellTokens - 1)) / kCellTokens);
}

// A thread's cell. Its token j is row i0 + j of (b, h); rows [0, count) are
// cached rows, data of the cell is null where the cache has no such cell.
struct CellTask {
  int b, h;
  long long i0;
  int count;
  uint8_t *cell;
};

// The cell of task x = (b * heads + h) * cells_touched(n) + k. A position, page
// or count out of range is recorded.
template <int D>
__device__ __forceinline__ CellTask find(const CacheRowsParams &p, uint32_t x, uint32_t kernel) {
  CellTask task;
  const uint32_t cells = cells_touched(p.n);
  const uint32_t bh = x / cells, k = x - bh * cells;
  task.b = bh / p.pool.heads;
  task.h = bh - task.b * p.pool.heads;
  const long long start = p.start[task.b];
  const long long c = (start >> 4) + k;  // floor, for a negative start too
  task.i0 = c * kCellTokens - start;
  task.count = p.counts ? p.counts[task.b] : p.n;
  if (task.count < 0 || task.count > p.n) {
    atomicCAS(p.status, 0u, index_code(kernel, 3));
    task.count = task.count < 0 ? 0 : p.n;
  }
  task.cell = nullptr;
  if (task.i0 >= task.count || task.i0 + kCellTokens <= 0) return task;
  if (c < 0 || c >= p.pool.table_cells) {
    atomicCAS(p.status, 0u, index_code(kernel, 1));
    return task;
  }
  const int pi = p.pool.by_page_cells.div((int)c);
  const int page = p.pool.table[(size_t)((long long)task.b * p.pool.table_stride + pi)];
  if (!p.pool.page_ok(page)) {
    atomicCAS(p.status, 0u, index_code(kernel, 2));
    return task;
  }
  task.cell = p.pool.template cell_ptr<D>(page, task.h, (int)c - pi * p.pool.page_cells);
  return task;
}

template <bool kF16>
__device__ __forceinline__ uint32_t round16(float x) {
  return pack2<kF16>(x, 0.f) & 0xffffu;
}

// Four codes as the nibbles of 16 bits (exact in fp32), code 0 lowest.
__device__ __forceinline__ uint32_t nibbles(float a, float b, float c, float d) {
  const float v = fmaf(fmaf(fmaf(d, 16.f, c), 16.f, b), 16.f, a);
  return __float_as_uint(v + 8388608.f) & 0xffffu;  // 2^23: the sum's last bits are v
}

// Codes by division: for groups whose range or step is near the ends of the
// exponents, or not finite, or where the type's subnormals make the step so
// coarse that a code passes 15. Out of line, being rare.
__device__ __noinline__ uint32_t codes_by_division(float4 a, float4 b, float s) {
  const float d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    u[i] = s > 0.f && s < INFINITY ? fminf(rintf(__fdiv_rn(d[i], s)), 15.f) : 0.f;
  return nibbles(u[0], u[1], u[2], u[3]) | (nibbles(u[4], u[5], u[6], u[7]) << 16);
}

// The correctly rounded quotients a / b of normal numbers from inv, 1 / b to a
// few units of the last place, by one correction with the remainder (Markstein,
// IBM J. Res. Dev. 34, 1990): y = rn(a inv) is within 2^-21 of the quotient, so
// r = a - y b is exact for a b of few bits (11 here), and y + r inv differs
// from a / b by 2^-43 of it, less than the distance of a quotient by 11 bits
// from the middle of two floats (2^-36).
__device__ __forceinline__ uint64_t quotient2(uint64_t a, uint64_t neg_b, uint64_t inv) {
  const uint64_t y = fmul2(a, inv);
  return ffma2(ffma2(y, neg_b, a), inv, y);
}
__device__ __forceinline__ float quotient(float a, float b, float inv) {
  const float y = a * inv;
  return fmaf(fmaf(-y, b, a), inv, y);
}

// Codes of this thread's 8 channels (a quad of threads holds a group) as the
// nibbles of a word, and the group word. Whole warps call it: the quads shuffle.
template <bool kF16>
__device__ __forceinline__ uint32_t quantise(const uint4 w, uint32_t &group) {
  uint32_t low = min2_nan<kF16>(min2_nan<kF16>(w.x, w.y), min2_nan<kF16>(w.z, w.w));
  uint32_t high = max2_nan<kF16>(max2_nan<kF16>(w.x, w.y), max2_nan<kF16>(w.z, w.w));
  low = min2_nan<kF16>(low, __byte_perm(low, low, 0x1032));
  high = max2_nan<kF16>(high, __byte_perm(high, high, 0x1032));
  // (min, -max) in one word for the quad
  uint32_t both = __byte_perm(low, high ^ 0x80008000u, 0x5410);
  both = min2_nan<kF16>(both, __shfl_xor_sync(0xffffffffu, both, 1));
  both = min2_nan<kF16>(both, __shfl_xor_sync(0xffffffffu, both, 2));
  float lo, hi;
  unpack2<kF16>(both ^ 0x80000000u, lo, hi);
  // x - lo, in pairs of channels i and i + 4, whose codes fill the two halves
  float d[8];
  unpack2<kF16>(w.x, d[0], d[1]);
  unpack2<kF16>(w.y, d[2], d[3]);
  unpack2<kF16>(w.z, d[4], d[5]);
  unpack2<kF16>(w.w, d[6], d[7]);
  const uint64_t lo2 = f2pack(lo, lo);
  uint64_t d2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d2[i] = fsub2(f2pack(d[i], d[i + 4]), lo2);
  const float range = hi - lo;
  float s, unused;
  // s at least the type's smallest normal number (2^-14 for f16, whose largest
  // range is 2^17), and everything far from the ends of fp32's exponents
  constexpr float kFrom = kF16 ? 0x1p-10f : 0x1p-96f, kTo = 0x1p96f;
  if (range >= kFrom && range <= kTo) {
    const uint32_t s16 = round16<kF16>(quotient(range, 15.f, 1.f / 15.f));
    unpack2<kF16>(s16, s, unused);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const uint64_t inv2 = f2pack(inv, inv), neg2 = f2pack(-s, -s);
    const uint64_t round2 = f2pack(12582912.f, 12582912.f);  // adding 1.5 * 2^23 rounds to whole
    uint64_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = fsub2(fadd2(quotient2(d2[i], neg2, inv2), round2), round2);
    const uint64_t sixteen2 = f2pack(16.f, 16.f);
    uint64_t v = ffma2(ffma2(ffma2(u[3], sixteen2, u[2]), sixteen2, u[1]), sixteen2, u[0]);
    float v0, v1;
    f2unpack(fadd2(v, f2pack(8388608.f, 8388608.f)), v0, v1);  // 2^23: the last bits are the codes
    group = s16 | (both << 16);
    return __byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x5410);
  }
  const uint32_t s16 = round16<kF16>(__fdiv_rn(range, 15.f));
  unpack2<kF16>(s16, s, unused);
  group = s < INFINITY ? s16 | (both << 16) : 0x7fff0000u;
#pragma unroll
  for (int i = 0; i < 4; ++i) f2unpack(d2[i], d[i], d[i + 4]);
  return codes_by_division(make_float4(d[0], d[1], d[2], d[3]),
                           make_float4(d[4], d[5], d[6], d[7]), s);
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kBlock<D>)
    fa_cache_write_kernel(const __grid_constant__ CacheRowsParams p) {
  constexpr int kLanes = D / 8;
  const int in_cell = threadIdx.x % (D / 2);
  const int tok = in_cell / kLanes, part = in_cell % kLanes;  // tokens tok + 4 x
  const int g = part >> 2, t = part & 3;
  const uint32_t x = blockIdx.x * kCellsPerBlock<D> + threadIdx.x / (D / 2);
  const uint32_t tasks = (uint32_t)p.B * p.pool.heads * cells_touched(p.n);
  CellTask task;
  task.cell = nullptr;
  if (x < tasks) task = find<D>(p, x, kKernCacheWrite);
  uint4 wk[4], wv[4];
  bool live[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long i = task.cell ? task.i0 + tok + 4 * j : -1;
    live[j] = task.cell && i >= 0 && i < task.count;
    wk[j] = wv[j] = make_uint4(0, 0, 0, 0);
    if (live[j]) {
      wk[j] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.k) +
                                                     p.sk.row(task.b, task.h, (int)i) + part * 8));
      wv[j] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v) +
                                                     p.sv.row(task.b, task.h, (int)i) + part * 8));
    }
  }
  if (!__any_sync(0xffffffffu, live[0] || live[1] || live[2] || live[3])) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t group;
    const uint32_t word = quantise<kF16>(wk[j], group);
    const int slot = cell_slot(tok + 4 * j);
    if (live[j]) {
      *reinterpret_cast<uint32_t *>(task.cell + k_word<D>(slot, t, g)) = word;
      if (t == 0) *reinterpret_cast<uint16_t *>(task.cell + k_s<D>(slot, g)) = (uint16_t)group;
      if (t == 1) *reinterpret_cast<uint16_t *>(task.cell + k_lo<D>(slot, g)) = (uint16_t)(group >> 16);
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {  // tokens tok + 8 y and tok + 8 y + 4
    // codes, whose halves are those of r = 2 t and r = 2 t + 1, and groups
    uint32_t word[2], group[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) word[z] = quantise<kF16>(wv[2 * y + z], group[z]);
    // the low (q = 0) or high halves of a pair of words, to the pair's tokens
    auto store = [&](int off, const uint32_t (&w)[2], int q) {
      uint8_t *const at = task.cell + off;
      if (live[2 * y] && live[2 * y + 1])
        *reinterpret_cast<uint32_t *>(at) = __byte_perm(w[0], w[1], q ? 0x7632 : 0x5410);
      else if (live[2 * y])
        *reinterpret_cast<uint16_t *>(at) = (uint16_t)(w[0] >> (16 * q));
      else if (live[2 * y + 1])
        *reinterpret_cast<uint16_t *>(at + 2) = (uint16_t)(w[1] >> (16 * q));
    };
    store(v_word<D>(y, tok, 2 * t, g), word, 0);
    store(v_word<D>(y, tok, 2 * t + 1, g), word, 1);
    if (t == 2) store(v_s<D>(y, tok, g), group, 0);
    if (t == 3) store(v_lo<D>(y, tok, g), group, 1);
  }
}

// lo + s u rounded once to the 16-bit type (s u is exact in fp32), for two codes.
template <bool kF16>
__device__ __forceinline__ uint32_t value2(uint32_t ua, uint32_t ub, float s, float lo) {
  // 2^23 + u as a float, minus 2^23: no conversion instruction
  const float a = __uint_as_float(0x4b000000u | ua) - 8388608.f;
  const float b = __uint_as_float(0x4b000000u | ub) - 8388608.f;
  return pack2<kF16>(fmaf(a, s, lo), fmaf(b, s, lo));
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kBlock<D>)
    fa_cache_read_kernel(const __grid_constant__ CacheRowsParams p) {
  constexpr int kLanes = D / 8;
  const int in_cell = threadIdx.x % (D / 2);
  const int tok = in_cell / kLanes, part = in_cell % kLanes;  // tokens tok + 4 x
  const int g = part >> 2, t = part & 3;
  const uint32_t x = blockIdx.x * kCellsPerBlock<D> + threadIdx.x / (D / 2);
  const uint32_t tasks = (uint32_t)p.B * p.pool.heads * cells_touched(p.n);
  if (x >= tasks) return;
  const CellTask task = find<D>(p, x, kKernCacheRead);
  uint32_t kw[4] = {}, gk[4] = {}, vw[2][2] = {}, vs[2] = {}, vl[2] = {};
  if (task.cell) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int slot = cell_slot(tok + 4 * j);
      kw[j] = __ldg(reinterpret_cast<const uint32_t *>(task.cell + k_word<D>(slot, t, g)));
      gk[j] = __ldg(reinterpret_cast<const uint16_t *>(task.cell + k_s<D>(slot, g))) |
              ((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(task.cell + k_lo<D>(slot, g))) << 16);
      vw[j >> 1][j & 1] = __ldg(reinterpret_cast<const uint32_t *>(
          task.cell + v_word<D>(j >> 1, tok, 2 * t + (j & 1), g)));
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      vs[y] = __ldg(reinterpret_cast<const uint32_t *>(task.cell + v_s<D>(y, tok, g)));
      vl[y] = __ldg(reinterpret_cast<const uint32_t *>(task.cell + v_lo<D>(y, tok, g)));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long i = task.i0 + tok + 4 * j;
    if (i < 0 || i >= p.n) continue;
    uint4 wk = make_uint4(0, 0, 0, 0), wv = wk;  // rows without a token read zero
    if (task.cell && i < task.count) {
      float s, lo;
      unpack2<kF16>(gk[j], s, lo);
      const uint32_t c = kw[j];
      wk.x = value2<kF16>(c & 15, (c >> 4) & 15, s, lo);
      wk.y = value2<kF16>((c >> 8) & 15, (c >> 12) & 15, s, lo);
      wk.z = value2<kF16>((c >> 16) & 15, (c >> 20) & 15, s, lo);
      wk.w = value2<kF16>((c >> 24) & 15, c >> 28, s, lo);
      unpack2<kF16>(__byte_perm(vs[j >> 1], vl[j >> 1], (j & 1) ? 0x7632 : 0x5410), s, lo);
      const uint32_t a = vw[j >> 1][0] >> (16 * (j & 1)), b = vw[j >> 1][1] >> (16 * (j & 1));
      wv.x = value2<kF16>(a & 15, (a >> 4) & 15, s, lo);
      wv.y = value2<kF16>((a >> 8) & 15, (a >> 12) & 15, s, lo);
      wv.z = value2<kF16>(b & 15, (b >> 4) & 15, s, lo);
      wv.w = value2<kF16>((b >> 8) & 15, (b >> 12) & 15, s, lo);
    }
    uint16_t *k = static_cast<uint16_t *>(p.k), *v = static_cast<uint16_t *>(p.v);
    *reinterpret_cast<uint4 *>(k + p.sk.row(task.b, task.h, (int)i) + part * 8) = wk;
    *reinterpret_cast<uint4 *>(v + p.sv.row(task.b, task.h, (int)i) + part * 8) = wv;
  }
}

template <int D, bool kF16>
cudaError_t launch_rows(const CacheRowsParams &p, bool write, cudaStream_t stream) {
  const uint32_t tasks = (uint32_t)p.B * p.pool.heads * cells_touched(p.n);
  const unsigned grid = (tasks - 1) / kCellsPerBlock<D> + 1;
  LaunchProbe probe(write ? kKindCacheWrite : kKindCacheRead, stream);
  if (write)
    fa_cache_write_kernel<D, kF16><<<grid, kBlock<D>, 0, stream>>>(p);
  else
    fa_cache_read_kernel<D, kF16><<<grid, kBlock<D>, 0, stream>>>(p);
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
