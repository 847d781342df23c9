// Attention over the 4-bit K/V cache for many query rows (a chunk of a prompt,
// drafted tokens times the query heads of a K/V head): 128 or 256 rows a CTA on
// tcgen05, O = softmax(scale Q K^T) V with K and V expanded in shared memory.
//
// With this many rows the products no longer fit the time that the codes take
// to arrive, so they run on tcgen05, whose operands are 16-bit values: a tile
// of 128 keys (d = 256: 64) is expanded once for all rows of a CTA. The operands
// are f16 for bf16 caches too: f16 has three bits more than bf16, and a power of
// two for each tile (2^eK, 2^eV over its largest |lo|, |lo + 15 s|) takes the
// place of bf16's exponents: the scores are multiplied with 2^eK in fp32, and the
// weights P carry 2^eV. The running reference m follows max_j (score_j + eV), so P
// stays below 2^8 and the accumulators have one scale.
//   K: an error of a score is one of its weight, and of the log-sum-exp, so K is
//      not rounded: K = mid + s (u - 8), mid = lo + 8 s, and the operand is
//      s (u - 8), which fits f16's 11 bits for the 8 bits of a bf16 s; an f16 s is
//      cut into 8 bits and the rest, two operands (the chunk below: 222 -> 269 us).
//      mid meets only the sums of q over its group: a product of 16 columns (32
//      for d = 256), mid and the sums as two f16 terms each.
//   V^ = lo + s u is rounded once to f16, 2^-11 relative (of elements below 2^-22
//      of a tile's largest: 2^-25 of 2^-15 of that), and P for bf16 caches, whose
//      outputs are rounded to eight bits; for f16 P has two terms (269 -> 313 us;
//      O is off by 0.00028 relative against 0.00034, 0.00021 of it its own rounding).
//
// The order of the operands is that in which the cache holds its codes, so
// that they are stored to shared memory as they come out of the words:
//   K tile   [128 slots][d], K-major: a word's 8 channels are stored in the
//            order 0 4 1 5 2 6 3 7, and Q's alike;
//   V^T tile [d][128 slots], K-major: a word holds the two neighbouring slots,
//            and four words a 16-byte piece of a channel's row;
//   the columns of S and P are slots (cell_token gives their tokens).
//
// CTA: 20 warps, one CTA an SM, pieces of the axis of work as in
// fa_cache_fwd.cu (the same units, scratch and merge):
//   warp 0        bulk copies of cells into a ring of two tiles
//   warp 1        tcgen05 issuer (one lane) and tensor-memory owner
//   warps 4-7     softmax and output, t = 0 (thread = row = TMEM lane)
//   warps 8-11    softmax and output, t = 1
//   warps 12-15   expansion of K
//   warps 16-19   expansion of V
// The two softmax warpgroups take turns with the tensor cores, either (kNT = 2,
// more than 128 rows a K/V head) on 128 rows each, which share every expanded
// tile, or (kNT = 1) on the same 128 rows and every second tile of keys each,
// with an m, l and O of their own that they merge at the end. With d = 256 there
// is tensor memory for one O only, and the second warpgroup is idle.
// Tensor memory: S_t [128 t, +128), P_t over the first 64 of these columns (f16: all)
// once they have been read, O_t [256 + t d, +d). The issue order P_t V, next S_t, per
// t, makes the completion of S_t tell that O_t and P_t are free.
//
// NaN. A group of V with a non-finite element reads as NaN, but 0 times NaN
// would spread it to rows that do not see its token. So it enters V^ as 0,
// and rows that see the token remember the group and put NaN in its channels
// at the end. A NaN in K needs no such care: hidden scores are overwritten.
// Measured (GB300): 2 sequences of 9000 and 16384 keys, 1024 new tokens each, 16
// query heads on 4, d = 128: 222 us, with the merge 232 us a call (the kernel for few
// rows: 1020 us), 0.96 PFLOP/s. A tile of 128 keys for 256 rows takes 2 us: two
// expansions side by side and two softmaxes share the schedulers. What a piece
// needs besides its tiles, about 10 us the first time, was as much in fetching
// instructions that run once as in their work: their loops are kept short.
// d = 256, 2 sequences of 6000 and 9000 keys, 2048 rows on each of 2 heads: 121 us
// (f16 170 us; the kernel for few rows 359 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_work.cuh"

namespace fa {
namespace {

constexpr int kThreads = 640;
// registers a thread: at the launch, and after the warpgroups have moved them
// (the softmax holds 32 scores of a row at a time and reads them twice, for the
// maximum and for P; the output's rows are 32 columns at a time too)
constexpr int kRegsLaunch = 96, kRegsIssue = 48, kRegsSoftmax = 128, kRegsExpand = 88;
static_assert(kRegsIssue + 2 * kRegsSoftmax + 2 * kRegsExpand == 5 * kRegsLaunch, "register split");
static_assert(kRegsLaunch * kThreads <= 65536, "registers of an SM");
constexpr int kRows = 128;
// Keys of a tile: with d = 256, twice as many would not fit the shared memory.
constexpr int tile_keys(int d) { return d == 256 ? 64 : 128; }
constexpr float kRescaleThreshold = 8.0f;  // log2: m moves when P would pass 2^8

template <int D, int kNT, int kTerms>
struct TcLayout {
  static constexpr int kG = D / 32;
  static constexpr int kKeys = tile_keys(D);
  static constexpr int kChunks = (D + 63) / 64;         // 64-channel chunks of a Q or K row
  static constexpr int kQBytes = kChunks * kRows * 128;  // 128 rows of 128 bytes a chunk
  static constexpr int kKBytes = kChunks * kKeys * 128;  // of one term
  // the groups' sums: 32 bytes a row of Q or K, or 64
  static constexpr int kXGroups = kG <= 4 ? 4 : 8, kXBytes = kG <= 4 ? 32 : 64;
  static constexpr int kVChunk = D * 128;               // D rows of 64 slots
  static constexpr int kVBytes = kKeys / 64 * kVChunk;
  static constexpr int kPacked = kKeys / kCellTokens * cell_bytes(D);
  static constexpr int kQ = 0;
  // Buffers of K and V tiles: with 256 rows there is room for three. K's is free
  // as soon as both S have been issued, V's only after both P V, a step later
  // (measured with one of V and two of K: 2.5 us a tile, the expansion of V waiting
  // for the products and they for it). With two terms of K, one of V at d = 128.
  static constexpr int kKBufs = kNT == 2 || D == 256 || kTerms == 2 ? 1 : 2;
  static constexpr int kK = kQ + kNT * kQBytes;           // (kNT = 1: the merge's O later)
  static constexpr int kV = kK + kKBufs * kTerms * kKBytes;
  static constexpr int kVBufs = kTerms == 2 && kNT * D >= 256 ? 1 : 2;
  static constexpr int kRing = kV + kVBufs * kVBytes;     // two tiles of cells
  static constexpr int kQx = kRing + 2 * kPacked;         // sums of Q, and the middles of K
  static constexpr int kKx = kQx + kNT * kRows * kXBytes;
  static constexpr int kMetaK = kKx + kKBufs * kKeys * kXBytes;  // [g][slot]: s's terms in f16, twice
  static constexpr int kMetaV = kMetaK + kKeys * kG * 8;  // [cell][y][g][t]: s, then lo, of two slots
  static constexpr int kVLo = kMetaV + kKeys / 2 * kG * 4;
  static constexpr int kNan = kVLo + kKeys / 2 * kG * 4;  // [4][128] groups of V that are NaN
  static constexpr int kScales = kNan + 4 * 128;          // [4]: 2^eK, 2^eV, 2^-eV, eV
  static constexpr int kFlags = kScales + 4 * 16;         // [4] any NaN, [4] found cells, reductions
  static constexpr int kRowScale = kFlags + 32 + 48;      // [128] of the query rows (turns)
  static constexpr int kBars = kRowScale + 4 * kRows;
  static constexpr int kNumBars = 22;
  static constexpr int kTmem = kBars + kNumBars * 8;
  static constexpr int kMisc = (kTmem + 8 + 15) / 16 * 16;
  static constexpr int kBytes = kMisc + kWorkBytes;
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 B
  static_assert(kAlloc <= 232448, "shared memory budget");
  static_assert(kBars % 8 == 0 && kRing % 128 == 0 && kV % 1024 == 0, "alignment");
};

struct TcBars {
  uint32_t base;
  __device__ uint32_t packed_full(int s) const { return base + 8 * s; }
  __device__ uint32_t packed_empty(int s) const { return base + 8 * (2 + s); }
  __device__ uint32_t k_full(int s) const { return base + 8 * (4 + s); }
  __device__ uint32_t k_free(int s) const { return base + 8 * (6 + s); }
  __device__ uint32_t v_full(int s) const { return base + 8 * (8 + s); }
  __device__ uint32_t v_free(int s) const { return base + 8 * (10 + s); }
  __device__ uint32_t v_scale(int s) const { return base + 8 * (12 + s); }  // eV is known
  __device__ uint32_t s_full(int t) const { return base + 8 * (14 + t); }
  __device__ uint32_t p_full(int t) const { return base + 8 * (16 + t); }
  __device__ uint32_t pv_done(int t) const { return base + 8 * (18 + t); }
  __device__ uint32_t q_full() const { return base + 8 * 20; }
  __device__ uint32_t teardown() const { return base + 8 * 21; }
};

enum TcRole : uint32_t { kRoleLoad = 1, kRoleMma = 2, kRoleSoftmax = 3, kRoleExpand = 4 };
constexpr uint32_t code(uint32_t role, uint32_t site) {
  return status_code(kKernCacheFwdTc, role, site);
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  st_shared_v4(a, x, y, z, w);
}
// Copies 16 bytes (`bytes` = 0: writes zeros), without waiting.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)x) : "memory");
}

// lo + s u of the four pairs of codes of a word (nibble p of either half), with
// s and lo for the two halves: u is made by joining the bits to 1024 (in the
// second place 1024 + 16 u), both exact, and the result is rounded once.
template <int kPair>
__device__ __forceinline__ uint32_t expand(uint32_t w, uint32_t s2, uint32_t lo2) {
  if constexpr (kPair >= 2) w >>= 8;
  uint32_t u;
  if constexpr (kPair & 1)
    u = hfma2((w & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd400d400u);  // / 16, - 64
  else
    u = hadd2((w & 0x000f000fu) | 0x64006400u, 0xe400e400u);               // - 1024
  return hfma2(u, s2, lo2);
}

// u - 8 of the four pairs of codes of a word, exact.
template <int kPair>
__device__ __forceinline__ uint32_t centred(uint32_t w) {
  if constexpr (kPair >= 2) w >>= 8;
  if constexpr (kPair & 1)
    return hfma2((w & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd480d480u);  // / 16, - 72
  else
    return hadd2((w & 0x000f000fu) | 0x64006400u, 0xe408e408u);               // - 1032
}

// A barrier of kCount threads, and whether all of them are well: they give up
// together, since a warp that left alone would leave the others at it.
template <int kId, int kCount = 128>
__device__ __forceinline__ bool expand_sync(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "n"(kId), "n"(kCount)
      : "memory");
  return all != 0;
}

// The largest x of a warpgroup that expands, through `red` ([4] floats).
template <int kId>
__device__ __forceinline__ float expand_max(float x, volatile float *red, int dw) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) red[dw] = x;
  expand_sync<kId>(true);
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// Bits of the 16 slots of a cell whose token is one of the first `tokens`; none
// unless bit 0 of `found` is set. (Slots 0, 2, 4, 6 are tokens 0 - 3, slots 1, 3,
// 5, 7 tokens 4 - 7, and so on: cell_slot.)
__device__ __forceinline__ uint32_t seen_slots(int tokens, uint32_t found) {
  uint32_t bits = 0;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int four = min(max(tokens - 4 * x, 0), 4);
    bits |= ((0x55u >> (8 - 2 * four)) & 0x55u) << ((x & 1) + 8 * (x >> 1));
  }
  return (found & 1u) ? bits : 0u;
}

// The power of two at or below x > 0 times 2^-7, between 2^-120 and 2^120 (1 for 0): what
// brings values up to x below 2^8.
__device__ __forceinline__ int tile_exponent(float x) {
  return x > 0.f ? min(max((int)(__float_as_uint(x) >> 23) - 127 - 7, -120), 120) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <int D, bool kF16, int kNT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_cache_fwd_tc_kernel(const __grid_constant__ CacheFwdParams p) {
  constexpr int kTerms = kF16 ? 2 : 1;
  using L = TcLayout<D, kNT, kTerms>;
  constexpr int kG = L::kG, kKeys = L::kKeys, kTileCells = kKeys / kCellTokens;
  constexpr int kSCols = 128;           // tensor memory columns of S
  constexpr bool kTurns = kNT == 1 && D != 256;  // the softmax warpgroups take turns at the tiles
  // the threads of an expansion hold the groups of a slot, or parts of them
  constexpr int kParts = 128 / kKeys, kGp = kG / kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *const smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const TcBars bars{sb + L::kBars};
  int *const misc = reinterpret_cast<int *>(smem + L::kMisc);
  volatile int *const nan_flag = reinterpret_cast<int *>(smem + L::kFlags);      // [4]
  volatile int *const found_cells = reinterpret_cast<int *>(smem + L::kFlags) + 4;  // [4] bit masks
  volatile float *const red = reinterpret_cast<float *>(smem + L::kFlags + 32);  // [3][4]
  volatile float *const scales = reinterpret_cast<float *>(smem + L::kScales);   // [4][4]
  const StatusSlot st = {p.status, misc, p.wait_limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bars.packed_full(s), 1);
      mbar_init(bars.packed_empty(s), 256);
      mbar_init(bars.k_full(s), 128);
      mbar_init(bars.k_free(s), 1);
      mbar_init(bars.v_full(s), 128);
      mbar_init(bars.v_free(s), 1);
      mbar_init(bars.v_scale(s), 128);
      mbar_init(bars.s_full(s), 1);
      mbar_init(bars.p_full(s), 128);
      mbar_init(bars.pv_done(s), 1);
    }
    mbar_init(bars.q_full(), kNT * 128);
    mbar_init(bars.teardown(), 1);
    misc[0] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + L::kTmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  constexpr int kBlockRows = kNT * kRows;
  const Blocks blocks{p, (p.nq * p.group + kBlockRows - 1) / kBlockRows, kBlockRows};
  const Share mine = find_share<kThreads>(p, blocks, misc);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kTmem);
  const int heads = p.pool.heads;

  // Every role walks over the same pieces, tiles [piece.t0, piece.t0 + count) of
  // a segment; tile0 counts the tiles before a piece (buffers and parities), tile1
  // those of them in which the second 128 rows took part.
  // work(piece, count, tile0, tile1, pieces) ends with the barrier of all threads.
  int4 chain = make_int4(-1, 0, 0, 0);
  bool failed = false;
  auto has_second = [&](const Piece &piece) {
    return kNT == 2 && piece.row0 + kRows < p.nq * p.group;
  };
  auto walk = [&](auto work) {
    long long f = mine.f;
    uint32_t tile0 = 0, tile1 = 0, pieces = 0;
    while (mine.found && f < mine.f_end) {
      const Piece piece(p, blocks, misc, f, mine.f_end);
      if (piece.h < 0 || piece.h >= heads) break;
      constexpr int kPerUnit = kUnitTokens / kKeys;
      const int count = max(0, min(piece.t1 * kPerUnit, (piece.cells + kTileCells - 1) / kTileCells) -
                                   piece.t0 * kPerUnit);
      work(piece, count, tile0, tile1, pieces);
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      failed = *reinterpret_cast<volatile int *>(misc) != 0;
      if (failed) break;
      piece.link(chain, pieces == 0);
      tile0 += count;
      if (has_second(piece)) tile1 += count;
      ++pieces;
      f = piece.next(p);
      if (!piece.advance(p, blocks, misc, f)) break;
      __syncthreads();
    }
  };

  if (warp < 4) {
    setmaxnreg_dec<kRegsIssue>();
    walk([&](const Piece &piece, int count, uint32_t tile0, uint32_t tile1, uint32_t pieces) {
      const int cells = piece.cells, cell0 = piece.t0 * (kUnitTokens / kCellTokens);
    if (warp == 0) {
      // ---- copies ----------------------------------------------------------
      const int32_t *const table = p.pool.table + (size_t)((long long)piece.b * p.pool.table_stride);
      const bool one_copy = p.pool.page_cells % kTileCells == 0;
      auto page_of = [&](int k) {  // of this lane's cell of tile k
        const int c = cell0 + k * kTileCells + lane;
        return lane < kTileCells && k < count && c < cells ? table[p.pool.by_page_cells.div(c)] : -1;
      };
      int page = page_of(0);
      bool ok = true;
      int issued = 0;
      for (; issued < count; ++issued) {
        const uint32_t i = tile0 + issued;
        const int slot = i & 1;
        const int ahead = page_of(issued + 1);
        ok = __all_sync(0xffffffffu, mbar_wait_inl(bars.packed_empty(slot), ((i >> 1) & 1) ^ 1, st,
                                                   code(kRoleLoad, 1)));
        if (!ok || (p.debug_flags & kDebugSkipLoads)) break;
        const int c = cell0 + issued * kTileCells + lane;
        const bool wanted = lane < kTileCells && c < cells;
        const bool here = wanted && p.pool.page_ok(page);
        if (wanted && !here) atomicCAS(p.status, 0u, index_code(kKernCacheFwd, 2));
        const uint32_t found = __ballot_sync(0xffffffffu, here);
        // (one page: all cells of the tile are there, those behind the sequence too)
        const uint32_t bytes = one_copy ? (found ? (uint32_t)L::kPacked : 0u)
                                        : __popc(found) * cell_bytes(D);
        if (lane == 0) {
          found_cells[i & 3] = (int)found;
          mbar_arrive_expect_tx(bars.packed_full(slot), bytes);
        }
        __syncwarp();
        if (one_copy ? lane == 0 && found : here)
          bulk_load_1d(sb + L::kRing + slot * L::kPacked + lane * cell_bytes(D),
                       p.pool.template cell_ptr<D>(
                           page, piece.h, c - p.pool.by_page_cells.div(c) * p.pool.page_cells),
                       one_copy ? bytes : (uint32_t)cell_bytes(D), bars.packed_full(slot));
        page = ahead;
      }
      if (!(p.debug_flags & kDebugSkipLoads))  // every copy issued lands before the piece ends
        for (int k = max(0, issued - 2); k < issued; ++k)
          mbar_wait_drain_inl(bars.packed_full((tile0 + k) & 1), ((tile0 + k) >> 1) & 1, st,
                              code(kRoleLoad, 2));
      __syncwarp();
    } else if (warp == 1) {
      // ---- tcgen05 issuer --------------------------------------------------
      if (elect_one() && count > 0) {
        constexpr uint32_t kIdS = idesc_f32acc(kRows, kKeys, 0, 0, true);
        constexpr uint32_t kIdPV = idesc_f32acc(kRows, D, 0, 0, true);
        const bool two = has_second(piece);
        // (a descriptor's low bits are the address in units of 16 bytes)
        const uint64_t q_desc = sdesc_sw128(sb + L::kQ, 16, 1024);
        const uint64_t k_desc = sdesc_sw128(sb + L::kK, 16, 1024);
        const uint64_t v_desc = sdesc_sw128(sb + L::kV, 16, 1024);
        const uint64_t qx_desc = sdesc_plain(sb + L::kQx, 128, 8 * L::kXBytes);
        const uint64_t kx_desc = sdesc_plain(sb + L::kKx, 128, 8 * L::kXBytes);
        auto issue_s = [&](int t, uint32_t i) {
          const uint64_t q = q_desc + (kNT == 2 ? t : 0) * (L::kQBytes >> 4);
          const uint64_t k = k_desc + (i % L::kKBufs) * (kTerms * L::kKBytes >> 4);
          const uint64_t qx = qx_desc + (kNT == 2 ? t : 0) * (kRows * L::kXBytes >> 4);
          const uint64_t kx = kx_desc + (i % L::kKBufs) * (kKeys * L::kXBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < L::kXBytes / 32; ++kk)
            mma_f16kind_ss(tmem + t * kSCols, qx + kk * 16, kx + kk * 16, kIdS, kk > 0);
#pragma unroll 1
          for (int term = 0; term < kTerms; ++term)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int q_off = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
              const int k_off = ((kk >> 2) * (kKeys * 128) + (kk & 3) * 32) >> 4;
              mma_f16kind_ss(tmem + t * kSCols, q + q_off, k + term * (L::kKBytes >> 4) + k_off,
                             kIdS, 1u);
            }
          mma_commit(bars.s_full(t));
        };
        auto issue_pv = [&](int t, uint32_t i, bool first) {
          const uint64_t v = v_desc + (i % L::kVBufs) * (L::kVBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
#pragma unroll
            for (int term = 0; term < kTerms; ++term)
              mma_f16kind_ts(tmem + 256 + t * D,
                             tmem + t * kSCols +
                                 (kTerms == 1 ? kk * 8 : (kk >> 1) * 32 + (kk & 1) * 8 + term * 16),
                             v + (((kk >> 2) * L::kVChunk + (kk & 3) * 32) >> 4), kIdPV,
                             (!first || kk > 0 || term > 0) ? 1u : 0u);
          mma_commit(bars.pv_done(t));
        };
        auto k_here = [&](uint32_t i) {
          const bool here = mbar_wait_inl(bars.k_full(i % L::kKBufs), (i / L::kKBufs) & 1, st,
                                          code(kRoleMma, 2));
          tc_fence_after();
          return here;
        };
        bool ok = mbar_wait_inl(bars.q_full(), pieces & 1, st, code(kRoleMma, 1)) && k_here(tile0);
        if constexpr (!kTurns) {
          if (ok) {
            issue_s(0, tile0);
            if (two) issue_s(1, tile0);
            mma_commit(bars.k_free(0));
          }
          for (int k = 0; k < count && ok; ++k) {
            const uint32_t i = tile0 + k;
            const bool more = k + 1 < count;
            ok = mbar_wait_inl(bars.v_full(i & 1), (i >> 1) & 1, st, code(kRoleMma, 3));
            for (int t = 0; t < (two ? 2 : 1) && ok; ++t) {
              ok = mbar_wait_inl(bars.p_full(t), (t ? tile1 + k : i) & 1, st, code(kRoleMma, 4 + t));
              if (!ok) break;
              tc_fence_after();
              issue_pv(t, i, k == 0);
              if (!more) continue;
              ok = t > 0 || k_here(i + 1);
              if (ok) issue_s(t, i + 1);
            }
            if (!ok) break;
            mma_commit(bars.v_free(i & 1));
            if (more) mma_commit(bars.k_free(0));
          }
        } else {
          // S of tile i for the t whose turn it is
          auto issue_turn = [&](uint32_t i) {
            issue_s(i & 1, i);
            mma_commit(bars.k_free(i % L::kKBufs));
          };
          if (ok) issue_turn(tile0);
          if (ok && count > 1) {
            ok = k_here(tile0 + 1);
            if (ok) issue_turn(tile0 + 1);
          }
          for (int k = 0; k < count && ok; ++k) {
            const uint32_t i = tile0 + k;
            const int t = i & 1;
            ok = mbar_wait_inl(bars.v_full(t), (i >> 1) & 1, st, code(kRoleMma, 3)) &&
                 mbar_wait_inl(bars.p_full(t), (i >> 1) & 1, st, code(kRoleMma, 4));
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, i, k < 2);
            mma_commit(bars.v_free(t));
            if (k + 2 < count) {
              ok = k_here(i + 2);
              if (ok) issue_turn(i + 2);
            }
          }
        }
        if (!ok) {  // gave up: what was issued ends before the tensor memory goes
          mma_commit(bars.teardown());
          mbar_wait_drain_inl(bars.teardown(), 0, st, code(kRoleMma, 7));
        }
      }
      __syncwarp();
    }
    });
  } else if (warp >= 12) {
    setmaxnreg_dec<kRegsExpand>();
    const int dt = threadIdx.x & 127, dw = warp & 3;
    if (warp < 16) {
      // ---- expansion of K ---------------------------------------------------
      walk([&](const Piece &piece, int count, uint32_t tile0, uint32_t, uint32_t) {
        bool ok = true;
        for (int k = 0; k < count; ++k) {
          const uint32_t i = tile0 + k;
          const int slot2 = i & 1;
          const uint32_t parity = (i >> 1) & 1;
          const uint32_t ring = sb + L::kRing + slot2 * L::kPacked;
          ok = expand_sync<1>(
              ok && mbar_wait_inl(bars.packed_full(slot2), parity, st, code(kRoleExpand, 1)));
          if (!ok) break;
          const uint32_t found = (uint32_t)found_cells[i & 3];
          uint32_t mid[4] = {0, 0, 0, 0};  // the groups' middles: four f16, and what they lack
          {
            // s and lo of a slot's groups g0 .. g0 + kGp - 1
            const int own = dt % kKeys, g0 = dt / kKeys * kGp, cell = own >> 4;
            const uint32_t at = ring + cell * cell_bytes(D) + k_lo<D>(own & 15, g0);
            float s[kGp], lo[kGp];
            uint32_t w[kGp];  // kGp lo, then kGp s, in pairs
            if constexpr (kG == 3) {
              lds_words<3>(at, w);
              unpack2<kF16>(w[0], lo[0], lo[1]);
              unpack2<kF16>(w[1], lo[2], s[0]);
              unpack2<kF16>(w[2], s[1], s[2]);
            } else {
              if constexpr (kParts == 1) {
                lds_words<kGp>(at, w);
              } else {
                lds_words<kGp / 2>(at, w);
                lds_words<kGp / 2>(at + D / 16, w + kGp / 2);
              }
#pragma unroll
              for (int x = 0; x < kGp / 2; ++x) {
                unpack2<kF16>(w[x], lo[2 * x], lo[2 * x + 1]);
                unpack2<kF16>(w[kGp / 2 + x], s[2 * x], s[2 * x + 1]);
              }
            }
            const bool live = ((found >> cell) & 1) &&
                              piece.t0 * kUnitTokens + k * kKeys + cell * kCellTokens +
                                      cell_token(own & 15) <
                                  piece.vis;
            float top = 0.f;
#pragma unroll
            for (int g = 0; g < kGp; ++g) {
              if (!live) s[g] = lo[g] = 0.f;
              // (a NaN does not enter the maximum)
              top = fmaxf(top, fmaxf(fabsf(lo[g]), fabsf(fmaf(15.f, s[g], lo[g]))));
            }
            const int e = tile_exponent(expand_max<1>(top, red, dw));
            const float down = pow2(-e);
#pragma unroll
            for (int g = 0; g < kGp; ++g) {
              const uint32_t at_s = sb + L::kMetaK + ((g0 + g) * kKeys + own) * (4 * kTerms);
              const uint32_t s2 = pack_f16x2(s[g] * down, s[g] * down);
              if constexpr (kTerms == 2) {  // 8 bits, and the rest
                const uint32_t high = s2 & 0xfff8fff8u;
                sts64(at_s, high, hadd2(s2, high ^ 0x80008000u));
              } else {
                sts32(at_s, s2);
              }
            }
#pragma unroll
            for (int x = 0; x < (kGp + 1) / 2; ++x) {
              float m0 = fmaf(8.f, s[2 * x], lo[2 * x]) * (down * 64.f), m1 = 0.f, h0, h1;
              if (2 * x + 1 < kGp) m1 = fmaf(8.f, s[2 * x + 1], lo[2 * x + 1]) * (down * 64.f);
              mid[x] = pack_f16x2(m0, m1);
              unpack2<true>(mid[x], h0, h1);
              mid[2 + x] = pack_f16x2(m0 - h0, m1 - h1);
            }
            if (dt == 0) scales[(i & 3) * 4] = pow2(e);
          }
          // the buffer that S of an earlier tile has read
          ok = expand_sync<1>(
              mbar_wait_inl(bars.k_free(i % L::kKBufs), ((i / L::kKBufs) & 1) ^ 1, st,
                            code(kRoleExpand, 2)));
          if (!ok) break;
          {
            const int own = dt % kKeys, part = dt / kKeys;
            const uint32_t at = sb + L::kKx + (i % L::kKBufs) * (kKeys * L::kXBytes) +
                                (own >> 3) * (8 * L::kXBytes) + (own & 7) * 16;
            if constexpr (L::kXGroups == 4) {
              sts128(at, mid[0], mid[1], mid[0], mid[1]);
              sts128(at + 128, mid[2], mid[3], 0u, 0u);
            } else {
              sts64(at + part * 8, mid[0], mid[1]);
              sts64(at + 128 + part * 8, mid[0], mid[1]);
              sts64(at + 256 + part * 8, mid[2], mid[3]);
              sts64(at + 384 + part * 8, 0u, 0u);
            }
          }
          const uint32_t dst = sb + L::kK + (i % L::kKBufs) * (kTerms * L::kKBytes);
          // eight lanes that load and store together: the four t, and two slots that
          // differ in bit 0 (words of other banks) and in bit 2 (pieces of other banks)
          const int t = lane & 3, low = (lane >> 3) ^ (((lane >> 2) & 1) * 5);
          // (loops of the roles stay rolled: together they are more code than the
          // instruction cache holds; measured 12 % on a chunk of 1024 tokens)
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            constexpr int kEights = kKeys / 32;  // of slots a warp
            const int slot = (dw * kEights + x % kEights) * 8 + low, g0 = x / kEights * kGp;
            uint32_t w[kGp];
            lds_words<kGp>(ring + (slot >> 4) * cell_bytes(D) + k_word<D>(slot & 15, t, g0), w);
#pragma unroll
            for (int y = 0; y < kGp; ++y) {
              const int g = g0 + y;
              uint32_t s2[2];
              if constexpr (kTerms == 2)
                lds64(sb + L::kMetaK + (g * kKeys + slot) * 8, s2[0], s2[1]);
              else
                s2[0] = lds32(sb + L::kMetaK + (g * kKeys + slot) * 4);
              const int block = (g & 1) * 4 + t;
              const uint32_t v0 = centred<0>(w[y]), v1 = centred<1>(w[y]);
              const uint32_t v2 = centred<2>(w[y]), v3 = centred<3>(w[y]);
#pragma unroll
              for (int term = 0; term < kTerms; ++term)
                sts128(dst + term * L::kKBytes + (g >> 1) * (kKeys * 128) + slot * 128 +
                           ((block ^ (slot & 7)) << 4),
                       hmul2(v0, s2[term]), hmul2(v1, s2[term]), hmul2(v2, s2[term]),
                       hmul2(v3, s2[term]));
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(bars.k_full(i % L::kKBufs));
          mbar_arrive(bars.packed_empty(slot2));
        }
      });
    } else {
      // ---- expansion of V ---------------------------------------------------
      walk([&](const Piece &piece, int count, uint32_t tile0, uint32_t, uint32_t) {
        bool ok = true;
        for (int k = 0; k < count; ++k) {
          const uint32_t i = tile0 + k;
          const int slot2 = i & 1;
          const uint32_t parity = (i >> 1) & 1;
          const uint32_t ring = sb + L::kRing + slot2 * L::kPacked;
          // the cells, and the buffer that P V of two tiles ago has read (whose
          // softmax has then seen its own scales: their barrier has two places)
          ok = expand_sync<2>(
              ok && mbar_wait_inl(bars.packed_full(slot2), parity, st, code(kRoleExpand, 3)) &&
              (L::kVBufs == 1 ||
               mbar_wait_inl(bars.v_free(slot2), parity ^ 1, st, code(kRoleExpand, 4))));
          if (!ok) break;
          const uint32_t found = (uint32_t)found_cells[i & 3];
          {
            // s and lo of groups g0 .. of one token: half z of pair (cell, y, t)
            const int own = dt % kKeys, part = dt / kKeys, g0 = part * kGp;
            const int cell = own >> 4, y = (own >> 3) & 1, t = (own >> 1) & 3, z = own & 1;
            const uint32_t at = ring + cell * cell_bytes(D);
            const int token = t + 8 * y + 4 * z;
            const bool live = ((found >> cell) & 1) &&
                              piece.t0 * kUnitTokens + k * kKeys + cell * kCellTokens + token <
                                  piece.vis;
            uint32_t ws[kGp], wl[kGp];
            lds_words<kGp>(at + v_s<D>(y, t, g0), ws);
            lds_words<kGp>(at + v_lo<D>(y, t, g0), wl);
            float s[kGp], lo[kGp], top = 0.f;
            uint32_t nans = 0;
#pragma unroll
            for (int g = 0; g < kGp; ++g) {
              unpack2<kF16>(__byte_perm(ws[g], wl[g], z ? 0x7632 : 0x5410), s[g], lo[g]);
              if (!live) s[g] = lo[g] = 0.f;
              if (!(lo[g] == lo[g])) {
                nans |= 1u << g;
                s[g] = lo[g] = 0.f;
              }
              top = fmaxf(top, fmaxf(fabsf(lo[g]), fabsf(fmaf(15.f, s[g], lo[g]))));
            }
            const bool any_nan = __any_sync(0xffffffffu, nans != 0);
            if (lane == 0) red[8 + dw] = any_nan ? 1.f : 0.f;
            const int e = tile_exponent(expand_max<2>(top, red + 4, dw));
            const float down = pow2(-e);
#pragma unroll
            for (int g = 0; g < kGp; ++g) {
              const uint32_t o = ((((cell * 2 + y) * kG + g0 + g) * 4 + t) * 2 + z) * 2;
              sts16(sb + L::kMetaV + o, pack_f16x2(s[g] * down, 0.f));
              sts16(sb + L::kVLo + o, pack_f16x2(lo[g] * down, 0.f));
            }
            smem[L::kNan + (i & 3) * 128 + part * kKeys + cell * 16 + cell_slot(token)] = (uint8_t)nans;
            if (dt == 0) {
              nan_flag[i & 3] = red[8] + red[9] + red[10] + red[11] > 0.f;
              scales[(i & 3) * 4 + 1] = down;
              scales[(i & 3) * 4 + 2] = (float)e;
            }
          }
          mbar_arrive(bars.v_scale(slot2));
          // (one buffer: P V of the last tile has read it)
          ok = expand_sync<2>(L::kVBufs == 2 ||
                              mbar_wait_inl(bars.v_free(slot2 ^ 1), ((i - 1) >> 1) & 1, st,
                                            code(kRoleExpand, 4)));
          if (!ok) break;
          const uint32_t dst = sb + L::kV + (i % L::kVBufs) * L::kVBytes;
          // eight lanes that store together: four blocks of 8 slots, two r
          const int kb = (lane & 3) | (dw % (kKeys / 32) << 2);  // block of 8 slots: cell * 2 + y
          const int g0 = dw / (kKeys / 32) * kGp;
          const int r = lane >> 2;
          const uint32_t from = ring + (kb >> 1) * cell_bytes(D);
#pragma unroll 1
          for (int gi = 0; gi < kGp; ++gi) {
            // (the four blocks of a warp lie 128-byte rows apart: at different groups
            // their words are in different banks)
            const int g =
                g0 + (kGp == 3 ? (gi + (lane & 3)) % 3 : (gi + (lane & 3)) & (kGp - 1));
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = lds32(from + v_word<D>(kb & 1, t, r, g));
            uint32_t s2[4], lo2[4];
            lds128(sb + L::kMetaV + (kb * kG + g) * 16, s2[0], s2[1], s2[2], s2[3]);
            lds128(sb + L::kVLo + (kb * kG + g) * 16, lo2[0], lo2[1], lo2[2], lo2[3]);
            auto row = [&](auto pair) {  // channel 32 g + 4 r + pair
              constexpr int kPair = decltype(pair)::value;
              const int c = 32 * g + 4 * r + kPair;
              sts128(dst + (kb >> 3) * L::kVChunk + c * 128 + (((kb & 7) ^ (c & 7)) << 4),
                     expand<kPair>(w[0], s2[0], lo2[0]), expand<kPair>(w[1], s2[1], lo2[1]),
                     expand<kPair>(w[2], s2[2], lo2[2]), expand<kPair>(w[3], s2[3], lo2[3]));
            };
            row(std::integral_constant<int, 0>{});
            row(std::integral_constant<int, 1>{});
            row(std::integral_constant<int, 2>{});
            row(std::integral_constant<int, 3>{});
          }
          fence_proxy_async_smem();
          mbar_arrive(bars.v_full(slot2));
          mbar_arrive(bars.packed_empty(slot2));
        }
      });
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    walk([&](const Piece &piece, int count, uint32_t tile0, uint32_t tile1, uint32_t pieces) {
      const int n = piece.n, len = piece.len, vis = piece.vis;
      // keys before `all` are visible to every row that is a token
      const int all = p.causal ? min(vis, len - n + p.by_group.div(piece.row0) + 1) : vis;
      // ---- Q, softmax, output ------------------------------------------------
      const int t = (warp - 4) >> 2, r = threadIdx.x & 127;
      const int tile_row0 = piece.row0 + (kNT == 2 ? t * kRows : 0), row = tile_row0 + r;
      const int tok = p.by_group.div(row), hq = piece.h * p.group + (row - tok * p.group);
      const bool live = tok < n;
      const bool warp_live = p.by_group.div(tile_row0 + (warp & 3) * 32) < n;  // its first row's token
      const bool has_rows = kTurns || t == 0 || has_second(piece);
      const uint32_t own0 = t == 0 ? tile0 : tile1;  // this warpgroup's tiles before (no turns)
      // The row scaled by a power of two, its largest element below 2^11. The rows
      // are copied to where the product reads them and scaled there, each by its own
      // thread: all of it is on its way at once, in little code (code that runs once
      // a piece costs most in fetching it).
      float c_row = 0.f;
      float *const row_scale = reinterpret_cast<float *>(smem + L::kRowScale);
      if (kNT == 2 || t == 0) {
        const uint16_t *const src = static_cast<const uint16_t *>(p.q) +
                                    (live ? p.sq.row(piece.b, hq, tok) : (size_t)0);
        const uint32_t own = sb + L::kQ + (kNT == 2 ? t : 0) * L::kQBytes + r * 128;
        auto at = [&](int x) {
          return own + (x >> 3) * (kRows * 128) + (((x & 7) ^ (r & 7)) << 4);
        };
        // eight lanes copy 128 bytes of a row, four rows at a time
        const uint32_t rows32 = sb + L::kQ + (kNT == 2 ? t : 0) * L::kQBytes + (warp & 3) * 4096;
#pragma unroll 2
        for (int y = 0; y < 8; ++y) {
          const int rr = 4 * y + (lane >> 3);
          const uint16_t *const row_src = reinterpret_cast<const uint16_t *>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), rr));
          const bool row_live = __shfl_sync(0xffffffffu, (int)live, rr);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
            if (c * 8 + (lane & 7) < D / 8)
              cp_async16(rows32 + c * (kRows * 128) + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4),
                         row_src + c * 64 + (lane & 7) * 8, row_live ? 16 : 0);
        }
        cp_async_wait_all();
        __syncwarp();
        uint32_t top2 = 0;  // the largest magnitudes of the even and the odd channels
#pragma unroll 8
        for (int x = 0; x < D / 8; ++x) {
          uint32_t w[4];
          lds128(at(x), w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int y = 0; y < 4; ++y) top2 = max2_nan<kF16>(top2, w[y] & 0x7fff7fffu);
        }
        float big, big1;
        unpack2<kF16>(top2, big, big1);
        const bool finite = big < INFINITY && big1 < INFINITY;
        big = fmaxf(big, big1);
        const int e = max((int)(__float_as_uint(big) >> 23), 11);  // (c_row is a normal number)
        const bool scaled = big > 0.f && finite;
        // (a row with an infinity or a NaN is NaN throughout: so are its scores)
        const float up = scaled ? __uint_as_float((uint32_t)(264 - e) << 23) : 1.f;
        c_row = scaled ? __uint_as_float((uint32_t)(e - 10) << 23) : 1.f;
        // and the sums of its groups, as two f16 terms each, for the middles of K
        const uint32_t sums = sb + L::kQx + (kNT == 2 ? t : 0) * (kRows * L::kXBytes) +
                              (r >> 3) * (8 * L::kXBytes) + (r & 7) * 16;
#pragma unroll
        for (int x = 0; x < L::kXBytes / 16; ++x) sts128(sums + x * 128, 0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int g = 0; g < kG; ++g) {
          float sum = 0.f;
#pragma unroll
          for (int x = 4 * g; x < 4 * g + 4; ++x) {
            uint32_t w[4];
            lds128(at(x), w[0], w[1], w[2], w[3]);
            float q[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              unpack2<kF16>(w[y], q[2 * y], q[2 * y + 1]);
              sum += q[2 * y] * up + q[2 * y + 1] * up;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              w[y] = pack_f16x2(q[y] * up, q[y + 4] * up);
              if (!finite) w[y] = 0x7fff7fffu;
            }
            sts128(at(x), w[0], w[1], w[2], w[3]);
          }
          sum = finite ? sum * 0x1p-6f : 0.f;
          float high, unused;
          const uint32_t sum_high = pack_f16x2(sum, 0.f);
          unpack2<true>(sum_high, high, unused);
          auto put = [&](int column, uint32_t x) {
            sts16(sums + (column >> 3) * 128 + (column & 7) * 2, x);
          };
          put(g, sum_high);
          put(L::kXGroups + g, pack_f16x2(sum - high, 0.f));
          put(2 * L::kXGroups + g, sum_high);
        }
        if (kTurns) row_scale[r] = c_row;
        fence_proxy_async_smem();
        mbar_arrive(bars.q_full());
      }
      bool ok = true;
      if (kTurns && t == 1) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait_inl(bars.q_full(), pieces & 1, st, code(kRoleSoftmax, 6)));
        c_row = row_scale[r];
      }
      const int lim = p.causal && live ? len - n + tok + 1 : len;
      const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
      const uint32_t tS = lanes + t * kSCols, tO = lanes + 256 + t * D;
      float m_used = -INFINITY, l = 0.f;
      uint32_t nan_groups = 0;
      bool any = false;
      for (int k = kTurns ? ((tile0 ^ t) & 1) : 0; k < count && has_rows && ok; k += kTurns ? 2 : 1) {
        const uint32_t i = tile0 + k;
        const uint32_t parity = (kTurns ? i >> 1 : own0 + k) & 1;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_inl(bars.s_full(t), parity, st, code(kRoleSoftmax, 1)));
        if (!ok) break;
        tc_fence_after();
        if (!warp_live) {  // no row of this warp is a token: nothing of it is read
          mbar_arrive(bars.p_full(t));
          any = true;
          continue;
        }
        const float ct = c_row * scales[(i & 3) * 4] * p.scale_log2;
        const uint32_t found = (uint32_t)found_cells[i & 3];
        const int key0 = piece.t0 * kUnitTokens + k * kKeys;
        const bool masked = key0 + kKeys > all || found != (1u << kTileCells) - 1;
        const int left = min(lim, vis) - key0;
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int q = 0; q < kKeys / 32; ++q) {
          uint32_t x32[32];
          tmem_ld32(tS + q * 32, x32);
          tmem_wait_ld();
          if (masked) {  // hidden scores become -inf, for the second reading too
            const uint32_t seen = seen_slots(left - q * 32, found >> (2 * q)) |
                                  seen_slots(left - q * 32 - 16, found >> (2 * q + 1)) << 16;
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(seen & (1u << x))) x32[x] = 0xff800000u;
            tmem_st32(tS + q * 32, x32);
          }
#pragma unroll
          for (int x = 0; x < 32; x += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mp[y] = fmax3(mp[y], __uint_as_float(x32[x + 2 * y]),
                            __uint_as_float(x32[x + 2 * y + 1]));
        }
        if (masked) tmem_wait_st();
        ok = __all_sync(0xffffffffu, mbar_wait_inl(bars.v_scale(i & 1), (i >> 1) & 1, st,
                                                   code(kRoleSoftmax, 5)));
        if (!ok) break;
        const float fv = scales[(i & 3) * 4 + 1], ev = scales[(i & 3) * 4 + 2];
        if (nan_flag[i & 3])
          for (int x = 0; x < 128; ++x)
            if ((x % kKeys & ~15) + cell_token(x & 15) < left)
              nan_groups |= (uint32_t)smem[L::kNan + (i & 3) * 128 + x] << (x / kKeys * kGp);
        const float m_tile = fmaf(fmax3(mp[0], mp[1], fmaxf(mp[2], mp[3])), ct, ev);
        const bool need = m_tile > m_used + kRescaleThreshold;
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m_used - m_tile);  // 0 on the first tile (m_used = -inf)
          m_used = m_tile;
        }
        // P = 2^(score - m + eV), over columns of S that have been read twice
        const float sub = ev - (m_used == -INFINITY ? 0.f : m_used);
        const uint64_t ct2 = f2pack(ct, ct), sub2 = f2pack(sub, sub);
        uint64_t sum[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll 1
        for (int q = 0; q < kKeys / 32; ++q) {
          uint32_t x32[32];
          tmem_ld32(tS + q * 32, x32);
          tmem_wait_ld();
          uint32_t pk[16 * kTerms];  // (f16: what the first sixteen lack in the others)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float a, b;
            f2unpack(ffma2(f2pack(__uint_as_float(x32[2 * x]), __uint_as_float(x32[2 * x + 1])), ct2,
                           sub2),
                     a, b);
            a = ex2_approx(a);
            b = ex2_approx(b);
            sum[x & 1] = fadd2(sum[x & 1], f2pack(a, b));
            pk[x] = pack_f16x2(a, b);
            if constexpr (kTerms == 2) {
              float a0, b0;
              unpack2<true>(pk[x], a0, b0);
              f2unpack(fsub2(f2pack(a, b), f2pack(a0, b0)), a, b);
              pk[16 + x] = pack_f16x2(a, b);
            }
          }
          if constexpr (kTerms == 2)
            tmem_st32(tS + 32 * q, pk);
          else
            tmem_st16(tS + 16 * q, pk);
        }
        float la, lb;
        f2unpack(fadd2(sum[0], sum[1]), la, lb);
        l = l * alpha + (la + lb) * fv;  // fv = 2^-eV
        if (any && __any_sync(0xffffffffu, need)) {
          // O *= alpha: P V of this t's previous tile is in it, having been issued
          // before this tile's S
#pragma unroll 1
          for (int q = 0; q < kG; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + q * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
            tmem_st32(tO + q * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bars.p_full(t));
        any = true;
      }
      tmem_wait_st();
      // ---- O / l and the log-sum-exp -------------------------------------------
      if constexpr (!kTurns) {
        if (ok && any)
          ok = __all_sync(0xffffffffu, mbar_wait_inl(bars.pv_done(t), (own0 + count - 1) & 1, st,
                                                     code(kRoleSoftmax, 2)));
        tc_fence_after();
      } else {
        // the last tiles of both warpgroups: O is complete, K's buffers are free
        for (int back = 1; back <= 2 && back <= count && ok; ++back) {
          const uint32_t i = tile0 + count - back;
          ok = __all_sync(0xffffffffu, mbar_wait_inl(bars.pv_done(i & 1), (i >> 1) & 1, st,
                                                     code(kRoleSoftmax, 3)));
        }
        tc_fence_after();
        // t = 1 hands m, l, O and the NaN groups over, [column / 4][row]
        float4 *const hand = reinterpret_cast<float4 *>(smem + L::kK);
        float *const stat = reinterpret_cast<float *>(smem + L::kMetaK);  // [3][row]
        if (t == 1 && ok) {
          stat[r] = any && warp_live ? m_used : -INFINITY;
          stat[kRows + r] = l;
          stat[2 * kRows + r] = __uint_as_float(nan_groups);
          if (any && warp_live) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(tO + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 4; ++x)
                hand[(q * 4 + x) * kRows + r] =
                    make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
            }
          }
        }
        ok = expand_sync<3, 256>(ok);
        if (t == 0 && ok && warp_live) {
          const float m1 = stat[r], l1 = stat[kRows + r];
          nan_groups |= __float_as_uint(stat[2 * kRows + r]);
          const float top = fmaxf(m_used, m1);  // (-inf: no key, or only NaN scores)
          const float w0 = top == m_used ? 1.f : ex2_approx(m_used - top);
          const float w1 = top == m1 ? 1.f : ex2_approx(m1 - top);
          const bool other = count > 1 || !any;  // t = 1 had a tile
          if (other) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(tO + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float4 a = hand[(q * 4 + x) * kRows + r];
                const float b4[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const float own = any ? __uint_as_float(o[4 * x + y]) : 0.f;
                  o[4 * x + y] = __float_as_uint(own * w0 + b4[y] * w1);
                }
              }
              tmem_st16(tO + q * 16, o);
            }
            tmem_wait_st();
            l = (any ? l * w0 : 0.f) + l1 * w1;
          }
          m_used = top;
        }
      }
      if (ok && has_rows && (kNT == 2 || t == 0)) {
        const bool whole = piece.t0 == 0 && piece.t1 == piece.tiles;
        const bool none = count == 0 || !live || l == 0.f;  // sees no key, or is no token
        const float inv = 1.f / l;
        const float lse2 = none ? -INFINITY : m_used + lg2_approx(l);
        const size_t prow = ((size_t)blockIdx.x * 2 + (pieces ? 1 : 0)) * kBlockRows + (row - piece.row0);
        const bool store = tok < p.nq;  // (nothing reads the other rows)
        const size_t at = store && whole ? p.so.row(piece.b, hq, tok) : 0;
        // a lane's row goes through shared memory (Q's, which nothing reads now), 32
        // columns at a time, so that eight lanes store 128 bytes of a row: 32 rows
        // a store would take 32 cycles
        const bool wide = !whole || p.o_f32;
        uint8_t *const to =
            !store   ? nullptr
            : !whole ? reinterpret_cast<uint8_t *>(p.part + prow * D)
                     : static_cast<uint8_t *>(p.o) + at * (p.o_f32 ? 4 : 2);
        const uint32_t mine32 = sb + L::kQ + (kNT == 2 ? t : 0) * L::kQBytes + (warp & 3) * 4096;
        const int piece4 = lane & 7;  // columns 4 piece4 .. of the 32
        uint8_t *row_to[8];           // of rows 4 y + lane / 8
#pragma unroll
        for (int y = 0; y < 8; ++y)
          row_to[y] = reinterpret_cast<uint8_t *>(__shfl_sync(
              0xffffffffu, reinterpret_cast<unsigned long long>(to), 4 * y + (lane >> 3)));
#pragma unroll 1
        for (int q = 0; q < kG; ++q) {
          uint32_t o[32];
          if (count > 0) {
            tmem_ld32(tO + q * 32, o);
            tmem_wait_ld();
          }
          // (a NaN among V's group spoils all of its channels)
          const float by = (nan_groups >> q) & 1 ? __uint_as_float(0x7fffffffu) : inv;
#pragma unroll
          for (int x = 0; x < 32; ++x)
            o[x] = none ? 0u : __float_as_uint(__uint_as_float(o[x]) * by);
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 8; ++x)
            sts128(mine32 + lane * 128 + ((x ^ (lane & 7)) << 4), o[4 * x], o[4 * x + 1],
                   o[4 * x + 2], o[4 * x + 3]);
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = 4 * y + (lane >> 3);
            lds128(mine32 + rr * 128 + ((piece4 ^ (rr & 7)) << 4), o[4 * y], o[4 * y + 1],
                   o[4 * y + 2], o[4 * y + 3]);
          }
          if (wide) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              if (row_to[y])
                reinterpret_cast<uint4 *>(row_to[y])[q * 8 + piece4] =
                    make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          } else {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              if (row_to[y])
                reinterpret_cast<uint2 *>(row_to[y])[q * 8 + piece4] = make_uint2(
                    pack2<kF16>(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1])),
                    pack2<kF16>(__uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3])));
          }
        }
        if (store) {
          if (whole)
            p.lse[((size_t)piece.b * p.hq + hq) * p.nq + tok] = lse2 * kLn2;
          else
            p.part_lse[prow] = lse2;
        }
      }
    });
  }
  if (threadIdx.x == 0 && !p.whole) p.chain[blockIdx.x] = failed ? make_int4(-1, 0, 0, 1) : chain;
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kF16, int kNT>
cudaError_t launch_tc(const CacheFwdParams &p, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // per device
  const cudaError_t e =
      allow_shared_memory(fa_cache_fwd_tc_kernel<D, kF16, kNT>, TcLayout<D, kNT, kF16 ? 2 : 1>::kAlloc, configured);
  if (e != cudaSuccess) return e;
  static const cudaError_t regs = check_kernel_regs(fa_cache_fwd_tc_kernel<D, kF16, kNT>, kRegsLaunch);
  if (regs != cudaSuccess) return regs;
  LaunchProbe probe(kKindCacheFwdTc, stream);
  fa_cache_fwd_tc_kernel<D, kF16, kNT><<<p.ctas, kThreads, TcLayout<D, kNT, kF16 ? 2 : 1>::kAlloc, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tc_rows(const CacheFwdParams &p, cudaStream_t stream) {
  const bool f16 = p.pool.f16 != 0;
  if constexpr (D != 256)
    if (p.block_rows == 256) return f16 ? launch_tc<D, true, 2>(p, stream) : launch_tc<D, false, 2>(p, stream);
  return f16 ? launch_tc<D, true, 1>(p, stream) : launch_tc<D, false, 1>(p, stream);
}

}  // namespace

cudaError_t launch_cache_forward_tc(const CacheFwdParams &p, cudaStream_t stream) {
  switch (p.pool.d) {
    case 64: return launch_tc_rows<64>(p, stream);
    case 96: return launch_tc_rows<96>(p, stream);
    case 128: return launch_tc_rows<128>(p, stream);
    case 256: return launch_tc_rows<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
