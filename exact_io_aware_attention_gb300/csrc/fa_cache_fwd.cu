// Attention over the 4-bit K/V cache: O = softmax(scale Q K^T) V where row j
// of K and V is lo_j + s_j u_j per group of 32 channels.
//
// Mathematics. The groups' s and lo stay out of the matrix products:
//     q . k_j = sum_g  s_jg (sum_{c in g} q_c u_jc) + lo_jg (sum_{c in g} q_c)
//     o_c     = sum_j (p_j s_jg) u_jc  +  sum_j p_j lo_jg          (c in g)
// so the operands of the products are the bare codes u, which an AND turns
// into f16 subnormals u * 2^-24 (or u * 2^-20: the query channels and the
// outputs concerned carry the factor), and s, lo are applied in fp32 to the
// small side: 16 tokens x 8 query rows. The products run S^T = U Q^T and
// O^T = U^T P^T with the tokens and the channels in the 16 rows of an m16n8k16
// product and the query rows in its 8 columns, since a decoding step has few
// query rows (the query heads of one K/V head times the new tokens).
//
// Why register operands and not tcgen05: a decoding step reads each code once
// for at most 16 query rows, so HBM bounds it, and a tcgen05 operand would
// have to pass through shared memory again as 16-bit values, four times the
// bytes; mma.sync takes the expanded codes from the registers they are
// expanded in.
//
// Numbers. Q is scaled per row by a power of two and converted to f16
// (exactly, down to 2^-24 of the row's largest element). The sums of q over
// the groups meet lo in one more product, each split into two or three 16-bit
// terms (2^-17 relative or better). P s is rounded to f16 (2^-11 relative), P~.
// What the codes lose to that rounding shows in a 16-bit f16 result, and for
// f16 they are measured from their middle,
//     o_c = sum_j P~_jg u_jc - 7.5 sum_j P~_jg + sum_j p_j (lo_jg + 7.5 s_jg),
// the sum of P~ from the tensor cores and the last one in fp32. For bf16, whose
// exponents hold any p, sum_j p_j lo_jg goes through the tensor cores with p
// split into two bf16 terms (2^-17). So that P~ neither overflows nor
// underflows whatever the size of V, the running reference m of the softmax
// follows max_j (score_j + log2 |v_j|) and not the maximum score. m, l and all
// sums are fp32. m moves only when p s would pass 2^8 (the result does not
// depend on m), so that a cell costs a vote, no reduction.
//
// Work. The cells of a (query block, K/V head) are one segment; all segments
// lie end to end on one axis, in units of eight cells, and every CTA takes an
// equal share of it, whatever the lengths. (Where the page table holds so few
// tokens that a merge would cost more than it saves, segments stay whole.)
// A CTA's four warps take every fourth pair of cells, each with its own ring of
// bulk copies and its own m, l and O, merged when the CTA leaves the segment. A
// segment within one CTA's share is written out at once; parts of a segment go to scratch and
// fa_cache_combine_kernel merges them in the order of the axis: the results
// do not depend on timing.
// Measured (GB300, ncu): 32 sequences of 1000 .. 16384 keys, 32 query heads on 8,
// d = 128, bf16: 75.6 us for 357 MB (4.7 TB/s, 0.70 of the copy rate). The same
// kernel without the arithmetic takes 62 us, without the copies 77 us at the time:
// what bounds it is the issue of the expansion (0.57 instructions a cycle and
// scheduler, the integer pipe, at half rate, 55 %). A warp more or less per
// scheduler, two cells at a time, or the copies' number in flight change nothing;
// fewer integer instructions do (groups in token pairs, lo through the tensor
// cores: 87 -> 75 us). One sequence of 65536 keys, 16 heads: 36 us and the merge.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "fa_cache.cuh"
#include "fa_cache_work.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
static_assert(kUnitTokens == 2 * kWarps * kCellTokens, "a pair of cells for each warp");
constexpr float kNoMax = -3e38f;   // m before the first visible key
constexpr float kMid = 7.5f;       // the middle of the codes
// m keeps p s below kMaxWeight, and p below kMaxWeight / kSmallStep unless V
// is as small as that; |v| counts from 2^-90 (p and its sum stay finite).
constexpr float kMaxWeight = 256.f, kSmallStep = 0x1p-32f;
constexpr float kMinSize = 0x1p-90f, kMaxSize = 0x1p100f;

// Ring of a warp: pairs of cells in flight, what the SM's shared memory holds
// for its CTAs: 150-200 KB an SM, the bytes in flight that HBM's latency needs.
template <int D, int NT>
constexpr int kStages = (220 * 1024 / cache_forward_ctas_per_sm(D, 8 * NT) - 2048) /
                        (kWarps * 2 * cell_bytes(D));

template <int D, int NT>
struct Layout {
  static constexpr int kNs = kStages<D, NT>;
  static constexpr int kRing = kNs * 2 * cell_bytes(D);
  static constexpr int kOutPitch = D + 4;  // floats: rows 4 banks apart
  static constexpr int kOut = 8 * NT * kOutPitch * 4;  // a warp's outputs reuse its ring
  static constexpr int kWarp = ((kRing > kOut ? kRing : kOut) + 127) / 128 * 128;
  static constexpr int kBars = kWarps * kWarp;                       // [warp][stage] mbarriers
  static constexpr int kStat = kBars + (kWarps * kNs * 8 + 15) / 16 * 16;  // [warp][8 NT] m, then l
  static constexpr int kMisc = kStat + 2 * kWarps * 8 * NT * 4;      // scan and flags
  static constexpr int kBytes = kMisc + kWorkBytes;
  static_assert(kNs >= 2 && kBars % 8 == 0 && kMisc % 16 == 0, "ring and alignment");
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same product of the cache's own type.
template <bool kF16>
__device__ __forceinline__ void mma16816_own(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    mma16816(d, a0, a1, a2, a3, b0, b1);
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NT, bool kF16>
__global__ void __launch_bounds__(kThreads, cache_forward_ctas_per_sm(D, 8 * NT))
    fa_cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  using L = Layout<D, NT>;
  constexpr int kG = D / 32, kNs = L::kNs, kRows = 8 * NT, kF = 1;
  constexpr uint32_t kPairBytes = 2 * cell_bytes(D);
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, t = lane & 3;
  const uint32_t ring = sbase + warp * L::kWarp;
  const uint32_t bars = sbase + L::kBars + warp * kNs * 8;
  float *const stat = reinterpret_cast<float *>(smem + L::kStat);
  int *const misc = reinterpret_cast<int *>(smem + L::kMisc);
  const StatusSlot st = {p.status, misc, p.wait_limit_ns};

  // the merge kernel may be set up meanwhile; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0)
    for (int s = 0; s < kNs; ++s) mbar_init(bars + s * 8, 1);
  if (threadIdx.x == 0) misc[0] = 0;
  fence_mbar_init();

  const Blocks blocks{p, (p.nq * p.group + kRows - 1) / kRows, kRows};
  const int heads = p.pool.heads;

  const Share mine = find_share<kThreads>(p, blocks, misc);
  long long f = mine.f;
  const long long f_end = mine.f_end;
  int4 chain = make_int4(-1, 0, 0, 0);

  uint32_t stage = 0, phase = 0;  // ring position of the next pair to consume
  bool first_piece = true;
  while (mine.found && f < f_end) {
    // ---- the piece: units [t0, t1) of a segment --------------------------
    const Piece piece(p, blocks, misc, f, f_end);
    const int n = piece.n, len = piece.len, vis = piece.vis, h = piece.h, b = piece.b;
    const int row0 = piece.row0, t0 = piece.t0, t1 = piece.t1, cells = piece.cells;
    if (h < 0 || h >= heads) break;
    // this warp's pairs of cells: cells 2 (p0 + 4 k) and the next, k < nk
    const int p0 = t0 * kWarps + warp;
    const int p_end = min(t1 * kWarps, (cells + 1) / 2);
    const int nk = p0 < p_end ? (p_end - p0 + kWarps - 1) / kWarps : 0;

    // This thread's part of the query rows, on its way while the cells are
    // looked up: row r of each n-tile, channels 8 t .. 8 t + 7 of every group.
    uint4 w[NT][kG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 8 + r;
      const int tok = p.by_group.div(row), hq = h * p.group + (row - tok * p.group);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        w[nt][g] = make_uint4(0, 0, 0, 0);
        if (tok < n)
          w[nt][g] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) +
                                                      p.sq.row(b, hq, tok) + g * 32 + t * 8);
      }
    }

    // Places of pair k's cells, as cell numbers of the pool: lane k % 32 looks
    // up those of 32 pairs at a time, a batch ahead. A page holds an even
    // number of cells, and the pair is one copy, or the two are found apart.
    const int32_t *const table = p.pool.table + (size_t)((long long)b * p.pool.table_stride);
    const bool apart = p.pool.page_cells & 1;
    constexpr uint32_t kNoCell = 0xffffffffu;
    bool bad_page = false;  // some page of this piece was not found
    int page0 = 0, page1 = 0;  // pages of the batch ahead
    uint32_t at0 = kNoCell, at1 = kNoCell;
    auto look_up = [&](int k) {
      const int c = 2 * (p0 + kWarps * (k + lane));
      if (k + lane < nk) page0 = table[p.pool.by_page_cells.div(c)];
      if (apart && k + lane < nk && c + 1 < cells) page1 = table[p.pool.by_page_cells.div(c + 1)];
    };
    auto place = [&](int page, int c) {
      if (!p.pool.page_ok(page)) {
        bad_page = true;
        atomicCAS(p.status, 0u, index_code(kKernCacheFwd, 2));
        return kNoCell;
      }
      return ((uint32_t)page * heads + h) * p.pool.page_cells +
             (c - p.pool.by_page_cells.div(c) * p.pool.page_cells);
    };
    auto take_over = [&](int k) {  // the batch ahead, of pairs k + lane
      const int c = 2 * (p0 + kWarps * (k + lane));
      at0 = k + lane < nk ? place(page0, c) : kNoCell;
      at1 = apart && k + lane < nk && c + 1 < cells ? place(page1, c + 1) : kNoCell;
      bad_page = __any_sync(0xffffffffu, bad_page);
    };
    look_up(0);
    take_over(0);
    int issued = 0;
    uint32_t issue_stage = stage;
    auto issue = [&]() {
      const int k = issued;
      if ((k & 31) == 0 && k > 0) {
        take_over(k);
        look_up(k + 32);
      }
      const uint32_t c0 = __shfl_sync(0xffffffffu, at0, k & 31);
      const uint32_t c1 = apart ? __shfl_sync(0xffffffffu, at1, k & 31) : kNoCell;
      if (lane == 0 && !(p.debug_flags & kDebugSkipLoads)) {
        const uint32_t bar = bars + issue_stage * 8, dst = ring + issue_stage * kPairBytes;
        const uint32_t bytes0 = c0 == kNoCell ? 0u : apart ? kPairBytes / 2 : kPairBytes;
        const uint32_t bytes1 = c1 == kNoCell ? 0u : kPairBytes / 2;
        mbar_arrive_expect_tx(bar, bytes0 + bytes1);
        if (bytes0) bulk_load_1d(dst, p.pool.data + (size_t)c0 * cell_bytes(D), bytes0, bar);
        if (bytes1)
          bulk_load_1d(dst + kPairBytes / 2, p.pool.data + (size_t)c1 * cell_bytes(D), bytes1, bar);
      }
      if (++issue_stage == kNs) issue_stage = 0;
      ++issued;
    };
    while (issued < min(nk, kNs)) issue();
    look_up(32);

    // ---- Q as the B operand of S^T -----------------------------------------
    // Of a group's 8 channels: pairs (0,4), (1,5) for the group's first 16-deep
    // product, (2,6), (3,7) for the second; the pairs that meet nibbles 1 and 3 of a
    // half word (codes * 2^-20) are scaled by 2^-4. qs: the sums of q over the
    // groups as the B operand of the product with lo, whose 16 columns are the
    // groups (two, four or eight) repeated, with one term of a sum each.
    constexpr int kGp = kG == 3 ? 4 : kG;
    constexpr float kSumScale = kF16 ? 0x1p-6f : 0x1p-24f;  // f16 has no room for 2^-24
    uint32_t qb[NT][kG][4];
    uint32_t qs[NT][2];
    constexpr bool kThird = D == 256 && !kF16;  // 16 columns hold two terms of eight groups
    [[maybe_unused]] uint32_t qs3[NT];           // (two of bf16: 2^-17, a third 2^-25)
    float c_row[NT][2];      // score = (products * c_row) * (2^24 scale), in log2 units
    int lim[NT][2];          // visible keys of the row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float big = 0.f;
      bool finite = true;
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        float x[8];
        unpack2<kF16>(w[nt][g].x, x[0], x[1]);
        unpack2<kF16>(w[nt][g].y, x[2], x[3]);
        unpack2<kF16>(w[nt][g].z, x[4], x[5]);
        unpack2<kF16>(w[nt][g].w, x[6], x[7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          big = fmaxf(big, fabsf(x[i]));
          finite = finite && fabsf(x[i]) < INFINITY;
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      finite = __shfl_xor_sync(0xffffffffu, (int)finite, 1) && finite;
      finite = __shfl_xor_sync(0xffffffffu, (int)finite, 2) && finite;
      // 2^(e - 127) <= big < 2^(e - 126), e its exponent field: q * up is below 2^11
      const int e = max((int)(__float_as_uint(big) >> 23), 11);  // (back is a normal number)
      const float up = big > 0.f && finite ? __uint_as_float((uint32_t)(264 - e) << 23) : 1.f;
      const float back = big > 0.f && finite ? __uint_as_float((uint32_t)(e - 10) << 23) : 1.f;
      float sum[kGp] = {};
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        float q8[8];
        unpack2<kF16>(w[nt][g].x, q8[0], q8[1]);
        unpack2<kF16>(w[nt][g].y, q8[2], q8[3]);
        unpack2<kF16>(w[nt][g].z, q8[4], q8[5]);
        unpack2<kF16>(w[nt][g].w, q8[6], q8[7]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float a = finite ? q8[x] * up : 0.f, c = finite ? q8[x + 4] * up : 0.f;
          sum[g] += a + c;
          const float f4 = (x & 1) ? 0x1p-4f : 1.f;
          qb[nt][g][x] = pack_f16x2(a * f4, c * f4);
        }
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        // a row with an infinity or a NaN has no finite scores: they become NaN
        sum[g] = finite ? sum[g] * kSumScale : __uint_as_float(0x7fffffffu);
      }
      // column k holds term k / kGp of group k % kGp; this thread's columns
      // are 2 t, 2 t + 1 and the same plus 8
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t word = 0;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const int k = half * 8 + 2 * tt;
          float a = sum[k % kGp], c = sum[(k + 1) % kGp];
          uint32_t pair = 0;
#pragma unroll
          for (int term = 0; term <= k / kGp; ++term) {
            float ra, rc;
            pair = term < 3 ? pack2<kF16>(a, c) : 0u;
            unpack2<kF16>(pair, ra, rc);
            a -= ra;
            c -= rc;
          }
          word = tt == t ? pair : word;
        }
        qs[nt][half] = word;
      }
      if constexpr (kThird) {
        uint32_t word = 0;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          float a = sum[2 * tt], c = sum[2 * tt + 1];
          uint32_t pair = 0;
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            float ra, rc;
            pair = pack2<kF16>(a, c);
            unpack2<kF16>(pair, ra, rc);
            a -= ra;
            c -= rc;
          }
          word = tt == t ? pair : word;
        }
        qs3[nt] = word;
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        c_row[nt][y] = __shfl_sync(0xffffffffu, back, (2 * t + y) * 4);
        const int tk = p.by_group.div(row0 + nt * 8 + 2 * t + y);
        lim[nt][y] = p.causal && tk < n ? len - n + tk + 1 : len;
      }
    }
    // keys before `all` are visible to every row (rows behind the last new
    // token see what they like and are written as zeros)
    const int all = p.causal ? min(vis, len - n + p.by_group.div(row0) + 1) : vis;

    float acc[kG][2][NT][4];  // O^T: channels 32 g + 4 r + 2 half + {0 (c0, c1), 1 (c2, c3)}
    // bf16: row g (c0, c1 of the threads r = g): sum of p lo of group g.
    // f16: row g: sum of P~ of group g; and the sums of p (lo + 7.5 s) over this
    // thread's slots r, r + 8 (a pair)
    float acc_g[NT][4];
    uint64_t acc_lo[NT][2][kF16 ? kG : 1];
    float m[NT][2], l[NT][2];
    const float scale24 = p.scale_log2 * 0x1p24f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        m[nt][y] = kNoMax;
        l[nt][y] = 0.f;
        acc_g[nt][2 * y] = acc_g[nt][2 * y + 1] = 0.f;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          if constexpr (kF16) acc_lo[nt][y][g] = 0;  // (0.f, 0.f)
          acc[g][0][nt][2 * y] = acc[g][0][nt][2 * y + 1] = 0.f;
          acc[g][1][nt][2 * y] = acc[g][1][nt][2 * y + 1] = 0.f;
        }
      }

    // kF cells, in shared memory at `at`, of which the first is cell c of the
    // sequence. kMasked: some of their keys may be hidden from some row.
    auto step = [&](uint32_t at, int c, auto masked_tag) {
      constexpr bool kMasked = decltype(masked_tag)::value;
      float sc[kF][NT][4];              // products, then scores
      float va[kF][kG], vb[kF][kG];     // V's steps s of slots r, r + 8
      int end_of[kF];                   // kMasked: keys of the sequence in the cell end here
      uint32_t vw[kF][2][kG];           // V's codes of slots 2t, 2t + 1, and of 2t + 8, 2t + 9
      // 16-bit steps of one slot, one after the other
      auto load_steps = [&](uint32_t from, float (&s)[kG]) {
        uint32_t w[kG / 2 + 1];
        if constexpr (kG == 3) {  // begins with the high half of a word
          float unused;
          w[0] = lds32(from - 2);
          w[1] = lds32(from + 2);
          unpack2<kF16>(w[0], unused, s[0]);
          unpack2<kF16>(w[1], s[1], s[2]);
        } else {
          if constexpr (kG == 2)
            w[0] = lds32(from);
          else
            lds_words<kG / 2>(from, w);
#pragma unroll
          for (int x = 0; x < kG / 2; ++x) unpack2<kF16>(w[x], s[2 * x], s[2 * x + 1]);
        }
      };
      // s or lo of V's groups, of slots r and r + 8: the halves r % 2 of the
      // words (0, r / 2) and (1, r / 2)
      auto load_own_token = [&](uint32_t from, float (&a)[kG], float (&b2)[kG]) {
        uint32_t w[2][kG];
#pragma unroll
        for (int y = 0; y < 2; ++y) lds_words<kG>(from + (4 * y + (r >> 1)) * (kG * 4), w[y]);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          if constexpr (kF16) {
            float unused;
            unpack2<true>(__byte_perm(w[0][g], 0u, (r & 1) ? 0x4432 : 0x4410), a[g], unused);
            unpack2<true>(__byte_perm(w[1][g], 0u, (r & 1) ? 0x4432 : 0x4410), b2[g], unused);
          } else {
            a[g] = __uint_as_float(__byte_perm(w[0][g], 0u, (r & 1) ? 0x3244 : 0x1044));
            b2[g] = __uint_as_float(__byte_perm(w[1][g], 0u, (r & 1) ? 0x3244 : 0x1044));
          }
        }
      };
      auto load_v = [&](int x2, uint32_t cell) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int sb = 0; sb < (kG + 3) / 4; ++sb)
            lds_words<(kG < 4 ? kG : 4)>(cell + v_word<D>(y, t, r, 4 * sb), vw[x2][y] + 4 * sb);
      };
#pragma unroll
      for (int x2 = 0; x2 < kF; ++x2) {
        const uint32_t cell = at + x2 * cell_bytes(D);
        // S^T: rows = slots r, r + 8; columns = query rows 2t, 2t + 1. First lo
        // times the sums of q: columns 2t, 2t+1 (mod kGp) are two groups
        // (d = 96: what stands in the fourth's place is an s, finite, and meets a 0)
        const uint32_t la = lds32(cell + k_lo<D>(r, 0) + 4 * (t % (kGp / 2)));
        const uint32_t lb = lds32(cell + k_lo<D>(r + 8, 0) + 4 * (t % (kGp / 2)));
        float ks[2][kG];  // K's steps of slots r, r + 8
        load_steps(cell + k_s<D>(r, 0), ks[0]);
        load_steps(cell + k_s<D>(r + 8, 0), ks[1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[x2][nt][x] = 0.f;
          mma16816_own<kF16>(sc[x2][nt], la, lb, la, lb, qs[nt][0], qs[nt][1]);
          if constexpr (kThird)
            mma16816_own<kF16>(sc[x2][nt], la, lb, 0u, 0u, qs3[nt], 0u);
          if constexpr (kF16)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[x2][nt][x] *= 0x1p-18f;
        }
#pragma unroll
        for (int sb = 0; sb < (kG + 3) / 4; ++sb) {
          constexpr int kW = kG < 4 ? kG : 4;
          uint32_t wa[kW], wb[kW];
          lds_words<kW>(cell + k_word<D>(r, t, 4 * sb), wa);
          lds_words<kW>(cell + k_word<D>(r + 8, t, 4 * sb), wb);
#pragma unroll
          for (int x = 0; x < kW; ++x) {
            const int g = 4 * sb + x;
            const uint32_t wa8 = wa[x] >> 8, wb8 = wb[x] >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(d, wa[x] & 0x000f000fu, wb[x] & 0x000f000fu, wa[x] & 0x00f000f0u,
                       wb[x] & 0x00f000f0u, qb[nt][g][0], qb[nt][g][1]);
              mma16816(d, wa8 & 0x000f000fu, wb8 & 0x000f000fu, wa8 & 0x00f000f0u,
                       wb8 & 0x00f000f0u, qb[nt][g][2], qb[nt][g][3]);
              sc[x2][nt][0] = fmaf(ks[0][g], d[0], sc[x2][nt][0]);
              sc[x2][nt][1] = fmaf(ks[0][g], d[1], sc[x2][nt][1]);
              sc[x2][nt][2] = fmaf(ks[1][g], d[2], sc[x2][nt][2]);
              sc[x2][nt][3] = fmaf(ks[1][g], d[3], sc[x2][nt][3]);
            }
          }
        }
        // (rounded before m is taken off: with one rounding for both, a score
        // beyond 2^24 could come out above the m that it set; by two factors, as their
        // product overflows for q beyond 2^116)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; x += 2)
            f2unpack(fmul2(fmul2(f2pack(sc[x2][nt][x], sc[x2][nt][x + 1]),
                                 f2pack(c_row[nt][0], c_row[nt][1])),
                           f2pack(scale24, scale24)),
                     sc[x2][nt][x], sc[x2][nt][x + 1]);
        load_own_token(cell + v_s<D>(0, 0, 0), va[x2], vb[x2]);
        if constexpr (kMasked) {
          const int cc = c + x2;
          const bool there =
              cc < cells && !(bad_page && !p.pool.page_ok(table[p.pool.by_page_cells.div(cc)]));
          // rows behind the sequence may hold anything: s = lo = 0 keeps it out
          const int end = end_of[x2] = there ? vis : 0;
          const int ka = cc * kCellTokens + cell_token(r), kb = ka + 8;
          float lo_a[kG], lo_b[kG];
          load_own_token(cell + v_lo<D>(0, 0, 0), lo_a, lo_b);
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            // bf16: a NaN lo is moved to s, where it meets no row that hides its token
            const float nan = __uint_as_float(0x7fffffffu);
            if (!kF16 && !(lo_a[g] == lo_a[g])) va[x2][g] = nan;
            if (!kF16 && !(lo_b[g] == lo_b[g])) vb[x2][g] = nan;
            va[x2][g] = ka < end ? va[x2][g] : 0.f;
            vb[x2][g] = kb < end ? vb[x2][g] : 0.f;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if ((x < 2 ? ka : kb) >= min(end, lim[nt][x & 1])) sc[x2][nt][x] = -INFINITY;
        }
      }

      float pr[kF][NT][4];
      bool over = false;
      auto weights = [&] {
#pragma unroll
        for (int x2 = 0; x2 < kF; ++x2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              float a, b2;
              f2unpack(fsub2(f2pack(sc[x2][nt][x], sc[x2][nt][x + 1]),
                             f2pack(m[nt][0], m[nt][1])), a, b2);
              pr[x2][nt][x] = ex2_approx(a);
              pr[x2][nt][x + 1] = ex2_approx(b2);
            }
      };
      weights();
#pragma unroll
      for (int x2 = 0; x2 < kF; ++x2) {
        // the largest p times the largest s of this thread's two slots: at
        // least the largest p s, which is what must stay in f16's range
        float top_s = kSmallStep;
#pragma unroll
        for (int g = 0; g < kG; ++g) top_s = fmax3(top_s, va[x2][g], vb[x2][g]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float top_p = fmaxf(fmax3(pr[x2][nt][0], pr[x2][nt][1], pr[x2][nt][2]), pr[x2][nt][3]);
          over = over || top_p * top_s > kMaxWeight;
        }
      }
      if (__any_sync(0xffffffffu, over)) {
        // the sizes of the tokens' values, in log2: steps, and lo as far as it
        // stands out
        float size[kF][2];
#pragma unroll
        for (int x2 = 0; x2 < kF; ++x2) {
          float sa = kMinSize, sb = kMinSize, lo_a[kG], lo_b[kG];
          load_own_token(at + x2 * cell_bytes(D) + v_lo<D>(0, 0, 0), lo_a, lo_b);
#pragma unroll
          for (int g = 0; g < kG; ++g) {  // (a hidden token's lo counts for nothing: its score is -inf)
            sa = fmaxf(sa, fmaxf(va[x2][g], fabsf(lo_a[g]) * 0x1p-10f));
            sb = fmaxf(sb, fmaxf(vb[x2][g], fabsf(lo_b[g]) * 0x1p-10f));
          }
          size[x2][0] = lg2_approx(fminf(sa, kMaxSize));
          size[x2][1] = lg2_approx(fminf(sb, kMaxSize));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = kNoMax;
#pragma unroll
            for (int x2 = 0; x2 < kF; ++x2)
              top = fmaxf(top, fmaxf(sc[x2][nt][y] + size[x2][0], sc[x2][nt][2 + y] + size[x2][1]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float m_new = fmaxf(m[nt][y], top);
            const float corr = ex2_approx(m[nt][y] - m_new);
            const uint64_t corr2 = f2pack(corr, corr);
            m[nt][y] = m_new;
            l[nt][y] *= corr;
            acc_g[nt][y] *= corr;
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              if constexpr (kF16) acc_lo[nt][y][g] = fmul2(acc_lo[nt][y][g], corr2);
              acc[g][0][nt][y] *= corr;
              acc[g][0][nt][2 + y] *= corr;
              acc[g][1][nt][y] *= corr;
              acc[g][1][nt][2 + y] *= corr;
            }
          }
        weights();
      }

#pragma unroll
      for (int x2 = 0; x2 < kF; ++x2) {
        const uint32_t cell = at + x2 * cell_bytes(D);
        uint64_t p2[NT][2];  // the weights of slots r, r + 8 of query row 2t + y
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            p2[nt][y] = f2pack(pr[x2][nt][y], pr[x2][nt][2 + y]);
            l[nt][y] += pr[x2][nt][y] + pr[x2][nt][2 + y];
          }
        load_v(x2, cell);
        [[maybe_unused]] float lo_a[kG], lo_b[kG];  // f16 only
        if constexpr (kF16) {
          load_own_token(cell + v_lo<D>(0, 0, 0), lo_a, lo_b);
          if constexpr (kMasked) {
            const int ka = (c + x2) * kCellTokens + cell_token(r);
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              lo_a[g] = ka < end_of[x2] ? lo_a[g] : 0.f;
              lo_b[g] = ka + 8 < end_of[x2] ? lo_b[g] : 0.f;
            }
          }
        } else {
          // sum of p lo: row g of the product takes lo of group g (rows from kG
          // on go nowhere), p as two bf16 terms, 2^-17 of it or better
          const int row = min(r, kG - 1);
          uint32_t l0 = lds32(cell + v_lo<D>(0, t, 0) + 4 * row);
          uint32_t l8 = lds32(cell + v_lo<D>(1, t, 0) + 4 * row);
          if constexpr (kMasked) {
            // out: tokens behind the sequence, and NaNs, which are in s now
            auto clean = [&](uint32_t w, int tok) {
              float a, b2;
              unpack2<kF16>(w, a, b2);
              const int key = (c + x2) * kCellTokens + tok;
              return (key < end_of[x2] && a == a ? w & 0xffffu : 0u) |
                     (key + 4 < end_of[x2] && b2 == b2 ? w & 0xffff0000u : 0u);
            };
            l0 = clean(l0, t);
            l8 = clean(l8, t + 8);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float *pv = pr[x2][nt];
            const uint32_t h0 = pack_bf16x2(pv[0], pv[1]), h8 = pack_bf16x2(pv[2], pv[3]);
            float a, b2;
            unpack2<false>(h0, a, b2);
            f2unpack(fsub2(f2pack(pv[0], pv[1]), f2pack(a, b2)), a, b2);
            const uint32_t e0 = pack_bf16x2(a, b2);
            unpack2<false>(h8, a, b2);
            f2unpack(fsub2(f2pack(pv[2], pv[3]), f2pack(a, b2)), a, b2);
            const uint32_t e8 = pack_bf16x2(a, b2);
            mma16816_own<false>(acc_g[nt], l0, 0u, l8, 0u, transpose8x8(h0), transpose8x8(h8));
            mma16816_own<false>(acc_g[nt], l0, 0u, l8, 0u, transpose8x8(e0), transpose8x8(e8));
          }
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const uint64_t s2 = f2pack(va[x2][g], vb[x2][g]);
          const uint32_t xa = vw[x2][0][g], xb = vw[x2][1][g];
          const uint32_t xa8 = xa >> 8, xb8 = xb >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w0, w8, y0, y8;
            f2unpack(fmul2(p2[nt][0], s2), w0, w8);
            f2unpack(fmul2(p2[nt][1], s2), y0, y8);
            if constexpr (kMasked && !kF16) {  // a hidden key's p is 0, but its s may be NaN
              w0 = pr[x2][nt][0] == 0.f ? 0.f : w0;
              y0 = pr[x2][nt][1] == 0.f ? 0.f : y0;
              w8 = pr[x2][nt][2] == 0.f ? 0.f : w8;
              y8 = pr[x2][nt][3] == 0.f ? 0.f : y8;
            }
            const uint32_t b0 = transpose8x8(pack_f16x2(w0, y0));
            const uint32_t b1 = transpose8x8(pack_f16x2(w8, y8));
            if constexpr (kF16) {
              const uint64_t mid2 =
                  ffma2(f2pack(kMid, kMid), s2, f2pack(lo_a[g], lo_b[g]));
              // a hidden key's p is 0, but its lo may be NaN
              float m0, m8;
              f2unpack(mid2, m0, m8);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                if constexpr (kMasked)
                  acc_lo[nt][y][g] =
                      fadd2(acc_lo[nt][y][g],
                            f2pack(pr[x2][nt][y] == 0.f ? 0.f : pr[x2][nt][y] * m0,
                                   pr[x2][nt][2 + y] == 0.f ? 0.f : pr[x2][nt][2 + y] * m8));
                else
                  acc_lo[nt][y][g] = ffma2(p2[nt][y], mid2, acc_lo[nt][y][g]);
              }
              mma16816(acc_g[nt], r == g ? 0x3c003c00u : 0u, 0u, r == g ? 0x3c003c00u : 0u, 0u, b0,
                       b1);
            }
            mma16816(acc[g][0][nt], xa & 0x000f000fu, xa & 0x00f000f0u, xb & 0x000f000fu,
                     xb & 0x00f000f0u, b0, b1);
            mma16816(acc[g][1][nt], xa8 & 0x000f000fu, xa8 & 0x00f000f0u, xb8 & 0x000f000fu,
                     xb8 & 0x00f000f0u, b0, b1);
          }
        }
      }
    };

    // ---- the pairs of cells ----------------------------------------------------
    int done = 0;
    for (; done < nk; ++done) {
      if (!__all_sync(0xffffffffu, mbar_wait(bars + stage * 8, phase, st,
                                             status_code(kKernCacheFwd, 1, 1))))
        break;
      const int c = 2 * (p0 + kWarps * done);
      const uint32_t at = ring + stage * kPairBytes;
      if ((c + 2) * kCellTokens > all || bad_page) {
#pragma unroll 1
        for (int x = 0; x < 2; x += kF) step(at + x * cell_bytes(D), c + x, std::true_type{});
      } else {
        // both at once where the registers allow (bf16, d up to 128: 3 % faster)
        if constexpr (kF16 || D == 256) {
#pragma unroll 1
          for (int x = 0; x < 2; x += kF) step(at + x * cell_bytes(D), c + x, std::false_type{});
        } else {
#pragma unroll
          for (int x = 0; x < 2; x += kF) step(at + x * cell_bytes(D), c + x, std::false_type{});
        }
      }
      __syncwarp();  // every lane has read the stage
      if (++stage == kNs) {
        stage = 0;
        phase ^= 1;
      }
      if (issued < nk) issue();
    }
    if (done < nk && !(p.debug_flags & kDebugSkipLoads)) {  // gave up: copies in flight still land
      for (int k = done; k < issued; ++k) {
        mbar_wait_drain(bars + stage * 8, phase, st, status_code(kKernCacheFwd, 1, 2));
        if (++stage == kNs) {
          stage = 0;
          phase ^= 1;
        }
      }
    }

    // ---- merge of the four warps ---------------------------------------------
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nt][y] += __shfl_xor_sync(0xffffffffu, l[nt][y], o);
        }
    float sum_lo[NT][2][kG];  // what the codes' sums lack: the lo terms over all slots
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const float row_g = __shfl_sync(0xffffffffu, acc_g[nt][y], g * 4 + t);
          sum_lo[nt][y][g] = row_g;
          if constexpr (kF16) {
            float a, c;
            f2unpack(acc_lo[nt][y][g], a, c);
            a += c;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            sum_lo[nt][y][g] = a - kMid * row_g;
          }
        }
    float *const out = reinterpret_cast<float *>(smem + warp * L::kWarp);  // [8 NT][kOutPitch]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = nt * 8 + 2 * t + y;
        if (r == 0) {
          stat[warp * kRows + row] = m[nt][y];
          stat[(kWarps + warp) * kRows + row] = l[nt][y];
        }
#pragma unroll
        for (int g = 0; g < kG; ++g)
          *reinterpret_cast<float4 *>(out + row * L::kOutPitch + g * 32 + r * 4) = make_float4(
              fmaf(acc[g][0][nt][y], 0x1p24f, sum_lo[nt][y][g]),
              fmaf(acc[g][0][nt][2 + y], 0x1p20f, sum_lo[nt][y][g]),
              fmaf(acc[g][1][nt][y], 0x1p24f, sum_lo[nt][y][g]),
              fmaf(acc[g][1][nt][2 + y], 0x1p20f, sum_lo[nt][y][g]));
      }
    __syncthreads();
    if (*(volatile int *)misc) {  // a wait gave up: nothing of this piece is written
      if (threadIdx.x == 0 && !p.whole) p.chain[blockIdx.x] = make_int4(-1, 0, 0, 1);
      return;
    }

    const bool whole = t0 == 0 && t1 == piece.tiles;
    const int slot = first_piece ? 0 : 1;
    constexpr int kChunks = D / 4;  // 4 columns a thread
    for (int x = threadIdx.x; x < kRows * kChunks; x += kThreads) {
      const int row = x / kChunks, col = (x - row * kChunks) * 4;
      float mm = kNoMax, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stat[w * kRows + row]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = ex2_approx(stat[w * kRows + row] - mm);
        const float4 a = *reinterpret_cast<const float4 *>(smem + w * L::kWarp +
                                                           (row * L::kOutPitch + col) * 4);
        ll = fmaf(wt, stat[(kWarps + w) * kRows + row], ll);
        o.x = fmaf(wt, a.x, o.x);
        o.y = fmaf(wt, a.y, o.y);
        o.z = fmaf(wt, a.z, o.z);
        o.w = fmaf(wt, a.w, o.w);
      }
      const int tok = p.by_group.div(row0 + row), hq = h * p.group + (row0 + row - tok * p.group);
      const bool none = ll == 0.f || tok >= n;  // sees no key, or is no token
      const float inv = 1.f / ll;
      o = none ? make_float4(0.f, 0.f, 0.f, 0.f)
               : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      const float lse2 = none ? -INFINITY : mm + lg2_approx(ll);
      if (!whole) {
        const size_t prow = ((size_t)blockIdx.x * 2 + slot) * kRows + row;
        *reinterpret_cast<float4 *>(p.part + prow * D + col) = o;
        if (col == 0) p.part_lse[prow] = lse2;
      } else if (tok < p.nq) {
        const size_t at = p.so.row(b, hq, tok) + col;
        if (p.o_f32)
          *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = o;
        else
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at) =
              make_uint2(pack2<kF16>(o.x, o.y), pack2<kF16>(o.z, o.w));
        if (col == 0) p.lse[((size_t)b * p.hq + hq) * p.nq + tok] = lse2 * kLn2;
      }
    }
    piece.link(chain, first_piece);
    first_piece = false;
    f = piece.next(p);
    if (!piece.advance(p, blocks, misc, f)) break;
    fence_proxy_async_smem();  // the next piece's copies overwrite the merge's reads and writes
    __syncthreads();
  }
  if (threadIdx.x == 0 && !p.whole) p.chain[blockIdx.x] = chain;
}

// Merge of the parts of the segments that more than one CTA worked on: blocks
// (x, y) merge the rows of the segment that begins in attention CTA x, if there
// is one:  LSE = log sum_s 2^LSE_s,  O = sum_s 2^(LSE_s - LSE) O_s.
// A thread holds 4 columns; kSub threads share a column's parts, each every
// kSub-th, so that a chain over the whole GPU is a few loads deep.
constexpr int kCombineThreads = 256, kCombineRows = 32;  // blocks of a segment at most

template <int D, int kRows, bool kF16>
__global__ void __launch_bounds__(kCombineThreads)
    fa_cache_combine_kernel(const __grid_constant__ CacheFwdParams p) {
  constexpr int kChunks = D / 4, kSub = kCombineThreads / kChunks;
  __shared__ float4 s_o[kSub][kChunks];
  __shared__ float s_top[kSub], s_sum[kSub];
  __shared__ int s_last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = blockIdx.x;
  const int4 c = p.chain[x];
  if (c.x < 0) return;
  const int row_blocks = (p.nq * p.group + kRows - 1) / kRows;
  const int b = p.by_row_blocks.div(c.x), row0 = (c.x - b * row_blocks) * kRows;
  // the first later CTA in which the segment ends
  if (threadIdx.x == 0) s_last = p.ctas - 1;
  __syncthreads();
  for (int s = x + 1; s < p.ctas; s += kCombineThreads) {
    const int y = s + threadIdx.x;
    if (y < p.ctas && p.chain[y].w != 0) atomicMin(&s_last, y);
    __syncthreads();
    if (s_last < s + kCombineThreads) break;
    __syncthreads();
  }
  const int last = s_last;
  const int sub = threadIdx.x / kChunks, chunk = threadIdx.x - sub * kChunks;

  // every `step`-th part from `from` on: their largest LSE, and sums scaled by it
  float top, sum;
  float4 o;
  auto add_parts = [&](int row, int from, int step) {
    top = -INFINITY;
    sum = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = D == 256 ? 8 : 4;  // (d = 256: 4 sequences of 76 parts 12.4 -> 10.3 us)
    for (int s0 = from; s0 <= last; s0 += kBatch * step) {
      float lse2[kBatch];
      float4 a[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = s0 + i * step;
        const size_t prow = ((size_t)s * 2 + (s == x ? c.z : 0)) * kRows + row;
        lse2[i] = s <= last ? p.part_lse[prow] : -INFINITY;
        a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s <= last) a[i] = *reinterpret_cast<const float4 *>(p.part + prow * D + chunk * 4);
      }
      float high = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) high = fmaxf(high, lse2[i]);
      if (top != -INFINITY) {
        const float corr = ex2_approx(top - high);
        sum *= corr;
        o = make_float4(o.x * corr, o.y * corr, o.z * corr, o.w * corr);
      }
      top = high;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        // (a part without keys counts nothing; a NaN goes on)
        const float w = lse2[i] == -INFINITY ? 0.f : ex2_approx(lse2[i] - top);
        sum += w;
        o = make_float4(fmaf(w, a[i].x, o.x), fmaf(w, a[i].y, o.y), fmaf(w, a[i].z, o.z),
                        fmaf(w, a[i].w, o.w));
      }
    }
  };
  auto store = [&](int row, int tok) {  // 4 columns of the row, by the threads of its chunks
    const int hq = c.y * p.group + (row0 + row - tok * p.group);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t at = p.so.row(b, hq, tok) + chunk * 4;
    if (p.o_f32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    else
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at) =
          make_uint2(pack2<kF16>(o.x * inv, o.y * inv), pack2<kF16>(o.z * inv, o.w * inv));
    if (chunk == 0)
      p.lse[((size_t)b * p.hq + hq) * p.nq + tok] =
          sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * kLn2;
  };

  // Few parts: the threads of a column merge them by themselves, and the kSub
  // sets of threads take rows of their own (a chunk of 1024 tokens, two or three
  // parts each: 47 -> 17 us; 128 rows in 19 parts 16 -> 12 us).
  if (last - x < (kRows >= 128 ? 40 : 4)) {
    if (sub >= kSub) return;
    for (int row = blockIdx.y + sub * gridDim.y; row < kRows; row += kSub * gridDim.y) {
      const int tok = p.by_group.div(row0 + row);
      if (tok >= p.nq) return;  // (nor are the rows behind it tokens)
      add_parts(row, x, 1);
      store(row, tok);
    }
    return;
  }
  for (int row = blockIdx.y; row < kRows; row += gridDim.y) {
    const int tok = p.by_group.div(row0 + row);
    if (tok >= p.nq) return;
    if (sub < kSub) {
      add_parts(row, x + sub, kSub);
      s_o[sub][chunk] = o;
      if (chunk == 0) {
        s_top[sub] = top;
        s_sum[sub] = sum;
      }
    }
    __syncthreads();
    if (sub == 0) {
      top = -INFINITY;
      sum = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kSub; ++i) top = fmaxf(top, s_top[i]);
#pragma unroll
      for (int i = 0; i < kSub; ++i) {
        if (s_sum[i] == 0.f) continue;
        // a NaN among a thread's parts leaves its top finite or at -inf and its sum NaN
        const float w = s_top[i] == -INFINITY ? 1.f : ex2_approx(s_top[i] - top);
        const float4 a = s_o[i][chunk];
        sum = fmaf(w, s_sum[i], sum);
        o = make_float4(fmaf(w, a.x, o.x), fmaf(w, a.y, o.y), fmaf(w, a.z, o.z),
                        fmaf(w, a.w, o.w));
      }
      store(row, tok);
    }
    __syncthreads();
  }
}

template <int D, int kRows, bool kF16>
cudaError_t launch_combine(const CacheFwdParams &p, cudaStream_t stream) {
  // set up while the attention kernel runs (programmatic dependent launch)
  LaunchProbe probe(kKindCacheCombine, stream);
  const long long rows = (long long)p.nq * p.group;
  cudaLaunchConfig_t cfg = {};
  const long long used = rows < kRows ? rows : kRows;
  cfg.gridDim = dim3(p.ctas, (unsigned)(used < kCombineRows ? used : kCombineRows));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_cache_combine_kernel<D, kRows, kF16>, p);
}

template <int D, int NT, bool kF16>
cudaError_t launch_d(const CacheFwdParams &p, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // per device
  cudaError_t e = allow_shared_memory(fa_cache_fwd_kernel<D, NT, kF16>, Layout<D, NT>::kBytes,
                                      configured);
  if (e != cudaSuccess) return e;
  LaunchProbe probe(kKindCacheFwd, stream);
  fa_cache_fwd_kernel<D, NT, kF16><<<p.ctas, kThreads, Layout<D, NT>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool kF16>
cudaError_t launch_t(const CacheFwdParams &all, cudaStream_t stream) {
  CacheFwdParams p = all;
  const int rows = p.block_rows;
  const int row_blocks = (p.nq * p.group + rows - 1) / rows;
  p.by_row_blocks = FastDiv(row_blocks);
  // no more CTAs than shares of sequences as long as the table could have
  const double segments = (double)p.B * row_blocks * p.pool.heads;
  const double shares =
      p.whole ? segments
              : segments * ((p.pool.table_cells * kCellTokens + kUnitTokens - 1) / kUnitTokens) /
                    kMinShare;
  if (shares < (double)p.ctas) p.ctas = (int)shares + 1;
  cudaError_t e;
  if (rows >= 128)
    e = launch_cache_forward_tc(p, stream);
  else if constexpr (D == 256)
    e = launch_d<D, 1, kF16>(p, stream);
  else
    e = rows == 16 ? launch_d<D, 2, kF16>(p, stream) : launch_d<D, 1, kF16>(p, stream);
  if (e != cudaSuccess || p.whole) return e;
  switch (rows) {
    case 8: return launch_combine<D, 8, kF16>(p, stream);
    case 128: return launch_combine<D, 128, kF16>(p, stream);
  }
  if constexpr (D != 256)
    return rows == 16 ? launch_combine<D, 16, kF16>(p, stream)
                      : launch_combine<D, 256, kF16>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_forward(const CacheFwdParams &p, cudaStream_t stream) {
  const bool f16 = p.pool.f16 != 0;
  switch (p.pool.d) {
    case 64: return f16 ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
    case 96: return f16 ? launch_t<96, true>(p, stream) : launch_t<96, false>(p, stream);
    case 128: return f16 ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
    case 256: return f16 ? launch_t<256, true>(p, stream) : launch_t<256, false>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
