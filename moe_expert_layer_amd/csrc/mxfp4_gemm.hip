// Grouped product of MXFP4 rows with MXFP4 weights (E2M1 values, one UE8M0 scale per 32 along K):
//   C[r, n] = sum_k A[r, k] * B[e, n, k]   for the rows r of group e, offsets[e] <= r < offsets[e + 1]
// on the scaled FP4 matrix instructions, which multiply the codes, apply both blocks' scales and sum
// in float32 (measured: within 2e-7 of the exact sum, as a sequential float32 sum is, for scales
// spread over 2^20).  The result is rounded once to C's type.
//
// A lane of the 16x16x128 instruction holds one 32-wide block of one row: row lane % 16, block
// lane / 16 of four.  Since the sum over K takes its blocks in any order, as long as both operands
// take the same, quarter q of the lanes works through the four blocks of the 128-wide scale word q of
// a 512-wide stretch in four instructions: a lane then needs one scale word and one 64-byte run of
// codes per operand row and stretch, and names the byte of the word in the instruction.
#include <hip/hip_runtime.h>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "device_common.hpp"
#include "elem.hpp"
#include "lds_dma.hpp"
#include "moe_internal.hpp"
#include "operators.hpp"

namespace moe {

// the rows of group e, inside [0, rows) whatever the offsets hold
__device__ __forceinline__ int2 group_rows(const int32_t* __restrict__ offsets, int e, int rows) {
  if (offsets == nullptr) return make_int2(0, rows);
  const int lo = min(max(offsets[e], 0), rows);
  return make_int2(lo, min(max(offsets[e + 1], lo), rows));
}

__device__ __forceinline__ v8i fp4_operand(uint4 q) {
  return v8i{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

// Groups with few rows: the weights are what is read.  One workgroup takes 16 * NS weight rows of one
// group; its NW waves take every NW-th 512-wide stretch of K, each lane straight from global memory into
// the matrix instruction's registers (a weight is used once per 16 rows: nothing to gain from LDS), and
// their partial sums meet in LDS, in wave order.  Rows go 16, 32 or 64 at a time (MT); a group with
// more is walked again, or by other workgroups (the grid's z).  Bound by HBM: 4 rows for each of 32
// groups of 4096 x 7168 take 89 us, 5.6 TB/s of weights, as the layer's own decode FC1 reads them (93 to 96 us a
// call in a captured graph).
template <typename T, int NW, int NS, int MAXR, int MT>
__device__ __forceinline__ void gemm_rows(const Mxfp4GemmArgs& g, float (*part)[MAXR][NS * 16 + 1], int e, int n0,
                                          int m0, int m_end) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int nblk = g.K / 32, nwords = (nblk + 3) / 4, nst = (nwords + 3) / 4;
  const long long ld = g.K / 2;
  const uint8_t *ap[MT], *as[MT], *bp[NS], *bs[NS];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const long long row = min(m0 + m * 16 + r16, m_end - 1);
    ap[m] = g.A + row * ld;
    as[m] = g.A_sf + row * g.a_row_mul;
  }
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const long long row = (long long)e * g.N + min(n0 + s * 16 + r16, g.N - 1);
    bp[s] = g.B + row * ld;
    bs[s] = g.B_sf + row * g.b_row_mul;
  }
  v4f acc[MT][NS];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int st = wave; st < nst; st += NW) {
    const int j = st * 4 + q;  // this lane's scale word
    const int jc = min(j, nwords - 1);
    const int left = nblk - 4 * j;  // blocks of the word inside K (<= 0: none)
    int sa[MT], sb[NS];
    uint4 a[MT][4], b[NS][4];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      sb[s] = *reinterpret_cast<const int*>(bs[s] + (long long)jc * g.b_word_mul);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[s][i] = *reinterpret_cast<const uint4*>(bp[s] + (i < left ? (long long)j * 64 + i * 16 : 0));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      sa[m] = *reinterpret_cast<const int*>(as[m] + (long long)jc * g.a_word_mul);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[m][i] = *reinterpret_cast<const uint4*>(ap[m] + (i < left ? (long long)j * 64 + i * 16 : 0));
    }
    if (left < 4) {  // past K: zero codes, and scales of 1 whatever the padding holds
      const int keep = left <= 0 ? 0 : (1 << (8 * left)) - 1;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sa[m] = (sa[m] & keep) | (0x7f7f7f7f & ~keep);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i >= left) a[m][i] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) sb[s] = (sb[s] & keep) | (0x7f7f7f7f & ~keep);
    }
    // the scale byte's index is an immediate
#define MOE_MX_STEP(I)                                                                                            \
  _Pragma("unroll") for (int s = 0; s < NS; ++s) _Pragma("unroll") for (int m = 0; m < MT; ++m) acc[m][s] =       \
      __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][I]), fp4_operand(b[s][I]), acc[m][s], 4, \
                                                       4, I, sa[m], I, sb[s]);
    MOE_MX_STEP(0)
    MOE_MX_STEP(1)
    MOE_MX_STEP(2)
    MOE_MX_STEP(3)
#undef MOE_MX_STEP
  }
  // lane holds rows 4 q + i, column r16 of each 16 x 16 tile
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][m * 16 + 4 * q + i][s * 16 + r16] = acc[m][s][i];
  __syncthreads();
  const int rows = min(MT * 16, m_end - m0);
  for (int i = tid; i < rows * NS * 16; i += NW * 64) {
    const int r = i / (NS * 16), c = i % (NS * 16);
    float v = part[0][r][c];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += part[w][r][c];
    if (n0 + c < g.N) static_cast<T*>(g.C)[(long long)(m0 + r) * g.c_stride + n0 + c] = Elem<T>::put(v);
  }
  __syncthreads();
}

template <typename T, int NW, int NS, int MAXR>
__global__ __launch_bounds__(NW * 64) void mxfp4_gemm_rows_kernel(Mxfp4GemmArgs g) {
  __shared__ float part[NW][MAXR][NS * 16 + 1];
  const int e = blockIdx.y, n0 = blockIdx.x * (NS * 16);
  const int2 rr = group_rows(g.offsets, e, g.rows);
  for (int m0 = rr.x + blockIdx.z * MAXR; m0 < rr.y; m0 += gridDim.z * MAXR) {
    const int rows = rr.y - m0;
    if (rows <= 16) gemm_rows<T, NW, NS, MAXR, 1>(g, part, e, n0, m0, rr.y);
    else if (MAXR == 32 || rows <= 32) gemm_rows<T, NW, NS, MAXR, 2>(g, part, e, n0, m0, rr.y);
    else gemm_rows<T, NW, NS, MAXR, MAXR / 16>(g, part, e, n0, m0, rr.y);
  }
}

// ---------------------------------------------------------------------------------------
// Tiles of BM rows x BN columns: 256 x 256 by eight waves of 64 x 128 where there are many, 128 x 128 by four waves of
// 32 x 128, two workgroups on a CU, where they would fill the GPU badly (the results of one are then stored while
// the other multiplies; its waves read 5 fragments for 4 instructions, where the large ones read 6 for 8).
//
// K advances 256 values a stage: 128 bytes (a cache line) of codes per operand row, brought from
// global memory straight into one of two LDS slots, and two scale words per row, into one of four.
// The NW waves each own a WTM x WTN part as 32 x 32 accumulators.  A lane of the 32x32x64 instruction
// holds one block of 32 of row lane % 32; half kb = lane / 32 of the lanes works through the four
// blocks of the stage's scale word kb in four steps, so it reads one scale word per row and stage.
// The fragments of the next step are read from LDS while the matrix instructions of this one run;
// the stage boundary (wait for the next stage's codes, barrier, loads of the stage after it into the
// slot just read) sits before the last step's instructions, when every wave holds its last fragments.
//
// Loads of a wave complete in order, so what is issued behind a stage's codes may stay in flight when
// those are waited for: the scales, which are asked for two stages earlier than the codes (every stage
// takes them from lines of their own, which come from HBM).
//
// Weights are the instruction's first operand, so a lane's results are runs of four columns of one
// row; a wave puts them in type T into its part of the second slot, 32 rows x 256 bytes at a time, and
// stores whole 16-byte chunks, while the next tile's first stage lands in the first slot.  Workgroups
// are persistent: each XCD has a contiguous range of tiles, whose rows and columns of operands meet in
// its L2, and its workgroups take them in turn.
//
// Measured: 32500 rows x 4096 x 7168 in 32 groups 500 to 570 us by box and clock, 3.3 to 3.8 PFLOP/s; 8192 x 8192 x
// 8192 260 us, 4.2; 4096 x 4096 x 57344, where the K loop is all there is, 410 to 430 us, 4.5 to 4.65.  On the last
// the matrix cores are busy 60 to 64% of the cycles at 1.75 to 1.8 GHz (2.4 GHz with nothing to multiply), so that
// half of every cycle saved is lost to the power limit (897K cycles 452 us, 727K 409 us).  On the first they are busy
// 47% of the cycles, at 1.9 to 2.0 GHz, and 34% of the L2's requests miss: about 12 of the 32 groups end with a tile
// of a few rows, which costs about as much as a full one (32 groups of 1024 rows 500 us, of 1030 rows 578 us), and a
// tile's results cost 7 us, all workgroups storing at once.  Not kept: 128 x 128 per
// wave, four waves (656 us on the last shape: one wave a SIMD waits for its own loads to issue); half-line
// stages, four of them (472 us, twice the L2 requests); results stored from the registers, 32 bytes a row
// at a time (680 against 525 us on the first shape); lines of later stages touched ahead, by every wave
// (3% slower) or by waves with no other loads; 128 x 128 tiles with four stages in flight, one workgroup on a CU (8
// groups of 4096 x 7168, 64 rows each: 27 against 34 us, but the same where the weights are not what is waited for:
// there a stage is 80 KB of fragments read from LDS and 32 KB written, 0.55 us).

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kTileGroupN = 8;  // column tiles that go together in the tile order

template <int BM, int BN, int NW, int WTM, int WTN>
struct TileCfg {
  static constexpr int NT = NW * 64, WM = BM / WTM, MI = WTM / 32, NI = WTN / 32;
  static constexpr int kRowB = 128;                  // bytes of codes per row and stage
  static constexpr int kSlot = (BM + BN) * kRowB;    // A's rows, then B's
  static constexpr int kScales = 2 * kSlot;          // four slots of [word][A's rows], [word][B's rows]
  static constexpr int kScaleSlot = (BM + BN) * 8;
  static constexpr int kPlan = kScales + 4 * kScaleSlot;
  static constexpr int lds_bytes(int groups) { return kPlan + (3 * groups + 1 + NW) * 4; }
  // workgroups that a CU's LDS holds: of the 128 x 128 tiles' two with up to 681 groups, one with more
  static constexpr int per_cu(int groups) { return 160 * 1024 / lds_bytes(groups); }
  static constexpr int kADma = BM / 8 / NW, kBDma = BN / 8 / NW;  // 1 KB loads per wave and stage
  static constexpr int kSDma = (BM + BN) * 2 / 64 / NW;           // 256-byte loads of scale words
  static constexpr int kPer = kADma + kBDma + kSDma;              // loads per wave and stage
  static_assert(WM * (BN / WTN) == NW && kADma * NW * 8 == BM && kBDma * NW * 8 == BN, "");
  static_assert(kSDma * NW * 32 == BM + BN && BM % 64 == 0 && BN % 64 == 0, "");
  static_assert(NW * 32 * 256 <= kSlot && WTN == 128, "the results' staging fits a slot, in passes of 256 bytes");
};

using Tiles256 = TileCfg<256, 256, 8, 64, 128>;
using Tiles128 = TileCfg<128, 128, 4, 32, 128>;

template <typename T, int BM, int BN, int NW, int WTM, int WTN>
__global__ __launch_bounds__(NW * 64, 1) void mxfp4_gemm_tile_kernel(Mxfp4GemmArgs g) {
  using C = TileCfg<BM, BN, NW, WTM, WTN>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  // the first row tile of each group [groups + 1], unsigned: where groups overlap (offsets that are not what they
  // should be), 512 of 1024 can have all of at most 2^30 rows, 2^32 tiles of 128 rows, which count as none
  unsigned* s_plan = reinterpret_cast<unsigned*>(lds + C::kPlan);
  int* s_lo = reinterpret_cast<int*>(s_plan + g.groups + 1);  // [groups] first row
  int* s_hi = s_lo + g.groups;                                // [groups] end
  unsigned* s_wsum = reinterpret_cast<unsigned*>(s_hi + g.groups);  // [NW]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  {  // the plan, by a scan over the groups
    const int per = (g.groups + C::NT - 1) / C::NT, beg = tid * per;
    unsigned sum = 0;
    for (int i = beg; i < min(beg + per, g.groups); ++i) {
      const int2 r = group_rows(g.offsets, i, g.rows);
      s_lo[i] = r.x;
      s_hi[i] = r.y;
      s_plan[i] = sum;
      sum += (r.y - r.x + BM - 1) / BM;
    }
    const unsigned inc = (unsigned)wave_inclusive_scan((int)sum);
    if (lane == 63) s_wsum[wave] = inc;
    __syncthreads();
    unsigned base = inc - sum;
    for (int w = 0; w < wave; ++w) base += s_wsum[w];
    for (int i = beg; i < min(beg + per, g.groups); ++i) s_plan[i] += base;
    if (tid == C::NT - 1) s_plan[g.groups] = base + sum;
    __syncthreads();
  }
  const int n_tiles = (g.N + BN - 1) / BN;
  const long long total = (long long)s_plan[g.groups] * n_tiles;
  // XCD x = blockIdx % 8 has tiles [x q + min(x, r), ...) of q = total / 8, r = total % 8
  const long long xq = total >> 3;
  const int x = blockIdx.x & 7, xr = (int)(total & 7);
  const long long x_cnt = xq + (x < xr ? 1 : 0), x_base = x * xq + (x < xr ? x : xr), x_step = gridDim.x >> 3;

  const int ld = g.K / 2, nblk = g.K / 32, nwords = (nblk + 3) / 4, nst = (nwords + 1) / 2;
  const bool ktail = (nblk & 7) != 0;
  const uint32_t ring0 = lds_addr(lds);

  // a tile's operands: buffers that end with its rows and columns
  struct Tile {
    v4i_srd a, b;
    const uint8_t* s;          // scale word 0 of the first row of the operand whose scales this wave loads
    uint32_t s_len;
    int row0, rows, n0, cols;
  };
  auto locate = [&](long long p) {
    const long long L = x_base + p;
    int e = 0, hi = g.groups - 1;
    const unsigned mt = (unsigned)(L / n_tiles);
    while (e < hi) {  // the last group that starts at or before this row tile (it has rows)
      const int mid = (e + hi + 1) >> 1;
      if (s_plan[mid] <= mt) e = mid; else hi = mid - 1;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    const unsigned first = __builtin_amdgcn_readfirstlane(s_plan[e]);
    const int m_tiles = (int)(__builtin_amdgcn_readfirstlane(s_plan[e + 1]) - first);
    const int li = (int)(L - (long long)first * n_tiles);
    const int grp = li / (kTileGroupN * m_tiles);
    const int gsz = min(n_tiles - grp * kTileGroupN, kTileGroupN);
    const int idx = li - grp * kTileGroupN * m_tiles, m = idx / gsz, n = idx % gsz;
    Tile t;
    t.row0 = __builtin_amdgcn_readfirstlane(s_lo[e]) + m * BM;
    t.rows = min(BM, __builtin_amdgcn_readfirstlane(s_hi[e]) - t.row0);
    t.n0 = (grp * kTileGroupN + n) * BN;
    t.cols = min(BN, g.N - t.n0);
    const long long brow = (long long)e * g.N + t.n0;
    t.a = buffer_srd(g.A + (long long)t.row0 * ld, (long long)t.rows * ld);
    t.b = buffer_srd(g.B + brow * ld, (long long)t.cols * ld);
    t.s = wave * C::kSDma < BM / 32 ? g.A_sf + t.row0 * g.a_row_mul : g.B_sf + brow * g.b_row_mul;
    t.s_len = (uint32_t)(wave * C::kSDma < BM / 32 ? (t.rows - 1) * g.a_row_mul + 4 : (t.cols - 1) * g.b_row_mul + 4);
    return t;
  };

  // load offsets of this lane: 16-byte chunk c of row r goes to chunk c ^ swz(r) of its LDS row
  uint32_t a_off[C::kADma], b_off[C::kBDma], s_off[C::kSDma];
#pragma unroll
  for (int i = 0; i < C::kADma; ++i) {
    const int r = (wave * C::kADma + i) * 8 + lane / 8;
    a_off[i] = (uint32_t)r * (uint32_t)ld + (((lane & 7) ^ swz<8>(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < C::kBDma; ++i) {
    const int r = (wave * C::kBDma + i) * 8 + lane / 8;
    b_off[i] = (uint32_t)r * (uint32_t)ld + (((lane & 7) ^ swz<8>(r)) << 4);
  }
  // the wave's scale loads are of one operand and one of its two words a stage
  static_assert(BM / 64 % C::kSDma == 0 && BN / 64 % C::kSDma == 0, "");
  const bool s_is_a = wave * C::kSDma < BM / 32;
  const int s_q = s_is_a ? wave * C::kSDma : wave * C::kSDma - BM / 32;  // in loads of 64 rows of one word
  const int s_word = s_is_a ? s_q / (BM / 64) : s_q / (BN / 64);
  const long long s_word_mul = s_is_a ? g.a_word_mul : g.b_word_mul;
#pragma unroll
  for (int i = 0; i < C::kSDma; ++i)
    s_off[i] = s_is_a ? (uint32_t)(((s_q + i) * 64 + lane) % BM) * (uint32_t)g.a_row_mul
                      : (uint32_t)(((s_q + i) * 64 + lane) % BN) * (uint32_t)g.b_row_mul;

  // load i of this wave for the stages that follow stage ks: codes of stage ks + 2 (past K they are the
  // next row's, or lie past the buffer; they are cut below), scales of stage ks + 4 (of the last again
  // where there is none)
  auto issue = [&](const Tile& t, int i, int ks) {
    if (i < C::kADma) {
      dma16_buffer(t.a, a_off[i], (uint32_t)(ks + 2) * C::kRowB,
                   ring0 + (uint32_t)(ks & 1) * C::kSlot + (wave * C::kADma + i) * 1024);
    } else if (i < C::kADma + C::kBDma) {
      const int k = i - C::kADma;
      dma16_buffer(t.b, b_off[k], (uint32_t)(ks + 2) * C::kRowB,
                   ring0 + (uint32_t)(ks & 1) * C::kSlot + BM * C::kRowB + (wave * C::kBDma + k) * 1024);
    } else {
      const int k = i - C::kADma - C::kBDma, q = wave * C::kSDma + k;
      const int j = min(2 * (ks + 4) + s_word, nwords - 1);
      dma4_buffer(buffer_srd(t.s + j * s_word_mul, t.s_len), s_off[k], 0u,
                  ring0 + C::kScales + (uint32_t)(ks & 3) * C::kScaleSlot + q * 256);
    }
  };

  // fragment addresses in a slot: chunk 4 kb + s of row r; rows 32 apart differ in bit 2 of the swizzle
  const int lrow = lane & 31, kb = lane >> 5;
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int ra = wm * WTM + lrow, rb = wn * WTN + lrow;
  const uint32_t fa_ = ra * C::kRowB + (((4 * kb) ^ swz<8>(ra)) << 4);
  const uint32_t fb_ = (BM + rb) * C::kRowB + (((4 * kb) ^ swz<8>(rb)) << 4);
  const uint32_t wa = C::kScales + (kb * BM + ra) * 4, wb = C::kScales + (2 * BM + kb * BN + rb) * 4;

  struct Frags {
    v4i a[C::MI], b[C::NI];
  };
  struct Scales {
    int a[C::MI], b[C::NI];
  };
  auto load = [&](int ks, int s, Frags& f) {
    const uint8_t* st = lds + (ks & 1) * C::kSlot;
    uint32_t fa = fa_, fb = fb_;
    asm volatile("" : "+v"(fa), "+v"(fb));  // an address is one instruction: made anew rather than kept in registers
#pragma unroll
    for (int m = 0; m < C::MI; ++m)
      f.a[m] = *reinterpret_cast<const v4i*>(st + (fa ^ (uint32_t)((s << 4) ^ ((m & 1) << 6))) + m * 32 * C::kRowB);
#pragma unroll
    for (int n = 0; n < C::NI; ++n)
      f.b[n] = *reinterpret_cast<const v4i*>(st + (fb ^ (uint32_t)((s << 4) ^ ((n & 1) << 6))) + n * 32 * C::kRowB);
  };
  auto load_scales = [&](int ks, Scales& c) {
    const uint8_t* st = lds + (ks & 3) * C::kScaleSlot;
#pragma unroll
    for (int m = 0; m < C::MI; ++m) c.a[m] = *reinterpret_cast<const int*>(st + wa + m * 128);
#pragma unroll
    for (int n = 0; n < C::NI; ++n) c.b[n] = *reinterpret_cast<const int*>(st + wb + n * 128);
  };
  // the last stage, where it lies past K for this lane: zero codes, and scales of 1 whatever the
  // padding holds
  auto cut = [&](int s, Frags& f) {
    if (ktail && ((nst - 1) * 2 + kb) * 4 + s >= nblk) {
#pragma unroll
      for (int m = 0; m < C::MI; ++m) f.a[m] = v4i{0, 0, 0, 0};
    }
  };
  auto cut_scales = [&](Scales& c) {
    if (ktail) {
      const int left = nblk - ((nst - 1) * 2 + kb) * 4;
      const int keep = left >= 4 ? -1 : left <= 0 ? 0 : (1 << (8 * left)) - 1;
#pragma unroll
      for (int m = 0; m < C::MI; ++m) c.a[m] = (c.a[m] & keep) | (0x7f7f7f7f & ~keep);
#pragma unroll
      for (int n = 0; n < C::NI; ++n) c.b[n] = (c.b[n] & keep) | (0x7f7f7f7f & ~keep);
    }
  };
  auto mma = [&](auto& acc, const Frags& f, const Scales& c, auto step) {
    constexpr int S = decltype(step)::value;
    auto wide = [](v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };
#pragma unroll
    for (int n = 0; n < C::NI; ++n)
#pragma unroll
      for (int m = 0; m < C::MI; ++m)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(f.b[n]), wide(f.a[m]), acc[m][n], 4, 4, S,
                                                                    c.b[n], S, c.a[m]);
  };
  auto mma1 = [&](auto& acc, const Frags& f, const Scales& c, auto step, int i) {  // its i-th instruction
    constexpr int S = decltype(step)::value;
    auto wide = [](v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };
    const int n = i / C::MI, m = i % C::MI;
    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(f.b[n]), wide(f.a[m]), acc[m][n], 4, 4, S, c.b[n],
                                                                S, c.a[m]);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;

  // loads [lo, hi) of the list above
  auto issue_range = [&](const Tile& t, int ks, auto lo, auto hi) {
#pragma unroll
    for (int i = decltype(lo)::value; i < decltype(hi)::value; ++i) issue(t, i, ks);
  };
  constexpr int kCodes = C::kADma + C::kBDma, kBehind = C::kSDma;
  using N0 = std::integral_constant<int, 0>;
  using NCodes = std::integral_constant<int, kCodes>;
  using NAll = std::integral_constant<int, C::kPer>;
  auto start = [&](const Tile& t) {  // codes of stage 0, scales of stages 0 to 2
    issue_range(t, -2, N0{}, NCodes{});
#pragma unroll
    for (int i = 0; i < 3; ++i) issue_range(t, i - 4, NCodes{}, NAll{});
  };
  auto second = [&](const Tile& t) {  // codes of stage 1, scales of stage 3
    if (nst > 1) issue_range(t, -1, N0{}, NCodes{});
    issue_range(t, -1, NCodes{}, NAll{});
  };

  long long p = blockIdx.x >> 3;
  if (p >= x_cnt) return;
  Tile t = locate(p);
  start(t);
  second(t);
  for (;;) {
    const bool more = p + x_step < x_cnt;
    if (nst > 1) wait_vm_barrier<kCodes + kBehind>();  // the first stage has landed
    else wait_vm_barrier<0>();
    Tile next = t;
    if (wm * WTM < t.rows && wn * WTN < t.cols) {
      v16f acc[C::MI][C::NI];
#pragma unroll
      for (int m = 0; m < C::MI; ++m)
#pragma unroll
        for (int n = 0; n < C::NI; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
      Frags f0, f1;
      Scales c, c2;
      load(0, 0, f0);
      load_scales(0, c);
      // the order of a step: the next step's fragments are asked for, then this one's instructions run.
      // The scheduler would sink the reads to their use and wait for each
      auto step = [&](int ks, auto s, Frags& now, Frags& then) {
        load(ks, decltype(s)::value + 1, then);
        __builtin_amdgcn_sched_barrier(0);
        mma(acc, now, c, s);
        __builtin_amdgcn_sched_barrier(0);
      };
#pragma unroll 1
      for (int ks = 0; ks + 2 < nst; ++ks) {
        step(ks, I0{}, f0, f1);
        step(ks, I1{}, f1, f0);
        step(ks, I2{}, f0, f1);
        wait_vm_barrier<kBehind>();  // stage ks + 1 has landed
        load(ks + 1, 0, f0);
        load_scales(ks + 1, c2);
        __builtin_amdgcn_sched_barrier(0);
        // the last step's instructions, the loads between them
        constexpr int kM = C::MI * C::NI;
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          mma1(acc, f1, c, I3{}, i);
#pragma unroll
          for (int l = i * C::kPer / kM; l < (i + 1) * C::kPer / kM; ++l) issue(t, l, ks);
          __builtin_amdgcn_sched_barrier(0);
        }
        c = c2;
      }
      if (nst > 1) {  // the last boundary: nothing more to load
        const int ks = nst - 2;
        step(ks, I0{}, f0, f1);
        step(ks, I1{}, f1, f0);
        step(ks, I2{}, f0, f1);
        wait_vm_barrier<0>();
        load(ks + 1, 0, f0);
        load_scales(ks + 1, c2);
        mma(acc, f1, c, I3{});
        c = c2;
      }
      cut(0, f0);
      cut_scales(c);
      load(nst - 1, 1, f1);
      cut(1, f1);
      mma(acc, f0, c, I0{});
      load(nst - 1, 2, f0);
      cut(2, f0);
      mma(acc, f1, c, I1{});
      load(nst - 1, 3, f1);
      cut(3, f1);
      mma(acc, f0, c, I2{});
      mma(acc, f1, c, I3{});
      wait_vm_barrier<0>();  // every wave is past its last fragment, no load is on its way to a slot
      if (more) {
        next = locate(p + x_step);
        start(next);
      }

      // lane: row lrow of row tile m, columns 8 q + 4 kb + 0..3 of column tile n; 16-byte chunks swizzled
      // by row.  The wave's own part of the slot: LDS operations of a wave stay in order
      // (made from a lane index the compiler cannot see through, or it would keep these addresses in
      // registers, and then in scratch memory, across the whole K loop)
      int el = lane;
      asm volatile("" : "+v"(el));
      constexpr int es = sizeof(T), kPassCols = 256 / es, kPassN = kPassCols / 32;  // columns, tiles per pass
      uint8_t* out = lds + C::kSlot + wave * (32 * 256);
      const int er = el & 31, ekb = el >> 5, ech = el & 15, erow = el >> 4;
      uint8_t* const put_at = out + er * 256;
      // 8 loads of 4 rows x 256 bytes: row 4 i + erow, chunk ech ^ (row & 15); (4 i + erow) & 15 has bits 2
      // and 3 from i
      const uint8_t* const get_at = out + erow * 256 + (((ech ^ erow) & 3) << 4);
#pragma unroll
      for (int m = 0; m < C::MI; ++m)
#pragma unroll
        for (int h = 0; h < (WTN + kPassCols - 1) / kPassCols; ++h) {
#pragma unroll
          for (int nn = 0; nn < kPassN; ++nn) {
            const int n = h * kPassN + nn;
            if (n < C::NI) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int at = (nn * 32 + 8 * q) * es;  // byte of the quarter-wave's run in the 256, kb = 0
                T v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = Elem<T>::put(acc[m][n][4 * q + j]);
                // 4 kb columns further: es = 2: bit 3 of the byte; es = 4: bit 4
                uint8_t* to = put_at + (((at + 4 * es * ekb) ^ ((er & 15) << 4)));
                __builtin_memcpy(__builtin_assume_aligned(to, 4 * es), v, 4 * es);
              }
            }
          }
          const int col = wn * WTN + h * kPassCols + ech * (16 / es), row = wm * WTM + m * 32 + erow;
          T* dst = static_cast<T*>(g.C) + (long long)(t.row0 + row) * g.c_stride + t.n0 + col;
          const long long step = 4 * g.c_stride;
          auto chunk = [&](int i) {
            return *reinterpret_cast<const u32x4*>(get_at + i * 1024 + (((ech & 12) ^ ((i & 3) << 2)) << 4));
          };
          if (t.cols == BN) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const u32x4 v = chunk(i);
              if (row + 4 * i < t.rows) store16(dst, v);
              dst += step;
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              if (row + 4 * i < t.rows) {
                const u32x4 v = chunk(i);
                if (col + 16 / es <= t.cols) {
                  store16(dst, v);
                } else {
                  T one[16 / es];
                  __builtin_memcpy(one, &v, 16);
#pragma unroll
                  for (int j = 0; j < 16 / es; ++j)
                    if (col + j < t.cols) dst[j] = one[j];
                }
              }
              dst += step;
            }
          }
        }
    } else {
      // a wave whose part lies past the group's rows or the columns only moves data: the same loads and
      // barriers
#pragma unroll 1
      for (int ks = 0; ks + 2 < nst; ++ks) {
        wait_vm_barrier<kBehind>();
        issue_range(t, ks, N0{}, NAll{});
      }
      if (nst > 1) wait_vm_barrier<0>();
      wait_vm_barrier<0>();
      if (more) {
        next = locate(p + x_step);
        start(next);
      }
    }
    if (!more) return;
    __syncthreads();  // the second slot is free
    second(next);
    t = next;
    p += x_step;
  }
}

template <typename T, int BM, int BN, int NW, int WTM, int WTN>
static hipError_t launch_tiles(const Mxfp4GemmArgs& g, hipStream_t s) {
  using C = TileCfg<BM, BN, NW, WTM, WTN>;
  auto kern = mxfp4_gemm_tile_kernel<T, BM, BN, NW, WTM, WTN>;
  constexpr int kMaxGroups = 1024;
  static std::atomic<uint64_t> ready{0};  // the LDS limit is raised once per device
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::lds_bytes(kMaxGroups));
    if (e != hipSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  // at most this many tiles; as many workgroups as fit the GPU at once, in whole rows of 8 XCDs
  const long long most = (((long long)g.rows + (long long)g.groups * (BM - 1)) / BM) * ((g.N + BN - 1) / BN);
  const long long room = (long long)device_cus() * C::per_cu(g.groups);
  const unsigned grid = (unsigned)(((most < room ? most : room) + 7) / 8 * 8);
  kern<<<dim3(grid), dim3(C::NT), C::lds_bytes(g.groups), s>>>(g);
  return hipGetLastError();
}

template <typename T, int NW, int NS, int MAXR>
static hipError_t launch_rows(const Mxfp4GemmArgs& g, hipStream_t s) {
  const unsigned x = (unsigned)((g.N + 16 * NS - 1) / (16 * NS)), y = (unsigned)g.groups;
  // few columns: the passes over rows spread over the grid up to 4096 waves, 16 per CU (one group may have all the
  // rows).  5826 rows x 32 x 4768 in 7 groups 87 -> 8 us, 334 rows x 1744 x 6592 37 -> 18; with half the waves
  // 1197 rows x 508 x 1728 in 7 groups 8.2 instead of 6.6 us, with twice as many 6.9.
  const long long room = 4096 / NW / ((long long)x * y), most = (g.rows + MAXR - 1) / MAXR;
  const unsigned z = (unsigned)(room < 1 ? 1 : room < most ? room : most);
  mxfp4_gemm_rows_kernel<T, NW, NS, MAXR><<<dim3(x, y, z), NW * 64, 0, s>>>(g);
  return hipGetLastError();
}

// Rows kernel (0), 256 x 256 tiles (1) or 128 x 128 tiles (2), by estimates in microseconds from the sizes alone
// (the groups' rows are on the device: their average stands for them).  Each is the larger of the weights' bytes at
// 5.5 TB/s (a kernel whose tiles are all resident at once reaches less) and of its own work: the rows kernel's
// latency grows with K and its time with the multiplications of its 16-row tiles, the tile kernels take their tiles
// in rounds, each a fixed time plus one for each stage of 256 along K, the longer the fuller the GPU is.  Where there
// are fewer rows than groups, only as many groups as rows count, and the rows kernel needs at least the time that
// its workgroups without rows take to come and go, 0.25 us a thousand (1 row in 256 groups of 7168 x 2048: 18 us,
// with 128 x 128 tiles 11; in 32 groups of 4096 x 7168 9.6 and 21 us).  The figures are fitted to 501 shapes (1 to 32
// groups of 1 to 2048 rows, all alike, nine N x K from 300 x 64 to 8192 x 8192), where the choice is on average 0.2%
// off the fastest; on 170 with fewer rows than groups (2 to 1024 of them) it is 0.1% off, on 60 with 720 and 1024 groups,
// where one workgroup of the 128 x 128 tiles fits a CU, 1% (4 rows each in 720 groups of 512 x 4096: 142 / 167 / 203
// us), on 90 with 64 to 640 groups 2.8%.  Groups of very different sizes, which the host does not see, cost more:
// Zipf shares 3.6% up to 32 groups, 15 to 20% from 64 on, most where K is short and a few groups have many rows
// (25600 in 640 groups of 256 x 512: 127 / 27 / 21 us).  Measured, rows / 256 / 128: one group of 8192 x 8192: 64 rows
// 15 / 44 / 24 us, 200 rows 42 / 46 / 25 us; 8 groups of 4096 x 4096: 64 rows each 35 / 26 / 16 us; 32 groups of
// 4096 x 7168: 4 rows each 93 / 96 / 85 us, 32 rows 133 / 102 / 89 us, 128 rows 366 / 119 / 130 us; 8192 x 8192 x 8192
// - / 265 / 344 us.
static int choose(const Mxfp4GemmArgs& g) {
  const int active = g.rows < g.groups ? g.rows : g.groups;  // groups that can have rows
  const double avg = (double)((g.rows + active - 1) / active), cus = device_cus(), stages = (g.K + 255) / 256;
  const double weights_us = 0.53 / 5.5e6 * active * g.N * g.K;
  const auto tiles_us = [&](int size, double slots, double fixed, double stage_idle, double stage_full) {
    const double m = (double)(((int)avg + size - 1) / size), n = (double)((g.N + size - 1) / size);
    const double full = active * m * n / slots, rounds = __builtin_ceil(full);
    const double stage = stage_idle + (stage_full - stage_idle) * (full < 1 ? full : 1);
    const double bytes_us = weights_us * (rounds <= 1 ? 1.15 : 1.0), work_us = rounds * (fixed + stage * stages);
    return bytes_us > work_us ? bytes_us : work_us;
  };
  const double empty_us = 3.5 + 0.25e-3 * (g.groups - active) * ((g.N + 31) / 32), fixed_us = 5.3 + 0.5e-3 * g.K;
  const double base_us = empty_us > fixed_us ? empty_us : fixed_us;
  const double rows_us = (weights_us > base_us ? weights_us : base_us) +
                         2.7e-9 * (avg <= 16 ? avg : (double)(((int)avg + 15) / 16 * 16)) * active * g.N * g.K;
  const double us256 = tiles_us(256, cus * Tiles256::per_cu(g.groups), 7.1, 0.98, 1.7);
  const double us128 = tiles_us(128, cus * Tiles128::per_cu(g.groups), 5.5, 0.77, 1.3);
  if (rows_us <= us256 && rows_us <= us128) return 0;
  return us256 <= us128 ? 1 : 2;
}

template <typename T>
static hipError_t launch(const Mxfp4GemmArgs& g, int variant, hipStream_t s) {
  if (variant < 0) variant = choose(g);
  if (variant == 1) return launch_tiles<T, 256, 256, 8, 64, 128>(g, s);
  if (variant == 2) return launch_tiles<T, 128, 128, 4, 32, 128>(g, s);
  // K within one 512-wide stretch: nothing to split over waves, so each is a workgroup (5838 rows x 1027 x 96 in
  // 4 groups 12 against 22 us, 8241 rows x 625 x 160 in 24 groups 9 against 15 us)
  if (g.K <= 512) return launch_rows<T, 1, 2, 32>(g, s);
  // up to 16 rows a group: half the registers, twice the waves (32 groups of 7168 x 2048, 4 rows each: 43
  // against 55 us); above: 64 rows a pass (one group of 8192 x 8192, 64 rows: 16 against 27 us)
  if ((long long)g.rows <= 16LL * g.groups) {
    // fewer workgroups than CUs: half the columns, eight waves along K (one row, 4099 x 7168: 5.6 against 7.3 us;
    // one group of 8192 x 8192, which has enough: 12.2 against 10.0 us).  Workgroups of groups without rows count:
    // they take their time too (1 row in 256 groups of 1024 x 1024 10.4 against 5.0 us)
    if ((long long)g.groups * ((g.N + 31) / 32) < device_cus()) return launch_rows<T, 8, 1, 32>(g, s);
    return launch_rows<T, 4, 2, 32>(g, s);
  }
  return launch_rows<T, 4, 2, 64>(g, s);
}

hipError_t launch_mxfp4_gemm(const Mxfp4GemmArgs& g, int out_dtype, int variant, hipStream_t s) {
  if (out_dtype == 0) return launch<Bf16>(g, variant, s);
  if (out_dtype == 1) return launch<F16>(g, variant, s);
  return launch<float>(g, variant, s);
}

}  // namespace moe
