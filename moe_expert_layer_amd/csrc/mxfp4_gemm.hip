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

// One group's 16 * NS weight rows against MT * 16 token rows at a time; the NW waves take every
// NW-th 512-wide stretch of K and their partial sums meet in LDS, in wave order.
template <typename T, int NW, int NS, int MT>
__global__ __launch_bounds__(NW * 64) void mxfp4_gemm_rows_kernel(Mxfp4GemmArgs g) {
  __shared__ float part[NW][MT * 16][NS * 16 + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.y, n0 = blockIdx.x * (NS * 16);
  const int2 rr = group_rows(g.offsets, e, g.rows);
  const int r16 = lane & 15, q = lane >> 4;
  const int nblk = g.K / 32, nwords = (nblk + 3) / 4, nst = (nwords + 3) / 4;
  const long long ld = g.K / 2;
  const uint8_t* bp[NS];
  const uint8_t* bs[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const long long row = (long long)e * g.N + min(n0 + s * 16 + r16, g.N - 1);
    bp[s] = g.B + row * ld;
    bs[s] = g.B_sf + row * g.b_row_mul;
  }
  for (int m0 = rr.x; m0 < rr.y; m0 += MT * 16) {
    const uint8_t* ap[MT];
    const uint8_t* as[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const long long row = min(m0 + m * 16 + r16, rr.y - 1);
      ap[m] = g.A + row * ld;
      as[m] = g.A_sf + row * g.a_row_mul;
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
#pragma unroll
      for (int m = 0; m < MT; ++m) sa[m] = *reinterpret_cast<const int*>(as[m] + (long long)jc * g.a_word_mul);
#pragma unroll
      for (int s = 0; s < NS; ++s) sb[s] = *reinterpret_cast<const int*>(bs[s] + (long long)jc * g.b_word_mul);
      uint4 a[MT][4], b[NS][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long at = i < left ? (long long)j * 64 + i * 16 : 0;
#pragma unroll
        for (int m = 0; m < MT; ++m) a[m][i] = *reinterpret_cast<const uint4*>(ap[m] + at);
#pragma unroll
        for (int s = 0; s < NS; ++s) b[s][i] = *reinterpret_cast<const uint4*>(bp[s] + at);
      }
      if (left < 4) {  // past K: zero codes and scales of 1
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
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          // the scale byte's index is an immediate
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][0]), fp4_operand(b[s][0]),
                                                                       acc[m][s], 4, 4, 0, sa[m], 0, sb[s]);
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][1]), fp4_operand(b[s][1]),
                                                                       acc[m][s], 4, 4, 1, sa[m], 1, sb[s]);
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][2]), fp4_operand(b[s][2]),
                                                                       acc[m][s], 4, 4, 2, sa[m], 2, sb[s]);
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][3]), fp4_operand(b[s][3]),
                                                                       acc[m][s], 4, 4, 3, sa[m], 3, sb[s]);
        }
    }
    // lane holds rows 4 q + i, column r16 of each 16 x 16 tile
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][m * 16 + 4 * q + i][s * 16 + r16] = acc[m][s][i];
    __syncthreads();
    for (int i = tid; i < MT * 16 * NS * 16; i += NW * 64) {
      const int r = i / (NS * 16), c = i % (NS * 16);
      float v = part[0][r][c];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += part[w][r][c];
      if (m0 + r < rr.y && n0 + c < g.N)
        static_cast<T*>(g.C)[(long long)(m0 + r) * g.c_stride + n0 + c] = Elem<T>::put(v);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
// Tiles of BM rows x BN columns for groups with many rows.
//
// K advances 256 values a stage: 128 bytes (a cache line) of codes per operand row, brought from
// global memory straight into one of two LDS slots, with the stage's two scale words per row.  The
// NW waves each own a WTM x WTN part as 32 x 32 accumulators.  A lane of the 32x32x64 instruction
// holds one block of 32 of row lane % 32; half kb = lane / 32 of the lanes works through the four
// blocks of the stage's scale word kb in four steps, so it reads one scale word per row and stage.
// The fragments of the next step are read from LDS while the matrix instructions of this one run;
// the stage boundary (wait for the next stage's loads, barrier, next loads issued into the slot just
// read) sits before the last step's instructions, when every wave holds its last fragments.
//
// Weights are the instruction's first operand, so a lane's results are runs of four columns of one
// row; a wave puts its part in type T into LDS (its own 32 KB of the slots) and stores whole 16-byte
// chunks, 256 contiguous bytes a row.  Workgroups are persistent: each XCD has a contiguous range of
// tiles, whose rows and columns of operands meet in its L2, and its workgroups take them in turn.

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kTileGroupN = 8;  // column tiles that go together in the tile order

template <int BM, int BN, int NW, int WTM, int WTN>
struct TileCfg {
  static constexpr int NT = NW * 64, WM = BM / WTM, MI = WTM / 32, NI = WTN / 32;
  static constexpr int kRowB = 128;                       // bytes of codes per row and stage
  static constexpr int kA = BM * kRowB, kB = BN * kRowB;  // offsets in a stage: A, B, A's words, B's words
  static constexpr int kSA = kA + kB, kSB = kSA + BM * 8;
  static constexpr int kStage = kSB + BN * 8;
  static constexpr int kPlan = 2 * kStage;
  static constexpr int kADma = BM / 8 / NW, kBDma = BN / 8 / NW;                // 1 KB loads per wave and stage
  static constexpr int kSaDma = BM * 2 / 64 / NW, kSbDma = BN * 2 / 64 / NW;  // 256-byte scale loads
  static constexpr int kOutB = NW * WTM * 256;                                   // results staged in LDS
  static_assert(WM * (BN / WTN) == NW && kADma * NW * 8 == BM && kBDma * NW * 8 == BN, "");
  static_assert(kSaDma * NW * 32 == BM && kSbDma * NW * 32 == BN, "");
  static_assert(kOutB <= 2 * kStage, "");
};

template <typename T, int BM, int BN, int NW, int WTM, int WTN>
__global__ __launch_bounds__(NW * 64, 1) void mxfp4_gemm_tile_kernel(Mxfp4GemmArgs g) {
  using C = TileCfg<BM, BN, NW, WTM, WTN>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  int* s_plan = reinterpret_cast<int*>(lds + C::kPlan);  // [groups + 1] first row tile of each group
  int* s_lo = s_plan + g.groups + 1;                     // [groups] first row
  int* s_hi = s_lo + g.groups;                           // [groups] end
  int* s_wsum = s_hi + g.groups;                         // [NW]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  {  // the plan, by a scan over the groups
    const int per = (g.groups + C::NT - 1) / C::NT, beg = tid * per;
    int sum = 0;
    for (int i = beg; i < min(beg + per, g.groups); ++i) {
      const int2 r = group_rows(g.offsets, i, g.rows);
      s_lo[i] = r.x;
      s_hi[i] = r.y;
      s_plan[i] = sum;
      sum += (r.y - r.x + BM - 1) / BM;
    }
    const int inc = wave_inclusive_scan(sum);
    if (lane == 63) s_wsum[wave] = inc;
    __syncthreads();
    int base = inc - sum;
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
  const long long x_cnt = xq + (x < xr ? 1 : 0), x_base = x * xq + (x < xr ? x : xr);

  const int lrow = lane & 31, kb = lane >> 5;
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int ld = g.K / 2, nblk = g.K / 32, nwords = (nblk + 3) / 4, nst = (nwords + 1) / 2;
  const bool ktail = (nblk & 7) != 0;
  const uint32_t ring0 = lds_addr(lds);
  // fragment addresses in a stage: chunk 4 kb + s of row r lies at (chunk ^ swz(r)); rows 32 apart
  // differ in bit 2 of the swizzle
  const int ra = wm * WTM + lrow, rb = wn * WTN + lrow;
  const uint32_t fa = ra * C::kRowB + (((4 * kb) ^ swz<8>(ra)) << 4);
  const uint32_t fb = C::kA + rb * C::kRowB + (((4 * kb) ^ swz<8>(rb)) << 4);
  const uint32_t wa = C::kSA + (kb * BM + ra) * 4, wb = C::kSB + (kb * BN + rb) * 4;

  for (long long p = blockIdx.x >> 3; p < x_cnt; p += gridDim.x >> 3) {
    const long long L = x_base + p;
    int e = 0;
    {
      int hi = g.groups - 1;  // the last group that starts at or before this row tile (it has rows)
      const int mt = (int)(L / n_tiles);
      while (e < hi) {
        const int mid = (e + hi + 1) >> 1;
        if (s_plan[mid] <= mt) e = mid; else hi = mid - 1;
      }
    }
    const int m_tiles = s_plan[e + 1] - s_plan[e];
    const long long li = L - (long long)s_plan[e] * n_tiles;
    const int grp = (int)(li / ((long long)kTileGroupN * m_tiles));
    const int gsz = min(n_tiles - grp * kTileGroupN, kTileGroupN);
    const int idx = (int)(li - (long long)grp * kTileGroupN * m_tiles);
    const int row0 = s_lo[e] + idx / gsz * BM, rows = min(BM, s_hi[e] - row0);
    const int n0 = (grp * kTileGroupN + idx % gsz) * BN, cols = min(BN, g.N - n0);

    // sources; rows and columns past the end repeat the last one
    const long long brow0 = (long long)e * g.N + n0;
    const uint8_t* a_base = g.A + (long long)row0 * ld;
    const uint8_t* b_base = g.B + brow0 * ld;
    const uint8_t* sa_base = g.A_sf + row0 * g.a_row_mul;
    const uint8_t* sb_base = g.B_sf + brow0 * g.b_row_mul;
    uint32_t a_off[C::kADma], b_off[C::kBDma], a_c, sa_off[C::kSaDma], sb_off[C::kSbDma];
    {
      // load i of the wave covers rows 8 (wave * n + i) .. + 7: the swizzle of a row 8 further differs,
      // so the chunk is computed per load and folded into the offset
#pragma unroll
      for (int i = 0; i < C::kADma; ++i) {
        const int r = (wave * C::kADma + i) * 8 + lane / 8;
        a_off[i] = (uint32_t)min(r, rows - 1) * (uint32_t)ld + (((lane & 7) ^ swz<8>(r)) << 4);
      }
#pragma unroll
      for (int i = 0; i < C::kBDma; ++i) {
        const int r = (wave * C::kBDma + i) * 8 + lane / 8;
        b_off[i] = (uint32_t)min(r, cols - 1) * (uint32_t)ld + (((lane & 7) ^ swz<8>(r)) << 4);
      }
      a_c = 0;
#pragma unroll
      for (int i = 0; i < C::kSaDma; ++i)
        sa_off[i] = (uint32_t)min(((wave * C::kSaDma + i) * 64 + lane) % BM, rows - 1) * (uint32_t)g.a_row_mul;
#pragma unroll
      for (int i = 0; i < C::kSbDma; ++i)
        sb_off[i] = (uint32_t)min(((wave * C::kSbDma + i) * 64 + lane) % BN, cols - 1) * (uint32_t)g.b_row_mul;
    }
    (void)a_c;

    auto issue = [&](int ks) {
      const uint32_t st = ring0 + (uint32_t)(ks & 1) * C::kStage;
      const long long k0 = (long long)ks * C::kRowB;
      if (ktail && ks == nst - 1) {  // chunks past the row's end repeat the row's first of the stage
#pragma unroll
        for (int i = 0; i < C::kADma; ++i) {
          const int r = (wave * C::kADma + i) * 8 + lane / 8;
          const uint32_t c = ((lane & 7) ^ swz<8>(r)) << 4;
          dma16(a_base + k0, k0 + c < ld ? a_off[i] : a_off[i] - c, uniform(st + (wave * C::kADma + i) * 1024));
        }
#pragma unroll
        for (int i = 0; i < C::kBDma; ++i) {
          const int r = (wave * C::kBDma + i) * 8 + lane / 8;
          const uint32_t c = ((lane & 7) ^ swz<8>(r)) << 4;
          dma16(b_base + k0, k0 + c < ld ? b_off[i] : b_off[i] - c, uniform(st + C::kA + (wave * C::kBDma + i) * 1024));
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::kADma; ++i)
          dma16(a_base + k0, a_off[i], uniform(st + (wave * C::kADma + i) * 1024));
#pragma unroll
        for (int i = 0; i < C::kBDma; ++i)
          dma16(b_base + k0, b_off[i], uniform(st + C::kA + (wave * C::kBDma + i) * 1024));
      }
#pragma unroll
      for (int i = 0; i < C::kSaDma; ++i) {
        const int t = wave * C::kSaDma + i, j = min(2 * ks + t / (BM / 64), nwords - 1);
        dma4(sa_base + j * g.a_word_mul, sa_off[i], uniform(st + C::kSA + t * 256));
      }
#pragma unroll
      for (int i = 0; i < C::kSbDma; ++i) {
        const int t = wave * C::kSbDma + i, j = min(2 * ks + t / (BN / 64), nwords - 1);
        dma4(sb_base + j * g.b_word_mul, sb_off[i], uniform(st + C::kSB + t * 256));
      }
    };

    struct Frags {
      v4i a[C::MI], b[C::NI];
    };
    int sa[C::MI], sb[C::NI];
    auto load = [&](int ks, int s, Frags& f) {
      const uint8_t* st = lds + (ks & 1) * C::kStage;
#pragma unroll
      for (int m = 0; m < C::MI; ++m)
        f.a[m] = *reinterpret_cast<const v4i*>(st + (fa ^ (uint32_t)((s << 4) ^ ((m & 1) << 6))) + m * 32 * C::kRowB);
#pragma unroll
      for (int n = 0; n < C::NI; ++n)
        f.b[n] = *reinterpret_cast<const v4i*>(st + (fb ^ (uint32_t)((s << 4) ^ ((n & 1) << 6))) + n * 32 * C::kRowB);
    };
    // the last stage's step s, where it lies past K for this lane: zero codes
    auto cut = [&](int s, Frags& f) {
      if (ktail && ((nst - 1) * 2 + kb) * 4 + s >= nblk) {
#pragma unroll
        for (int m = 0; m < C::MI; ++m) f.a[m] = v4i{0, 0, 0, 0};
      }
    };
    auto load_scales = [&](int ks) {
      const uint8_t* st = lds + (ks & 1) * C::kStage;
#pragma unroll
      for (int m = 0; m < C::MI; ++m) sa[m] = *reinterpret_cast<const int*>(st + wa + m * 128);
#pragma unroll
      for (int n = 0; n < C::NI; ++n) sb[n] = *reinterpret_cast<const int*>(st + wb + n * 128);
    };
    auto cut_scales = [&]() {  // the last stage's, past K: scales of 1, whatever the padding holds
      if (ktail) {
        const int left = nblk - ((nst - 1) * 2 + kb) * 4;
        const int keep = left >= 4 ? -1 : left <= 0 ? 0 : (1 << (8 * left)) - 1;
#pragma unroll
        for (int m = 0; m < C::MI; ++m) sa[m] = (sa[m] & keep) | (0x7f7f7f7f & ~keep);
#pragma unroll
        for (int n = 0; n < C::NI; ++n) sb[n] = (sb[n] & keep) | (0x7f7f7f7f & ~keep);
      }
    };
    auto mma = [&](auto& acc, const Frags& f, auto step) {
      constexpr int S = decltype(step)::value;
      auto wide = [](v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };
#pragma unroll
      for (int n = 0; n < C::NI; ++n)
#pragma unroll
        for (int m = 0; m < C::MI; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(f.b[n]), wide(f.a[m]), acc[m][n], 4, 4, S,
                                                                      sb[n], S, sa[m]);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;

    __syncthreads();  // every wave is done with the slots (the previous tile's results)
    issue(0);
    wait_vm_barrier<0>();
    if (nst > 1) issue(1);
    // a wave whose part lies past the group's rows or the columns only moves data
    const bool live = wm * WTM < rows && wn * WTN < cols;
    if (!live) {
      for (int ks = 0; ks + 1 < nst; ++ks) {
        wait_vm_barrier<0>();
        if (ks + 2 < nst) issue(ks + 2);
      }
      __syncthreads();
    } else {
      v16f acc[C::MI][C::NI];
#pragma unroll
      for (int m = 0; m < C::MI; ++m)
#pragma unroll
        for (int n = 0; n < C::NI; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;

      Frags f0, f1;
      load(0, 0, f0);
      load_scales(0);
      for (int ks = 0; ks + 1 < nst; ++ks) {
        load(ks, 1, f1);
        mma(acc, f0, I0{});
        load(ks, 2, f0);
        mma(acc, f1, I1{});
        load(ks, 3, f1);
        mma(acc, f0, I2{});
        wait_vm_barrier<0>();
        if (ks + 2 < nst) issue(ks + 2);
        load(ks + 1, 0, f0);
        mma(acc, f1, I3{});
        load_scales(ks + 1);
      }
      cut(0, f0);
      cut_scales();
      load(nst - 1, 1, f1);
      cut(1, f1);
      mma(acc, f0, I0{});
      load(nst - 1, 2, f0);
      cut(2, f0);
      mma(acc, f1, I1{});
      load(nst - 1, 3, f1);
      cut(3, f1);
      mma(acc, f0, I2{});
      mma(acc, f1, I3{});
      __syncthreads();  // every wave is past its last fragment read

      // lane: row ra + 32 m, columns 8 (i / 4) + 4 kb + i % 4 of column tile n; 256 bytes of each row
      // at a time, 16-byte chunks swizzled by row
      constexpr int es = sizeof(T), kPassCols = 256 / es;  // columns per pass
      constexpr int kPassN = kPassCols / 32;               // column tiles per pass
      uint8_t* out = lds + wave * (WTM * 256);
#pragma unroll
      for (int h = 0; h < (WTN + kPassCols - 1) / kPassCols; ++h) {
#pragma unroll
        for (int m = 0; m < C::MI; ++m)
#pragma unroll
          for (int nn = 0; nn < kPassN; ++nn) {
            const int n = h * kPassN + nn;
            if (n < C::NI) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int r = m * 32 + lrow, at = (nn * 32 + 8 * q + 4 * kb) * es;  // byte in the 256-byte run
                T v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = Elem<T>::put(acc[m][n][4 * q + j]);
                uint8_t* to = out + r * 256 + ((((at >> 4) ^ (r & 15)) << 4) | (at & 15));
                __builtin_memcpy(__builtin_assume_aligned(to, 4 * es), v, 4 * es);
              }
            }
          }
        // read back row by row (the wave's own part: no barrier, LDS operations stay in order)
        const int c = lane & 15;
        const int col = wn * WTN + h * kPassCols + c * (16 / es);
#pragma unroll 4
        for (int r = lane >> 4; r < WTM; r += 4) {
          Chunk16<es> v;
          __builtin_memcpy(&v, __builtin_assume_aligned(out + r * 256 + ((c ^ (r & 15)) << 4), 16), 16);
          if (wm * WTM + r < rows && h * kPassCols + c * (16 / es) < WTN) {
            T* dst = static_cast<T*>(g.C) + (long long)(row0 + wm * WTM + r) * g.c_stride + n0 + col;
            if (col + 16 / es <= cols) {
              *reinterpret_cast<Chunk16<es>*>(dst) = v;
            } else {
              T one[16 / es];
              __builtin_memcpy(one, &v, 16);
#pragma unroll
              for (int j = 0; j < 16 / es; ++j)
                if (col + j < cols) dst[j] = one[j];
            }
          }
        }
      }
    }
  }
}

template <typename T, int BM, int BN, int NW, int WTM, int WTN>
static hipError_t launch_tiles(const Mxfp4GemmArgs& g, hipStream_t s) {
  using C = TileCfg<BM, BN, NW, WTM, WTN>;
  auto kern = mxfp4_gemm_tile_kernel<T, BM, BN, NW, WTM, WTN>;
  constexpr int kMaxGroups = 1024;
  const size_t bytes = C::kPlan + (size_t)(3 * g.groups + 1 + NW) * 4;
  static std::atomic<uint64_t> ready{0};  // the LDS limit is raised once per device
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize,
                            C::kPlan + (3 * kMaxGroups + 1 + NW) * 4);
    if (e != hipSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  // at most this many tiles; one workgroup per CU, in whole rows of 8 XCDs
  const long long most = (((long long)g.rows + (long long)g.groups * (BM - 1)) / BM) * ((g.N + BN - 1) / BN);
  const long long cus = device_cus();
  const unsigned grid = (unsigned)(((most < cus ? most : cus) + 7) / 8 * 8);
  kern<<<dim3(grid), dim3(C::NT), bytes, s>>>(g);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch(const Mxfp4GemmArgs& g, int variant, hipStream_t s) {
  const long long avg = g.rows / g.groups;
  if (variant == 1 || (variant < 0 && avg > 64)) return launch_tiles<T, 256, 256, 4, 128, 128>(g, s);
  mxfp4_gemm_rows_kernel<T, 4, 2, 2><<<dim3((unsigned)((g.N + 31) / 32), (unsigned)g.groups), 256, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_mxfp4_gemm(const Mxfp4GemmArgs& g, int out_dtype, int variant, hipStream_t s) {
  if (out_dtype == 0) return launch<Bf16>(g, variant, s);
  if (out_dtype == 1) return launch<F16>(g, variant, s);
  return launch<float>(g, variant, s);
}

}  // namespace moe
