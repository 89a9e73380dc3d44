// Matrix product of two 8-bit block-scaled operands:
//   Y[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a8[m, k] w8[n, k],
// blocks of 128 channels, e4m3 codes, fp32 scales (any positive numbers), Y fp16 or bf16.
//
// One v_mfma_f32_16x16x128_f8f6f4 covers exactly one scale block, so its result is the block's
// inner sum; the scales multiply it in fp32 as it is added to the accumulator (one fma per value
// and block). The weight is the MFMA's row operand and the activation its column operand: a lane
// then holds one activation row's results, so sa is one value per lane and sw one per wave. Which
// channel sits at which of the 32 bytes a lane supplies does not matter as long as both operands
// agree; lane group lg (lane / 16) supplies the 16-byte chunks lg and lg + 4 of a block.
//
//   few rows  fp8_skinny_kernel (up to 8, or 48 on small weights): bound by the weight's bytes,
//             which go from memory straight into the MFMA's registers; 8 waves of a workgroup share
//             16 weight rows and split K.
//   else      fp8_tiled_kernel: tiles of 64, 128 or 256 rows, both operands through LDS, moved there
//             by the buffer unit; with fewer tiles than CUs K is split over workgroups and the fp32
//             partials are added in slice order by fp8_sum_slices_kernel.
// Measured per call: 1 x 28672 x 8192 42 us (5.6 TB/s); 77 x 11000 x 4112 21 us (two launches);
// 8192 x 11008 x 4096 400 us (1.85 PFLOP/s; matrix units busy 40% of the cycles at 2.0 GHz, the
// scaling's vector instructions 31%).
// Rounding: the instruction adds the channels in groups of 8 (of a lane's consecutive bytes), each
// product cut 13 bits below the group's largest sum of operand exponents, and the groups in fp32
// (measured; random normal operands end within 2e-5 of the exact sum, relative norm). That is the
// price of the 8-bit rate: far below the rounding of a bf16 or fp16 output. Everything else is fp32,
// and Y is rounded once.
#include "fp8_format.h"
#include "kernels.h"
#include "tile_order.h"

namespace awq {

namespace {

constexpr int kSkWaves = 8;

__device__ __forceinline__ intx8 frag_of(uint4 a, uint4 b) {
  return intx8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
__device__ __forceinline__ floatx4 mfma_fp8(intx8 a, intx8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ uint16_t to16(float f) {
  return DT == kF16 ? f2h(f) : f2bf(f);
}
// four consecutive outputs of row m from column n on
template <int DT>
__device__ __forceinline__ void store4(uint16_t* Y, int64_t N, int64_t m, int64_t n, floatx4 v) {
  uint16_t* p = Y + m * N + n;
  if (n + 3 < N && (N & 3) == 0) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2((uint32_t)to16<DT>(v[0]) | ((uint32_t)to16<DT>(v[1]) << 16),
                   (uint32_t)to16<DT>(v[2]) | ((uint32_t)to16<DT>(v[3]) << 16));
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) p[r] = to16<DT>(v[r]);
  }
}

}  // namespace

// MT blocks of 16 activation rows (M <= 16 MT; rows past M read row M - 1 and are not stored, as
// are weight rows past N). Wave w takes the blocks w, w + 8, ...; U of them have their loads in
// flight together. The waves' sums are added in wave order through LDS.
template <int MT, int U, int DT>
__global__ __launch_bounds__(64 * kSkWaves) void fp8_skinny_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ sa, const uint8_t* __restrict__ W,
    const float* __restrict__ sw, int64_t M, int64_t N, int64_t K, uint16_t* __restrict__ Y) {
  __shared__ floatx4 red[kSkWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int KB = (int)((K + 127) / 128);
  const int64_t nr = n0 + li < N ? n0 + li : N - 1;
  const uint8_t* wr = W + nr * K + 16 * lg;
  const float* swr = sw + (n0 >> 7) * KB;
  const uint8_t* ar[MT];
  const float* sar[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = 16 * t + li < M ? 16 * t + li : M - 1;
    ar[t] = A + m * K + 16 * lg;
    sar[t] = sa + m * KB;
  }
  floatx4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};

  // 16 bytes at p + k, zeros when the chunk lies past the row's K channels
  auto chunk = [&](const uint8_t* p, int64_t k) {
    return k + 16 * lg < K ? *reinterpret_cast<const uint4*>(p + k) : make_uint4(0u, 0u, 0u, 0u);
  };
  for (int kb0 = wave; kb0 < KB; kb0 += kSkWaves * U) {
    uint4 w[U][2], a[U][MT][2];
    float s[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + kSkWaves * u;
      const int64_t k = (int64_t)kb * 128;          // past K: zeros
      w[u][0] = chunk(wr, k);
      w[u][1] = chunk(wr, k + 64);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + kSkWaves * u;
      const int kc = kb < KB ? kb : KB - 1;
      const float swv = swr[kc];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        a[u][t][0] = chunk(ar[t], (int64_t)kb * 128);
        a[u][t][1] = chunk(ar[t], (int64_t)kb * 128 + 64);
        s[u][t] = sar[t][kc] * swv;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const floatx4 p = mfma_fp8(frag_of(w[u][0], w[u][1]), frag_of(a[u][t][0], a[u][t][1]),
                                   floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(p[r], s[u][t], acc[t][r]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * MT; e += 64 * kSkWaves) {
    const int t = e >> 6, l = e & 63;
    floatx4 v = red[0][t][l];
#pragma unroll
    for (int w = 1; w < kSkWaves; ++w) v = v + red[w][t][l];
    const int64_t m = 16 * t + (l & 15), n = n0 + 4 * (l >> 4);
    if (m < M) store4<DT>(Y, N, m, n, v);
  }
}

// Tile BM (activation rows) x BN (weight rows), one scale block of K per step, WM x WN waves. The
// tiles of a step (rows of 128 bytes) are moved into one of two LDS stages by the buffer unit
// while the other stage is multiplied.
// Chunk c (16 bytes) of LDS row r sits at position c ^ ((r >> 1) & 7): the 16 rows a fragment read
// touches at once then cover all 64 banks. The step's activation scales (one per row, gathered)
// go to LDS the same way. Rows past M or N, and channels past K, read as zeros.
template <int BM, int BN, int WM, int WN, int DT>
__global__ __launch_bounds__(64 * WM * WN) void fp8_tiled_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ sa, const uint8_t* __restrict__ W,
    const float* __restrict__ sw, int64_t M, int64_t N, int64_t K, uint16_t* __restrict__ Y,
    uint32_t tilesM, uint32_t tilesN, int steps_per_slice,
    float* __restrict__ partials, int64_t slice_stride) {
  constexpr int kWaves = WM * WN;
  constexpr int kTiles = (BM + BN) * 128, kStage = kTiles + 4 * BM;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16;   // 16 x 16 blocks of a wave
  constexpr int kLoads = (BM + BN) / 8 / kWaves;        // 1 KiB loads per wave and step
  static_assert(kLoads % 2 == 0, "a load's 8-row group has the parity of its index");
  extern __shared__ __attribute__((aligned(1024))) char smem[];   // two stages
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave / WN, wn = wave % WN;
  const int li = lane & 15, lg = lane >> 4;

  const TileAt at = tile_order<8>(tilesM, tilesN);
  const int64_t m0 = (int64_t)at.tm * BM, n0 = (int64_t)at.tn * BN;
  const int KB = (int)((K + 127) / 128);
  const int b0 = (int)at.slice * steps_per_slice;
  const int b1 = b0 + steps_per_slice < KB ? b0 + steps_per_slice : KB;

  // ---- loads: LDS rows 0 .. BM - 1 are activation rows, BM .. BM + BN - 1 weight rows; load j of
  // wave w fills rows 8 (kLoads w + j) .. + 7, lane l the position l % 8 of row l / 8 ------------
  const rsrc_t ra = make_rsrc(A + m0 * K, (uint32_t)((M - m0 < BM ? M - m0 : BM) * K));
  const rsrc_t rw = make_rsrc(W + n0 * K, (uint32_t)((N - n0 < BN ? N - n0 : BN) * K));
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  uint32_t voff[2], chunk[2];   // by the parity of the 8-row group (the swizzle key's bit 2)
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    chunk[p] = (uint32_t)((lane & 7) ^ ((4 * p + (lane >> 4)) & 7));
    voff[p] = (uint32_t)(lane >> 3) * (uint32_t)K + chunk[p] * 16u;
  }
  auto issue = [&](int b, int st) {
    const uint32_t k = (uint32_t)b * 128u;
    const bool tail = k + 128u > (uint32_t)K;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int g = kLoads * wave + j;              // 8-row group (wave-uniform)
      const bool isw = g >= BM / 8;
      const uint32_t so = (uint32_t)(8 * (isw ? g - BM / 8 : g)) * (uint32_t)K + k;
      uint32_t vo = voff[j & 1];                    // g and j have the same parity
      if (tail && k + chunk[j & 1] * 16u >= (uint32_t)K) vo = 0x80000000u;   // past every range
      buffer_load16_lds_so(isw ? rw : ra, lds0 + (uint32_t)(st * kStage + g * 1024), vo, so);
    }
  };

  // ---- scales: wave w < BM / 64 gathers sa of rows 64 w .. 64 w + 63; sw is one value per wave ----
  const rsrc_t rs = make_rsrc(sa + m0 * KB, (uint32_t)((M - m0 < BM ? M - m0 : BM) * KB * 4));
  const uint32_t soff = (uint32_t)(64 * wave + lane) * (uint32_t)KB * 4u;
  auto issue_scales = [&](int b, int st) {
    if (wave < BM / 64)
      buffer_load4_lds(rs, lds0 + (uint32_t)(st * kStage + kTiles + 256 * wave), soff,
                       (uint32_t)b * 4u);
  };
  const int64_t nw = n0 + wn * NB * 16;             // the wave's first column
  const float* swr = sw + ((nw < N ? nw : N - 1) >> 7) * KB;
  static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0, "one weight scale per wave and step");

  // ---- fragments: row r at r * 128, chunks lg and lg + 4 --------------------------------------
  const int key = (li >> 1) & 7;
  const uint32_t f0 = (uint32_t)(li * 128 + ((lg ^ key) << 4));
  const uint32_t f1 = (uint32_t)(li * 128 + (((lg + 4) ^ key) << 4));
  auto frag = [&](const char* rows) {
    return frag_of(*reinterpret_cast<const uint4*>(rows + f0),
                   *reinterpret_cast<const uint4*>(rows + f1));
  };
  floatx4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  // Step b: the matrix instructions of one 16-row block after another. While block i's run, block
  // i + 2's fragment is read (one block ahead is less than an LDS read takes) and block i - 1's
  // results are scaled and added. Two blocks before the end the wave waits for step b + 1's loads
  // and passes the barrier (its own reads of this stage are done, everyone's loads have landed): the
  // last blocks' instructions then cover the issue of step b + 2's loads into this stage and the
  // reads of step b + 1's first fragments.
  // The last steps load the last block again, so that no wait stands behind a branch.
  static_assert(MB % 2 == 0, "the fragment registers take turns");
  intx8 wf[NB], af[2];
  floatx4 part[NB];           // results not yet added, and their row block's scale
  float psc = 0.0f, asc[2];   // scales of the blocks in af
#pragma unroll
  for (int j = 0; j < NB; ++j) part[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto wrows = [&](int st) { return smem + st * kStage + (BM + wn * NB * 16) * 128; };
  auto arows = [&](int st) { return smem + st * kStage + wm * MB * 16 * 128; };
  auto scale_at = [&](int st, int i) {
    return reinterpret_cast<const float*>(smem + st * kStage + kTiles)[(wm * MB + i) * 16 + li];
  };
  auto step = [&](int b, int st, float sw0, float sw1) {
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int ip = i == 0 ? MB - 1 : i - 1;
      if (i == MB - 2) {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        __syncthreads();
        issue(b + 2 < b1 ? b + 2 : b1 - 1, st);
        issue_scales(b + 2 < b1 ? b + 2 : b1 - 1, st);
      }
      float sc;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const floatx4 p = mfma_fp8(wf[j], af[i & 1], floatx4{0.f, 0.f, 0.f, 0.f});
        if (i == MB - 1) wf[j] = frag(wrows(st ^ 1) + j * 16 * 128);
        if (j == NB - 1) {   // the block's fragment is used: read the next but one
          sc = asc[i & 1];
          const int st2 = i + 2 < MB ? st : st ^ 1, i2 = i + 2 < MB ? i + 2 : i + 2 - MB;
          af[i & 1] = frag(arows(st2) + i2 * 16 * 128);
          asc[i & 1] = scale_at(st2, i2) * (i + 2 < MB ? sw0 : sw1);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[ip][j][r] = __builtin_fmaf(part[j][r], psc, acc[ip][j][r]);
        // here, not later: the sums would otherwise pile up behind the matrix instructions
        asm volatile("" : "+v"(acc[ip][j]));
        part[j] = p;
        __builtin_amdgcn_sched_barrier(0);
      }
      psc = sc;
    }
  };
  auto weight_scale = [&](int b) { return swr[b < b1 ? b : b1 - 1]; };
  issue(b0, 0);
  issue_scales(b0, 0);
  issue(b0 + 1 < b1 ? b0 + 1 : b0, 1);
  issue_scales(b0 + 1 < b1 ? b0 + 1 : b0, 1);
  float sw0 = weight_scale(b0), sw1 = weight_scale(b0 + 1);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NB; ++j) wf[j] = frag(wrows(0) + j * 16 * 128);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    af[i] = frag(arows(0) + i * 16 * 128);
    asc[i] = scale_at(0, i) * sw0;
  }
  int b = b0;
  for (; b + 1 < b1; b += 2) {
    const float sw2 = weight_scale(b + 2), sw3 = weight_scale(b + 3);
    step(b, 0, sw0, sw1);
    step(b + 1, 1, sw1, sw2);
    sw0 = sw2;
    sw1 = sw3;
  }
  if (b < b1) step(b, 0, sw0, sw1);
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[MB - 1][j][r] = __builtin_fmaf(part[j][r], psc, acc[MB - 1][j][r]);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));   // no load may land in LDS that is no longer ours

  // ---- store ----------------------------------------------------------------------------------
  if (!partials && (N & 7) == 0) {
    // Through LDS, 64 rows of the wave's columns at a time (a region per wave), so that a row's columns
    // leave in whole lines (8192x11008x4096: 396 us, 404 in 8-byte pieces straight from the
    // accumulators).
    static_assert(MB % 4 == 0, "blocks of 64 rows");
    constexpr int kPitch = NB * 32 + 16, kChunks = NB * 2;   // bytes and 16-byte chunks of a row
    __syncthreads();   // the stages are read
    char* reg = smem + wave * 64 * kPitch;
#pragma unroll
    for (int i0 = 0; i0 < MB; i0 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const floatx4 v = acc[i0 + i][j];
          *reinterpret_cast<uint2*>(reg + (16 * i + li) * kPitch + j * 32 + lg * 8) =
              make_uint2((uint32_t)to16<DT>(v[0]) | ((uint32_t)to16<DT>(v[1]) << 16),
                         (uint32_t)to16<DT>(v[2]) | ((uint32_t)to16<DT>(v[3]) << 16));
        }
#pragma unroll
      for (int e = 0; e < kChunks; ++e) {
        const int row = (64 * e + lane) / kChunks, c = lane % kChunks;
        const uint4 v = *reinterpret_cast<const uint4*>(reg + row * kPitch + c * 16);
        const int64_t m = m0 + (wm * MB + i0) * 16 + row, n = nw + 8 * c;
        if (m < M && n < N) *reinterpret_cast<uint4*>(Y + m * N + n) = v;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t m = m0 + (wm * MB + i) * 16 + li;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t n = nw + j * 16 + 4 * lg;
      if (partials) {
        float* P = partials + (int64_t)at.slice * slice_stride + m * N + n;
        if (n + 3 < N && (N & 3) == 0) {
          *reinterpret_cast<floatx4*>(P) = acc[i][j];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < N) P[r] = acc[i][j][r];
        }
      } else {
        store4<DT>(Y, N, m, n, acc[i][j]);
      }
    }
  }
}

// Y = round(sum of the S slices' partials), added in slice order; four elements per thread.
template <int DT>
__global__ __launch_bounds__(256) void fp8_sum_slices_kernel(const float* __restrict__ P, int S,
                                                             int64_t stride, int64_t MN,
                                                             uint16_t* __restrict__ Y) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= MN) return;
  const floatx4 t = sum_slices(P + e, S, stride);   // within the padded slice
  if (e + 3 < MN) {
    *reinterpret_cast<uint2*>(Y + e) =
        make_uint2((uint32_t)to16<DT>(t[0]) | ((uint32_t)to16<DT>(t[1]) << 16),
                   (uint32_t)to16<DT>(t[2]) | ((uint32_t)to16<DT>(t[3]) << 16));
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (e + r < MN) Y[e + r] = to16<DT>(t[r]);
  }
}

// Which kernel. A workgroup of the skinny kernel reads all activations for 16 weight rows, which
// costs more than the weight's bytes as M grows; the tiled one with K slices is two launches, a few
// us, which small weights do not earn back. Skinny and tiled, us:
//   28672 x 8192: M = 8 57 and 57, M = 16 70 and 58, M = 64 178 and 66
//   11008 x 4096: M = 8 14.5 and 14.5, M = 16 17.7 and 15.1, M = 64 41 and 21
//   4096 x 4096:  M = 16 9.3 and 13.8, M = 48 13.7 and 13.9, M = 64 15.5 and 13.8
static bool skinny(int64_t M, int64_t N, int64_t K) {
  return M <= 8 || (M <= 48 && N * K <= (int64_t(1) << 24));
}

Fp8GemmPlan fp8_gemm_plan(int64_t M, int64_t N, int64_t K) {
  Fp8GemmPlan p{};
  const int64_t KB = (K + 127) / 128;
  p.S = 1;
  p.steps = KB;
  if (skinny(M, N, K)) return p;
  const int64_t t256 = ((M + 255) / 256) * ((N + 255) / 256);
  // 256-row tiles while they fill the CUs and are not half empty (128 rows instead, us:
  // 100 x 65536 x 4096 79 to 74, 77 x 80000 x 2048 62 to 49)
  p.tile = t256 >= 256 && M > 128 ? 256 : M > 64 ? 128 : 64;
  const int64_t bn = p.tile == 256 ? 256 : 128;
  const int64_t tiles = ((M + p.tile - 1) / p.tile) * ((N + bn - 1) / bn);
  if (p.tile != 256 && tiles < 256) {
    int64_t S = 512 / tiles;
    const int64_t smax = KB / 4;
    S = S > smax ? smax : S;
    S = S < 1 ? 1 : S;
    p.steps = (KB + S - 1) / S;
    p.S = (KB + p.steps - 1) / p.steps;
  }
  p.stride = (M * N + 3) / 4 * 4;
  p.ws_bytes = p.S > 1 ? (size_t)(p.S * p.stride * 4) : 0;
  return p;
}

template <int DT>
static hipError_t fp8_gemm_dt(const uint8_t* A, const float* sa, const uint8_t* W, const float* sw,
                              int64_t M, int64_t N, int64_t K, uint16_t* Y, void* ws,
                              hipStream_t stream) {
  if (skinny(M, N, K)) {
    const unsigned grid = (unsigned)((N + 15) / 16);
#define AWQ_SK(MT_, U_)                                                                \
  fp8_skinny_kernel<MT_, U_, DT><<<grid, 64 * kSkWaves, 0, stream>>>(A, sa, W, sw, M, N, K, Y)
    if (M <= 16) AWQ_SK(1, 4); else if (M <= 32) AWQ_SK(2, 2); else AWQ_SK(4, 1);
#undef AWQ_SK
    return hipGetLastError();
  }
  const Fp8GemmPlan p = fp8_gemm_plan(M, N, K);
  const uint32_t tm = (uint32_t)((M + p.tile - 1) / p.tile);
  const int64_t bn = p.tile == 256 ? 256 : 128;
  const uint32_t tn = (uint32_t)((N + bn - 1) / bn);
  const uint32_t tiles = tm * tn;
  float* P = p.S > 1 ? static_cast<float*>(ws) : nullptr;
#define AWQ_FT(BM_, BN_, WM_, WN_)                                                             \
  fp8_tiled_kernel<BM_, BN_, WM_, WN_, DT><<<tiles * (unsigned)p.S, 64 * WM_ * WN_,            \
                                             2 * ((BM_ + BN_) * 128 + 4 * BM_), stream>>>(     \
      A, sa, W, sw, M, N, K, Y, tm, tn, (int)p.steps, P, p.stride)
  if (p.tile == 256) AWQ_FT(256, 256, 2, 4);
  else if (p.tile == 128) AWQ_FT(128, 128, 2, 2);
  else AWQ_FT(64, 128, 1, 4);
#undef AWQ_FT
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.S == 1) return e;
  const int64_t MN = M * N;
  fp8_sum_slices_kernel<DT><<<(unsigned)((MN + 1023) / 1024), 256, 0, stream>>>(
      P, (int)p.S, p.stride, MN, Y);
  return hipGetLastError();
}

hipError_t launch_fp8_gemm(const uint8_t* A, const float* sa, const uint8_t* W, const float* sw,
                           int64_t M, int64_t N, int64_t K, int dtype, uint16_t* Y, void* ws,
                           hipStream_t stream) {
  return dtype == kF16 ? fp8_gemm_dt<kF16>(A, sa, W, sw, M, N, K, Y, ws, stream)
                       : fp8_gemm_dt<kBF16>(A, sa, W, sw, M, N, K, Y, ws, stream);
}

}  // namespace awq
