// The gated feed-forward block on packed 4-bit weights,
//   g = A Wg^T,  u = A Wu^T,  H = act(g) u,   W[n, k] = c(q[n, k]) step[n, k / G],
// both projections, the activation and the product in one pass over A and the codes; optionally
// g and u are kept in 8 bits (fp8_format.h, blocks of 1 x 128) for the backward pass. Gate and up
// read one input, whose s is folded into the operator before them, so there is no s here.
//
// Every kernel multiplies the exact codes c(q) (integers, exact in fp16) with the fp16
// activations, sums in fp32 and applies the fp32 step to each group's partial sum; g and u are
// fp32 until H is rounded once, and until they are cut to 8 bits.
//   M <= 2    w4a16_gated_gemv_kernel: bound by the codes' bytes; a wave owns one output channel,
//             its gate row and its up row.
//   few rows  w4a16_gated_skinny_kernel (up to 16, or 32 on small weights): MFMA, codes from memory
//             to registers, K over 8 waves.
//   else      w4a16_gated_tiled_kernel: 128 (64, 32) rows x 128 output channels; with few tiles K is
//             split over workgroups and w4a16_gated_finish_kernel adds the slices in order and applies
//             the activation. The 8-bit form always takes this path: 128 output channels of a
//             tile are one block of the format.
// Measured per call: 1 row of 11008 x 4096 11.6 us (46.5 MB, 4.0 TB/s); 16 rows 21.5 us; 512 rows,
// groups of 64 with zero points, 148 us (0.62 PFLOP/s); 4096 rows with the 8-bit form 746 us (0.99
// PFLOP/s; matrix units busy 46% of the cycles at 2.0 GHz, the decode's and scaling's vector
// instructions 44%).
#include "fp8_format.h"
#include "gated_act.h"
#include "kernels.h"
#include "tile_order.h"

namespace awq {

namespace {
constexpr int kGvPos = 2;         // chunk positions per lane whose loads are in flight together
constexpr int kChunkBytes = 80;   // LDS bytes per 32-channel chunk: 64 of activations, 16 padding
constexpr int kGvWaves = 8;
constexpr int kSkWaves = 8;
constexpr int kTN = 128;          // output channels of a tile of the tiled kernel
}  // namespace

// ---------------------------------------------------------------------------------------------
// One or two rows. The activations go to LDS once per workgroup in the decode order (channel t
// next to t + 4 of each 8); lane l of a wave takes the 32-channel chunks l, l + 64, ... of the
// channel's gate row and up row. ONE: all chunks fit one load batch (K <= 4096). TI: table
// entries of 8 channels per thread (K <= 4096 TI), loaded before the codes.
template <int GS, bool ZP, int ACT, bool ONE, int TI, int MB>
__global__ __launch_bounds__(64 * kGvWaves) void w4a16_gated_gemv_kernel(
    const uint16_t* __restrict__ A, int64_t M, int64_t N, int64_t K, GatedWeights W,
    uint16_t* __restrict__ H) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * kGvWaves + wave;
  const int64_t n = n0 < N ? n0 : N - 1;          // past N: row N - 1, not stored
  const int nch = (int)(K / 32);
  const int64_t ngr = K / GS, wpr = K / 8;
  const int npos = (nch + 63) / 64;
  const size_t tbytes = (size_t)nch * kChunkBytes;

  uint4 araw[MB][TI];
  const int nq8 = (int)(K / 8);
#pragma unroll
  for (int it = 0; it < TI; ++it) {
    const int q8 = tid + 64 * kGvWaves * it;
    const int qc = q8 < nq8 ? q8 : 0;
#pragma unroll
    for (int m = 0; m < MB; ++m)
      araw[m][it] = *reinterpret_cast<const uint4*>(A + (m < M ? m : M - 1) * K + (int64_t)qc * 8);
  }
  struct Buf {
    uint4 w[kGvPos][2];
    uint32_t st[kGvPos][2], z[kGvPos][2];
  };
  auto load = [&](int p0, Buf& b) {
#pragma unroll
    for (int j = 0; j < kGvPos; ++j) {
      const int c = lane + 64 * (p0 + j);
      const int cc = c < nch ? c : 0;             // a chunk past the row adds nothing (see below)
      const int64_t g = n * ngr + ((int64_t)cc * 32) / GS;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        b.w[j][r] = *reinterpret_cast<const uint4*>(W.q[r] + n * wpr + 4 * cc);
        b.st[j][r] = W.s[r][g];
        if (ZP) b.z[j][r] = W.z[r][g];
      }
    }
  };
  Buf wb[ONE ? 1 : 2];
  load(0, wb[0]);
  __builtin_amdgcn_sched_barrier(0);              // the code loads stay ahead of the table

#pragma unroll
  for (int it = 0; it < TI; ++it) {
    const int q8 = tid + 64 * kGvWaves * it;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const uint4 a = araw[m][it];                // channels (0,1) (2,3) (4,5) (6,7)
      const uint32_t p0 = __builtin_amdgcn_perm(a.z, a.x, 0x05040100u);   // (0, 4)
      const uint32_t p1 = __builtin_amdgcn_perm(a.z, a.x, 0x07060302u);   // (1, 5)
      const uint32_t p2 = __builtin_amdgcn_perm(a.w, a.y, 0x05040100u);   // (2, 6)
      const uint32_t p3 = __builtin_amdgcn_perm(a.w, a.y, 0x07060302u);   // (3, 7)
      if (q8 < nq8)
        *reinterpret_cast<uint4*>(lds + m * tbytes + (size_t)(q8 >> 2) * kChunkBytes +
                                  (q8 & 3) * 16) = make_uint4(p0, p1, p2, p3);
    }
  }
  __syncthreads();

  float part[2][MB];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int m = 0; m < MB; ++m) part[r][m] = 0.0f;
  auto process = [&](int p0, const Buf& b) {
#pragma unroll
    for (int j = 0; j < kGvPos; ++j) {
      const int c = lane + 64 * (p0 + j);
      const bool ok = c < nch;
      const int cc = ok ? c : 0;
      half2_t lo[2], hi[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float zc = ZP ? (float)b.z[j][r] : 8.0f;
        const _Float16 a = (_Float16)(1024.0f + zc), d = (_Float16)(-64.0f - zc);
        lo[r] = half2_t{a, a};
        hi[r] = half2_t{d, d};
      }
      float acc[2][MB][2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[r][m][0] = acc[r][m][1] = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint4 a4[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m)
          a4[m] = *reinterpret_cast<const uint4*>(lds + m * tbytes + (size_t)cc * kChunkBytes +
                                                  16 * v);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t wv = v == 0 ? b.w[j][r].x : v == 1 ? b.w[j][r].y
                            : v == 2 ? b.w[j][r].z : b.w[j][r].w;
          half2_t qp[4];
          unpack_word8<ZP>(wv, lo[r], hi[r], qp);
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const uint32_t ap[4] = {a4[m].x, a4[m].y, a4[m].z, a4[m].w};
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
              acc[r][m][jj & 1] = __builtin_amdgcn_fdot2(
                  qp[jj], __builtin_bit_cast(half2_t, ap[jj]), acc[r][m][jj & 1], false);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float st = h2f((uint16_t)b.st[j][r]);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          const float t = __builtin_fmaf(st, acc[r][m][0] + acc[r][m][1], part[r][m]);
          part[r][m] = ok ? t : part[r][m];
        }
      }
    }
  };
  if constexpr (ONE) {
    process(0, wb[0]);
  } else {
    for (int p = 0; p < npos; p += 2 * kGvPos) {
      if (p + kGvPos < npos) load(p + kGvPos, wb[ONE ? 0 : 1]);
      process(p, wb[0]);
      if (p + kGvPos < npos) {
        if (p + 2 * kGvPos < npos) load(p + 2 * kGvPos, wb[0]);
        process(p + kGvPos, wb[ONE ? 0 : 1]);
      }
    }
  }
  // lanes 0..31 end with the gate's sum, lanes 32..63 with the up row's, in a fixed order
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const bool hi = lane >= 32;
    float v = (hi ? part[1][m] : part[0][m]) + __shfl_xor(hi ? part[0][m] : part[1][m], 32);
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) v += __shfl_xor(v, mk);
    const float u = __shfl_xor(v, 32);
    if (lane == 0 && n0 < N && m < M) H[m * N + n0] = f2h(act_f<ACT>(v) * u);
  }
}

namespace {

// Pair j (channels 2j, 2j + 1) of a word's 8 codes as exact fp16 values: byte j is spread to bytes 0
// and 2; with the exponent bits around them, and bit 3 of signed codes flipped, the pair is
// (1024 + u, 1024 + 16 u'), and one packed fma with (1, 1/16) and -(1024 + zc, 64 + zc) gives
// (c, c'); zc = 8 for signed codes (u = c + 8) or the zero point.
template <bool ZP>
__device__ __forceinline__ void decode_pair(uint32_t w, int j, half2_t nsub, half8_t& f) {
  constexpr uint32_t kExp = ZP ? 0x64006400u : 0x64806408u;
  const uint32_t t = __builtin_amdgcn_perm(w, w, 0x0C000C00u | (uint32_t)j | ((uint32_t)j << 16));
  const half2_t q = __builtin_elementwise_fma(
      __builtin_bit_cast(half2_t, (t & 0x00F0000Fu) ^ kExp),
      half2_t{(_Float16)1.0f, (_Float16)0.0625f}, nsub);
  f[2 * j] = q[0];
  f[2 * j + 1] = q[1];
}
template <bool ZP>
__device__ __forceinline__ half8_t decode8(uint32_t w, half2_t nsub) {
  half8_t f;
#pragma unroll
  for (int j = 0; j < 4; ++j) decode_pair<ZP>(w, j, nsub, f);
  return f;
}
__device__ __forceinline__ half2_t decode_nsub(float zc) {
  return half2_t{(_Float16)(-1024.0f - zc), (_Float16)(-64.0f - zc)};
}

// Which 8-channel chunk of a 128-channel block lane group lg feeds to MFMA kk (0..3). Groups of
// 128: 4 lg + kk (the lane's four words are one 16-byte load). Groups of 64: MFMAs 0, 1 cover
// the first group and 2, 3 the second, chunk 8 (kk / 2) + 2 lg + kk % 2 (two 8-byte loads).
template <int GS>
__device__ __forceinline__ int chunk_of(int lg, int kk) {
  return GS == 128 ? 4 * lg + kk : 8 * (kk >> 1) + 2 * lg + (kk & 1);
}
template <int GS>
__device__ __forceinline__ void load_block(const uint32_t* row, int lg, uint32_t (&w)[4]) {
  if (GS == 128) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + 4 * lg);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(row + 2 * lg);
    const uint2 b = *reinterpret_cast<const uint2*>(row + 8 + 2 * lg);
    w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
  }
}

}  // namespace

// ---------------------------------------------------------------------------------------------
// Up to 16 MT rows: a workgroup owns 16 output channels (their gate and up rows), its 8 waves
// split the 128-channel blocks of K; the waves' sums are added in wave order through LDS. The
// activations are the MFMA's row operand, the codes its column operand, so that a lane's results
// all belong to one output channel and the step is one value per lane and group.
template <int GS, bool ZP, int ACT, int MT>
__global__ __launch_bounds__(64 * kSkWaves) void w4a16_gated_skinny_kernel(
    const uint16_t* __restrict__ A, int64_t M, int64_t N, int64_t K, GatedWeights W,
    uint16_t* __restrict__ H) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  floatx4* red = reinterpret_cast<floatx4*>(lds);   // [wave][matrix][MT][lane]
  constexpr int kG = 128 / GS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t n = n0 + li < N ? n0 + li : N - 1;
  const int KB = (int)(K / 128);
  const uint16_t* ar[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) ar[t] = A + (16 * t + li < M ? 16 * t + li : M - 1) * K;
  floatx4 acc[2][MT];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[r][t] = floatx4{0.f, 0.f, 0.f, 0.f};

  struct Block {
    uint32_t w[2][4];
    half8_t a[MT][4];
  };
  auto load = [&](int kb, Block& b) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      load_block<GS>(W.q[r] + n * (K / 8) + (int64_t)kb * 16, lg, b.w[r]);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        b.a[t][kk] = *reinterpret_cast<const half8_t*>(ar[t] + (int64_t)kb * 128 +
                                                       8 * chunk_of<GS>(lg, kk));
  };
  // group steps and zero points of four of the wave's blocks at a time, one per lane group (groups of
  // 64: both of a block in one load), handed to all lane groups when their block comes
  struct Steps {
    uint32_t st[2], z[2];
  };
  Steps sv;
  auto load_steps = [&](int kb) {
    const int kl = kb + kSkWaves * lg < KB ? kb + kSkWaves * lg : KB - 1;
    const int64_t g = n * (K / GS) + (int64_t)kl * kG;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (GS == 128) {
        sv.st[r] = W.s[r][g];
        if (ZP) sv.z[r] = W.z[r][g];
      } else {
        sv.st[r] = *reinterpret_cast<const uint32_t*>(W.s[r] + g);
        if (ZP) sv.z[r] = *reinterpret_cast<const uint16_t*>(W.z[r] + g);
      }
    }
  };
  auto spread = [&](int j) {
    Steps g;
    const int from = 4 * (16 * (j & 3) + li);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      g.st[r] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)sv.st[r]);
      if (ZP) g.z[r] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)sv.z[r]);
    }
    return g;
  };
  auto compute = [&](const Block& b, const Steps& g) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < kG; ++h) {
        const half2_t nsub = decode_nsub(ZP ? (float)((g.z[r] >> (8 * h)) & 0xFFu) : 8.0f);
        floatx4 part[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) part[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = h * 4 / kG; kk < (h + 1) * 4 / kG; ++kk) {
          const half8_t wf = decode8<ZP>(b.w[r][kk], nsub);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            part[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.a[t][kk], wf, part[t], 0, 0, 0);
        }
        const float st = h2f((uint16_t)(g.st[r] >> (16 * h)));
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][t][e] = __builtin_fmaf(part[t][e], st, acc[r][t][e]);
      }
  };
  // two blocks of the wave in flight
  Block b0, b1;
  if (wave < KB) {
    load_steps(wave);
    load(wave, b0);
  }
  for (int kb = wave, j = 0; kb < KB; kb += 2 * kSkWaves, j += 2) {
    if (kb + kSkWaves < KB) load(kb + kSkWaves, b1);
    compute(b0, spread(j));
    if (kb + kSkWaves < KB) {
      const Steps g = spread(j + 1);
      if (kb + 2 * kSkWaves < KB) {
        if ((j & 3) == 2) load_steps(kb + 2 * kSkWaves);
        load(kb + 2 * kSkWaves, b0);
      }
      compute(b1, g);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) red[((wave * 2 + r) * MT + t) * 64 + lane] = acc[r][t];
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * MT; e += 64 * kSkWaves) {
    const int t = e >> 6, l = e & 63;
    floatx4 v[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      v[r] = red[(r * MT + t) * 64 + l];
#pragma unroll
      for (int w = 1; w < kSkWaves; ++w) v[r] = v[r] + red[((w * 2 + r) * MT + t) * 64 + l];
    }
    const int64_t nn = n0 + (l & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = 16 * t + 4 * (l >> 4) + i;
      if (m < M && nn < N) H[m * N + nn] = f2h(act_f<ACT>(v[0][i]) * v[1][i]);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Tile of TM rows x 128 output channels, 128 channels of K per step, 4 waves; wave w owns the
// output channels 32 w .. 32 w + 31 (their gate and up rows: four 16-column blocks) for all TM
// rows, so every code is decoded once per tile. The activation tile (TM rows of 256 bytes) is
// moved into one of two LDS stages by the buffer unit, chunk c of row r at position c ^ (r & 15);
// each wave loads its codes, steps and zero points into registers one step ahead. Step b waits
// for its loads, passes a barrier, issues step b + 1's loads and computes.
//
// The steps change with the group, so they cannot be left to the end; instead of a second set of
// registers for the group's partial sums, the accumulators hold sum / (the current group's step):
// at a group's start they are multiplied by (last step / this step), and by the last step at the
// end. Each such factor is within 2^-22 of the quotient. A group whose step is 0 decodes to zeros
// and keeps the step before it.
// Rows past M and output channels past N read as zeros; neither is stored.
struct GatedOut {
  uint16_t* H;
  uint8_t *g8, *u8;        // nullptr: not kept
  float *gs, *us;
  uint32_t* flags;
};

template <int GS, bool ZP, int ACT, bool CKPT, int TM>
__global__ __launch_bounds__(256, 2) void w4a16_gated_tiled_kernel(
    const uint16_t* __restrict__ A, int64_t M, int64_t N, int64_t K, GatedWeights W, GatedOut O,
    uint32_t tilesM, uint32_t tilesN, int steps_per_slice, float* __restrict__ partials,
    int64_t Np) {
  constexpr int kG = 128 / GS;
  constexpr int kStage = TM * 256;
  constexpr int MB = TM / 16;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const TileAt at = tile_order<8>(tilesM, tilesN);
  const int64_t m0 = (int64_t)at.tm * TM, n0 = (int64_t)at.tn * kTN;
  const int KB = (int)(K / 128);
  const int b0 = (int)at.slice * steps_per_slice;
  const int b1 = b0 + steps_per_slice < KB ? b0 + steps_per_slice : KB;

  const rsrc_t ra = make_rsrc(A + m0 * K, (uint32_t)((M - m0 < TM ? M - m0 : TM) * K * 2));
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  uint32_t voff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)   // load j of wave w: rows TM / 4 w + 4 j + lane / 16
    voff[j] = (uint32_t)(lg * K * 2) +
              (uint32_t)((li ^ (4 * ((TM / 16 * wave + j) & 3) + lg)) << 4);
  auto issue = [&](int b, int st) {
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int r0 = TM / 4 * wave + 4 * j;
      buffer_load16_lds_so(ra, lds0 + (uint32_t)(st * kStage + r0 * 256), voff[j & 3],
                           (uint32_t)(r0 * K * 2) + (uint32_t)b * 256u);
    }
  };
  // column blocks t = 2 matrix + half: output channels n0 + 32 wave + 16 half + li, read through buffer
  // descriptors that start at the tile's first channel (a lane's offsets then never change, and
  // channels past N read as zeros)
  const uint32_t nrows = (uint32_t)(N - n0 < kTN ? N - n0 : kTN);
  rsrc_t rq[2], rst[2], rz[2];
  uint32_t qoff[2], goff[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    rq[r] = make_rsrc(W.q[r] + n0 * (K / 8), nrows * (uint32_t)(K / 2));
    rst[r] = make_rsrc(W.s[r] + n0 * (K / GS), nrows * (uint32_t)(K / GS) * 2u);
    if (ZP) rz[r] = make_rsrc(W.z[r] + n0 * (K / GS), nrows * (uint32_t)(K / GS));
    const uint32_t row = (uint32_t)(32 * wave + 16 * r + li);
    qoff[r] = row * (uint32_t)(K / 2) + (uint32_t)lg * (GS == 128 ? 16u : 8u);
    goff[r] = (row * (uint32_t)(K / GS) + (uint32_t)(lg * kG));
  }
  struct Codes {
    uint32_t w[4][4];
  };
  auto load_codes = [&](int b, Codes& c) {
    const uint32_t qs = (uint32_t)b * 64u;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = t >> 1, h = t & 1;
      if (GS == 128) {
        const uint4 v = buffer_load16(rq[r], qoff[h], qs);
        c.w[t][0] = v.x; c.w[t][1] = v.y; c.w[t][2] = v.z; c.w[t][3] = v.w;
      } else {
        const uint2 v = buffer_load8(rq[r], qoff[h], qs), x = buffer_load8(rq[r], qoff[h] + 32u, qs);
        c.w[t][0] = v.x; c.w[t][1] = v.y; c.w[t][2] = x.x; c.w[t][3] = x.y;
      }
    }
  };
  // Group steps and zero points of four K steps at a time, K step b + lg in lane group lg; spread(j)
  // hands those of the j-th to all lane groups. Every lane loading the step that it uses was four times
  // the loads, each of two bytes in 16 rows, and they bound the kernel (17 rows of 28672 x 8192, groups
  // of 64 with zero points: 167 us that way, 110 this way, 82 with none of them).
  struct Steps {
    uint32_t st[4], z[4];   // groups of 64: both groups' values
  };
  Steps sv;
  auto load_steps = [&](int b) {
    const uint32_t gs = (uint32_t)b * (uint32_t)kG;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = t >> 1, h = t & 1;
      if (GS == 128) {
        sv.st[t] = buffer_load2(rst[r], 2u * goff[h], 2u * gs);
        if (ZP) sv.z[t] = buffer_load1(rz[r], goff[h], gs);
      } else {
        sv.st[t] = buffer_load4(rst[r], 2u * goff[h], 2u * gs);
        if (ZP) sv.z[t] = buffer_load2(rz[r], goff[h], gs);
      }
    }
  };
  auto spread = [&](int j, Steps& c) {
    const int from = 4 * (16 * j + li);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (GS == 128) {   // one word: the step below the zero point
        const uint32_t v = (uint32_t)__builtin_amdgcn_ds_bpermute(
            from, (int)(ZP ? sv.st[t] | sv.z[t] << 16 : sv.st[t]));
        c.st[t] = ZP ? v & 0xFFFFu : v;
        if (ZP) c.z[t] = v >> 16;
      } else {
        c.st[t] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)sv.st[t]);
        if (ZP) c.z[t] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)sv.z[t]);
      }
    }
  };
  floatx4 acc[4][MB];   // [column block][16-row block]
  float prev[4];        // the step the accumulators are divided by
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    prev[t] = 1.0f;
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[t][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  // One group: its decode and scale factors, then kK channel blocks of 32. Groups of 64 decode a
  // block ahead, among the matrix instructions of the block before (512 rows of 11008 x 4096 with zero
  // points: 167 us, 203 without); groups of 128 have no registers left for that (1100 us instead
  // of 830 for 4096 rows), and half as much scaling per instruction.
  auto compute = [&](int st, const Codes& c, const Steps& g) {
    const char* sa = smem + st * kStage;
    constexpr int kK = 4 / kG;
    constexpr bool kAhead = GS == 64;
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      half2_t nsub[4];
      bool none[4];   // a step of 0: the codes are taken as ones that decode to 0
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float s = h2f((uint16_t)(h == 0 ? g.st[t] & 0xFFFFu : g.st[t] >> 16));
        const float z = ZP ? (float)(GS == 128 ? g.z[t] : h == 0 ? g.z[t] & 0xFFu : g.z[t] >> 8) : 8.0f;
        none[t] = s == 0.0f;
        nsub[t] = decode_nsub(ZP && none[t] ? 0.0f : z);
        const float now = none[t] ? prev[t] : s;
        const float ratio = prev[t] * __builtin_amdgcn_rcpf(now);
        prev[t] = now;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][i][e] *= ratio;
      }
      half8_t wf[2][4];
      auto decode = [&](int k) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          wf[kAhead ? k & 1 : 0][t] = decode8<ZP>(none[t] ? 0u : c.w[t][h * kK + k], nsub[t]);
      };
      if (kAhead) {
        decode(0);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int ch = chunk_of<GS>(lg, h * kK + k);
        if (!kAhead) decode(k);
        if (kAhead && k + 1 < kK) decode(k + 1);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const half8_t af =
              *reinterpret_cast<const half8_t*>(sa + (16 * i + li) * 256 + ((ch ^ li) << 4));
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, wf[kAhead ? k & 1 : 0][t],
                                                               acc[t][i], 0, 0, 0);
        }
        if (kAhead) {
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);       // LDS reads
#pragma unroll
          for (int i = 0; i < MB; ++i) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);   // vector ALU
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
            }
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  Codes cb[2];
  issue(b0, 0);
  load_codes(b0, cb[0]);
  load_steps(b0);
  auto step = [&](int b, int st, const Codes& cur, Codes& nxt) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    const int j = (b - b0) & 3;
    Steps g;
    spread(j, g);
    if (b + 1 < b1) {
      issue(b + 1, st ^ 1);
      load_codes(b + 1, nxt);
      if (j == 3) load_steps(b + 1);
    }
    compute(st, cur, g);
  };
  for (int b = b0; b < b1; b += 2) {
    step(b, 0, cb[0], cb[1]);
    if (b + 1 < b1) step(b + 1, 1, cb[1], cb[0]);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][i][e] *= prev[t];

  // a lane holds, for block i and element e, row m0 + 16 i + 4 lg + e of its output channels
  if (partials) {   // [slice][matrix][M][Np], Np = whole tiles; stores past the last row are dropped
    const uint32_t rows = (uint32_t)(M - m0 < TM ? M - m0 : TM), ld = (uint32_t)Np * 4u;
    const uint32_t off = (uint32_t)(4 * lg) * ld + (uint32_t)(32 * wave + li) * 4u;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const rsrc_t rp = make_rsrc(partials + (((int64_t)at.slice * 2 + r) * M + m0) * Np + n0,
                                  rows * ld - (uint32_t)n0 * 4u);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            buffer_store4(rp, off + 64u * h, (uint32_t)(16 * i + e) * ld,
                          __float_as_uint(acc[2 * r + h][i][e]));
    }
    return;
  }
  __syncthreads();   // the last step's reads of the stages are done
  // H (TM x 256 B), and the codes of g and u (TM x 128 B each), go through LDS to whole-row stores
  char* hl = smem;
  char* cl = smem + TM * 256;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * i + 4 * lg + e, col = 32 * wave + 16 * h + li;
        *reinterpret_cast<uint16_t*>(hl + row * 256 + col * 2) =
            f2h(act_f<ACT>(acc[h][i][e]) * acc[2 + h][i][e]);
      }
  if constexpr (CKPT) {
    __shared__ float wmax[2][4][TM];
    bool any = false;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t mx = 0u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool col = n0 + 32 * wave + 16 * h + li < N;
            const uint32_t a = __float_as_uint(acc[2 * r + h][i][e]) & 0x7FFFFFFFu;
            const bool bad = a >= 0x7F800000u;
            any |= bad && col && m0 + 16 * i + 4 * lg + e < M;
            mx = (bad || !col) ? mx : max(mx, a);
          }
          const float w = group_absmax<16>(__uint_as_float(mx));
          if (li == 0) wmax[r][wave][16 * i + 4 * lg + e] = w;
        }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + 4 * lg + e;
          const Fp8Scale s = fp8_scale(fmaxf(fmaxf(wmax[r][0][row], wmax[r][1][row]),
                                             fmaxf(wmax[r][2][row], wmax[r][3][row])));
          const int64_t m = m0 + row;
          if (wave == 0 && li == 0 && m < M)
            (r == 0 ? O.gs : O.us)[m * (int64_t)tilesN + at.tn] = s.scale;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float v = acc[2 * r + h][i][e];
            uint32_t code = fp8_pack4(v * s.inv, 0.0f, 0.0f, 0.0f) & 0xFFu;
            if ((__float_as_uint(v) & 0x7FFFFFFFu) >= 0x7F800000u) code = 0x7Fu;
            cl[r * TM * 128 + row * 128 + 32 * wave + 16 * h + li] = (char)code;
          }
        }
    if (O.flags) wave_flag(O.flags, any, kFlagNonfiniteAct);
  }
  __syncthreads();
  for (int e = tid; e < TM * 16; e += 256) {   // 16 bytes of H each
    const int row = e >> 4;
    const int64_t m = m0 + row, n = n0 + 8 * (e & 15);
    if (m >= M || n >= N) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(hl + row * 256 + (e & 15) * 16);
    uint16_t* p = O.H + m * N + n;
    if (n + 8 <= N && (N & 7) == 0) {
      *reinterpret_cast<uint4*>(p) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < N) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
  if constexpr (CKPT) {
    for (int e = tid; e < 2 * TM * 8; e += 256) {   // 16 codes each; N % 16 == 0 here
      const int r = e / (TM * 8), row = (e >> 3) % TM;
      const int64_t m = m0 + row, n = n0 + 16 * (e & 7);
      if (m < M && n < N)
        *reinterpret_cast<uint4*>((r == 0 ? O.g8 : O.u8) + m * N + n) =
            *reinterpret_cast<const uint4*>(cl + r * TM * 128 + row * 128 + (e & 7) * 16);
    }
  }
}

// The K slices' partials [S][2][M][Np] added in slice order, then the activation, the product and
// the 8-bit blocks; 16 lanes hold the 128 output channels of one block of one row, 8 each.
template <int ACT, bool CKPT>
__global__ __launch_bounds__(256) void w4a16_gated_finish_kernel(
    const float* __restrict__ P, int S, int64_t M, int64_t N, int64_t Np, GatedOut O) {
  const uint32_t nb = (uint32_t)(Np / 128);
  const uint32_t b = blockIdx.x * 16u + (threadIdx.x >> 4);
  const bool in = b < (uint32_t)(M * nb);
  const uint32_t row = in ? b / nb : 0u, kb = in ? b - row * nb : 0u;
  const int64_t n = (int64_t)kb * 128 + 8 * (threadIdx.x & 15);
  float v[2][8];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float* p = P + (r * M + row) * Np + n;
    const floatx4 a = sum_slices(p, S, 2 * M * Np), c = sum_slices(p + 4, S, 2 * M * Np);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v[r][t] = n + t < N ? a[t] : 0.0f;
      v[r][4 + t] = n + 4 + t < N ? c[t] : 0.0f;
    }
  }
  if (in) {
    uint16_t* p = O.H + (int64_t)row * N + n;
    uint16_t h[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) h[t] = f2h(act_f<ACT>(v[0][t]) * v[1][t]);
    if (n + 8 <= N && (N & 7) == 0) {
      *reinterpret_cast<uint4*>(p) =
          make_uint4((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16),
                     (uint32_t)h[4] | ((uint32_t)h[5] << 16), (uint32_t)h[6] | ((uint32_t)h[7] << 16));
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (n + t < N) p[t] = h[t];
    }
  }
  if constexpr (CKPT) {
    uint32_t any = 0u;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float amax;
      const uint32_t bad = fp8_absmax8(v[r], amax);
      any |= bad;
      const Fp8Scale s = fp8_scale(group_absmax<16>(amax));
      if (in && n < N)
        *reinterpret_cast<uint2*>((r == 0 ? O.g8 : O.u8) + (int64_t)row * N + n) =
            fp8_pack8(v[r], s.inv, bad);
      if (in && (threadIdx.x & 15) == 0) (r == 0 ? O.gs : O.us)[b] = s.scale;
    }
    if (O.flags) wave_flag(O.flags, in && any != 0u, kFlagNonfiniteAct);
  }
}

// ---- plans and launches ---------------------------------------------------------------------

// Which kernel. The skinny one decodes 16 output channels' codes once for up to 32 rows but reads the
// activations once per 16 channels; the tiled one with K slices is two launches. Skinny and
// tiled, us (groups of 128):
//   28672 x 8192: M = 8 72 and 75, M = 16 89 and 78
//   11008 x 4096: M = 8 17.8 and 22.5, M = 16 21.5 and 23.2
//   4096 x 4096:  M = 16 11.9 and 16.8, M = 32 12.5 and 16.8
// (above 16 rows, before either loaded several steps' group steps at once: 17 x 28672 x 8192 124 and
// 103, 17 x 11008 x 4096 30.7 and 28.4.)
static bool skinny(int64_t M, int64_t N, int64_t K) {
  return M <= 16 || (M <= 32 && N * K <= (int64_t(1) << 24));
}

GatedPlan w4a16_gated_plan(int64_t M, int64_t N, int64_t K, bool ckpt) {
  GatedPlan p{};
  p.S = 1;
  if (!ckpt && skinny(M, N, K)) return p;
  p.tn = (N + kTN - 1) / kTN;
  // 128 rows share a decoded weight tile (64 against 128 rows, us, groups of 128 and groups of 64 with
  // zero points: 128 x 28672 x 8192 158 and 145, 224 and 185; 1024 x 11008 x 4096 198 and 179, 303
  // and 229); with 64 such tiles or fewer the finer split of rows fills more CUs (256 x 4096 x 4096
  // 33 and 40, 41 and 44; 256 x 1024 x 4096 23 and 27, 25 and 29). 32 rows where that is all: fewer
  // registers, more workgroups per CU (17 x 11008 x 4096 23.6 and 26.2, 29.8 and 34.5 with 64).
  p.bm = M > 64 && (M + 127) / 128 * p.tn > 64 ? 128 : M > 32 ? 64 : 32;
  p.tm = (M + p.bm - 1) / p.bm;
  p.Np = p.tn * kTN;
  const int64_t KB = K / 128, tiles = p.tm * p.tn;
  if (tiles < 256) {   // two workgroups per CU (four of 32 rows), at least 4 steps each
    p.S = (p.bm == 32 ? 1024 : 512) / tiles;
    const int64_t smax = KB / 4;
    p.S = p.S > smax ? smax : p.S;
    p.S = p.S < 1 ? 1 : p.S;
  }
  p.steps = (KB + p.S - 1) / p.S;
  p.S = (KB + p.steps - 1) / p.steps;
  p.ws_bytes = p.S > 1 ? (size_t)(p.S * 2 * M * p.Np * 4) : 0;
  return p;
}

template <int GS, bool ZP, int ACT>
static hipError_t gated(const uint16_t* A, int64_t M, int64_t N, int64_t K, const GatedWeights& W,
                        const GatedOut& O, void* ws, hipStream_t stream) {
  const bool ckpt = O.g8 != nullptr;
  if (!ckpt && (M == 1 || (M == 2 && K <= 28672))) {
    const unsigned grid = (unsigned)((N + kGvWaves - 1) / kGvWaves);
    const size_t lds = (size_t)M * (size_t)(K / 32) * kChunkBytes;
#define AWQ_GG(ONE_, TI_, MB_)                                                                \
  w4a16_gated_gemv_kernel<GS, ZP, ACT, ONE_, TI_, MB_><<<grid, 64 * kGvWaves, lds, stream>>>( \
      A, M, N, K, W, O.H)
#define AWQ_GM(MB_)                                       \
  do {                                                    \
    if (K <= 4096) AWQ_GG(true, 1, MB_);                  \
    else if (K <= 8192) AWQ_GG(false, 2, MB_);            \
    else if (K <= 16384) AWQ_GG(false, 4, MB_);           \
    else AWQ_GG(false, 8, MB_);                           \
  } while (0)
    if (M == 1) AWQ_GM(1); else AWQ_GM(2);
#undef AWQ_GM
#undef AWQ_GG
    return hipGetLastError();
  }
  if (!ckpt && skinny(M, N, K)) {
    const unsigned grid = (unsigned)((N + 15) / 16);
    const int mt = M <= 16 ? 1 : 2;
    const size_t lds = (size_t)kSkWaves * 2 * mt * 64 * sizeof(floatx4);
    if (mt == 1)
      w4a16_gated_skinny_kernel<GS, ZP, ACT, 1><<<grid, 64 * kSkWaves, lds, stream>>>(A, M, N, K, W,
                                                                                      O.H);
    else
      w4a16_gated_skinny_kernel<GS, ZP, ACT, 2><<<grid, 64 * kSkWaves, lds, stream>>>(A, M, N, K, W,
                                                                                      O.H);
    return hipGetLastError();
  }
  const GatedPlan p = w4a16_gated_plan(M, N, K, ckpt);
  float* P = p.S > 1 ? static_cast<float*>(ws) : nullptr;
  const unsigned grid = (unsigned)(p.tm * p.tn * p.S);
#define AWQ_GT(CKPT_, TM_)                                                    \
  w4a16_gated_tiled_kernel<GS, ZP, ACT, CKPT_, TM_><<<grid, 256, 0, stream>>>( \
      A, M, N, K, W, O, (uint32_t)p.tm, (uint32_t)p.tn, (int)p.steps, P, p.Np)
  if (p.bm == 128) {
    if (ckpt) AWQ_GT(true, 128); else AWQ_GT(false, 128);
  } else if (p.bm == 64) {
    if (ckpt) AWQ_GT(true, 64); else AWQ_GT(false, 64);
  } else {
    if (ckpt) AWQ_GT(true, 32); else AWQ_GT(false, 32);
  }
#undef AWQ_GT
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.S == 1) return e;
  const unsigned fgrid = (unsigned)((M * p.tn + 15) / 16);
  if (ckpt)
    w4a16_gated_finish_kernel<ACT, true><<<fgrid, 256, 0, stream>>>(P, (int)p.S, M, N, p.Np, O);
  else
    w4a16_gated_finish_kernel<ACT, false><<<fgrid, 256, 0, stream>>>(P, (int)p.S, M, N, p.Np, O);
  return hipGetLastError();
}

hipError_t launch_w4a16_gated(const uint16_t* A, int64_t M, int64_t N, int64_t K, int group,
                              int act, const GatedWeights& W, uint16_t* H, uint8_t* g8, float* gs,
                              uint8_t* u8, float* us, uint32_t* flags, void* ws,
                              hipStream_t stream) {
  const GatedOut O{H, g8, u8, gs, us, flags};
  const bool zp = W.z[0] != nullptr;
#define AWQ_GA(GS_, ZP_)                                                            \
  (act == kSilu ? gated<GS_, ZP_, kSilu>(A, M, N, K, W, O, ws, stream)              \
                : gated<GS_, ZP_, kGelu>(A, M, N, K, W, O, ws, stream))
  if (group == 64) return zp ? AWQ_GA(64, true) : AWQ_GA(64, false);
  return zp ? AWQ_GA(128, true) : AWQ_GA(128, false);
#undef AWQ_GA
}

}  // namespace awq
