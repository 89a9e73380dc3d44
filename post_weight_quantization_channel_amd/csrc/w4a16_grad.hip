// Gradients through packed 4-bit weights, W[n, k] = c(q[n, k]) step[n, k / G]:
//   one matrix (launch_w4a16_gemm_backward):    dA[m, k] = sum_n dY[m, n] W[n, k] / s[k]
//   gated block (launch_w4a16_gated_backward):  g, u from their 8-bit blocks,
//     dg = dH u act'(g), du = dH act(g),  dA = dg Wg + du Wu.
//
// The sum runs over the output channels n, and the step changes with n and with the group of the
// column k, so it can be applied neither to the accumulators nor to a whole operand. It goes onto
// the gradient, once per group of columns: for the columns of one group the operands are
//   P[m, n] = fp16(d[m, n] step[n, group])   and   c(q[n, k])  (an integer, exact in fp16).
// fp16 has few exponents, so both factors are brought to a common range with powers of two
// (exact): step' = step 2^-f[group] <= 1, 2^f at or above the group's largest step over all n; and
// d' = d 2^e[m] with the row's largest |d'| in [2^14, 2^15). 2^(f - e) comes back on the fp32 sums.
// Nothing overflows, and only products more than 2^29 below a column group's largest possible one
// lose bits to fp16's subnormals. In the gated form d' has more than 11 bits and is kept as hi + lo
// (two fp16 numbers): P = fma(hi, step', lo step') is then rounded once, as in the one-matrix form,
// where d' is dY itself. So the result carries two fp16 roundings, P's and the output's: sqrt(2)
// times the error of the output's alone. (Rounding d' to fp16 and the weight to fp16(c step) would
// make it 1.67 times.)
//
// 4096 rows, 2 x 11008 x 4096 (gated): 869 us for the call, 0.85 PFLOP/s; in a kernel trace the rows
// take 128 us (541 MB, 4.2 TB/s), the steps 6, the product the rest, its matrix units busy 47% of
// the cycles at the 1.9 GHz that the power limit leaves. 16 rows of 4096 x 4096: four launches of 4,
// 6, 11 and 4 us.
//
// Launches: the rows (d', in blocks of 32 channels: [n / 32][m][32], so that a tile of a step is
// contiguous) beside the largest steps of 64 parts of n; the steps (step' with n contiguous); the
// product; and with several slices of n their sum in slice order.
#include "fp8_format.h"
#include "gated_act.h"
#include "kernels.h"
#include "tile_order.h"

namespace awq {

namespace {

// Layout of the contraction: matrix 0's channels at 0 .. N - 1, matrix 1's at Nc .. Nc + N - 1, Nc
// = N rounded up to 32; the channels between carry d' = 0 and step' = 0.
struct GradShape {
  int64_t M, N, K, Nc, C;   // C = all contraction entries (a multiple of 32)
};

constexpr int kParts = 64;        // parts of n whose largest steps are found side by side
constexpr int kMaxGroups = 512;   // K <= 32768, groups of 64

// ---- steps ----------------------------------------------------------------------------------
// Part `part` of `kParts`: pmax[group][part] = the largest |step| (fp16 bits, which order like the
// numbers) of its channels, both matrices. Called by a workgroup of 512 threads, `wide` (a power of
// two) of which hold the groups of one channel.
__device__ __forceinline__ void grad_step_maxima(const GatedWeights& W, const GradShape& S,
                                                 int matrices, int groups, int part,
                                                 uint32_t* __restrict__ pmax, uint32_t* lds) {
  const int wide = groups > 256 ? 512 : groups > 128 ? 256 : groups > 64 ? 128 : groups > 32 ? 64 : 32;
  const int g = threadIdx.x & (wide - 1), r0 = threadIdx.x / wide, rows = 512 / wide;
  lds[threadIdx.x] = 0u;
  __syncthreads();
  const int64_t per = (S.N + kParts - 1) / kParts;
  const int64_t n0 = per * part;
  const int64_t n1 = n0 + per < S.N ? n0 + per : S.N;
  uint32_t mx = 0u;
  if (g < groups) {
    for (int mat = 0; mat < matrices; ++mat) {
      const uint16_t* s = W.s[mat] + g;
#pragma unroll 8
      for (int64_t n = n0 + r0; n < n1; n += rows) mx = max(mx, (uint32_t)(s[n * groups] & 0x7FFFu));
    }
    atomicMax(&lds[g], mx);
  }
  __syncthreads();
  if ((int)threadIdx.x < groups) pmax[threadIdx.x * kParts + part] = lds[threadIdx.x];
}

// One workgroup: 32 channels of the contraction, up to 128 groups of columns at a time (read along
// the rows, written along the channels, through LDS). st [groups][C] fp16 step', sub [groups][C]
// fp16 -(1024 + z) (ZP), colscale [groups] fp32 2^f.
template <bool ZP>
__global__ __launch_bounds__(256) void grad_steps_kernel(GatedWeights W, GradShape S, int groups,
                                                         const uint32_t* __restrict__ pmax,
                                                         uint16_t* __restrict__ st,
                                                         uint16_t* __restrict__ sub,
                                                         float* __restrict__ colscale) {
  constexpr int kTG = 128;
  __shared__ uint32_t expo[kTG];   // biased exponent of 2^f
  __shared__ uint16_t tile[32 * kTG];
  __shared__ uint8_t ztile[ZP ? 32 * kTG : 1];
  const int64_t c0 = (int64_t)blockIdx.x * 32;
  const int mat = c0 >= S.Nc ? 1 : 0;
  const int64_t n0 = c0 - mat * S.Nc;
  const int rows = (int)(S.N - n0 < 32 ? S.N - n0 : 32);
  for (int g0 = 0; g0 < groups; g0 += kTG) {
    const int ng = groups - g0 < kTG ? groups - g0 : kTG;
    if (g0) __syncthreads();
    for (int e = threadIdx.x; e < rows * ng; e += 256) {
      const int r = e / ng, g = e - r * ng;
      const int64_t at = (n0 + r) * groups + g0 + g;
      tile[r * kTG + g] = W.s[mat][at];
      if (ZP) ztile[r * kTG + g] = W.z[mat][at];
    }
    // 16 lanes per group: four parts each, then the maximum over the lanes
    for (int g = threadIdx.x >> 4; g < ng; g += 16) {
      const uint4 p = *reinterpret_cast<const uint4*>(pmax + (g0 + g) * kParts + 4 * (threadIdx.x & 15));
      const uint32_t bits = max(max(p.x, p.y), max(p.z, p.w));
      const float top = group_absmax<16>(h2f((uint16_t)bits));
      const uint32_t u = __float_as_uint(top);
      // the power of two at or above the largest step; 1 for 0 and for a non-finite step
      if ((threadIdx.x & 15) == 0) {
        expo[g] = (u == 0u || u >= 0x7F800000u) ? 127u : (u + 0x7FFFFFu) >> 23;
        if (blockIdx.x == 0) colscale[g0 + g] = __uint_as_float(expo[g] << 23);
      }
    }
    __syncthreads();
    const int r = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < ng; g += 8) {
      const int64_t at = (int64_t)(g0 + g) * S.C + c0 + r;
      const float inv = __uint_as_float((254u - expo[g]) << 23);
      st[at] = r < rows ? f2h(h2f(tile[r * kTG + g]) * inv) : (uint16_t)0;
      if (ZP) sub[at] = f2h(-1024.0f - (r < rows ? (float)ztile[r * kTG + g] : 0.0f));
    }
  }
}

// ---- rows -----------------------------------------------------------------------------------
struct GatedSaved {
  const uint8_t *g8, *u8;
  const float *gs, *us;
};

// 8 values of a row of N halves from channel n on (a multiple of 8); channels past N give 0.
__device__ __forceinline__ void load8_halves(const uint16_t* p, int64_t n, int64_t N, float (&v)[8]) {
  if (n + 8 <= N && ((reinterpret_cast<uintptr_t>(p + n)) & 15u) == 0) {
    load8_f32<kF16>(p + n, v);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = n + t < N ? h2f(p[n + t]) : 0.0f;
  }
}

// One workgroup of 512 threads per row, which first finds the row's largest |d|. IT > 0: the row is at
// most IT x 4096 channels and stays in registers meanwhile; IT = 0: any length, the values are
// formed twice (gated, 4096 rows of 11008: 190 us that way, 128 in registers). Consecutive rows go
// to one XCD, whose L2 then joins their 64-byte pieces of a line. The last kParts workgroups find
// the largest steps instead.
template <bool GATED, int ACT, int IT>
__global__ __launch_bounds__(512) void grad_rows_kernel(
    const uint16_t* __restrict__ dY, GatedSaved V, GatedWeights W, GradShape S, int groups,
    uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, float* __restrict__ unscale,
    uint32_t* __restrict__ pmax) {
  __shared__ uint32_t wmax[8];
  __shared__ uint32_t gmax[kMaxGroups];
  const uint32_t M = (uint32_t)S.M;
  if (blockIdx.x >= M) {
    grad_step_maxima(W, S, GATED ? 2 : 1, groups, (int)(blockIdx.x - M), pmax, gmax);
    return;
  }
  const uint32_t xcd = blockIdx.x & 7u, rem = M & 7u;
  const int64_t m = xcd * (M >> 3) + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t KB = (S.N + 127) / 128;
  const uint16_t* row = dY + m * S.N;

  auto values = [&](int64_t n, float (&d0)[8], float (&d1)[8]) {
    float d[8];
    load8_halves(row, n, S.N, d);
    if constexpr (GATED) {
      float g[8], u[8];
      if (n < S.N) {   // N % 16 == 0: all eight are there
        const uint2 gw = *reinterpret_cast<const uint2*>(V.g8 + m * S.N + n);
        const uint2 uw = *reinterpret_cast<const uint2*>(V.u8 + m * S.N + n);
        const float gs = V.gs[m * KB + (n >> 7)], us = V.us[m * KB + (n >> 7)];
        float t[4];
        fp8_unpack4(gw.x, t);
        for (int i = 0; i < 4; ++i) g[i] = t[i] * gs;
        fp8_unpack4(gw.y, t);
        for (int i = 0; i < 4; ++i) g[4 + i] = t[i] * gs;
        fp8_unpack4(uw.x, t);
        for (int i = 0; i < 4; ++i) u[i] = t[i] * us;
        fp8_unpack4(uw.y, t);
        for (int i = 0; i < 4; ++i) u[4 + i] = t[i] * us;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = u[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float df;
        const float f = act_f_df<ACT>(g[i], df);
        d0[i] = d[i] * u[i] * df;
        d1[i] = d[i] * f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) d0[i] = d[i];
    }
  };

  uint32_t mx = 0u;
  auto largest = [&](const float (&d)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(d[i]) & 0x7FFFFFFFu);
  };
  const int64_t first = 8 * (int64_t)threadIdx.x;
  constexpr int kIt = IT > 0 ? IT : 1, kMat = GATED ? 2 : 1;
  float d[kMat][kIt][8];
  if constexpr (IT > 0) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (first + 4096 * it >= S.Nc) continue;
      values(first + 4096 * it, d[0][it], d[kMat - 1][it]);
      largest(d[0][it]);
      if (GATED) largest(d[kMat - 1][it]);
    }
  } else {
    for (int64_t n = first; n < S.Nc; n += 4096) {
      values(n, d[0][0], d[kMat - 1][0]);
      largest(d[0][0]);
      if (GATED) largest(d[kMat - 1][0]);
    }
  }
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, k));
  if (lane == 0) wmax[wave] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mx = max(mx, wmax[w]);
  const int e = escale_for_max(__uint_as_float(mx));   // 0 for 0 and for Inf or NaN
  const float sc = ldexpf(1.0f, e);
  if (threadIdx.x == 0) unscale[m] = ldexpf(1.0f, -e);

  auto put = [&](int64_t c, const float (&v)[8]) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[2 * i] * sc, b = v[2 * i + 1] * sc;
      h[i] = f2h2(a, b);
      if (GATED) {
        const float ha = h2f((uint16_t)(h[i] & 0xFFFFu)), hb = h2f((uint16_t)(h[i] >> 16));
        // an infinite or NaN value has no low part
        l[i] = f2h2(fabsf(ha) <= 65504.0f ? a - ha : 0.0f, fabsf(hb) <= 65504.0f ? b - hb : 0.0f);
      }
    }
    const int64_t at = ((c >> 5) * S.M + m) * 32 + (c & 31);
    *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    if (GATED) *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
  };
  if constexpr (IT > 0) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int64_t n = first + 4096 * it;
      if (n >= S.Nc) continue;
      put(n, d[0][it]);
      if (GATED) put(S.Nc + n, d[kMat - 1][it]);
    }
  } else {
    for (int64_t n = first; n < S.Nc; n += 4096) {
      values(n, d[0][0], d[kMat - 1][0]);
      put(n, d[0][0]);
      if (GATED) put(S.Nc + n, d[kMat - 1][0]);
    }
  }
}

// ---- the product ----------------------------------------------------------------------------
// Tile BM rows x two groups of columns, 32 channels of the contraction per step, two LDS stages.
// A stage holds P for the tile's rows, once per column group ([group][row][32]), and the decoded
// codes of the tile's columns ([column][32]), rows of 64 bytes whose 16-byte chunk c sits at
// c ^ ((row >> 2) & 3): the 16 rows a fragment read touches at once cover all 64 banks. Half the
// waves take each column group (with its P), BM / (waves / 2) rows each.
// A thread decodes words in pairs, (channel n, channel n + 1) of the same 8 columns: byte j of both
// words gives the fp16 pairs of columns 2j and 2j + 1, so the transposed tile costs no more than a
// plain one. LDS column i * WPG + w is column 8 w + i of its group (WPG = words per group), which
// spreads a wave's writes over all banks.
// Step t computes from one stage while the values of step t + 1, loaded during step t - 1, are
// folded and decoded into the other; one barrier per step.
// Rows past M read as zeros and columns past K as the last word; neither is stored.
template <int G, bool ZP, bool LO, int BM>
__global__ __launch_bounds__(BM == 256 ? 512 : 256) void grad_gemm_kernel(
    GatedWeights W, GradShape S, const uint16_t* __restrict__ hi, const uint16_t* __restrict__ lo,
    const uint16_t* __restrict__ st, const uint16_t* __restrict__ sub,
    const float* __restrict__ unscale, const float* __restrict__ colscale,
    const uint16_t* __restrict__ s16, uint16_t* __restrict__ dA, uint32_t tilesM, uint32_t tilesK, int steps_per_slice,
    float* __restrict__ partials) {
  constexpr int NT = BM == 256 ? 512 : 256, kWaves = NT / 64;
  constexpr int KT = 2 * G, WPG = G / 8;
  constexpr int RM = BM / (kWaves / 2), MBLK = RM / 32, NBLK = G / 32;
  constexpr int kP = BM * 64;                       // bytes of one group's P
  constexpr int kStage = 2 * kP + KT * 64;
  constexpr int kAT = BM * 4 / NT;                  // 16-byte chunks of d' per thread
  constexpr int kBT = (4 * G + NT - 1) / NT;        // word pairs per thread
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int vg = wave / (kWaves / 2), mq = wave % (kWaves / 2);
  const TileAt at = tile_order<2>(tilesM, tilesK);
  const int64_t m0 = (int64_t)at.tm * BM, k0 = (int64_t)at.tn * KT;
  const int T = (int)(S.C / 32);
  const int s0 = (int)at.slice * steps_per_slice;
  const int s1 = s0 + steps_per_slice < T ? s0 + steps_per_slice : T;
  const int64_t wpr = S.K / 8;
  const int mat_step = (int)(S.Nc / 32);            // first step of matrix 1

  // Each step's values are read through buffer descriptors that start at the step's first entry, so
  // that a thread's offset never changes and entries past the end (rows past M, channels past N)
  // read as zeros.
  // This thread's chunks of d': row tid / 4 (+ NT / 4), chunk tid % 4.
  const int ac = tid & 3;
  const uint32_t rows = (uint32_t)(S.M - m0 < BM ? S.M - m0 : BM);
  uint32_t aoff[kAT], awr[kAT];                     // byte offsets: global, within P
#pragma unroll
  for (int i = 0; i < kAT; ++i) {
    const int row = (tid >> 2) + i * (NT / 4);
    aoff[i] = (uint32_t)(row * 64 + ac * 16);
    awr[i] = (uint32_t)(row * 64 + ((ac ^ ((row >> 2) & 3)) << 4));
  }
  const int64_t grp0 = k0 / G, groups = S.K / G;
  const uint16_t* sp[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) sp[v] = st + (grp0 + v < groups ? grp0 + v : groups - 1) * S.C;
  // this thread's word pairs: channels 2 (t % 16), word t / 16 of the tile
  int bn[kBT];
  uint32_t boff[kBT], bwr[kBT];
  const uint16_t* bsub[kBT];
#pragma unroll
  for (int i = 0; i < kBT; ++i) {
    // with fewer pairs than threads the upper threads repeat the lower ones' (a branch would cost more)
    const int t = (tid + i * NT) % (4 * G);
    const int w = t >> 4;
    bn[i] = 2 * (t & 15);
    const int64_t word = k0 / 8 + w < wpr ? k0 / 8 + w : wpr - 1;
    boff[i] = (uint32_t)((bn[i] * wpr + word) * 4);
    bsub[i] = ZP ? sub + (word / WPG) * S.C + bn[i] : nullptr;
    // column i8 * WPG + w % WPG of group w / WPG, i8 = 0..7: row offset added at the write
    bwr[i] = (uint32_t)((w / WPG) * G + w % WPG);
  }
  // one step's values in flight
  uint4 rh[kAT], rl[kAT], rs[2];
  uint32_t rq[kBT][2], rz[kBT];
  auto entries = [&](const uint16_t* p, int t) {    // step t of hi or lo, from row m0 on
    return make_rsrc(p + ((int64_t)t * S.M + m0) * 32, rows * 64u);
  };
  auto codes = [&](int t) {                          // step t's rows of its matrix
    const int mat = t >= mat_step ? 1 : 0;
    const int64_t n = (int64_t)(t - mat * mat_step) * 32;
    const int64_t left = S.N - n < 32 ? S.N - n : 32;
    return make_rsrc(W.q[mat] + n * wpr, (uint32_t)(left * wpr * 4));
  };
  auto load_a = [&](int t, int i) {
    rh[i] = buffer_load16(entries(hi, t), aoff[i]);
    if (LO) rl[i] = buffer_load16(entries(lo, t), aoff[i]);
  };
  auto load_s = [&](int t) {
#pragma unroll
    for (int v = 0; v < 2; ++v) rs[v] = buffer_load16(make_rsrc(sp[v] + (int64_t)t * 32, 64u), ac * 16u);
  };
  auto load_b = [&](int t, int i) {
    const rsrc_t r = codes(t);
    rq[i][0] = buffer_load4(r, boff[i]);
    rq[i][1] = buffer_load4(r, boff[i] + (uint32_t)(wpr * 4));
    if (ZP) rz[i] = *reinterpret_cast<const uint32_t*>(bsub[i] + (int64_t)t * 32);
  };
  // chunk i of d' folded with column group v's steps, into P
  auto fold = [&](char* base, int i, int v) {
    const uint32_t h[4] = {rh[i].x, rh[i].y, rh[i].z, rh[i].w};
    const uint32_t l[4] = {LO ? rl[i].x : 0u, LO ? rl[i].y : 0u, LO ? rl[i].z : 0u, LO ? rl[i].w : 0u};
    const uint32_t s[4] = {rs[v].x, rs[v].y, rs[v].z, rs[v].w};
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const half2_t hv = __builtin_bit_cast(half2_t, h[j]);
      const half2_t sv = __builtin_bit_cast(half2_t, s[j]);
      half2_t pv;
      if constexpr (LO)
        pv = __builtin_elementwise_fma(hv, sv, __builtin_bit_cast(half2_t, l[j]) * sv);
      else
        pv = hv * sv;
      p[j] = __builtin_bit_cast(uint32_t, pv);
    }
    *reinterpret_cast<uint4*>(base + v * kP + awr[i]) = make_uint4(p[0], p[1], p[2], p[3]);
  };
  // byte j (columns 2j, 2j + 1) of word pair i
  auto decode = [&](char* base, int i, int j) {
    constexpr uint32_t kLo = ZP ? 0x64006400u : 0x64086408u;   // exponent, and the flip of bit 3
    constexpr uint32_t kHi = ZP ? 0x64006400u : 0x64806480u;
    const half2_t sixteenth = half2_t{(_Float16)0.0625f, (_Float16)0.0625f};
    // subtrahends: -(1024 + zc) for the low nibbles, -(64 + zc) for the high ones
    const half2_t nlo = ZP ? __builtin_bit_cast(half2_t, rz[i])
                           : half2_t{(_Float16)-1032.0f, (_Float16)-1032.0f};
    const half2_t nhi = nlo + half2_t{(_Float16)960.0f, (_Float16)960.0f};
    const uint32_t x = __builtin_amdgcn_perm(rq[i][1], rq[i][0],
                                             0x0C040C00u + (uint32_t)j * 0x00010001u);
    const half2_t a = __builtin_bit_cast(half2_t, (x & 0x000F000Fu) ^ kLo) + nlo;
    const half2_t b = __builtin_elementwise_fma(
        __builtin_bit_cast(half2_t, (x & 0x00F000F0u) ^ kHi), sixteenth, nhi);
    const int chunk = bn[i] >> 3, within = (bn[i] & 7) * 2;
    const uint32_t ra = bwr[i] + (uint32_t)(2 * j * WPG), rb = ra + WPG;
    char* d = base + 2 * kP + within;
    *reinterpret_cast<uint32_t*>(d + ra * 64 + ((chunk ^ ((ra >> 2) & 3)) << 4)) =
        __builtin_bit_cast(uint32_t, a);
    *reinterpret_cast<uint32_t*>(d + rb * 64 + ((chunk ^ ((rb >> 2) & 3)) << 4)) =
        __builtin_bit_cast(uint32_t, b);
  };
  // the staging of a step in pieces: folds of the chunks, then bytes of the word pairs; each set of
  // registers is loaded again, for step `t`, as soon as its last piece is done
  constexpr int kPieces = 2 * kAT + 4 * kBT;
  auto piece = [&](char* base, int x, int t) {
    if (x < 2 * kAT) {
      fold(base, x >> 1, x & 1);
      if (x & 1) load_a(t, x >> 1);
      if (x == 2 * kAT - 1) load_s(t);
    } else if (x < kPieces) {
      const int y = x - 2 * kAT;
      decode(base, y >> 2, y & 3);
      if ((y & 3) == 3) load_b(t, y >> 2);
    }
  };

  const int l32 = lane & 31, lh = lane >> 5;
  floatx16 acc[MBLK][NBLK];
#pragma unroll
  for (int i = 0; i < MBLK; ++i)
#pragma unroll
    for (int j = 0; j < NBLK; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  uint32_t foff[2];                                  // fragment offset of sub-step 0, 1 in a row block
#pragma unroll
  for (int h = 0; h < 2; ++h)
    foff[h] = (uint32_t)(l32 * 64 + (((2 * h + lh) ^ ((l32 >> 2) & 3)) << 4));
  // Step t computes from stage `cur` while step t + 1's values go into the other stage and step
  // t + 2's are loaded. The pieces stand between the matrix instructions of the step's first half,
  // which run in their shadow (left to the compiler, they all came first). The barrier stands in the
  // middle: the other stage is then written and `cur` read, so the second half's matrix instructions
  // cover the reads of the next step's first fragments (with the barrier between the steps, every
  // wave waited there for its fragments). Nothing is conditional (the last step loads the slice's
  // last step again and writes a stage nobody reads): behind a branch the compiler has to wait for
  // the newest loads before it uses the older ones. 4096 rows, 2 x 11008 x 4096: 1285 us without
  // any of this, 1040 without branches, 840 with the pieces; the barrier in the middle then took a
  // kernel trace's 878 to 848.
  constexpr int kH = MBLK * NBLK, kPer = (kPieces + kH - 1) / kH;
  const int last = s1 - 1;
  const char* pa = smem + vg * kP + mq * RM * 64;
  const char* pb = smem + 2 * kP + vg * G * 64;
  half8_t a[2][MBLK], b[2][NBLK];
  auto read_a = [&](int stage, int h, int i) {
    a[h][i] = *reinterpret_cast<const half8_t*>(pa + stage * kStage + i * 32 * 64 + foff[h]);
  };
  auto read_b = [&](int stage, int h, int j) {
    b[h][j] = *reinterpret_cast<const half8_t*>(pb + stage * kStage + j * 32 * 64 + foff[h]);
  };
  auto step = [&](int t, int cur) {
    char* other = smem + (cur ^ 1) * kStage;
    const int tl = t + 2 < last ? t + 2 : last;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1) __syncthreads();
#pragma unroll
      for (int x = 0; x < kH; ++x) {
        const int j = x / MBLK, i = x % MBLK;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[h][i], b[h][j], acc[i][j], 0, 0, 0);
        // fragments of the other half: this step's second, or the next step's first
        const int stage = h == 0 ? cur : cur ^ 1;
        if (x < MBLK) read_a(stage, h ^ 1, x);
        if (x < NBLK) read_b(stage, h ^ 1, x);
        if (h == 0) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) piece(other, x * kPer + k, tl);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // prologue: step s0 staged and its first fragments read, step s0 + 1 in the registers
  const int second = s0 < last ? s0 + 1 : last;
#pragma unroll
  for (int i = 0; i < kAT; ++i) load_a(s0, i);
  load_s(s0);
#pragma unroll
  for (int i = 0; i < kBT; ++i) load_b(s0, i);
#pragma unroll
  for (int x = 0; x < kPieces; ++x) piece(smem, x, second);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MBLK; ++i) read_a(0, 0, i);
#pragma unroll
  for (int j = 0; j < NBLK; ++j) read_b(0, 0, j);
  int t = s0;
  for (; t + 1 < s1; t += 2) {
    step(t, 0);
    step(t + 1, 1);
  }
  if (t < s1) step(t, 0);

  // ---- store: a lane's block j holds column 8 w + i8, w = lane % WPG -------------------------
  const int64_t kl = k0 + vg * G + 8 * (l32 % WPG) + l32 / WPG;   // of block 0; + 32 / WPG per block
  const int64_t ml = m0 + mq * RM + 4 * lh;
  const bool live = k0 + vg * G < S.K;   // a whole group of columns: K % G == 0
  if (partials) {
    if (!live) return;
    float* P = partials + (int64_t)at.slice * S.M * S.K + kl;
#pragma unroll
    for (int i = 0; i < MBLK; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t m = ml + 32 * i + 8 * (e >> 2) + (e & 3);
        if (m < S.M) {
#pragma unroll
          for (int j = 0; j < NBLK; ++j) P[m * S.K + (32 / WPG) * j] = acc[i][j][e];
        }
      }
    return;
  }
  // Through LDS, 32 rows of the wave's columns at a time (a region per wave), so that a row's columns
  // leave as whole lines.
  constexpr int kPitch = 2 * G + 16;
  static_assert(kWaves * 32 * kPitch <= 2 * kStage, "the regions fit the stages");
  const float cs = live ? colscale[kl / G] : 1.0f;
  float sv[NBLK];
#pragma unroll
  for (int j = 0; j < NBLK; ++j) sv[j] = live && s16 ? h2f(s16[kl + (32 / WPG) * j]) : 1.0f;
  __syncthreads();   // the stages are read
  if (!live) return;
  char* reg = smem + wave * 32 * kPitch;
#pragma unroll
  for (int i = 0; i < MBLK; ++i) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int r = 8 * (e >> 2) + (e & 3) + 4 * lh;
      const int64_t m = m0 + mq * RM + 32 * i + r;
      const float us = unscale[m < S.M ? m : S.M - 1] * cs;
#pragma unroll
      for (int j = 0; j < NBLK; ++j) {
        float v = acc[i][j][e] * us;
        if (s16) v = v / sv[j];
        *reinterpret_cast<uint16_t*>(reg + r * kPitch +
                                     2 * (8 * (l32 % WPG) + l32 / WPG + (32 / WPG) * j)) = f2h(v);
      }
    }
#pragma unroll
    for (int e = 0; e < G / 16; ++e) {   // 32 rows of G / 8 chunks of 16 bytes
      const int x = 64 * e + lane, r = x / (G / 8), c = x % (G / 8);
      const uint4 v = *reinterpret_cast<const uint4*>(reg + r * kPitch + c * 16);
      const int64_t m = m0 + mq * RM + 32 * i + r;
      if (m < S.M) *reinterpret_cast<uint4*>(dA + m * S.K + k0 + vg * G + 8 * c) = v;
    }
  }
}

// dA = round(sum of the slices' partials [slices][M][K] times 2^(f - e) (/ s[k])), slices in order.
__global__ __launch_bounds__(256) void grad_finish_kernel(const float* __restrict__ P, int slices,
                                                          GradShape S, int group,
                                                          const float* __restrict__ unscale,
                                                          const float* __restrict__ colscale,
                                                          const uint16_t* __restrict__ s16,
                                                          uint16_t* __restrict__ dA) {
  const int64_t MK = S.M * S.K;
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;   // K % 128 == 0: one row
  if (e >= MK) return;
  const int64_t m = e / S.K, k = e - m * S.K;
  const floatx4 t = sum_slices(P + e, slices, MK);
  const float us = unscale[m] * colscale[k / group];
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = t[i] * us;
    if (s16) v[i] = v[i] / h2f(s16[k + i]);
  }
  *reinterpret_cast<uint2*>(dA + e) = make_uint2(f2h2(v[0], v[1]), f2h2(v[2], v[3]));
}

constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

GradPlan w4a16_grad_plan(int64_t M, int64_t N, int64_t K, int group, bool gated, bool zp) {
  GradPlan p{};
  p.Nc = (N + 31) / 32 * 32;
  p.C = gated ? 2 * p.Nc : p.Nc;
  p.bm = M > 128 ? 256 : 64;
  p.tm = (M + p.bm - 1) / p.bm;
  p.tk = (K + 2 * group - 1) / (2 * group);
  const int64_t T = p.C / 32, tiles = p.tm * p.tk;
  // one large workgroup per CU, or two small; at least 8 or 4 steps each
  const int64_t want = p.bm == 256 ? 256 : 512, least = p.bm == 256 ? 8 : 4;
  int64_t S = want / tiles;
  S = S > T / least ? T / least : S;
  S = S < 1 ? 1 : S;
  p.steps = (T + S - 1) / S;
  p.S = (T + p.steps - 1) / p.steps;
  const int64_t groups = K / group;
  size_t off = 0;
  p.off_st = off;       off += up256((size_t)(groups * p.C * 2));
  p.off_sub = off;      off += zp ? up256((size_t)(groups * p.C * 2)) : 0;
  p.off_pmax = off;     off += up256((size_t)(kParts * groups * 4));
  p.off_col = off;      off += up256((size_t)(groups * 4));
  p.off_unscale = off;  off += up256((size_t)(M * 4));
  p.off_hi = off;       off += up256((size_t)(M * p.C * 2));
  p.off_lo = off;       off += gated ? up256((size_t)(M * p.C * 2)) : 0;
  p.off_part = off;     off += p.S > 1 ? up256((size_t)(p.S * M * K * 4)) : 0;
  p.ws_bytes = off;
  return p;
}

template <int G, bool ZP, bool GATED>
static hipError_t grad(const uint16_t* dY, const GatedSaved& V, int act, const GatedWeights& W,
                       const uint16_t* s16, int64_t M, int64_t N, int64_t K, uint16_t* dA,
                       char* ws, hipStream_t stream) {
  const GradPlan p = w4a16_grad_plan(M, N, K, G, GATED, ZP);
  const GradShape S{M, N, K, p.Nc, p.C};
  uint16_t* st = reinterpret_cast<uint16_t*>(ws + p.off_st);
  uint16_t* sub = reinterpret_cast<uint16_t*>(ws + p.off_sub);
  uint32_t* pmax = reinterpret_cast<uint32_t*>(ws + p.off_pmax);
  float* col = reinterpret_cast<float*>(ws + p.off_col);
  float* unscale = reinterpret_cast<float*>(ws + p.off_unscale);
  uint16_t* hi = reinterpret_cast<uint16_t*>(ws + p.off_hi);
  uint16_t* lo = reinterpret_cast<uint16_t*>(ws + p.off_lo);
  float* part = p.S > 1 ? reinterpret_cast<float*>(ws + p.off_part) : nullptr;
  hipError_t e;
#define AWQ_GR1(ACT_, IT_)                                                           \
  grad_rows_kernel<GATED, ACT_, IT_><<<(unsigned)M + kParts, 512, 0, stream>>>(      \
      dY, V, W, S, (int)(K / G), hi, lo, unscale, pmax)
#define AWQ_GR(ACT_)                                                                 \
  do {                                                                               \
    if (p.Nc <= 4096) AWQ_GR1(ACT_, 1);                                              \
    else if (p.Nc <= 2 * 4096) AWQ_GR1(ACT_, 2);                                     \
    else if (p.Nc <= 3 * 4096) AWQ_GR1(ACT_, 3);                                     \
    else if (p.Nc <= 5 * 4096) AWQ_GR1(ACT_, 5);                                     \
    else if (p.Nc <= 7 * 4096) AWQ_GR1(ACT_, 7);                                     \
    else AWQ_GR1(ACT_, 0);                                                           \
  } while (0)
  if (!GATED || act == kSilu) AWQ_GR(kSilu); else AWQ_GR(kGelu);
#undef AWQ_GR
#undef AWQ_GR1
  if ((e = hipGetLastError()) != hipSuccess) return e;
  grad_steps_kernel<ZP><<<(unsigned)(p.C / 32), 256, 0, stream>>>(W, S, (int)(K / G), pmax, st, sub,
                                                                  col);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned grid = (unsigned)(p.tm * p.tk * p.S);
  const auto lds = [](int bm) { return (size_t)2 * (2 * bm * 64 + 2 * G * 64); };
  if (p.bm == 256)
    grad_gemm_kernel<G, ZP, GATED, 256><<<grid, 512, lds(256), stream>>>(
        W, S, hi, lo, st, sub, unscale, col, s16, dA, (uint32_t)p.tm, (uint32_t)p.tk, (int)p.steps, part);
  else
    grad_gemm_kernel<G, ZP, GATED, 64><<<grid, 256, lds(64), stream>>>(
        W, S, hi, lo, st, sub, unscale, col, s16, dA, (uint32_t)p.tm, (uint32_t)p.tk, (int)p.steps, part);
  if ((e = hipGetLastError()) != hipSuccess || p.S == 1) return e;
  grad_finish_kernel<<<(unsigned)((M * K / 4 + 255) / 256), 256, 0, stream>>>(
      part, (int)p.S, S, G, unscale, col, s16, dA);
  return hipGetLastError();
}

hipError_t launch_w4a16_gemm_backward(const uint16_t* dY, const uint32_t* qweight,
                                      const uint16_t* scales16, const uint8_t* zeros,
                                      const uint16_t* s16, int64_t M, int64_t N, int64_t K,
                                      int group, uint16_t* dA, void* ws, hipStream_t stream) {
  const GatedWeights W{{qweight, qweight}, {scales16, scales16}, {zeros, zeros}};
  const GatedSaved V{};
  char* w = static_cast<char*>(ws);
#define AWQ_G(GS_, ZP_) grad<GS_, ZP_, false>(dY, V, kSilu, W, s16, M, N, K, dA, w, stream)
  if (group == 64) return zeros ? AWQ_G(64, true) : AWQ_G(64, false);
  return zeros ? AWQ_G(128, true) : AWQ_G(128, false);
#undef AWQ_G
}

hipError_t launch_w4a16_gated_backward(const uint16_t* dH, const uint8_t* g8, const float* gs,
                                       const uint8_t* u8, const float* us, const GatedWeights& W,
                                       int64_t M, int64_t N, int64_t K, int group, int act,
                                       uint16_t* dA, void* ws, hipStream_t stream) {
  const GatedSaved V{g8, u8, gs, us};
  char* w = static_cast<char*>(ws);
  const bool zp = W.z[0] != nullptr;
#define AWQ_G(GS_, ZP_) grad<GS_, ZP_, true>(dH, V, act, W, nullptr, M, N, K, dA, w, stream)
  if (group == 64) return zp ? AWQ_G(64, true) : AWQ_G(64, false);
  return zp ? AWQ_G(128, true) : AWQ_G(128, false);
#undef AWQ_G
}

}  // namespace awq
