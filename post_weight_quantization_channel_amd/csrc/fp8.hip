// The 8-bit block quantizer and its inverse (format: fp8_format.h).
//
// Both are streaming passes: 16-bit input gives 2 bytes read and 1 written per value, and nothing
// is read twice, so memory bounds them. Blocks by 1 row: 16 lanes hold one block (8 channels
// each), its maximum is four DPP steps. Blocks by 128 rows: one workgroup holds one block in
// registers (8 rows of 8 channels per thread). Measured: 28672 x 8192 fp16 in 128 x 128 blocks 129 us
// (705 MB, 5.4 TB/s), back to bf16 126 us; a large copy reaches 5.0 TB/s.
#include "fp8_format.h"
#include "kernels.h"

namespace awq {

namespace {

// 8 values at X + idx (all in bounds), or zeros
template <int DT>
__device__ __forceinline__ void load8_or_zero(const void* X, int64_t idx, bool ok, float (&v)[8]) {
  if (ok) {
    load8_f32<DT>(static_cast<const char*>(X) + idx * (DT == kF32 ? 4 : 2), v);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = 0.0f;
  }
}

}  // namespace

// One block of 128 channels of one row per 16 lanes. blocks = M ceil(K / 128) < 2^32.
template <int DT>
__global__ __launch_bounds__(256) void fp8_quantize_rows_kernel(
    const void* __restrict__ X, uint32_t blocks, uint32_t KB, int64_t K, int64_t ldx,
    uint8_t* __restrict__ q, float* __restrict__ scales, uint32_t* __restrict__ flags) {
  const uint32_t b = blockIdx.x * 16u + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const bool in = b < blocks;
  const uint32_t row = in ? b / KB : 0u;
  const int64_t k = in ? (int64_t)(b - row * KB) * 128 + 8 * l : K;
  float v[8];
  load8_or_zero<DT>(X, (int64_t)row * ldx + k, k < K, v);
  float amax;
  const uint32_t bad = fp8_absmax8(v, amax);
  const Fp8Scale s = fp8_scale(group_absmax<16>(amax));
  if (k < K) {
    *reinterpret_cast<uint2*>(q + (int64_t)row * K + k) = fp8_pack8(v, s.inv, bad);
  }
  if (in && l == 0) scales[b] = s.scale;
  if (flags) wave_flag(flags, bad != 0u, kFlagNonfiniteX);
}

// One 128 x 128 block per workgroup of 256 threads; blockIdx.x = row block * KB + column block.
template <int DT>
__global__ __launch_bounds__(256) void fp8_quantize_tiles_kernel(
    const void* __restrict__ X, int64_t M, uint32_t KB, int64_t K, int64_t ldx,
    uint8_t* __restrict__ q, float* __restrict__ scales, uint32_t* __restrict__ flags) {
  __shared__ float wmax[4];
  const uint32_t rb = blockIdx.x / KB, kb = blockIdx.x - rb * KB;
  const int64_t k = (int64_t)kb * 128 + 8 * (threadIdx.x & 15);
  const int64_t m0 = (int64_t)rb * 128 + (threadIdx.x >> 4);
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8_or_zero<DT>(X, (m0 + 16 * i) * ldx + k, k < K && m0 + 16 * i < M, v[i]);
  float amax = 0.0f;
  uint32_t bad[8], any = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a;
    bad[i] = fp8_absmax8(v[i], a);
    any |= bad[i];
    amax = fmaxf(amax, a);
  }
  amax = group_absmax<16>(amax);
  amax = fmaxf(amax, __shfl_xor(amax, 16));
  amax = fmaxf(amax, __shfl_xor(amax, 32));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
  __syncthreads();
  const Fp8Scale s = fp8_scale(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k < K && m0 + 16 * i < M) {
      *reinterpret_cast<uint2*>(q + (m0 + 16 * i) * K + k) = fp8_pack8(v[i], s.inv, bad[i]);
    }
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
  if (flags) wave_flag(flags, any != 0u, kFlagNonfiniteX);
}

// 16 codes per thread (K % 16 == 0, so they lie in one row and one block). units = M K / 16.
template <int DT>
__global__ __launch_bounds__(256) void fp8_dequantize_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ scales, int64_t units, int64_t upr,
    int64_t KB, int rows_shift, void* __restrict__ out) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int64_t row = (units >> 32) == 0 ? (int64_t)((uint32_t)u / (uint32_t)upr) : u / upr;
  const int64_t col = u - row * upr;
  const float s = scales[(row >> rows_shift) * KB + (col >> 3)];
  const uint4 w4 = *reinterpret_cast<const uint4*>(q + u * 16);
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  float v[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float t[4];
    fp8_unpack4(w[j], t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * j + i] = t[i] * s;
  }
  if constexpr (DT == kF32) {
    float4* o = reinterpret_cast<float4*>(out) + u * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      p[j] = DT == kF16 ? f2h2(v[2 * j], v[2 * j + 1])
                        : ((uint32_t)f2bf(v[2 * j]) | ((uint32_t)f2bf(v[2 * j + 1]) << 16));
    uint4* o = reinterpret_cast<uint4*>(out) + u * 2;
    o[0] = make_uint4(p[0], p[1], p[2], p[3]);
    o[1] = make_uint4(p[4], p[5], p[6], p[7]);
  }
}

hipError_t launch_fp8_quantize(const void* X, int dtype, int64_t M, int64_t K, int64_t ldx,
                               int block_rows, uint8_t* q, float* scales, uint32_t* flags,
                               hipStream_t stream) {
  const int64_t KB = (K + 127) / 128;
  if (block_rows == 1) {
    const uint32_t blocks = (uint32_t)(M * KB);
    const unsigned grid = (unsigned)((M * KB + 15) / 16);
#define AWQ_Q(DT_)                                                                      \
  fp8_quantize_rows_kernel<DT_><<<grid, 256, 0, stream>>>(X, blocks, (uint32_t)KB, K, ldx, q, \
                                                          scales, flags)
    if (dtype == kF32) AWQ_Q(kF32); else if (dtype == kF16) AWQ_Q(kF16); else AWQ_Q(kBF16);
#undef AWQ_Q
  } else {
    const unsigned grid = (unsigned)(((M + 127) / 128) * KB);
#define AWQ_Q(DT_)                                                                              \
  fp8_quantize_tiles_kernel<DT_><<<grid, 256, 0, stream>>>(X, M, (uint32_t)KB, K, ldx, q, scales, \
                                                           flags)
    if (dtype == kF32) AWQ_Q(kF32); else if (dtype == kF16) AWQ_Q(kF16); else AWQ_Q(kBF16);
#undef AWQ_Q
  }
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* q, const float* scales, int64_t M, int64_t K,
                                 int block_rows, int dtype, void* out, hipStream_t stream) {
  const int64_t upr = K / 16, units = M * upr;
  const unsigned grid = (unsigned)((units + 255) / 256);
#define AWQ_D(DT_)                                                                          \
  fp8_dequantize_kernel<DT_><<<grid, 256, 0, stream>>>(q, scales, units, upr, (K + 127) / 128, \
                                                       block_rows == 1 ? 0 : 7, out)
  if (dtype == kF32) AWQ_D(kF32); else if (dtype == kF16) AWQ_D(kF16); else AWQ_D(kBF16);
#undef AWQ_D
  return hipGetLastError();
}

}  // namespace awq
