// q8_gemm_simple.cu -- the grouped 8-bit products on the CUDA cores: 16 rows of one expert
// by 128 output features per block, one feature per thread, fp32 accumulation.
#include <cuda_fp8.h>

#include "kernels.h"
#include "q8.cuh"

namespace dsmoe {
namespace {
constexpr int kRows = 16;

__device__ __forceinline__ float e4m3(uint32_t b) {
  __nv_fp8_e4m3 v;
  v.__x = static_cast<uint8_t>(b);
  return static_cast<float>(v);
}
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u) : s == 0u ? __uint_as_float(1u << 22) : __uint_as_float(s << 23);
}

template <bool kGated>
__global__ void __launch_bounds__(128) q8_simple_kernel(const Q8GemmArgs a) {
  __shared__ float s_a[kRows][kQ8Block];
  __shared__ int s_e, s_row, s_end;
  __shared__ uint32_t s_max[4][kRows];
  if (threadIdx.x == 0) {
    int left = blockIdx.y, e = 0;
    s_e = -1;
    for (; e < a.E; ++e) {
      const int b = min(max(a.offsets[e], 0), a.R), t = min(max(a.offsets[e + 1], b), a.R);
      const int tiles = (t - b + kRows - 1) / kRows;
      if (left < tiles) {
        s_e = e;
        s_row = b + left * kRows;
        s_end = t;
        break;
      }
      left -= tiles;
    }
  }
  __syncthreads();
  if (s_e < 0) return;
  const int e = s_e, row0 = s_row, rows = min(kRows, s_end - s_row);
  const int S = q8_scale_cols(a.K), nnb = (a.N + kQ8Block - 1) / kQ8Block;
  const int n = blockIdx.x * kQ8Block + threadIdx.x;
  const bool ok = n < a.N;
  float acc[kGated ? 2 : 1][kRows] = {};
  for (int k0 = 0; k0 < a.K; k0 += kQ8Block) {
    __syncthreads();
    const int kn = min(kQ8Block, a.K - k0);
    for (int i = threadIdx.x; i < kRows * kQ8Block; i += 128) {
      const int r = i / kQ8Block, k = i % kQ8Block;
      float v = 0.f;
      if (r < rows && k < kn) {
        const int64_t row = row0 + r;
        v = e4m3(a.a[row * a.K + k0 + k]) * scale_value(a.a_scales[row * S + k0 / kQ8Block]);
      }
      s_a[r][k] = v;
    }
    __syncthreads();
    if (!ok) continue;
#pragma unroll
    for (int w = 0; w < (kGated ? 2 : 1); ++w) {
      const uint8_t* W = (w ? a.W1 : a.W) + (static_cast<int64_t>(e) * a.N + n) * a.K + k0;
      const float sc = scale_value((w ? a.W1_scales : a.W_scales)[(static_cast<int64_t>(e) * nnb + blockIdx.x) * S + k0 / kQ8Block]);
      for (int k = 0; k < kn; k += 4) {
        const uint32_t w4 = *reinterpret_cast<const uint32_t*>(W + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float wv = e4m3((w4 >> (8 * j)) & 255u) * sc;
#pragma unroll
          for (int r = 0; r < kRows; ++r) acc[w][r] = fmaf(s_a[r][k + j], wv, acc[w][r]);
        }
      }
    }
  }
  if (!kGated) {
    for (int r = 0; r < rows; ++r)
      if (ok) a.out[static_cast<int64_t>(row0 + r) * a.N + n] = __float2bfloat16_rn(acc[0][r]);
    return;
  }
  const int So = q8_scale_cols(a.N);
  float m[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float g = acc[0][r];
    m[r] = ok ? g / (1.0f + __expf(-g)) * acc[kGated ? 1 : 0][r] : 0.f;
    const uint32_t x = __reduce_max_sync(0xffffffffu, abs_bits(m[r]));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5][r] = x;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r >= rows) break;
    const uint32_t s = q8_scale_byte(max(max(s_max[0][r], s_max[1][r]), max(s_max[2][r], s_max[3][r])));
    const int64_t row = row0 + r;
    if (ok) a.q_out[row * a.N + n] = s == 255u ? 0x7F : static_cast<uint8_t>(q8_pack2(m[r] * q8_inv_scale(s), 0.f));
    if (threadIdx.x == 0) a.q_scales[row * So + blockIdx.x] = static_cast<uint8_t>(s);
    if (static_cast<int>(blockIdx.x) == nnb - 1 && static_cast<int>(threadIdx.x) < So - nnb)
      a.q_scales[row * So + nnb + threadIdx.x] = kQ8PadScale;
  }
}
}  // namespace

cudaError_t launch_q8_simple(const Q8GemmArgs& a, cudaStream_t s) {
  const dim3 grid((a.N + kQ8Block - 1) / kQ8Block, (a.R + kRows - 1) / kRows + a.E);
  if (grid.y > 65535) return cudaErrorInvalidValue;
  if (a.W1) q8_simple_kernel<true><<<grid, 128, 0, s>>>(a);
  else q8_simple_kernel<false><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}
}  // namespace dsmoe
