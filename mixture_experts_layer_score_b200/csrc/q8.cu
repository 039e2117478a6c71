// q8.cu -- the memory-bound operators of the 8-bit path: block quantisation of token rows
// (1 x 128 blocks) and of expert weights (128 x 128), and the RMSNorm in front of the
// layer, which adds the residual, writes the bf16 rows that the router reads and the 8-bit
// rows that the experts read, with its backward pass.
#include "kernels.h"
#include "q8.cuh"
#include "sm100_ptx.cuh"

namespace dsmoe {

namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16x2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  return m;
}

// The eight e4m3 values of f under scale byte s.
__device__ __forceinline__ uint2 encode8(const float (&f)[8], uint32_t s) {
  if (s == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float m = q8_inv_scale(s);
  return make_uint2(q8_pack4(f[0] * m, f[1] * m, f[2] * m, f[3] * m),
                    q8_pack4(f[4] * m, f[5] * m, f[6] * m, f[7] * m));
}

// Largest of v over the 16 lanes of this half warp (all 32 lanes call).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sixteen lanes hold one block of 128 values, eight each.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const bf16* __restrict__ x, int64_t R, int C,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  const int nb = (C + kQ8Block - 1) / kQ8Block, S = q8_scale_cols(C);
  const int64_t units = R * nb, step = static_cast<int64_t>(gridDim.x) * 16;
  const int sub = threadIdx.x & 15;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  // every lane of a warp runs the same number of rounds (the shuffles need them all)
  const int64_t warp_first = static_cast<int64_t>(blockIdx.x) * 16 + ((threadIdx.x >> 5) << 1);
  for (int64_t u0 = warp_first, u = first; u0 < units; u0 += step, u += step) {
    const bool row_ok = u < units;
    const int64_t r = row_ok ? u / nb : 0;
    const int b = row_ok ? static_cast<int>(u - r * nb) : 0;
    const int c = b * kQ8Block + sub * 8;
    const bool ok = row_ok && c < C;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) v = *reinterpret_cast<const uint4*>(x + r * C + c);
    float f[8];
    unpack8(v, f);
    const uint32_t s = q8_scale_byte(half_warp_max(amax8(f)));
    if (ok) *reinterpret_cast<uint2*>(q + r * C + c) = encode8(f, s);
    if (row_ok && sub == 0) scales[r * S + b] = static_cast<uint8_t>(s);
    if (row_ok && b == nb - 1 && sub < S - nb) scales[r * S + nb + sub] = kQ8PadScale;
  }
}

// One block of threads per 128 x 128 tile of one expert's matrix; the tile stays in registers
// between the maximum and the encoding (thread: eight columns of rows i, i + 16, ...).
__global__ void __launch_bounds__(256) quantize_weights_kernel(const bf16* __restrict__ W, int64_t tiles, int N, int K,
                                                               uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scales) {
  __shared__ uint32_t s_max[8];
  const int nkb = (K + kQ8Block - 1) / kQ8Block, nnb = (N + kQ8Block - 1) / kQ8Block, S = q8_scale_cols(K);
  const int col = (threadIdx.x & 15) * 8, row = threadIdx.x >> 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t en = tile / nkb;  // expert * nnb + row block
    const int kb = static_cast<int>(tile - en * nkb);
    const int64_t e = en / nnb;
    const int nb = static_cast<int>(en - e * nnb);
    const int k = kb * kQ8Block + col;
    const int64_t base = (e * N + static_cast<int64_t>(nb) * kQ8Block) * K + k;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = row + 16 * i;
      v[i] = make_uint4(0, 0, 0, 0);
      if (k < K && nb * kQ8Block + n < N) v[i] = *reinterpret_cast<const uint4*>(W + base + static_cast<int64_t>(n) * K);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
      unpack8(v[i], f);
      m = max(m, amax8(f));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();  // the previous tile's s_max has been read
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
    const uint32_t s = q8_scale_byte(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = row + 16 * i;
      float f[8];
      unpack8(v[i], f);
      if (k < K && nb * kQ8Block + n < N)
        *reinterpret_cast<uint2*>(q + base + static_cast<int64_t>(n) * K) = encode8(f, s);
    }
    if (threadIdx.x == 0) scales[en * S + kb] = static_cast<uint8_t>(s);
    if (kb == nkb - 1 && static_cast<int>(threadIdx.x) < S - nkb) scales[en * S + nkb + threadIdx.x] = kQ8PadScale;
  }
}

// Sum over the block in a fixed order (warp butterflies, then the warps' sums in order); every
// thread gets the result. `red` holds 32 floats and is free again after the next call's
// first barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < warps; ++i) t += red[i];
  return t;
}

// One row per block: r = bf16(x + residual) stays in registers (8 NV values per thread)
// between the sum of squares and the scaled row u = bf16((r rstd) w); the 8-bit row is
// that of u, so that it equals the quantisation of the bf16 row.
template <int NV>
__global__ void __launch_bounds__(1024) norm_q8_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int d = a.d, nv = d >> 3, S = q8_scale_cols(d), nb = (d + kQ8Block - 1) / kQ8Block;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = static_cast<int64_t>(t) * d;
    float f[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      uint4 v = make_uint4(0, 0, 0, 0), rv = make_uint4(0, 0, 0, 0);
      if (c < nv) {
        v = reinterpret_cast<const uint4*>(a.x + row)[c];
        if (a.residual) rv = reinterpret_cast<const uint4*>(a.residual + row)[c];
      }
      unpack8(v, f[i]);
      if (a.residual) {
        float g[8];
        unpack8(rv, g);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(f[i][2 * j] + g[2 * j], f[i][2 * j + 1] + g[2 * j + 1]);
        v = make_uint4(w[0], w[1], w[2], w[3]);
        unpack8(v, f[i]);
      }
      if (a.r && c < nv) reinterpret_cast<uint4*>(a.r + row)[c] = v;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
    }
    const float rstd = rsqrtf(block_sum(ss, red) / static_cast<float>(d) + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      float w[8];
      uint4 wv = make_uint4(0, 0, 0, 0);
      if (c < nv) wv = reinterpret_cast<const uint4*>(a.w)[c];
      unpack8(wv, w);
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[j] = pack_bf16x2(f[i][2 * j] * rstd * w[2 * j], f[i][2 * j + 1] * rstd * w[2 * j + 1]);
      const uint4 uv = make_uint4(p[0], p[1], p[2], p[3]);
      if (a.u && c < nv) reinterpret_cast<uint4*>(a.u + row)[c] = uv;
      if (a.q) {  // threads past the row hold zeros; a block of 128 is one half warp
        unpack8(uv, f[i]);
        const uint32_t s = q8_scale_byte(half_warp_max(c < nv ? amax8(f[i]) : 0u));
        if (c < nv) {
          reinterpret_cast<uint2*>(a.q + row)[c] = encode8(f[i], s);
          if ((c & 15) == 0) a.scales[static_cast<int64_t>(t) * S + (c >> 4)] = static_cast<uint8_t>(s);
        }
      }
    }
    if (a.q && static_cast<int>(threadIdx.x) < S - nb)
      a.scales[static_cast<int64_t>(t) * S + nb + threadIdx.x] = kQ8PadScale;
  }
}

// dx and this block's share of dw: rows blockIdx.x, blockIdx.x + gridDim.x, ... in order; the
// row's two sums (of r^2 and of w dy r) are reduced together.
template <int NV>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBwdArgs a) {
  __shared__ float red[32];
  const int d = a.d, nv = d >> 3;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    uint4 wv = make_uint4(0, 0, 0, 0);
    if (c < nv) wv = reinterpret_cast<const uint4*>(a.w)[c];
    unpack8(wv, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  const float inv_d = 1.0f / static_cast<float>(d);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = static_cast<int64_t>(t) * d;
    float dy[NV][8], r[NV][8];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      uint4 rv = make_uint4(0, 0, 0, 0);
      float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f), y1 = y0;
      if (c < nv) {
        rv = reinterpret_cast<const uint4*>(a.r + row)[c];
        y0 = reinterpret_cast<const float4*>(a.dy + row)[2 * c];
        y1 = reinterpret_cast<const float4*>(a.dy + row)[2 * c + 1];
      }
      unpack8(rv, r[i]);
      dy[i][0] = y0.x, dy[i][1] = y0.y, dy[i][2] = y0.z, dy[i][3] = y0.w;
      dy[i][4] = y1.x, dy[i][5] = y1.y, dy[i][6] = y1.z, dy[i][7] = y1.w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(r[i][j], r[i][j], ss);
        sg = fmaf(dy[i][j] * w[i][j], r[i][j], sg);
      }
    }
    const float rstd = rsqrtf(block_sum(ss, red) * inv_d + a.eps);
    const float k = block_sum(sg, red) * inv_d * rstd * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nv) {
        float e[8];
        uint4 ev = make_uint4(0, 0, 0, 0);
        if (a.dres) ev = reinterpret_cast<const uint4*>(a.dres + row)[c];
        unpack8(ev, e);
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] += rstd * (dy[i][j] * w[i][j]) - r[i][j] * k;
          dw[i][j] = fmaf(dy[i][j], r[i][j] * rstd, dw[i][j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = pack_bf16x2(e[2 * j], e[2 * j + 1]);
        reinterpret_cast<uint4*>(a.dx + row)[c] = make_uint4(p[0], p[1], p[2], p[3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nv) {
      float4* p = reinterpret_cast<float4*>(a.part + static_cast<int64_t>(blockIdx.x) * d) + 2 * c;
      p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw[c] = the blocks' shares added in a fixed order: 32 row groups of consecutive blocks,
// then the groups in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int G, int d,
                                                       float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int per = (G + 31) / 32, b0 = g * per, b1 = min(G, b0 + per);
  float v = 0.f;
  if (c < d)
    for (int b = b0; b < b1; ++b) v += part[static_cast<int64_t>(b) * d + c];
  s[g][lane] = v;
  __syncthreads();
  if (g == 0 && c < d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][lane];
    dw[c] = t;
  }
}

// Vectors of eight per thread and threads of a block that holds one row of d values.
int norm_vectors(int d) { return d <= 8192 ? 1 : d <= 16384 ? 2 : 4; }
int norm_threads(int d) {
  const int per = norm_vectors(d) * 8;
  return (((d + per - 1) / per) + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_quantize_rows(const bf16* x, int64_t R, int C, uint8_t* q, uint8_t* scales, int num_sms,
                                 cudaStream_t s) {
  const int64_t units = R * ((C + kQ8Block - 1) / kQ8Block);
  int64_t grid = (units + 15) / 16;
  if (grid > 8 * num_sms) grid = 8 * num_sms;
  if (grid < 1) return cudaSuccess;
  quantize_rows_kernel<<<static_cast<int>(grid), 256, 0, s>>>(x, R, C, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_quantize_weights(const bf16* W, int E, int N, int K, uint8_t* q, uint8_t* scales, int num_sms,
                                    cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>(E) * ((N + kQ8Block - 1) / kQ8Block) * ((K + kQ8Block - 1) / kQ8Block);
  int64_t grid = 8 * num_sms;
  if (grid > tiles) grid = tiles;
  if (grid < 1) return cudaSuccess;
  quantize_weights_kernel<<<static_cast<int>(grid), 256, 0, s>>>(W, tiles, N, K, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_norm_q8(const NormArgs& a, int num_sms, cudaStream_t s) {
  const int threads = norm_threads(a.d), nv = norm_vectors(a.d);
  const int grid = a.T;
  (void)num_sms;
  if (nv == 1) norm_q8_kernel<1><<<grid, threads, 0, s>>>(a);
  else if (nv == 2) norm_q8_kernel<2><<<grid, threads, 0, s>>>(a);
  else norm_q8_kernel<4><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

int norm_backward_blocks(int64_t T, int d, int num_sms) {
  const int threads = norm_threads(d);
  const int per_sm = threads >= 1024 ? 1 : 1024 / threads;
  const int64_t g = static_cast<int64_t>(num_sms < kNormMaxSms ? num_sms : kNormMaxSms) * per_sm;
  return static_cast<int>(g < T ? g : T);
}

cudaError_t launch_norm_backward(const NormBwdArgs& a, float* dw, int num_sms, cudaStream_t s) {
  const int threads = norm_threads(a.d), nv = norm_vectors(a.d);
  const int grid = norm_backward_blocks(a.T, a.d, num_sms);
  if (nv == 1) norm_backward_kernel<1><<<grid, threads, 0, s>>>(a);
  else if (nv == 2) norm_backward_kernel<2><<<grid, threads, 0, s>>>(a);
  else norm_backward_kernel<4><<<grid, threads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_dw_kernel<<<(a.d + 31) / 32, 1024, 0, s>>>(a.part, grid, a.d, dw);
  return cudaGetLastError();
}

}  // namespace dsmoe
