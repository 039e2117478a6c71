// q8.cu -- the memory-bound operators of the 8-bit path: block quantisation of token rows
// (1 x 128 blocks) and of expert weights (128 x 128), and the RMSNorm in front of the
// layer, which adds the residual, writes the bf16 rows that the router reads and the 8-bit
// rows that the experts read, with its backward pass.
#include <algorithm>

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

// Sixteen lanes hold one block of 128 values, eight each; every thread has kQuantUnits blocks in
// flight (8192 x 7168, repeated: 43 us with one, 35 with two or four, 41 with eight).
constexpr int kQuantUnits = 4;
__global__ void __launch_bounds__(256) quantize_rows_kernel(const bf16* __restrict__ x, uint32_t units, int C,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  const int nb = (C + kQ8Block - 1) / kQ8Block, S = q8_scale_cols(C), sub = threadIdx.x & 15;
  const uint32_t first = blockIdx.x * (16u * kQuantUnits) + (threadIdx.x >> 4);
  uint4 v[kQuantUnits];
  uint32_t row[kQuantUnits];
  int blk[kQuantUnits];
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const uint32_t u = first + 16u * i;
    row[i] = u / static_cast<uint32_t>(nb);
    blk[i] = static_cast<int>(u - row[i] * nb);
    const int c = blk[i] * kQ8Block + sub * 8;
    v[i] = make_uint4(0, 0, 0, 0);
    if (u < units && c < C) v[i] = *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row[i]) * C + c);
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const bool ok = first + 16u * i < units;
    const int c = blk[i] * kQ8Block + sub * 8;
    const int64_t r = row[i];
    float f[8];
    unpack8(v[i], f);
    const uint32_t s = q8_scale_byte(half_warp_max(amax8(f)));
    if (!ok) continue;
    if (c < C) *reinterpret_cast<uint2*>(q + r * C + c) = encode8(f, s);
    if (sub == 0) scales[r * S + blk[i]] = static_cast<uint8_t>(s);
    if (blk[i] == nb - 1 && sub < S - nb) scales[r * S + nb + sub] = kQ8PadScale;
  }
}

// One block of threads per 128 x 128 tile of one expert's matrix; the tile stays in registers
// between the maximum and the encoding (thread: eight columns of rows i, i + 16, ...). Three blocks
// an SM: 32 x 2048 x 7168 weights, calls repeated, take 244 us (5.8 TB/s) against 259 with four, 269
// with two and 306 with five.
__global__ void __launch_bounds__(256, 3) quantize_weights_kernel(const bf16* __restrict__ W, int64_t tiles, int N,
                                                                  int K, uint8_t* __restrict__ q,
                                                                  uint8_t* __restrict__ scales) {
  __shared__ uint32_t s_max[2][8];
  const int nkb = (K + kQ8Block - 1) / kQ8Block, nnb = (N + kQ8Block - 1) / kQ8Block, S = q8_scale_cols(K);
  const int col = (threadIdx.x & 15) * 8, row = threadIdx.x >> 4;
  uint32_t turn = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1u) {
    const int64_t en = tile / nkb;  // expert * nnb + row block
    const int kb = static_cast<int>(tile - en * nkb);
    const int64_t e = en / nnb;
    const int n0 = static_cast<int>(en - e * nnb) * kQ8Block + row, k = kb * kQ8Block + col;
    // rows n0, n0 + 16, ... of this thread's columns, as far as the matrix goes
    const int rows = k < K ? (N - n0 + 15) / 16 : 0;
    const int64_t base = (e * N + n0) * K + k, step = static_cast<int64_t>(16) * K;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = i < rows ? __ldcs(reinterpret_cast<const uint4*>(W + base + i * step)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
      unpack8(v[i], f);
      m = max(m, amax8(f));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[turn][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, s_max[turn][i]);
    const uint32_t s = q8_scale_byte(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= rows) break;
      float f[8];
      unpack8(v[i], f);
      __stcs(reinterpret_cast<uint2*>(q + base + i * step), encode8(f, s));
    }
    if (threadIdx.x == 0) scales[en * S + kb] = static_cast<uint8_t>(s);
    if (kb == nkb - 1 && static_cast<int>(threadIdx.x) < S - nkb) scales[en * S + nkb + threadIdx.x] = kQ8PadScale;
  }
}

// One warp per token: lanes k < K' claim a slot in their expert's segment (experts in
// [e_begin, e_end); the others get slot -1), then the warp copies the token's 8-bit row
// (16-byte vectors, four in flight per lane) and its scales (words) to each claimed slot.
__global__ void __launch_bounds__(256) permute_q8_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ scales,
                                                         const int32_t* __restrict__ topk_idx,
                                                         const int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ cursor, int T, int K, int N,
                                                         int e_begin, int e_end, int d,
                                                         int32_t* __restrict__ slot_of, uint8_t* __restrict__ q_out,
                                                         uint8_t* __restrict__ scales_out, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int gw = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, nw = (gridDim.x * blockDim.x) >> 5;
  const int d16 = d >> 4, S4 = q8_scale_cols(d) >> 2;
  for (int t = gw; t < T; t += nw) {
    int pos = -1;
    if (lane < K) {
      const int e = topk_idx[static_cast<int64_t>(t) * K + lane];
      if (e < 0 || e >= N) {
        atomicOr(status, kStatusBadIndex);
      } else if (e >= e_begin && e < e_end) {
        pos = offsets[e] + atomicAdd(&cursor[e], 1);
      }
      slot_of[static_cast<int64_t>(t) * K + lane] = pos;
    }
    int pk[16];  // every lane learns all K' slots (K' <= 16)
#pragma unroll
    for (int k = 0; k < 16; ++k) pk[k] = __shfl_sync(0xffffffffu, pos, k);
    const uint4* src = reinterpret_cast<const uint4*>(q) + static_cast<int64_t>(t) * d16;
    for (int c0 = lane; c0 < d16; c0 += 4 * 32) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + 32 * u < d16) v[u] = src[c0 + 32 * u];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + 32 * u < d16)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < K && pk[k] >= 0)
              reinterpret_cast<uint4*>(q_out)[static_cast<int64_t>(pk[k]) * d16 + c0 + 32 * u] = v[u];
    }
    for (int c = lane; c < S4; c += 32) {
      const uint32_t v = reinterpret_cast<const uint32_t*>(scales)[static_cast<int64_t>(t) * S4 + c];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k < K && pk[k] >= 0) reinterpret_cast<uint32_t*>(scales_out)[static_cast<int64_t>(pk[k]) * S4 + c] = v;
    }
  }
}

// Sums of n values over the block, in a fixed order (warp butterflies, then the warps' sums in
// order); every thread gets them. red holds 32 n floats that the block has zeroed once; two
// of them used in turn make one barrier per call enough.
template <int n>
__device__ __forceinline__ void block_sums(float (&v)[n], float* red) {
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < n; ++i) red[32 * i + warp] = v[i];
  __syncthreads();
  const int quads = (static_cast<int>(blockDim.x >> 5) + 3) >> 2;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= quads) break;
      const float4 p = reinterpret_cast<const float4*>(red + 32 * i)[j];
      s += (p.x + p.y) + (p.z + p.w);
    }
    v[i] = s;
  }
}

__device__ __forceinline__ uint4 add_bf16x8(const uint4& a, const uint4& b) {
  float x[8], y[8];
  unpack8(a, x);
  unpack8(b, y);
  return make_uint4(pack_bf16x2(x[0] + y[0], x[1] + y[1]), pack_bf16x2(x[2] + y[2], x[3] + y[3]),
                    pack_bf16x2(x[4] + y[4], x[5] + y[5]), pack_bf16x2(x[6] + y[6], x[7] + y[7]));
}

// One row at a time per block, 8 NV values per thread: r = bf16(x + residual) stays in
// registers between the sum of squares and the scaled row u = bf16((r rstd) w); the 8-bit
// row is that of u, so that it equals the quantisation of the bf16 row. The block loads
// its next row before it reduces this one. Bound by HBM: 9 bytes a value, 8192 x 7168 in
// 87 us in a burst, 89-90 repeated (5.9 TB/s).
template <int NV>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512) norm_q8_kernel(const NormArgs a) {
  __shared__ __align__(16) float red[2][32];
  const int d = a.d, nv = d >> 3, S = q8_scale_cols(d), nb = (d + kQ8Block - 1) / kQ8Block;
  if (threadIdx.x < 64) (&red[0][0])[threadIdx.x] = 0.f;
  if (blockDim.x < 64 && threadIdx.x + 32 < 64) (&red[0][0])[threadIdx.x + 32] = 0.f;
  __syncthreads();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 x[NV], y[NV];
  auto load = [&](int t) {
    const int64_t row = static_cast<int64_t>(t) * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      x[i] = y[i] = zero;
      if (c < nv) {
        x[i] = reinterpret_cast<const uint4*>(a.x + row)[c];
        if (a.residual) y[i] = reinterpret_cast<const uint4*>(a.residual + row)[c];
      }
    }
  };
  int t = blockIdx.x;
  if (t < a.T) load(t);
  for (uint32_t turn = 0; t < a.T; turn ^= 1u) {
    const int64_t row = static_cast<int64_t>(t) * d;
    uint4 r[NV];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      r[i] = a.residual ? add_bf16x8(x[i], y[i]) : x[i];
      if (a.r && c < nv) reinterpret_cast<uint4*>(a.r + row)[c] = r[i];
      float f[8];
      unpack8(r[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(f[j], f[j], ss[0]);
    }
    const int t_row = t;
    t += gridDim.x;
    if (t < a.T) load(t);
    block_sums<1>(ss, red[turn]);
    // rounded to nearest: rsqrtf moves 12% more of u's values across a bf16 border (8192 x 7168:
    // 490 against 440 of 5.9e7), in the same time
    const float rstd = __frsqrt_rn(ss[0] / static_cast<float>(d) + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      float f[8], w[8];
      unpack8(r[i], f);
      unpack8(c < nv ? __ldg(reinterpret_cast<const uint4*>(a.w) + c) : zero, w);
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = pack_bf16x2(f[2 * j] * rstd * w[2 * j], f[2 * j + 1] * rstd * w[2 * j + 1]);
      const uint4 u = make_uint4(p[0], p[1], p[2], p[3]);
      if (a.u && c < nv) reinterpret_cast<uint4*>(a.u + row)[c] = u;
      if (a.q) {  // a block of 128 is one half warp; threads past the row hold zeros
        unpack8(u, f);
        const uint32_t s = q8_scale_byte(half_warp_max(c < nv ? amax8(f) : 0u));
        if (c < nv) {
          reinterpret_cast<uint2*>(a.q + row)[c] = encode8(f, s);
          if ((c & 15) == 0) a.scales[static_cast<int64_t>(t_row) * S + (c >> 4)] = static_cast<uint8_t>(s);
        }
      }
    }
    if (a.q && static_cast<int>(threadIdx.x) < S - nb)
      a.scales[static_cast<int64_t>(t_row) * S + nb + threadIdx.x] = kQ8PadScale;
  }
}

// 16 bytes from global to shared memory, asynchronously; groups are waited for in order.
__device__ __forceinline__ void copy16_async(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// The part of the backward pass that follows a row's two sums: dx of eight columns, and their
// terms of dw.
__device__ __forceinline__ void norm_backward_columns(const float (&dy)[8], const float (&r)[8], const float (&w)[8],
                                                      const uint4& dres, float rstd, float m, float (&dw)[8],
                                                      bf16* dx) {
  float e[8];
  unpack8(dres, e);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    e[j] += rstd * (dy[j] * w[j]) - r[j] * m;
    dw[j] = fmaf(dy[j], r[j] * rstd, dw[j]);
  }
  *reinterpret_cast<uint4*>(dx) = make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]),
                                             pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7]));
}

__device__ __forceinline__ void store_share(float* part, int64_t at, const float (&dw)[8]) {
  float4* p = reinterpret_cast<float4*>(part + at);
  p[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
  p[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
}

// dx and this block's share of dw, for rows of at most 8192 values: eight columns per
// thread, rows t, t + grid, ... in order. The rows ahead are copied into a ring of kBwdStages
// rows in shared memory, so that loads stay in flight through the barrier of the row's sums
// (of r^2 and of w dy r); each warp reads only what it copied itself. Bound by HBM: 10 bytes a
// value, 16384 x 1280 in 40 us with the kernel that adds the shares (with the rows loaded into
// registers between the barriers it took a quarter longer).
constexpr int kBwdStages = 3;
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBwdArgs a) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ __align__(16) float red[2][64];
  const int d = a.d, nv = d >> 3, lane = threadIdx.x & 31, c = threadIdx.x, B = blockDim.x;
  for (int i = threadIdx.x; i < 128; i += B) (&red[0][0])[i] = 0.f;
  __syncthreads();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool on = c < nv;
  // dy leaves in the order of its lines: 64 units of 16 bytes per warp, two of them a lane's
  const int u0 = 2 * (c - lane) + lane;
  auto load = [&](int t, int stage) {
    if (t < a.T) {
      uint4* s = ring + static_cast<int64_t>(stage) * 4 * B;
      const int64_t row = static_cast<int64_t>(t) * d;
      const uint4* y = reinterpret_cast<const uint4*>(a.dy + row);
      if (u0 < 2 * nv) copy16_async(s + u0, y + u0);
      if (u0 + 32 < 2 * nv) copy16_async(s + u0 + 32, y + u0 + 32);
      if (on) {
        copy16_async(s + 2 * B + c, reinterpret_cast<const uint4*>(a.r + row) + c);
        if (a.dres) copy16_async(s + 3 * B + c, reinterpret_cast<const uint4*>(a.dres + row) + c);
      }
    }
    copy_commit();
  };
  float w[8], dw[8] = {};
  unpack8(on ? reinterpret_cast<const uint4*>(a.w)[c] : zero, w);
  const float inv_d = 1.0f / static_cast<float>(d);
#pragma unroll
  for (int i = 0; i < kBwdStages - 1; ++i) load(blockIdx.x + i * gridDim.x, i);
  int stage = 0;
  uint32_t turn = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1u) {
    // into the row before this one, which every warp has read before the last barrier
    load(t + (kBwdStages - 1) * gridDim.x, stage == 0 ? kBwdStages - 1 : stage - 1);
    copy_wait<kBwdStages - 1>();
    __syncwarp();
    const uint4* s = ring + static_cast<int64_t>(stage) * 4 * B;
    float dy[8] = {}, r[8] = {};
    uint4 dres = zero;
    if (on) {
      const float4 y0 = reinterpret_cast<const float4*>(s)[2 * c], y1 = reinterpret_cast<const float4*>(s)[2 * c + 1];
      dy[0] = y0.x, dy[1] = y0.y, dy[2] = y0.z, dy[3] = y0.w;
      dy[4] = y1.x, dy[5] = y1.y, dy[6] = y1.z, dy[7] = y1.w;
      unpack8(s[2 * B + c], r);
      if (a.dres) dres = s[3 * B + c];
    }
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[0] = fmaf(r[j], r[j], sums[0]);
      sums[1] = fmaf(dy[j] * w[j], r[j], sums[1]);
    }
    block_sums<2>(sums, red[turn]);
    const float rstd = rsqrtf(sums[0] * inv_d + a.eps);
    if (on)
      norm_backward_columns(dy, r, w, dres, rstd, sums[1] * inv_d * rstd * rstd * rstd, dw,
                            a.dx + static_cast<int64_t>(t) * d + 8 * c);
    stage = stage + 1 == kBwdStages ? 0 : stage + 1;
  }
  if (on) store_share(a.part, static_cast<int64_t>(blockIdx.x) * d + 8 * c, dw);
}

// The same for longer rows, which a ring in shared memory would not hold: 8 NV columns per
// thread, loaded into registers.
template <int NV>
__global__ void __launch_bounds__(512) norm_backward_long_kernel(const NormBwdArgs a) {
  __shared__ __align__(16) float red[2][64];
  const int d = a.d, nv = d >> 3;
  for (int i = threadIdx.x; i < 128; i += blockDim.x) (&red[0][0])[i] = 0.f;
  __syncthreads();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float dw[NV][8] = {};
  const float inv_d = 1.0f / static_cast<float>(d);
  uint32_t turn = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1u) {
    const int64_t row = static_cast<int64_t>(t) * d;
    float sums[2] = {0.f, 0.f};
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {  // the second pass reads the row again, from L2
      const float rstd = rsqrtf(sums[0] * inv_d + a.eps), m = sums[1] * inv_d * rstd * rstd * rstd;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nv) continue;
        float r[8], w[8];
        unpack8(reinterpret_cast<const uint4*>(a.r + row)[c], r);
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.w) + c), w);
        const float4 y0 = reinterpret_cast<const float4*>(a.dy + row)[2 * c];
        const float4 y1 = reinterpret_cast<const float4*>(a.dy + row)[2 * c + 1];
        const float dy[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        if (pass == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sums[0] = fmaf(r[j], r[j], sums[0]);
            sums[1] = fmaf(dy[j] * w[j], r[j], sums[1]);
          }
        } else {
          norm_backward_columns(dy, r, w, a.dres ? reinterpret_cast<const uint4*>(a.dres + row)[c] : zero, rstd, m,
                                dw[i], a.dx + row + 8 * c);
        }
      }
      if (pass == 0) block_sums<2>(sums, red[turn]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nv) store_share(a.part, static_cast<int64_t>(blockIdx.x) * d + 8 * c, dw[i]);
  }
}

// dw of eight columns per block: the blocks' shares are added in a fixed order, 128 groups of
// rows (two threads of four columns each) and then the groups. (32 columns per block keeps
// too few SMs busy.)
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ part, int G, int d,
                                                      float* __restrict__ dw) {
  __shared__ float s[128][9];
  const int g = threadIdx.x >> 1, c = (threadIdx.x & 1) * 4, col = blockIdx.x * 8 + c;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int b = g; b < G; b += 128) {
    const float4 p = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(b) * d + col);
    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
  }
  s[g][c] = v.x, s[g][c + 1] = v.y, s[g][c + 2] = v.z, s[g][c + 3] = v.w;
  __syncthreads();
  // warp w sums column w: four groups per lane, then a butterfly
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float t = (s[lane][w] + s[lane + 32][w]) + (s[lane + 64][w] + s[lane + 96][w]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) dw[blockIdx.x * 8 + w] = t;
}

// How a block holds rows of d values: vectors of eight per thread, threads.
int norm_vectors(int d) { return d <= 2048 ? 1 : d <= 8192 ? 2 : d <= 16384 ? 4 : 8; }
int norm_threads(int d) {
  const int per = norm_vectors(d) * 8;
  return ((d + per - 1) / per + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_quantize_rows(const bf16* x, int64_t R, int C, uint8_t* q, uint8_t* scales, cudaStream_t s) {
  const int64_t units = R * ((C + kQ8Block - 1) / kQ8Block);
  if (units == 0) return cudaSuccess;
  if (units > INT32_MAX - 64) return cudaErrorInvalidValue;  // more values than any GPU's memory holds
  const int grid = static_cast<int>((units + 16 * kQuantUnits - 1) / (16 * kQuantUnits));
  quantize_rows_kernel<<<grid, 256, 0, s>>>(x, static_cast<uint32_t>(units), C, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_quantize_weights(const bf16* W, int E, int N, int K, uint8_t* q, uint8_t* scales,
                                    cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>(E) * ((N + kQ8Block - 1) / kQ8Block) * ((K + kQ8Block - 1) / kQ8Block);
  // a block per tile: the blocks' phases drift apart and keep the memory busy (32 x 2048 x 7168
  // weights, repeated: 244 us, against 250 with as many blocks as are resident at once)
  const int64_t grid = std::min<int64_t>(tiles, 1 << 30);
  quantize_weights_kernel<<<static_cast<int>(grid), 256, 0, s>>>(W, tiles, N, K, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_permute_q8(const uint8_t* q, const uint8_t* scales, const int32_t* topk_idx,
                              const int32_t* offsets, int32_t* cursor, int T, int K, int N, int e_begin, int e_end,
                              int d, int32_t* slot_of, uint8_t* q_out, uint8_t* scales_out, uint32_t* status,
                              int num_sms, cudaStream_t s) {
  const int grid = std::max(1, std::min((T + 7) / 8, 8 * num_sms));
  permute_q8_kernel<<<grid, 256, 0, s>>>(q, scales, topk_idx, offsets, cursor, T, K, N, e_begin, e_end, d, slot_of,
                                         q_out, scales_out, status);
  return cudaGetLastError();
}

cudaError_t launch_norm_q8(const NormArgs& a, int num_sms, cudaStream_t s) {
  const int nv = norm_vectors(a.d), threads = norm_threads(a.d);
  // eight blocks per SM, more than are resident at once, so that their phases drift apart (8192
  // rows of 7168: 87 us against 94 with the resident two and 101 with a block per row)
  const int grid = static_cast<int>(std::min<int64_t>(a.T, 8 * num_sms));
  if (nv == 1) norm_q8_kernel<1><<<grid, threads, 0, s>>>(a);
  else if (nv == 2) norm_q8_kernel<2><<<grid, threads, 0, s>>>(a);
  else if (nv == 4) norm_q8_kernel<4><<<grid, threads, 0, s>>>(a);
  else norm_q8_kernel<8><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

namespace {
constexpr int kBwdRingMax = 8192;  // longest row of norm_backward_kernel
int bwd_threads(int d) { return d <= kBwdRingMax ? (d / 8 + 31) / 32 * 32 : 512; }
int bwd_ring_bytes(int d) { return d <= kBwdRingMax ? kBwdStages * bwd_threads(d) * 64 : 0; }
}  // namespace

// Blocks of the backward pass: about 512 threads per SM (16384 rows of 1280: 40 us, with 1024
// threads 47; fewer shares of dw to add too), 1024 where a row has more than 320, and about
// 200 KB of rings.
int norm_backward_blocks(int64_t T, int d, int num_sms) {
  int per_sm = (bwd_threads(d) > 320 ? 1024 : 512) / bwd_threads(d);
  if (d <= kBwdRingMax) per_sm = std::min(per_sm, 204800 / bwd_ring_bytes(d));
  const int64_t g = static_cast<int64_t>(std::min(num_sms, kNormMaxSms)) * std::max(per_sm, 1);
  return static_cast<int>(std::min(g, T));
}

// Up to so many rows one block takes them all and its share is dw (us a call: 1 x 1024 6.8, 2 x 7168
// 7.9, 4 x 3328 6.9 against 9.1-9.5 with a second launch; 4 x 7168 10.2 either way).
constexpr int kBwdSingleRows = 4;

cudaError_t launch_norm_backward(const NormBwdArgs& args, float* dw, int num_sms, cudaStream_t s, int* launches) {
  NormBwdArgs a = args;
  const int threads = bwd_threads(a.d), ring = bwd_ring_bytes(a.d);
  const bool single = a.T <= kBwdSingleRows;
  const int grid = single ? 1 : norm_backward_blocks(a.T, a.d, num_sms);
  if (single) a.part = dw;
  *launches = single ? 1 : 2;
  cudaError_t e = cudaSuccess;
  if (a.d <= kBwdRingMax) {
    if (ring > 40 * 1024)  // (with the static part, more than 48 KB needs leave)
      e = cudaFuncSetAttribute(norm_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kBwdStages * 1024 * 64);
    if (e != cudaSuccess) return e;
    norm_backward_kernel<<<grid, threads, ring, s>>>(a);
  } else if (a.d <= 16384) {
    norm_backward_long_kernel<4><<<grid, threads, 0, s>>>(a);
  } else {
    norm_backward_long_kernel<8><<<grid, threads, 0, s>>>(a);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess || single) return e;
  norm_dw_kernel<<<a.d / 8, 256, 0, s>>>(a.part, grid, a.d, dw);
  return cudaGetLastError();
}

}  // namespace dsmoe
