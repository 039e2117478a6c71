// gemm_q8_sm100.cu -- persistent grouped products of 8-bit rows with 8-bit expert weights on
// the 5th-generation tensor cores (tcgen05 kind::mxf8f6f4, block-scaled), operands staged by
// TMA, scales copied from shared into tensor memory.
//
//   out[r, n] = sum_b 2^(sa[r,b] + sw[n/128,b] - 254) sum_{k in block b} a[r,k] W[e,n,k]
//
// The scales are powers of two, so the tensor core applies them itself (one e8m0 byte per
// 32 values of K; a block of 128 uses the same byte for its four MMAs) and the fp32
// accumulator in tensor memory holds the scaled sum over all of K: no partial sum is ever
// read back to be rescaled. (A gated product with K > 2048 is summed in chains, see q8_chains.)
//
// Orientation as in the bf16 grouped GEMM (gemm_sm100.cu): M = 128 output features per chain,
// N = the tile's tokens rounded up to 16, two chains sharing the token operand (gated: the
// same 128 features of W_gate and W_up; plain: the even and the odd ones of 256 features, so
// that a thread's two accumulators are neighbours in the output row).
//
// One CTA per SM, 352 threads:
//   warp 0      TMA producer: per 128-wide K block two 128 x 128 weight tiles and a
//               kTok x 128 token tile (bytes, 128-byte swizzle) through a ring.
//   warp 1      one thread issues, per four K blocks, the copies of the scales into tensor
//               memory (32x128b.warpx4) and, per K block, 2 x 4 MMAs of K = 32.
//   warps 2-9   epilogue: two groups of four warps take alternate 8-token chunks; warp q of
//               a group reads TMEM lanes [32q, 32q+32) into registers and frees the
//               accumulator. The plain output is stored from there (a warp's pairs of
//               features make one line of a token's row). The gated output's scale is that
//               of 128 features, the lanes of four warps: the group transposes two chunks
//               at a time through shared memory and the maximum is one over a staged row.
//   warp 10     scale loader: a 32-bit word of a row's scales is four K blocks; the words
//               of the tile's tokens and of the two weight tiles go to a ring of slots
//               in the layout that the copy into tensor memory takes.
// Every wait is bounded; a role that gives up raises the abort flag and a status bit, the
// CTA drains its copies and MMAs and returns; the epilogue's groups decide together (through
// shared memory), so that none of their barriers is left waiting. Where a launch has few
// tiles (few rows, few features), the CTAs of a cluster share a tile along K: each sends its
// fp32 partial sums through distributed shared memory to the CTA that owns the token, which
// adds them in the order of K.
//
// What bounds it: with few rows the weights' bytes (48 experts of 7168 x 2048 and 144 rows: 109 us,
// 6.3 TB/s); with many the power limit (gate/up, 8192 rows, 32 experts, d = 7168, F = 2048:
// 300-312 us in a burst, 350-367 repeated, 1.3-1.6 PFLOP/s; 265 and 305 with one chain over K, whose
// sums are coarser) and each drain of a single accumulator (about 6 us of that for one a tile); with a
// short K loop a tile's start and end (32,768 rows, 64 experts, K = 704, N = 1024: 45-47 us, floor 21).
// An MMA of M = 128, K = 32 takes max(64 + 0.14 N, N / 2) cycles, hence the large N.
// The accumulation over K is the tensor core's: fp32, truncating (relative error 4e-7 at
// K = 7168, which a bf16 or fp32 output of the plain product carries).
#include <algorithm>

#include "kernels.h"
#include "q8.cuh"
#include "sm100_pair_ptx.cuh"
#include "sm100_ptx.cuh"

namespace dsmoe {

namespace {

constexpr int kBK = 128;    // K per ring stage: one 128-byte swizzled row, one scale block
constexpr int kFeat = 128;  // features per chain
constexpr int kMmaK = 32;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps + 1);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kWBytes = 2 * kFeat * kBK;
constexpr int kSfSlots = 2;
constexpr uint32_t kSfCols = 16;        // TMEM columns of one set: 4 + 4 (weights), 8 (tokens)
constexpr uint32_t kSfCol0 = kTmemCols - 2 * kSfCols;
constexpr int kChunk = 8;               // tokens per epilogue chunk
constexpr uint32_t kStgBytes = 2 * kChunk * kFeat * 4;

template <int kTok>
struct Geo {
  static constexpr uint32_t kAccCols = 2 * kTok;
  static constexpr int kBufs = 2 * kAccCols <= kSfCol0 ? 2 : 1;
  static constexpr int kAccs = kSfCol0 / kAccCols;  // that tensor memory holds
  static constexpr int kStages = kTok > 112 ? 3 : kTok > 32 ? 4 : 5;
  static constexpr uint32_t kXBytes = kTok * kBK;
  static constexpr uint32_t kBoxRows = q8_box_rows(kTok);
  static constexpr uint32_t kSfBytes = kTok > 128 ? 2048 : 1536;  // weight tiles 2 x 512, tokens 512 or 1024
  static constexpr uint32_t kOffW = 0;
  static constexpr uint32_t kOffX = kOffW + kStages * kWBytes;
  static constexpr uint32_t kOffSf = kOffX + kStages * kXBytes;
  static constexpr uint32_t kOffStg = kOffSf + kSfSlots * kSfBytes;
  static constexpr uint32_t kOffBars = kOffStg + 4 * kStgBytes;  // two groups, two buffers
  static constexpr uint32_t kNumBars = 2 * kStages + 2 * kSfSlots + 4 + 1;
  static constexpr uint32_t kOffMisc = kOffBars + kNumBars * 8;
  static constexpr uint32_t kOffTiles = kOffMisc + 32;
  // the clipped offsets, next to the tile prefix where there is room for them
  static constexpr bool kRowsInSmem = kTok < 240;
  static constexpr uint32_t kOffRows = kOffTiles + (512 + 1) * 4;
  static constexpr uint32_t kSmemUsed = kOffRows + (kRowsInSmem ? (512 + 1) * 4 : 0);
  static constexpr size_t kSmemBytes = kSmemUsed + 1024;  // slack to align the ring to 1024 bytes
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kAccCols <= kSfCol0 && kTok % 16 == 0 && kTok <= 256, "tile geometry");
  static_assert(kXBytes % 1024 == 0 && kTok % kBoxRows == 0 && kBoxRows % 8 == 0,
                "token boxes start on swizzle atoms");
};

// The tensor core truncates as it accumulates, so its error grows with the length of the sum: of
// SwiGLU's values in 8 bits (8192 rows, N = 2048, K = 7168) one chain of MMAs carries 275-332 across
// an e4m3 border and an fp32 sum 98-119 (K = 2048: 64-81 and 46-60); chains of at most 2048 values,
// added in fp32, carry 90-146. A gated sum over `quads` groups of four K blocks takes so many chains;
// chain_end is the K block after chain i's last (kq0, kq1: the CTA's groups, kb1: its end). Their
// lengths differ by at most one group.
constexpr int kChainQuads = 4;
__host__ __device__ __forceinline__ int q8_chains(int quads) { return (quads + kChainQuads - 1) / kChainQuads; }
__device__ __forceinline__ int chain_end(int kq0, int kq1, int chains, int i, int kb1) {
  return min(4 * (kq0 + (i + 1) * (kq1 - kq0) / chains), kb1);
}

// D[tmem] (+)= (A 2^sfa)(B 2^sfb)^T, e4m3 operands, e8m0 scales in tensor memory.
__device__ __forceinline__ void mma_q8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (format codes 0), e8m0 scales (bit
// 23), K-major, byte `id` of each 32-bit word of scales for both operands.
__device__ __forceinline__ uint32_t idesc_q8(int m, int n, uint32_t id) {
  return (id << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) |
         (id << 29);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// 512 bytes of shared memory (32 rows of 16 bytes) into four columns, the same for each
// quarter of the lanes: row i's word j is the scales of operand row i + 32 j.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;         // leading byte offset (one 16-byte column: unused)
  d |= static_cast<uint64_t>(128 >> 4) << 32;  // stride byte offset: next eight rows
  d |= static_cast<uint64_t>(1) << 46;         // descriptor version for sm_100
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// fp32 sums, rounded to nearest.
__device__ __forceinline__ void add8(uint32_t (&a)[8], const uint32_t (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) + __uint_as_float(b[i]));
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int half) {
  asm volatile("bar.sync %0, %1;" ::"r"(half + 1), "r"(128) : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// mbar_wait_bounded that looks at the limit after every poll.
__device__ __forceinline__ bool mbar_wait_checked(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                                  volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag || global_timer_ns() - t0 > limit_ns) return false;
  return true;
}

// mbar_wait_bounded for a converged warp: every lane polls, the decisions are the warp's.
__device__ __forceinline__ bool mbar_wait_converged(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                                    volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 63u) == 0 && __any_sync(0xffffffffu, *abort_flag != 0 || global_timer_ns() - t0 > limit_ns)) return false;
  }
}

struct Q8Tile {
  int expert, row0, m_valid, n_blk;
};

// Offset e, clipped to [0, R]; without offsets all rows are one group's.
__device__ __forceinline__ int clipped_offset(const Q8GemmArgs& a, int e) {
  if (!a.offsets) return e == 0 ? 0 : a.R;
  return min(max(__ldg(a.offsets + e), 0), a.R);
}

// Rows [b, t) of group e. Offsets that decrease count as their running maximum, so that the groups
// are disjoint and a launch has no more tiles than token_tiles allows for. rows: that maximum, or,
// where shared memory has no room for it, whether the offsets decrease at all.
template <int kTok>
__device__ __forceinline__ void group_rows(const Q8GemmArgs& a, const int32_t* rows, int e, int& b, int& t) {
  if (Geo<kTok>::kRowsInSmem) {
    b = rows[e];
    t = rows[e + 1];
  } else {
    b = clipped_offset(a, e);
    t = clipped_offset(a, e + 1);
    if (*rows)
      for (int i = 0; i < e; ++i) b = max(b, clipped_offset(a, i));
    t = max(t, b);
  }
}

template <int kTok>
__device__ __forceinline__ Q8Tile decode_tile(const Q8GemmArgs& a, const int32_t* tile_start, const int32_t* rows,
                                              int tile) {
  int lo = 0, hi = a.E - 1;
  while (lo < hi) {  // last group whose first tile is <= tile
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  int b, e;
  group_rows<kTok>(a, rows, lo, b, e);
  const int M = e - b, mt = (M + kTok - 1) / kTok, local = tile - tile_start[lo], m_blk = local % mt;
  // near-equal token tiles in granules of 16, token tiles fastest: the CTAs that share a
  // weight tile run at the same rate and find it in L2
  const int gr = (M + 15) >> 4, q = gr / mt, rem = gr - q * mt;
  const int g0 = m_blk * q + min(m_blk, rem);
  Q8Tile t;
  t.expert = lo;
  t.n_blk = local / mt;
  t.row0 = b + g0 * 16;
  t.m_valid = min((q + (m_blk < rem ? 1 : 0)) * 16, M - g0 * 16);
  return t;
}

// SiLU(g) u. The approximations that flush subnormals take half the instructions of those that
// do not, and the drain of a gated tile is bound by its instructions; what they flush is
// e^-g next to 1, and 1 / (1 + e^-g) below 2^-126 (g < -87, where |SiLU| < 1.1e-36 becomes 0).
__device__ __forceinline__ float swiglu(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

// The warp stores a block of 128 gated outputs in 8 bits for the first n of kRows rows in a row,
// four features per lane, and their scales (the last block of a row also the row's padding
// scales). The rows are worked on side by side: their maxima are reduced back to back.
template <int kRows>
__device__ __forceinline__ void store_gated_rows(const Q8GemmArgs& a, int64_t row, int n, int blk, int lane,
                                                 const float4 (&m)[kRows]) {
  const int So = q8_scale_cols(a.N), nb = (a.N + kFeat - 1) / kFeat, f = blk * kFeat + 4 * lane;
  uint32_t s[kRows], mine = 0;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    s[r] = __reduce_max_sync(0xffffffffu, max(max(abs_bits(m[r].x), abs_bits(m[r].y)),
                                              max(abs_bits(m[r].z), abs_bits(m[r].w))));
  uint8_t* q = a.q_out + row * a.N + f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    s[r] = q8_scale_byte(s[r]);
    if (lane == r) mine = s[r];
    const float k = q8_inv_scale(s[r]);
    const uint32_t v = s[r] == 255u ? 0x7F7F7F7Fu : q8_pack4(m[r].x * k, m[r].y * k, m[r].z * k, m[r].w * k);
    if (r < n && f < a.N) *reinterpret_cast<uint32_t*>(q + static_cast<int64_t>(r) * a.N) = v;
  }
  uint8_t* scales = a.q_scales + row * So;
  if (lane < n) scales[lane * So + blk] = static_cast<uint8_t>(mine);
  if (blk == nb - 1 && lane < So - nb)
    for (int r = 0; r < n; ++r) scales[r * So + nb + lane] = kQ8PadScale;
}

// Four fp32 outputs at `at`: added to the bf16 rows given, or to what is there.
__device__ __forceinline__ void add_f32(const Q8GemmArgs& a, int64_t at, float4 o) {
  if (a.add_bf16) {
    const uint2 x = *reinterpret_cast<const uint2*>(a.add_bf16 + at);
    const float2 x0 = unpack_bf16x2(x.x), x1 = unpack_bf16x2(x.y);
    o.x += x0.x, o.y += x0.y, o.z += x1.x, o.w += x1.y;
  } else {
    const float4 x = *reinterpret_cast<const float4*>(a.out_f32 + at);
    o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
  }
  *reinterpret_cast<float4*>(a.out_f32 + at) = o;
}

// kLong (gated): K is accumulated in several chains (q8_chains), which the epilogue adds in fp32,
// rounded to nearest, while the next one runs (160-token tiles have one accumulator: after it).
template <int kOut, int kTok, bool kSplit, bool kLong>
__global__ void __launch_bounds__(kThreads, 1) gemm_q8_kernel(const __grid_constant__ Q8GemmArgs a) {
  using G_ = Geo<kTok>;
  constexpr bool kGated = kOut == kQ8Gated;
  constexpr int kTileFeat = kGated ? kFeat : 2 * kFeat;  // output features of a tile
  constexpr int kHold = (kTok / kChunk + 1) / 2;         // chunks of an epilogue group
  constexpr int kRegChunks = kTok > 112 ? 6 : kHold;     // of them (kLong) with their sums in registers
  static_assert(kOut != kQ8F32 || G_::kBufs == 2, "the fp32 output leaves the accumulators late");
  static_assert(!kLong || (kGated && !kSplit), "chains are joined by the epilogue of one CTA");
  static_assert(!kLong || G_::kBufs * G_::kAccCols + 4 * kChunk * (kHold - kRegChunks) <= kSfCol0, "sums of chains");
  static_assert(!kSplit || (kTok % 8 == 0 && kTok * 2 * kFeat * 4 <= G_::kOffSf), "the ring holds the partial sums");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* base = smem_raw + pad;
  uint8_t* sW = base + G_::kOffW;
  uint8_t* sX = base + G_::kOffX;
  uint8_t* sSf = base + G_::kOffSf;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + G_::kOffBars);
  uint64_t* empty = full + G_::kStages;
  uint64_t* sf_full = empty + G_::kStages;
  uint64_t* sf_empty = sf_full + kSfSlots;
  uint64_t* acc_full = sf_empty + kSfSlots;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + G_::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + G_::kOffMisc + 4);
  volatile int* never_flag = reinterpret_cast<volatile int*>(base + G_::kOffMisc + 8);
  volatile int* group_ok = reinterpret_cast<volatile int*>(base + G_::kOffMisc + 16);  // [epilogue group][tile parity]
  int32_t* tile_start = reinterpret_cast<int32_t*>(base + G_::kOffTiles);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_tiles = (a.N + kTileFeat - 1) / kTileFeat;
  const int kb_all = (a.K + kBK - 1) / kBK, kq_all = (kb_all + 3) >> 2;
  // kSplit: the CTAs of a cluster share one tile, each a range of K in whole groups of four blocks
  const int splits = kSplit ? a.splits : 1, rank = kSplit ? static_cast<int>(pair::cta_rank()) : 0;
  const int kq0 = kSplit ? rank * kq_all / splits : 0, kq1 = kSplit ? (rank + 1) * kq_all / splits : kq_all;
  const int kb0 = 4 * kq0, kb1 = kSplit ? min(4 * kq1, kb_all) : kb_all;
  // chains of this CTA: in a cluster each stays in its accumulator until the join
  const int chains = kLong ? q8_chains(kq_all) : kSplit && kGated ? min(q8_chains(kq1 - kq0), G_::kAccs) : 1;
  const int tile0 = kSplit ? blockIdx.x / splits : blockIdx.x, tile_step = kSplit ? gridDim.x / splits : gridDim.x;

  int32_t* group_begin = reinterpret_cast<int32_t*>(base + (G_::kRowsInSmem ? G_::kOffRows : G_::kOffMisc + 12));
  bool decreases = false;
  for (int e = threadIdx.x; e <= a.E; e += kThreads) {
    const int at = clipped_offset(a, e);
    decreases |= e < a.E && clipped_offset(a, e + 1) < at;
    if (G_::kRowsInSmem) group_begin[e] = at;
  }
  if (threadIdx.x == kThreads - 1) {
    tma_prefetch_desc(&a.map_a);
    tma_prefetch_desc(&a.map_w0);
    if (kGated) tma_prefetch_desc(&a.map_w1);
  }
  if (threadIdx.x == 0) {
    tile_start[0] = 0;
    *abort_flag = 0;
    *never_flag = 0;
    for (int s = 0; s < G_::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], 32);
      mbar_init(&sf_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (__syncthreads_or(decreases)) {  // rare: the running maximum, or the mark that there is one to take
    if (!G_::kRowsInSmem) *group_begin = 1;
    else if (threadIdx.x == 0)
      for (int e = 1; e <= a.E; ++e) group_begin[e] = max(group_begin[e], group_begin[e - 1]);
    __syncthreads();
  } else if (!G_::kRowsInSmem) {
    *group_begin = 0;
  }
  if (warp == 0) {  // tile_start[1..E]: the groups' tiles and their inclusive prefix
    __syncwarp();
    int carry = 0;
    for (int b0 = 0; b0 < a.E; b0 += 32) {
      const int e = b0 + lane;
      int v = 0;
      if (e < a.E) {
        int b, t;
        group_rows<kTok>(a, group_begin, e, b, t);
        v = ((t - b + kTok - 1) / kTok) * n_tiles;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
      }
      if (e < a.E) tile_start[e + 1] = v + carry;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (kSplit) pair::cluster_sync();  // every CTA of the cluster is there to be written to
  const uint32_t tmem_base = *tmem_slot;
  const int total = tile_start[a.E];

  uint32_t issued_mask = 0, issued_parity = 0;  // producer bookkeeping for the abort drain

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------------ TMA producer
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < total; tile += tile_step) {
        const Q8Tile t = decode_tile<kTok>(a, tile_start, group_begin, tile);
        const int n0 = t.n_blk * kTileFeat;
        // only the boxes that hold rows of the tile (a full tile's bytes every time: 342 us for
        // the large gate/up, 329 so)
        const int boxes = (t.m_valid + G_::kBoxRows - 1) / G_::kBoxRows;
        const uint32_t stage_bytes = kWBytes + boxes * G_::kBoxRows * kBK;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, a.wait_limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], stage_bytes);
          uint8_t* w = sW + stage * kWBytes;
          if (kGated) {  // the same 128 rows of W_gate and W_up
            tma_load_3d(w, &a.map_w0, &full[stage], kb * kBK, n0, t.expert);
            tma_load_3d(w + kWBytes / 2, &a.map_w1, &full[stage], kb * kBK, n0, t.expert);
          } else {  // the even and the odd rows of 256
            tma_load_4d(w, &a.map_w0, &full[stage], kb * kBK, 0, n0 >> 1, t.expert);
            tma_load_4d(w + kWBytes / 2, &a.map_w0, &full[stage], kb * kBK, 1, n0 >> 1, t.expert);
          }
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(sX + stage * G_::kXBytes + i * G_::kBoxRows * kBK, &a.map_a, &full[stage], kb * kBK,
                        t.row0 + i * static_cast<int>(G_::kBoxRows));
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == G_::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(a.status, kStatusTimeoutProducer);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------------- MMA issuer
    // The whole warp walks the loop and one elected lane issues, so that the descriptors stay
    // in uniform registers: issued from a branch on the lane number, eight MMAs took
    // 950 cycles whatever their N (N = 128 needs 512).
    int stage = 0;
    uint32_t phase = 0;
    uint32_t quad = 0;  // groups of four K blocks so far
    bool ok = true;
    int it = 0;
    for (int tile = tile0; ok && tile < total; tile += tile_step, ++it) {
      const Q8Tile t = decode_tile<kTok>(a, tile_start, group_begin, tile);
      const int n_mma = (t.m_valid + 15) & ~15;
      const uint32_t idesc = idesc_q8(kFeat, n_mma, 0);
      int acc = it % G_::kBufs, chain = 0, first = kb0;
      if (!mbar_wait_converged(&acc_empty[acc], ((it / G_::kBufs) & 1) ^ 1u, a.wait_limit_ns, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t d0 = tmem_base + acc * G_::kAccCols;
      int last = kLong || kSplit ? chain_end(kq0, kq1, chains, 0, kb1) - 1 : kb1 - 1;  // of this chain
      uint32_t sf = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t id = kb & 3;
        if ((kLong || kSplit) && kb > last) {  // the next chain
          first = kb;
          last = chain_end(kq0, kq1, chains, ++chain, kb1) - 1;
          if (kLong) {
            ++it;
            acc = it % G_::kBufs;
            if (!mbar_wait_converged(&acc_empty[acc], ((it / G_::kBufs) & 1) ^ 1u, a.wait_limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            d0 = tmem_base + acc * G_::kAccCols;
          } else {
            d0 += G_::kAccCols;
          }
        }
        if (id == 0) {
          // the columns of this set were last read by the MMAs of two groups ago
          const uint32_t slot = quad % kSfSlots;
          if ((quad >= 2 && !mbar_wait_converged(&sf_empty[(quad - 2) % kSfSlots], ((quad - 2) / kSfSlots) & 1u,
                                                 a.wait_limit_ns, abort_flag)) ||
              !mbar_wait_converged(&sf_full[slot], (quad / kSfSlots) & 1u, a.wait_limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          sf = tmem_base + kSfCol0 + (quad & 1u) * kSfCols;
          const uint32_t s0 = smem_addr(sSf + slot * G_::kSfBytes);
          if (elect_one()) {
            tmem_copy_scales(sf, s0);
            if (kGated) tmem_copy_scales(sf + 4, s0 + 512);
            tmem_copy_scales(sf + 8, s0 + 1024);
            if (n_mma > 128) tmem_copy_scales(sf + 12, s0 + 1536);
          }
          __syncwarp();
        }
        if (!mbar_wait_converged(&full[stage], phase, a.wait_limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t w0 = smem_desc_kmajor_sw128(smem_addr(sW + stage * kWBytes));
        const uint64_t w1 = smem_desc_kmajor_sw128(smem_addr(sW + stage * kWBytes + kWBytes / 2));
        const uint64_t xd = smem_desc_kmajor_sw128(smem_addr(sX + stage * G_::kXBytes));
        const uint32_t di = idesc | (id << 4) | (id << 29);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBK / kMmaK; ++k) {
            const uint64_t dk = static_cast<uint64_t>(2 * k);
            const uint32_t accum = (kb > first || k) ? 1u : 0u;
            mma_q8_ss(d0, w0 + dk, xd + dk, di, sf, sf + 8, accum);
            mma_q8_ss(d0 + kTok, w1 + dk, xd + dk, di, kGated ? sf + 4 : sf, sf + 8, accum);
          }
          mma_commit(&empty[stage]);
          if (id == 3 || kb == kb1 - 1) mma_commit(&sf_empty[quad % kSfSlots]);
          if (kb == (kLong ? last : kb1 - 1)) mma_commit(&acc_full[acc]);
        }
        __syncwarp();
        if (id == 3 || kb == kb1 - 1) ++quad;
        if (++stage == G_::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(a.status, kStatusTimeoutMma);
    }
  } else if (warp == 2 + kEpiWarps) {
    // -------------------------------------------------------------------- scale loader
    const int S4 = q8_scale_cols(a.K) >> 2, nnb = (a.N + kFeat - 1) / kFeat;
    const uint32_t* as = reinterpret_cast<const uint32_t*>(a.a_scales);
    const uint32_t* ws0 = reinterpret_cast<const uint32_t*>(a.W_scales);
    const uint32_t* ws1 = reinterpret_cast<const uint32_t*>(kGated ? a.W1_scales : a.W_scales);
    constexpr uint32_t kOnes = 0x7F7F7F7Fu;
    constexpr int kWords = (kTok + 31) / 32;
    uint32_t quad = 0;
    bool ok = true;
    for (int tile = tile0; ok && tile < total; tile += tile_step) {
      const Q8Tile t = decode_tile<kTok>(a, tile_start, group_begin, tile);
      const int nb0 = kGated ? t.n_blk : 2 * t.n_blk, nb1 = kGated ? nb0 : nb0 + 1;
      const uint32_t* p0 = ws0 + (static_cast<int64_t>(t.expert) * nnb + nb0) * S4;
      const uint32_t* p1 = ws1 + (static_cast<int64_t>(t.expert) * nnb + nb1) * S4;
      uint32_t w[8], g0, g1;
      auto load = [&](int kq) {
        g0 = __ldg(p0 + kq);
        g1 = nb1 < nnb ? __ldg(p1 + kq) : kOnes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = kOnes;
          if (i < kWords && 32 * i + lane < t.m_valid)
            w[i] = __ldg(as + static_cast<int64_t>(t.row0 + 32 * i + lane) * S4 + kq);
        }
      };
      load(kq0);
      for (int kq = kq0; kq < kq1; ++kq, ++quad) {
        const uint32_t slot = quad % kSfSlots;
        if (!mbar_wait_warp(&sf_empty[slot], ((quad / kSfSlots) & 1u) ^ 1u, a.wait_limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        uint4* dst = reinterpret_cast<uint4*>(sSf + slot * G_::kSfBytes) + lane;
        if (kGated) {
          dst[0] = make_uint4(g0, g0, g0, g0);
          dst[32] = make_uint4(g1, g1, g1, g1);
        } else {  // both chains: rows 0-63 are of the first block of 128 features, 64-127 of the second
          dst[0] = make_uint4(g0, g0, g1, g1);
        }
        dst[64] = make_uint4(w[0], w[1], w[2], w[3]);
        if (kTok > 128) dst[96] = make_uint4(w[4], w[5], w[6], w[7]);
        fence_proxy_async();
        mbar_arrive(&sf_full[slot]);
        if (kq + 1 < kq1) load(kq + 1);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(a.status, kStatusTimeoutProducer);
    }
  } else {
    // -------------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;
    const bool leader = ((warp - 2) & 3) == 0 && lane == 0;
    uint8_t* stg = base + G_::kOffStg + half * 2 * kStgBytes;
    uint32_t buf = 0;  // staging buffer of the next chunk
    const int w4 = (warp - 2) & 3;  // this warp's rows of a staged chunk: 4 w4 .. 4 w4 + 3
    int it = 0;
    // the accumulator of turn `it` is complete: the same answer for the whole group (its warps are
    // at most one turn apart)
    auto filled = [&]() -> bool {
      const int acc = it % G_::kBufs;
      if (leader) {
        const bool ok = mbar_wait_checked(&acc_full[acc], (it / G_::kBufs) & 1, a.wait_limit_ns, abort_flag);
        group_ok[2 * half + (it & 1)] = ok;
        if (!ok) {
          *abort_flag = 1;
          atomicOr(a.status, kStatusTimeoutEpilogue);
        }
      }
      group_sync(half);
      if (!group_ok[2 * half + (it & 1)]) return false;
      (void)mbar_try_wait(&acc_full[acc], (it / G_::kBufs) & 1);
      tc_fence_after();
      return true;
    };
    for (int tile = tile0; tile < total; tile += tile_step, ++it) {
      const Q8Tile t = decode_tile<kTok>(a, tile_start, group_begin, tile);
      if (!filled()) break;
      const int acc = it % G_::kBufs;
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * G_::kAccCols;
      const int n_chunks = (t.m_valid + kChunk - 1) / kChunk;
      const int n0 = t.n_blk * kTileFeat;
      if constexpr (kSplit) {
        break;  // a cluster has one tile, joined below
      } else if constexpr (kOut == kQ8F32) {
        // A thread's two accumulators are neighbours in the output row: a warp's words of a token
        // make one line, stored as they come. What is added is on its way before the
        // accumulators are read.
        const int f = n0 + 2 * (q * 32 + lane);
        const bool on = f < a.N;
#pragma unroll 1
        for (int c = half; c < n_chunks; c += 2) {
          const int n = on ? t.m_valid - kChunk * c : 0;  // tokens of the chunk
          const int64_t at = static_cast<int64_t>(t.row0 + kChunk * c) * a.N + f;
          float2 add[kChunk];
#pragma unroll
          for (int j = 0; j < kChunk; ++j) {
            add[j] = make_float2(0.f, 0.f);
            if (j < n)
              add[j] = a.add_bf16 ? unpack_bf16x2(*reinterpret_cast<const uint32_t*>(a.add_bf16 + at +
                                                                                   static_cast<int64_t>(j) * a.N))
                                  : *reinterpret_cast<const float2*>(a.out_f32 + at + static_cast<int64_t>(j) * a.N);
          }
          uint32_t v0[kChunk], v1[kChunk];
          tmem_ld8(tb + kChunk * c, v0);
          tmem_ld8(tb + kTok + kChunk * c, v1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
            if (j < n)
              *reinterpret_cast<float2*>(a.out_f32 + at + static_cast<int64_t>(j) * a.N) =
                  make_float2(add[j].x + __uint_as_float(v0[j]), add[j].y + __uint_as_float(v1[j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
      } else {
        // First the accumulators move to registers (gated: through SwiGLU; plain: both chains
        // rounded into one register), so that the next tile's MMAs may overwrite them ...
        uint32_t hold[kHold][kChunk], v0[2][kChunk], v1[2][kChunk];
        if constexpr (kLong) {
          // ... with the sums of the chains before the last: those of the group's first kRegChunks
          // chunks in registers, of the others in the columns that the accumulators leave
          uint32_t u[kRegChunks][kChunk];
#pragma unroll
          for (int i = 0; i < kRegChunks; ++i)
#pragma unroll
            for (int j = 0; j < kChunk; ++j) hold[i][j] = u[i][j] = 0;
          const uint32_t spare = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + G_::kBufs * G_::kAccCols +
                                 half * (kHold - kRegChunks) * 2 * kChunk;
          uint32_t from = tb;
          bool ok = true;
#pragma unroll 1
          for (int chain = 0; chain + 1 < chains; ++chain) {
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
              if (2 * i + half >= n_chunks) break;
              const uint32_t at = from + kChunk * (2 * i + half), kept = spare + (i - kRegChunks) * 2 * kChunk;
              if (i < kRegChunks) {
                tmem_ld8(at, v0[0]);
                tmem_ld8(at + kTok, v1[0]);
                tmem_wait_ld();
                add8(hold[i], v0[0]);
                add8(u[i < kRegChunks ? i : 0], v1[0]);
              } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  tmem_ld8(at + k * kTok, v0[0]);
                  if (chain > 0) tmem_ld8(kept + k * kChunk, v1[0]);
                  tmem_wait_ld();
                  if (chain > 0) add8(v0[0], v1[0]);
                  tmem_st8(kept + k * kChunk, v0[0]);
                }
              }
            }
            if (kHold > kRegChunks) tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[it % G_::kBufs]);
            ++it;
            ok = filled();
            if (!ok) break;
            from = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + it % G_::kBufs * G_::kAccCols;
          }
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kHold; ++i) {
            if (2 * i + half >= n_chunks) break;
            const uint32_t at = from + kChunk * (2 * i + half), kept = spare + (i - kRegChunks) * 2 * kChunk;
            tmem_ld8(at, v0[0]);
            if (i >= kRegChunks) tmem_ld8(kept, hold[i]);
            tmem_ld8(at + kTok, v1[0]);
            if (i >= kRegChunks) tmem_ld8(kept + kChunk, u[0]);
            tmem_wait_ld();
            add8(hold[i], v0[0]);
            add8(v1[0], u[i < kRegChunks ? i : 0]);
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
              hold[i][j] = __float_as_uint(swiglu(__uint_as_float(hold[i][j]), __uint_as_float(v1[0][j])));
          }
        } else {
#pragma unroll
          for (int i = 0; i < kHold; i += 2) {  // two chunks at a time
            if (2 * i + half >= n_chunks) break;
            const uint32_t at = tb + kChunk * (2 * i + half);
            tmem_ld8(at, v0[0]);
            tmem_ld8(at + kTok, v1[0]);
            if (i + 1 < kHold) {  // (columns past the tile's tokens hold what nothing reads)
              tmem_ld8(at + 2 * kChunk, v0[1]);
              tmem_ld8(at + 2 * kChunk + kTok, v1[1]);
            }
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 2 * kChunk; ++j) {
              const int s = j >= kChunk ? 1 : 0;
              if (i + s >= kHold) break;
              const float x = __uint_as_float(v0[s][j & 7]), y = __uint_as_float(v1[s][j & 7]);
              hold[i + s][j & 7] = kGated ? __float_as_uint(swiglu(x, y)) : pack_bf16x2(x, y);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[it % G_::kBufs]);
        if constexpr (!kGated) {
          // ... then they are stored: a thread's two are neighbours in the output row, and a
          // warp's words of a token make one line
          const int f = n0 + 2 * (q * 32 + lane);
          const int n = f < a.N ? t.m_valid : 0;
          bf16* out = a.out + static_cast<int64_t>(t.row0) * a.N + f;
#pragma unroll
          for (int i = 0; i < kHold; ++i) {
            const int tok = kChunk * (2 * i + half);
            if (tok >= t.m_valid) break;
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
              if (tok + j < n) *reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(tok + j) * a.N) = hold[i][j];
          }
        } else {
          // ... then two chunks at a time are transposed through shared memory (a scale is that of
          // 128 features, four warps' lanes) and leave row by row, four rows per warp
#pragma unroll
          for (int i = 0; i < kHold; i += 2) {
            if (2 * i + half >= n_chunks) break;
            uint32_t* st = reinterpret_cast<uint32_t*>(stg + buf * kStgBytes);
#pragma unroll
            for (int j = 0; j < 2 * kChunk; ++j) {
              const int ii = i + (j >= kChunk ? 1 : 0);
              if (ii >= kHold) break;
              st[j * kFeat + q * 32 + lane] = hold[ii][j & 7];
            }
            group_sync(half);
            // this warp's four rows of the sixteen, neighbours in the output
            const int j0 = 4 * w4, tok = kChunk * (2 * (i + (j0 >= kChunk ? 1 : 0)) + half) + (j0 & (kChunk - 1));
            float4 m[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) m[r] = reinterpret_cast<const float4*>(st)[(j0 + r) * (kFeat / 4) + lane];
            if (tok < t.m_valid)
              store_gated_rows<4>(a, t.row0 + tok, min(t.m_valid - tok, 4), t.n_blk, lane, m);
            buf ^= 1u;
          }
        }
      }
    }
  }

  __syncthreads();
  if (*abort_flag) {
    // let every copy and MMA this CTA started finish before its memory is released
    if (warp == 0 && lane == 0) {
      for (int s = 0; s < G_::kStages; ++s)
        if ((issued_mask >> s) & 1u)
          if (!mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, drain_wait_limit(a.wait_limit_ns), never_flag))
            atomicOr(a.status, kStatusTimeoutDrain);
    }
    if (warp == 1) {  // by the lane that issued them: the same one is elected every time
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      if (!mbar_wait_converged(drain, 0, drain_wait_limit(a.wait_limit_ns), never_flag) && lane == 0)
        atomicOr(a.status, kStatusTimeoutDrain);
    }
  }
  if constexpr (kSplit) {
    // The partial sums of token t go to CTA t % splits, slot t / splits, to the place
    // [source CTA][slot][chain][feature] of its ring, which nothing uses any more once every
    // CTA of the cluster is here.
    __syncthreads();
    pair::cluster_sync();
    const bool epilogue = warp >= 2 && warp < 2 + kEpiWarps && tile0 < total;
    if (epilogue && !*abort_flag) {
      const Q8Tile t = decode_tile<kTok>(a, tile_start, group_begin, tile0);
      tc_fence_after();
      const int q = warp & 3;
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = (warp - 2) >> 2; kChunk * c < t.m_valid; c += 2) {
        uint32_t p0[kChunk], p1[kChunk];
        tmem_ld8(tb + kChunk * c, p0);
        tmem_ld8(tb + kTok + kChunk * c, p1);
        tmem_wait_ld();
        for (int chain = 1; chain < chains; ++chain) {
          uint32_t v0[kChunk], v1[kChunk];
          tmem_ld8(tb + chain * G_::kAccCols + kChunk * c, v0);
          tmem_ld8(tb + chain * G_::kAccCols + kTok + kChunk * c, v1);
          tmem_wait_ld();
          add8(p0, v0);
          add8(p1, v1);
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          const int tok = kChunk * c + j;
          if (tok >= t.m_valid) break;
          const uint32_t at =
              smem_addr(base) + ((rank * (kTok / splits) + tok / splits) * 2 * kFeat + q * 32 + lane) * 4;
          const uint32_t to = pair::map_to(at, tok % splits);
          pair::st_cluster_u32(to, p0[j]);
          pair::st_cluster_u32(to + kFeat * 4, p1[j]);
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
  if constexpr (kSplit) {
    __syncwarp();
    pair::cluster_sync();  // the partial sums have arrived
    if (tile0 >= total || warp < 2 || warp >= 2 + kEpiWarps) return;
    const Q8Tile t = decode_tile<kTok>(a, tile_start, group_begin, tile0);
    const int slots = kTok / splits;
    for (int slot = warp - 2; slot * splits + rank < t.m_valid; slot += kEpiWarps) {
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
      for (int s = 0; s < splits; ++s) {  // in the order of K
        const float4* p = reinterpret_cast<const float4*>(base) + (s * slots + slot) * (kFeat / 2) + lane;
        const float4 x = p[0], y = p[kFeat / 4];
        g.x += x.x, g.y += x.y, g.z += x.z, g.w += x.w;
        u.x += y.x, u.y += y.y, u.z += y.z, u.w += y.w;
      }
      const int64_t row = t.row0 + slot * splits + rank;
      const int n0 = t.n_blk * kTileFeat;
      if (kGated) {
        const float4 m[1] = {
            make_float4(swiglu(g.x, u.x), swiglu(g.y, u.y), swiglu(g.z, u.z), swiglu(g.w, u.w))};
        store_gated_rows<1>(a, row, 1, t.n_blk, lane, m);
      } else if (n0 + 8 * lane < a.N) {
        const int64_t at = row * a.N + n0 + 8 * lane;
        if (kOut == kQ8Bf16) {
          *reinterpret_cast<uint4*>(a.out + at) = make_uint4(pack_bf16x2(g.x, u.x), pack_bf16x2(g.y, u.y),
                                                             pack_bf16x2(g.z, u.z), pack_bf16x2(g.w, u.w));
        } else {
          add_f32(a, at, make_float4(g.x, u.x, g.y, u.y));
          add_f32(a, at + 4, make_float4(g.z, u.z, g.w, u.w));
        }
      }
    }
  }
}

template <int kOut, int kTok, bool kSplit, bool kLong>
cudaError_t launch_one(const Q8GemmArgs& a, int grid, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(gemm_q8_kernel<kOut, kTok, kSplit, kLong>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Geo<kTok>::kSmemBytes));
  if (e != cudaSuccess) return e;
  if (!kSplit) {
    gemm_q8_kernel<kOut, kTok, kSplit, kLong><<<grid, kThreads, Geo<kTok>::kSmemBytes, s>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = a.splits;
  cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Geo<kTok>::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_q8_kernel<kOut, kTok, kSplit, kLong>, a);
}

template <int kOut>
cudaError_t launch_tok(const Q8GemmArgs& a, const Q8Tiling& t, cudaStream_t s) {
  const int tok = t.tok, grid = t.grid;
  if (t.splits > 1)
    return tok == 32 ? launch_one<kOut, 32, true, false>(a, grid, s) : launch_one<kOut, 112, true, false>(a, grid, s);
  if constexpr (kOut == kQ8Gated)
    if (t.chains > 1)
      return tok == 32    ? launch_one<kOut, 32, false, true>(a, grid, s)
             : tok == 112 ? launch_one<kOut, 112, false, true>(a, grid, s)
                          : launch_one<kOut, 160, false, true>(a, grid, s);
  if (tok == 32) return launch_one<kOut, 32, false, false>(a, grid, s);
  if constexpr (kOut != kQ8F32)
    if (tok == 240) return launch_one<kOut, 240, false, false>(a, grid, s);
  return launch_one<kOut, 112, false, false>(a, grid, s);
}

// Tiles of `tok` rows that R rows in E groups make at most.
int64_t token_tiles(int64_t R, int E, int tok) { return (R + (tok - 1) * std::min<int64_t>(E, R)) / tok; }

// Token tile by rows per group g, measured over K = 256 .. 7168 on 32 groups (us, N = 2048
// unless said):
//   32   g <= 16 (plain, K = 7168, g = 8: 76.7 against 78.2 with 112; g = 24: 96 against 80), and
//        where even its tiles are no more than one per SM, each then the shorter (64 groups of
//        56 rows, N = 128, K = 256, gated, in a graph: 6.1 against 7.8).
//   240  one accumulator, so that the start of a tile's epilogue is exposed, but an MMA at
//        N = 240 costs 0.5 cycles a token and at N = 112 0.75: from g = 100 on where the K loop is
//        long enough to bury that start. Gated, 1024 <= K <= 2048 (K = 1024, g = 512: 87 against 99;
//        K = 2048, g = 120: 62.8 against 67.5; K = 704, g = 300: 61 against 57 the other way).
//        Plain, whose 112-token tiles run two accumulators over a cheaper epilogue, K >= 4096
//        (K = 7168, g = 100: 98.8 against 107), or g >= 240 with g K >= 350,000 (K = 1280,
//        g = 512: 53.8 against 61.1; K = 2048, g = 200: 45.4 against 43.3 and K = 448, g = 512:
//        35.2 against 33.4 the other way).
//   160  gated, K > 2048, from g = 110 on: the sums of two chains and more have to be kept, and those
//        of 240 tokens have no place in registers and tensor memory (of 160: 6 of a group's 10 chunks
//        in registers). K = 7168, g = 120: 187 against 223 with 112, g = 256: 315 against 343, g = 100:
//        176 against 166 the other way.
//   112  the rest, and in place of 32 where its clusters (q8_splits) shorten a CTA's K loop by 14
//        blocks or more (in a graph: 128 rows, gated, K = 7168: 17.2 against 19.9; 256 rows: 25.6
//        against 30.3; 4 groups of 169 rows, N = 600, K = 3968: 14.1 against 16.5; less than 14, 5 groups
//        of 184 rows, N = 512, K = 3280, gated: 21.4 against 16.9 the other way).
// Of an expert range (E of E_all groups) g and the tiles are those of the range's share of the rows.
int q8_splits(int64_t tiles, int tok, int K, bool gated, int num_sms);
int q8_token_tile(int64_t R, int E, int E_all, int N, int K, bool gated, int num_sms) {
  const int64_t n_tiles = gated ? (N + 127) / 128 : (N + 255) / 256, g = R / E_all;
  if (g <= 16) return 32;
  if (std::max<int64_t>(E, (R * E / E_all + 31) / 32) * n_tiles <= num_sms) {
    const int kb = (K + kBK - 1) / kBK;
    const int s32 = q8_splits(token_tiles(R, E, 32) * n_tiles, 32, K, gated, num_sms);
    const int s112 = q8_splits(token_tiles(R, E, 112) * n_tiles, 112, K, gated, num_sms);
    return kb / s32 - kb / s112 >= 14 ? 112 : 32;
  }
  if (gated && q8_chains((K + 511) / 512) > 1) return g >= 110 ? 160 : 112;
  const bool large = gated ? g >= 100 && K >= 1024 : (g >= 100 && K >= 4096) || (g >= 240 && g * K >= 350000);
  return large ? 240 : 112;
}

// CTAs that share a tile along K: the most of 8, 4, 2 whose clusters run side by side (of 148 SMs,
// 15 clusters of 8 CTAs, 33 of 4, 74 of 2) and that leave each CTA a group of four K blocks.
// One row, N = 128, K = 7168, gated, in a graph: 27.2 us alone, 16.2, 11.6 and 8.6 with 2, 4 and 8; 16
// tiles: 28.6, 18.5, 14.1 and 20.4 (the 16th cluster of 8 runs afterwards). Joining the sums of a
// 112-token tile takes longer, so there the K loop has to get 14 blocks shorter; two chains of a gated
// sum are what tensor memory holds of it (of 32 tokens seven, which any K can do with).
int q8_splits(int64_t tiles, int tok, int K, bool gated, int num_sms) {
  const int groups = (K + 511) / 512, kb = (K + kBK - 1) / kBK;
  if (tok > 112) return 1;
  for (int s = 8; s > 1; s >>= 1) {
    const int idle = s == 8 ? 28 : s == 4 ? 16 : 0;
    if (tiles * s <= num_sms - idle && groups >= s)
      return tok == 32 || (kb - kb / s >= 14 && (!gated || q8_chains((groups + s - 1) / s) <= 2)) ? s : 1;
  }
  return 1;
}

}  // namespace

Q8Tiling q8_tiling(int64_t R, int E, int E_all, int N, int K, int out, int num_sms) {
  const bool gated = out == kQ8Gated;
  const int64_t n_tiles = (N + (gated ? 127 : 255)) / (gated ? 128 : 256);
  Q8Tiling t;
  t.tok = q8_token_tile(R, E, E_all, N, K, gated, num_sms);
  if (out == kQ8F32) t.tok = std::min(t.tok, 112);  // its accumulators are read late: two of them
  const int64_t bound = token_tiles(R, E, t.tok) * n_tiles;
  t.splits = q8_splits(bound, t.tok, K, gated, num_sms);
  t.grid = static_cast<int>(t.splits > 1 ? bound * t.splits : std::min<int64_t>(bound, num_sms));
  t.chains = gated ? q8_chains(((K + 511) / 512 + t.splits - 1) / t.splits) : 1;
  if (t.splits > 1) t.chains = std::min(t.chains, t.tok == 32 ? Geo<32>::kAccs : Geo<112>::kAccs);
  return t;
}

cudaError_t launch_gemm_q8(const Q8GemmArgs& args, const Q8Tiling& t, cudaStream_t s) {
  Q8GemmArgs a = args;
  a.splits = t.splits;
  if (a.q_out) return launch_tok<kQ8Gated>(a, t, s);
  return a.out_f32 ? launch_tok<kQ8F32>(a, t, s) : launch_tok<kQ8Bf16>(a, t, s);
}

}  // namespace dsmoe
