// lily_mx4_linear: the product of 4-bit weights with 8- or 4-bit rows, both in blocks of 32 along K that
// share a power of two:
//   out[t][n] = sum over blocks of 2^(sw + sx - 254) * sum_k w[n][k] x[t][k]
//
// The tensor cores take this form as it is: tcgen05.mma kind::mxf8f6f4 (e2m1 weights, e4m3 rows, 32 of K an
// instruction) and kind::mxf4 (e2m1 both, 64 of K) multiply elements exactly, apply both scales to the product of
// a block and sum in fp32.  Weights are always the 128 rows of the M side and tokens the N side, NT of them
// (16 to 192, by the call): a single token then costs no more than its weights' bytes, which bound small
// calls, and large ones are bound by the tensor cores.
//
// One block an SM walks output tiles of 128 x NT.  Its warps: one that copies codes by TMA (128-byte rows of K,
// 128-byte swizzle: 128 elements of 8 bits, where 4-bit weights are spread to 16 elements in 16 bytes by the
// copy, or 256 elements of 4 bits), two that copy scales, one that issues the products, eight that write
// results from tensor memory, while the next tile's products run into the other half of it.  The scales of 128 rows
// and 128 elements of K are 512 bytes, row r's four at (r % 32) * 16 + (r / 32) * 4, and go to four columns of
// tensor memory ahead of the products that use them; tcgen05.cp and tcgen05.mma run in the order of their issue.
//
// Where there are tiles for two fifths of the SMs at most, a cluster of up to 8 blocks shares a tile: each takes a
// part of K, and their sums meet in shared memory in the order of the parts.  Such calls have tiles of 16 tokens (see tile_width).
//
// Measured on one GB300, 8-bit rows unless said otherwise: 16 x 151,936 x 2048 29.7 us (5.9 TB/s, 87% of the measured copy
// rate); 1 x 5120 x 2048 5.2 us (about 1.9 until the first weights and scales are there, 0.7 of products, 1.3 of the
// join); 8192 x 5120 x 2048 66 us (2.6 PFLOP/s) and 43 us with 4-bit rows (4.0), 8192 x 8192 x 8192 326 us (3.4) and
// 210 us (5.2).  Large 8-bit ones are bound by shared memory:
// a stage of 192 tokens writes and reads 80 KB there, some 640 of the 663 cycles that it takes, as 4-bit weights fill
// bytes beside 8-bit rows.
#include <cuda.h>

#include <algorithm>

#include "mx_device.cuh"
#include "tc_sm100.cuh"

namespace lq4 {

constexpr int kLinM = 128, kLinThreads = 384;
constexpr int kSfAhead = 3;  // fetches of scales of either warp that are on their way to L2

template <int BITS, int NT>
struct LinShape {
  static constexpr int KB = BITS == 8 ? 128 : 256;          // elements of K a stage: rows of 128 bytes
  __host__ __device__ static constexpr int k_blocks(int K) { return K / KB + (K % KB != 0); }  // (K + KB - 1 may pass 2^31)
  static constexpr int GROUPS = KB / 128;                    // of 128 elements: one word of scales a row
  static constexpr int XSF = (NT + 127) / 128;               // 512-byte blocks of the tokens' scales a group
  static constexpr int W_BYTES = kLinM * 128, X_BYTES = NT * 128;
  static constexpr int TX = (BITS == 8 ? W_BYTES / 2 : W_BYTES) + X_BYTES;  // the copy counts packed bytes
  static constexpr int STAGE = W_BYTES + X_BYTES;           // and its scales, which lie behind all stages
  static constexpr int SF_BYTES = GROUPS * 512 * (1 + XSF);
  static constexpr int FIT = (220 * 1024 - 1024) / (STAGE + SF_BYTES);
  static constexpr int STAGES = FIT < 10 ? FIT : 10;
  static constexpr int SMEM = STAGES * (STAGE + SF_BYTES) + 1024;
  static constexpr int SF_COLS = GROUPS * 4 * (1 + XSF);     // tensor memory columns of a stage's scales
  static constexpr int COLS = 2 * NT + 2 * SF_COLS;
  static constexpr int ALLOC = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  // Instruction descriptor: formats of W (e2m1: 5, or 1 among the 4-bit kinds) and x, N, E8M0 scales, M.
  static constexpr uint32_t IDESC = ((BITS == 8 ? 5u : 1u) << 7) | ((BITS == 8 ? 0u : 1u) << 10) |
                                    ((uint32_t)(NT >> 3) << 17) | (1u << 23) | ((uint32_t)(kLinM >> 4) << 24);
  static constexpr int PER = 4 / GROUPS;  // stages whose scales are read at once, by one of two warps in turns
  // A wait on a barrier's parity holds for one phase back.  A warp that copies scales skips the other's PER stages, and it
  // waited for the stage before those; with STAGES > PER the phase before the one it waits for next is over by then.
  static_assert(STAGES > PER, "a parity would be taken for the one two phases on");
  static constexpr bool SHARED = NT == 16;  // a cluster may share a tile
  static_assert(COLS <= 512 && (!SHARED || NT * kLinM * 4 <= STAGES * STAGE), "tile does not fit");
};

struct LinArgs {
  const uint8_t *w_scales, *x_scales;
  void *out;
  int64_t out_ts;
  int32_t *err;
  int N, T, K, dtype;
  int m_tiles, tiles, split;
};

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// The products and copies of a block in one piece each: the whole warp comes here and one elected lane issues them.  Elected
// for each instruction instead, what issues them takes longer than few tokens' products (40 cycles an instruction).
//
// N times 512 bytes of scales (32 rows of 16 bytes) to four columns of tensor memory, for each of its four quarters.
template <int N>
__device__ __forceinline__ void copy_scales_warp(uint32_t taddr, uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 32;  // eight rows of 16 bytes, then the next eight
  d |= (uint64_t)1 << 46;           // descriptor version; no swizzle
  static_assert(N == 2 || N == 3 || N == 4 || N == 6, "");
  if (N == 2)
    asm volatile(
        "{\n.reg .pred p;\n.reg .b32 t;\n.reg .b64 d;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n"
        "add.u32 t, %0, 4;\nadd.u64 d, %1, 32;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "}" ::"r"(taddr),
        "l"(d)
        : "memory");
  if (N == 3)
    asm volatile(
        "{\n.reg .pred p;\n.reg .b32 t;\n.reg .b64 d;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n"
        "add.u32 t, %0, 4;\nadd.u64 d, %1, 32;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 8;\nadd.u64 d, %1, 64;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "}" ::"r"(taddr),
        "l"(d)
        : "memory");
  if (N == 4)
    asm volatile(
        "{\n.reg .pred p;\n.reg .b32 t;\n.reg .b64 d;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n"
        "add.u32 t, %0, 4;\nadd.u64 d, %1, 32;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 8;\nadd.u64 d, %1, 64;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 12;\nadd.u64 d, %1, 96;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "}" ::"r"(taddr),
        "l"(d)
        : "memory");
  if (N == 6)
    asm volatile(
        "{\n.reg .pred p;\n.reg .b32 t;\n.reg .b64 d;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n"
        "add.u32 t, %0, 4;\nadd.u64 d, %1, 32;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 8;\nadd.u64 d, %1, 64;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 12;\nadd.u64 d, %1, 96;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 16;\nadd.u64 d, %1, 128;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "add.u32 t, %0, 20;\nadd.u64 d, %1, 160;\n@p tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n"
        "}" ::"r"(taddr),
        "l"(d)
        : "memory");
}
// The four products of 32 bytes of K each.  8-bit rows: 32 of K, the scales' bytes 0 to 3; 4-bit rows: 64 of K, byte pairs of
// one word of scales and then of the next (sb_step columns on), which is left out where K ends before it (second = 0).
template <int BITS>
__device__ __forceinline__ void mma_block_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                               uint32_t sb, uint32_t accumulate, uint32_t sb_step, uint32_t second) {
  if (BITS == 8)
    asm volatile(
        "{\n.reg .pred p, q, r;\n.reg .b64 a, b;\n.reg .b32 i, s, t;\nelect.sync _|p, 0xffffffff;\n"
        "setp.ne.b32 q, %6, 0;\nsetp.eq.b32 r, %6, %6;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], q;\n"
        "add.u64 a, %1, 2;\nadd.u64 b, %2, 2;\nadd.u32 i, %3, 536870928;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, i, [%4], [%5], r;\n"
        "add.u64 a, %1, 4;\nadd.u64 b, %2, 4;\nadd.u32 i, %3, 1073741856;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, i, [%4], [%5], r;\n"
        "add.u64 a, %1, 6;\nadd.u64 b, %2, 6;\nadd.u32 i, %3, 1610612784;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, i, [%4], [%5], r;\n"
        "}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(sb_step), "r"(second)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p, q, r;\n.reg .b64 a, b;\n.reg .b32 i, s, t;\nelect.sync _|p, 0xffffffff;\n"
        "setp.ne.b32 q, %6, 0;\nsetp.eq.b32 r, %6, %6;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], q;\n"
        "add.u64 a, %1, 2;\nadd.u64 b, %2, 2;\nadd.u32 i, %3, 1073741856;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, i, [%4], [%5], r;\n"
        "add.u32 s, %4, 4;\nadd.u32 t, %5, %7;\nsetp.ne.and.b32 p, %8, 0, p;\n"
        "add.u64 a, %1, 4;\nadd.u64 b, %2, 4;\nadd.u32 i, %3, 0;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, i, [s], [t], r;\n"
        "add.u64 a, %1, 6;\nadd.u64 b, %2, 6;\nadd.u32 i, %3, 1073741856;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, i, [s], [t], r;\n"
        "}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(sb_step), "r"(second)
        : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float peer_float(uint32_t saddr, int rank) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }
// One feature of up to 16 tokens.
template <typename O>
__device__ __forceinline__ void store_column(O *p, int64_t step, const float (&v)[16], int count) {
  if (count >= 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j, p += step) put(p, v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j, p += step)
      if (j < count) put(p, v[j]);
  }
}
__device__ __forceinline__ void store_out(const LinArgs &a, int t, int n, float v) {
  const int64_t at = t * a.out_ts + n;
  if (a.dtype == LILY_F32) put(static_cast<float *>(a.out) + at, v);
  else if (a.dtype == LILY_BF16) put(static_cast<__nv_bfloat16 *>(a.out) + at, v);
  else put(static_cast<__half *>(a.out) + at, v);
}

template <int BITS, int NT>
__global__ void __launch_bounds__(kLinThreads, 1)
    mx4_linear_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map, LinArgs a) {
  using S = LinShape<BITS, NT>;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bars[2 * S::STAGES + 4 + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t tiles_at = (tc::smem_u32(s_raw) + 1023u) & ~1023u, sf_at = tiles_at + S::STAGES * S::STAGE;
  const uint32_t bars = tc::smem_u32(s_bars);
  auto full = [&](int i) { return bars + 8 * i; };  // codes and scales are there
  auto empty = [&](int i) { return bars + 8 * (S::STAGES + i); };
  auto acc_full = [&](int i) { return bars + 8 * (2 * S::STAGES + i); };
  auto acc_empty = [&](int i) { return bars + 8 * (2 * S::STAGES + 2 + i); };
  const uint32_t drained = bars + 8 * (2 * S::STAGES + 4);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = S::SHARED ? a.split : 1;
  const int rank = blockIdx.x % split, group = blockIdx.x / split, groups = gridDim.x / split;
  const int blocks = S::k_blocks(a.K);
  const int k_begin = (int)((int64_t)blocks * rank / split), k_end = (int)((int64_t)blocks * (rank + 1) / split);
  volatile int *abort = &s_abort;

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < S::STAGES; ++i) tc::mbar_init(full(i), 2), tc::mbar_init(empty(i), 1);
    for (int i = 0; i < 2; ++i) tc::mbar_init(acc_full(i), 1), tc::mbar_init(acc_empty(i), 8);
    tc::mbar_init(drained, 1);
    tc::mbar_init_fence();
    asm volatile("prefetch.tensormap [%0];" ::"l"(&w_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&x_map) : "memory");
  }
  // The first weights and their scales start on their way to L2 while the kernel before this one still runs.  (If it is that
  // that writes them, L2 gets what it writes.  Norm, product, quantisation, product of one token, weights from memory: 13.6 ->
  // 13.1 us; 16 x 151,936 x 2048 of 4-bit rows 28.1 -> 27.3; products of one token in a row 5.1 -> 5.3.)
  if (group < a.tiles) {
    const int m = group % a.m_tiles * kLinM;
    if (warp == 1 && lane < S::STAGES && k_begin + lane < k_end) prefetch_2d(&w_map, (k_begin + lane) * 128, m);
    const int word = (k_begin / S::PER + warp - 2) * 4;
    if ((warp == 2 || warp == 3) && word < a.K / 128)
      for (int row = m + lane; row < min(m + kLinM, a.N); row += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w_scales + ((int64_t)row * (a.K / 128) + word) * 4));
  }
  pdl_wait();
  if (warp == 3) {
    tc::tmem_alloc(tc::smem_u32(&s_tmem), S::ALLOC);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, s_tmem, 0);
  next_may_start();  // not before: its tensor memory must not be what this block waits for

  if (warp == 0) {  // codes
    int stage = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int tile = group; ok && tile < a.tiles; tile += groups) {
      const int m = tile % a.m_tiles * kLinM, t = tile / a.m_tiles * NT;
      for (int kb = k_begin; kb < k_end; ++kb) {
        ok = tc::wait_bar(empty(stage), phase ^ 1, abort, a.err);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t at = tiles_at + stage * S::STAGE;
          tc::mbar_arrive_expect_tx(full(stage), S::TX);
          tma_2d(at, &w_map, kb * 128, m, full(stage));  // in elements of the map: 128 of 4 bits, or bytes
          tma_2d(at + S::W_BYTES, &x_map, kb * 128, t, full(stage));
        }
        __syncwarp();
        ++issued;
        if (++stage == S::STAGES) stage = 0, phase ^= 1;
      }
    }
    if (*abort) {  // the copies under way end before their memory is given back
      // (a stage whose scales never came does not fill: that wait ends by the limit, long after the copy)
      const long long t0 = clock64();
      for (int i = 0; i < S::STAGES && i < issued; ++i) {
        if (--stage < 0) stage = S::STAGES - 1, phase ^= 1;
        while (!tc::mbar_try_wait(full(stage), phase) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp == 2 || warp == 3) {
    // Scales: a lane reads four words (512 of K, up to four blocks) of rows lane, lane + 32, .. at once.  The two warps take
    // these fetches in turns: one's are under way while the other hands its own out.
    const int words = a.K / 128;
    const bool wide = words % 4 == 0 && ((uintptr_t)a.w_scales | (uintptr_t)a.x_scales) % 16 == 0;
    constexpr int PER = S::PER, XROWS = (NT + 31) / 32;
    auto load = [&](const uint8_t *scales, int row, int rows, int word) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(scales) + (int64_t)row * words + word;
        if (wide) {
          v = __ldg(reinterpret_cast<const uint4 *>(p));
        } else {
          v.x = __ldg(p);
          if (word + 1 < words) v.y = __ldg(p + 1);
          if (word + 2 < words) v.z = __ldg(p + 2);
          if (word + 3 < words) v.w = __ldg(p + 3);
        }
      }
      return v;
    };
    auto part = [](const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
    struct Place {  // a fetch: blocks kb .. end - 1 of a tile
      int tile, kb, end;
    };
    auto place = [&](int tile, int kb) { return Place{tile, kb, min(k_end, (kb / PER + 1) * PER)}; };
    auto after = [&](const Place &p) { return p.end < k_end ? place(p.tile, p.end) : place(p.tile + groups, k_begin); };
    uint4 w[4], x[XROWS];
    auto fetch = [&](const Place &p) {
      if (p.tile >= a.tiles) return;
      const int m = p.tile % a.m_tiles * kLinM, t = p.tile / a.m_tiles * NT, word = p.kb / PER * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = load(a.w_scales, m + 32 * j + lane, a.N, word);
#pragma unroll
      for (int i = 0; i < XROWS; ++i) x[i] = load(a.x_scales, t + 32 * i + lane, a.T, word);
    };
    // A fetch is under way long enough for L2 but not for memory: the weights' scales are brought to L2 ahead of it.
    Place far = place(group, k_begin);
    auto prefetch = [&]() {
      if (far.tile >= a.tiles) return;
      const int m = far.tile % a.m_tiles * kLinM;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = m + 32 * j + lane;
        if (row < a.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w_scales + ((int64_t)row * words + far.kb / PER * 4) * 4));
      }
      far = after(far), far = after(far);
    };
    int stage = 0, phase = 0;
    auto advance = [&](int n) {
      for (stage += n; stage >= S::STAGES; stage -= S::STAGES) phase ^= 1;
    };
    bool ok = k_begin < k_end;
    Place now = place(group, k_begin);
    if (warp == 3) {
      advance(now.end - now.kb);
      now = after(now), far = now;
    }
    for (int i = 0; i < kSfAhead; ++i) prefetch();
    fetch(now);
    while (ok && now.tile < a.tiles) {
      uint4 now_w[4], now_x[XROWS];
#pragma unroll
      for (int j = 0; j < 4; ++j) now_w[j] = w[j];
#pragma unroll
      for (int i = 0; i < XROWS; ++i) now_x[i] = x[i];
      const Place other = after(now), next = after(other);
      fetch(next);
      prefetch();
#pragma unroll
      for (int s = 0; s < PER; ++s) {
        const int kb = now.kb / PER * PER + s;
        if (kb < now.kb || kb >= now.end) continue;
        ok = ok && tc::wait_bar(empty(stage), phase ^ 1, abort, a.err);
        if (!ok) break;
        const uint32_t at = sf_at + stage * S::SF_BYTES + lane * 16;
#pragma unroll
        for (int g = 0; g < S::GROUPS; ++g) {
          const int c = s * S::GROUPS + g;
          st_shared4(at + g * 512, part(now_w[0], c), part(now_w[1], c), part(now_w[2], c), part(now_w[3], c));
#pragma unroll
          for (int i = 0; i < XROWS; i += 4)
            st_shared4(at + (S::GROUPS + g * S::XSF + i / 4) * 512, part(now_x[i], c),
                       i + 1 < XROWS ? part(now_x[i + 1 < XROWS ? i + 1 : i], c) : 0,
                       i + 2 < XROWS ? part(now_x[i + 2 < XROWS ? i + 2 : i], c) : 0,
                       i + 3 < XROWS ? part(now_x[i + 3 < XROWS ? i + 3 : i], c) : 0);
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full(stage));
        advance(1);
      }
      if (other.tile < a.tiles) advance(other.end - other.kb);
      now = next;
    }
  } else if (warp == 1) {  // products
    int stage = 0, buf = 0, buf_phase = 0, slot = 0;
    bool ok = true;
    // The vote makes what follows a wait the same for the whole warp to the compiler, which then keeps descriptors and addresses
    // in uniform registers; moved there for every instruction they cost more than few tokens' products (16 tokens of
    // 151,936 x 2048: 39.9 -> 32.8 us).
    auto wait = [&](uint32_t bar, int parity) { return __all_sync(~0u, tc::wait_bar(bar, parity, abort, a.err)); };
    // Scales go to tensor memory one stage ahead of the products that use them, so that no product waits for a copy issued
    // just before it.
    int64_t left = group < a.tiles ? (int64_t)((a.tiles - group + groups - 1) / groups) * (k_end - k_begin) : 0;
    int ahead = 0, ahead_phase = 0;
    auto copy_scales = [&](int to) {
      if (left == 0) return;
      --left;
      ok = wait(full(ahead), ahead_phase);
      if (!ok) return;
      tc::tc_fence_after();
      copy_scales_warp<S::GROUPS * (1 + S::XSF)>(tmem + 2 * NT + to * S::SF_COLS, sf_at + ahead * S::SF_BYTES);
      if (++ahead == S::STAGES) ahead = 0, ahead_phase ^= 1;
    };
    copy_scales(0);
    for (int tile = group; ok && tile < a.tiles; tile += groups) {
      ok = wait(acc_empty(buf), buf_phase ^ 1);
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t d = tmem + buf * NT;
      for (int kb = k_begin; kb < k_end; ++kb) {
        const uint32_t at = tiles_at + stage * S::STAGE, sf = tmem + 2 * NT + slot * S::SF_COLS;
        slot ^= 1;
        copy_scales(slot);
        if (!ok) break;
        mma_block_warp<BITS>(d, tc::desc_k128_sw128(at), tc::desc_k128_sw128(at + S::W_BYTES), S::IDESC, sf,
                             sf + 4 * S::GROUPS, kb > k_begin, 4 * S::XSF, BITS == 8 || kb * S::KB + 128 < a.K);
        tc::mma_commit_warp(empty(stage));
        if (++stage == S::STAGES) stage = 0;
      }
      if (!ok) break;
      tc::mma_commit_warp(acc_full(buf));
      if (++buf == 2) buf = 0, buf_phase ^= 1;
    }
    if (*abort) {  // the products under way end before tensor memory is given back
      tc::mma_commit_warp(drained);
      const long long t0 = clock64();
      while (!tc::mbar_try_wait(drained, 0) && clock64() - t0 < tc::kWaitCycles) {
      }
    }
  } else if (warp >= 4) {  // results: a thread has one row of the weights, and every other 16 tokens
    const int row = (warp & 3) * 32 + lane, half = (warp - 4) >> 2;
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);
    int buf = 0, buf_phase = 0;
    for (int tile = group; tile < a.tiles; tile += groups) {
      if (!tc::wait_bar(acc_full(buf), buf_phase, abort, a.err, 1000)) break;
      tc::tc_fence_after();
      const int n = tile % a.m_tiles * kLinM + row, t0 = tile / a.m_tiles * NT;
#pragma unroll 1
      for (int c = 16 * half; c < NT && t0 + c < a.T; c += 32) {
        float v[16];
        tc::tmem_ld16(mine + buf * NT + c, v);
        if (split > 1) {  // one tile: the stages are free, and take the sums
#pragma unroll
          for (int j = 0; j < 16; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(tiles_at + 4 * ((c + j) * kLinM + row)), "f"(v[j]) : "memory");
        } else if (n < a.N) {
          const int64_t at = (int64_t)(t0 + c) * a.out_ts + n;
          const int count = a.T - t0 - c;
          if (a.dtype == LILY_F32) store_column(static_cast<float *>(a.out) + at, a.out_ts, v, count);
          else if (a.dtype == LILY_BF16) store_column(static_cast<__nv_bfloat16 *>(a.out) + at, a.out_ts, v, count);
          else store_column(static_cast<__half *>(a.out) + at, a.out_ts, v, count);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(acc_empty(buf));
      if (++buf == 2) buf = 0, buf_phase ^= 1;
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();
    const int tile = group, n0 = tile % a.m_tiles * kLinM, t0 = tile / a.m_tiles * NT;
    const int cells = min(NT, a.T - t0) * kLinM;
    if (!*abort) {
      for (int i = rank * kLinThreads + threadIdx.x; i < cells; i += split * kLinThreads) {
        float v[8], sum = 0.f;  // all are asked for before the first is waited for
#pragma unroll
        for (int p = 0; p < 8; ++p) v[p] = p < split ? peer_float(tiles_at + 4 * i, p) : 0.f;
#pragma unroll
        for (int p = 0; p < 8; ++p) sum += p < split ? v[p] : 0.f;
        const int n = n0 + i % kLinM;
        if (n < a.N) store_out(a, t0 + i / kLinM, n, sum);
      }
    }
    cluster_sync();  // no block leaves while another reads its sums
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 3) tc::tmem_dealloc(tmem, S::ALLOC);
}

// ----------------------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
  static std::atomic<void *> found{nullptr};
  void *f = found.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// Rows of K elements as boxes of `rows` rows and 128 bytes of shared memory.
static bool encode(CUtensorMap *map, const uint8_t *codes, int64_t count, int K, int bits, bool spread, int rows) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(spread || bits == 8 ? K : K / 2), (cuuint64_t)count};
  const cuuint64_t stride[1] = {(cuuint64_t)K * bits / 8};
  const cuuint32_t box[2] = {128, (cuuint32_t)rows}, step[2] = {1, 1};
  return f(map, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
           const_cast<uint8_t *>(codes), dims, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Parts of K, one a block of a cluster.  A cluster's blocks have to find SMs in one corner of the GPU, so not all SMs can be
// counted on: with more than four fifths of them (two thirds by clusters over four) some clusters wait for a second
// round (1 x 2048 x 4096: 9.2 us with 16 clusters of 8, 5.6 of 6 or 4, 9.1 without; 40 x 2048 x 4096: 12.9 us with 48 clusters
// of 3, 8.1 of 2).
static int k_parts(int tiles, int blocks, int sms) {
  int parts = std::min(std::min(8, blocks), sms * 4 / 5 / tiles);
  if (parts > 4) parts = std::max(4, std::min(parts, sms * 2 / 3 / tiles));
  return std::max(1, parts);
}

template <int BITS, int NT>
static cudaError_t launch_tiles(const lily_mx_mat &W, const lily_mx_mat &x, LinArgs a, cudaStream_t st) {
  using S = LinShape<BITS, NT>;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem<S::SMEM>(mx4_linear_kernel<BITS, NT>, done);
  if (e != cudaSuccess) return e;
  CUtensorMap w_map, x_map;
  if (!encode(&w_map, W.codes, W.rows, W.cols, 4, BITS == 8, kLinM) ||
      !encode(&x_map, x.codes, x.rows, x.cols, BITS, false, NT))
    return cudaErrorInvalidValue;
  const int sms = std::max(1, sm_count()), blocks = S::k_blocks(a.K);
  a.m_tiles = (a.N + kLinM - 1) / kLinM;
  const int64_t tiles = (int64_t)a.m_tiles * ((a.T + NT - 1) / NT);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  a.tiles = (int)tiles;
  a.split = S::SHARED ? k_parts((int)tiles, blocks, sms) : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.split > 1 ? a.split * a.tiles : std::min(a.tiles, sms));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S::SHARED ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, mx4_linear_kernel<BITS, NT>, w_map, x_map, a);
}

// Tokens a tile.  What a tile costs goes with the rows that its stages bring to shared memory and the products read there,
// 128 of weights and NT of tokens, so the width is the one with the least of rows times rounds of tiles over the SMs.
// A wider tile costs more in one round, so one is taken only where the width before it needs a second: there are more tiles than SMs of
// that, and, as no width is more than twice the one before, more than half as many of the wider, too many for clusters.
// (3001 x 2048 x 4096 of 4-bit rows: 16.4 us with 192, two rounds of which the second is 68% full; 15.5 with 160.)
static int tile_width(int64_t T, int64_t m_tiles, int64_t sms) {
  int best = 16;
  int64_t least = INT64_MAX;
  for (const int nt : {16, 32, 64, 96, 128, 160, 192}) {
    const int64_t tiles = m_tiles * ((T + nt - 1) / nt), cost = (tiles + sms - 1) / sms * (128 + nt);
    if (cost < least) least = cost, best = nt;
  }
  return best;
}

template <int BITS>
static cudaError_t launch_bits(const lily_mx_mat &W, const lily_mx_mat &x, const LinArgs &a, cudaStream_t st) {
  switch (tile_width(a.T, (a.N + kLinM - 1) / kLinM, std::max(1, sm_count()))) {
    case 16: return launch_tiles<BITS, 16>(W, x, a, st);
    case 32: return launch_tiles<BITS, 32>(W, x, a, st);
    case 64: return launch_tiles<BITS, 64>(W, x, a, st);
    case 96: return launch_tiles<BITS, 96>(W, x, a, st);
    case 128: return launch_tiles<BITS, 128>(W, x, a, st);
    case 160: return launch_tiles<BITS, 160>(W, x, a, st);
    default: return launch_tiles<BITS, 192>(W, x, a, st);
  }
}

int launch_mx4_linear(const lily_mx_mat &W, const lily_mx_mat &x, int dtype, void *out, int64_t out_ts, void *ws,
                      cudaStream_t st) {
  LinArgs a = {};
  a.w_scales = W.scales, a.x_scales = x.scales;
  a.out = out, a.out_ts = out_ts, a.dtype = dtype;
  a.err = static_cast<int32_t *>(ws) + kHdrError;
  a.N = W.rows, a.T = x.rows, a.K = W.cols;
  const cudaError_t e = x.bits == 8 ? launch_bits<8>(W, x, a, st) : launch_bits<4>(W, x, a, st);
  return e == cudaSuccess ? LILY_Q4_OK : (cudaGetLastError(), LILY_Q4_ERR_CUDA);
}

}  // namespace lq4
