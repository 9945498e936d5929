// lily_kv8_attention, the form for many rows a sequence (prompt chunks): tcgen05 tiles.
//
// Bound by the tensor cores (4 * head_dim operations a visible query-key pair).  A block takes row
// tiles of 128 rows -- the group's heads of consecutive tokens of one key/value head, so that every
// code read serves all of them -- and walks their visible keys 128 at a time:
//   S = Q K^T (both in shared memory), P = 2^(S' - m) as fp16 written over S in tensor memory,
//   O += P V (P from tensor memory, V from shared memory), O in tensor memory throughout.
// One block an SM, which holds all 512 TMEM columns.  Warps: 8 of softmax (a thread owns a row: its
// maximum and sum need no exchange), 4 (head_dim 256: 8) that turn codes into fp16 operands, 1 that
// issues the products.
//
// Head_dim 64 and 128: two row tiles a block share each converted key tile (S 2 x 128 columns, O 2 x
// head_dim); K and V have two buffers.  While one tile's softmax runs, the other's products do.
// Head_dim 256: one row tile (O 256 columns), S twice: the next key tile's scores are computed under
// the softmax of the current one, and two softmax groups take the key tiles in turns, handing the
// running maximum on.  K and V have one buffer (64 KB each); K's four atoms of 64 elements and V's two
// halves of 64 keys are given back and refilled one by one.
//
// Operands.  K's codes keep their order; V's are transposed on the way (a lane holds 8 or 16 bytes of
// 8 consecutive tokens, byte permutes interleave the tokens), so both are K-major tiles with the
// 128-byte swizzle, written without bank conflicts.  Codes of the next tile are in flight in
// registers meanwhile; nothing is computed from a load before it is needed (a select after a load
// waits for it: 1449 -> 800 us came mostly from removing such waits).  fp16 holds the codes exactly and
// q after a scaling by a power of two; the weights are rounded to fp16 relative to the largest
// weight-times-magnitude (see kv8_attention.cu for the magnitudes' place in the exponent).
//
// A row's reference m is set 6 below the largest exponent there is (see kv8_device.cuh) and moves only when
// one grows to 15 above it (head_dim 64 and 128: to 11.9), where fp16 still holds its weight, because
// moving it rescales O in tensor memory.  Head_dim 64 and 128 need no maximum before
// the weights then: a tile is done in one pass to the reference there is, and done again where sixteen of a
// row's weights come to more than 65504 (ragged prompts below: 657 us with a pass for the maximum, 608 with
// the maximum beside the weights, 583 with a sum, which is there anyway, as the sign).  The pass
// holds a row's 64 words of weights until it is known to stand, so the softmax warps take registers
// from the issuing warp's group (160 a thread and 64: those 583 us; 168 and 40: 586; 152 and 80: 620; 144 and
// 96: 609).  Head_dim 256 has no registers for it.
//
// Measured on one GB300: 5 ragged prompts, 6.6k tokens over up to 8k keys each, 32 / 8 heads of 128: 578 us
// (1,101 TFLOP/s, 57% of the measured bf16 rate); a 4096-token chunk after 28,672, 16 / 2 heads of 256:
// 1.95 ms (1,058 TFLOP/s, 55%); 5 prompts of 1500 tokens after 3000, 16 / 4 heads of 64: 199 us (30%: its
// 450M exponentials alone take about 90 us).  What bounds it: at 128, the chain of one row tile (scores 540 cycles,
// weights about 1,750, product 870, hand-overs 700) against the other's, and the issue of
// the softmax's instructions (an eighth of the exponentials as polynomials instead: 657 -> 679 us, half
// of them 748); at 256 conversion and products about equally (without conversion 1.61 ms, with a
// quarter of the products 1.82 ms).  Tried without gain: four softmax groups of half a row each
// (751 us), issuing whichever row tile is ready (886 us), starting the product after half of the
// weights, longer suspension in barrier waits.
#include <algorithm>

#include "kv8_device.cuh"
#include "tc_sm100.cuh"

namespace lq4 {

constexpr int kRows = 128, kKeys = 128;
// A row's reference below the largest exponent when it is set.  More of it keeps smaller weights, less leaves
// more room before the reference has to move: 5 x 1500 prompts over 3000 keys, heads of 128, 460 us at 0 and 5,
// 462 at 6, 469 at 7; with scores four times as spread 631, 655, 658, 661.
constexpr int kBias = 6;

template <int D>
struct PromptShape {
  static constexpr int NQ = D == 256 ? 1 : 2;   // row tiles of a block
  static constexpr int KB = D == 256 ? 1 : 2;   // buffers of K and of V
  static constexpr int CW = D == 256 ? 8 : 4;   // converting warps
  static constexpr int THREADS = 32 * (8 + CW + (D == 256 ? 1 : 4));
  // Registers a thread after the split at head_dim 64, 128, of 128 at launch: 2 x 160 + 128 + 64 = 4 x 128
  static constexpr int SOFTMAX_REGS = 160, ISSUE_REGS = 64;
  static constexpr int ROWS = kRows * NQ;
  static constexpr int TILE = kKeys * D * 2;    // bytes of a K or V tile (and of 128 rows of Q)
  static constexpr int VW = D == 64 ? 2 : 4;    // words of a token a lane holds of V
  static constexpr int COLS = D == 256 ? 16 : 32;  // score columns a thread holds, twice
  // The exponent above a row's reference beyond which it moves.  fp16 holds weights below 2^16; sixteen whose
  // sum is above 65504 have one above 2^11.9, so that the one pass never finds too much and moves nothing.
  static constexpr float MOVE = D == 256 ? 15.f : 11.9f;
  static constexpr int SMEM = (NQ + 2 * KB) * TILE + 1024;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tm_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 columns in two steps, for work between them; the wait passes the registers through.
__device__ __forceinline__ void tm_ld16_start(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_ld16_wait(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// f(c, W columns) for each W-column part c of a row's 128, the next part's load under way.
template <int W, int UNROLL = W == 32 ? 2 : 1, typename F>
__device__ __forceinline__ void for_columns(uint32_t addr, F f) {
  uint32_t x[W], y[W];
  auto start = [&](int c, uint32_t *r) {
#pragma unroll
    for (int i = 0; i < W; i += 16) tm_ld16_start(addr + W * c + i, r + i);
  };
  auto wait = [&](uint32_t *r) {
#pragma unroll
    for (int i = 0; i < W; i += 16) tm_ld16_wait(r + i);
  };
  start(0, x);
  // Unrolled at 32 columns (five percent of the whole at head_dim 128); at 16, where a thread has
  // 96 registers, unrolling spills (half as fast again).
#pragma unroll(UNROLL)
  for (int c = 0; c < 128 / W; c += 2) {
    wait(x);
    start(c + 1, y);
    f(c, x);
    wait(y);
    if (c + 2 < 128 / W) start(c + 2, x);
    f(c + 1, y);
  }
}

__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 columns from registers, not waited for.
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

constexpr uint32_t idesc_f16(int N) {  // D fp32, A and B fp16, both K-major, 128 x N
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A bounded wait whose answer the whole warp shares: when one lane gives up they all leave together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *err) {
  return __all_sync(~0u, tc::wait_bar(bar, parity, abort_flag, err));
}

struct PromptItem {
  int row0, n, len;  // the sequence
  int rt;            // row tile (of ROWS)
  int lo, tiles;     // first key, key tiles
};

template <int D>
__global__ void __launch_bounds__(PromptShape<D>::THREADS, 1)
    kv8_prompt_kernel(AttnArgs a, int bf16, int splits) {
  using P = PromptShape<D>;
  constexpr int NQ = P::NQ, WARPS = P::THREADS / 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[24];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_count[WARPS], s_found[2];
  __shared__ float4 s_meta[8][8];
  __shared__ float s_max[kRows];        // head_dim 256: the rows' running maximum
  __shared__ float2 s_ml[2][kRows];     // head_dim 256: the two groups' maximum and sum
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *const mem = smem_raw + (base - tc::smem_u32(smem_raw));
  constexpr uint32_t kAt = NQ * P::TILE, vAt = (NQ + P::KB) * P::TILE;  // K and V buffers
  const uint32_t bar = tc::smem_u32(s_bar);
  const uint32_t k_full = bar, k_free = bar + 32;                                        // [KP]
  const uint32_t v_full = bar + 64, v_free = bar + 80;                                   // [2]
  const uint32_t s_full = bar + 96, p_full = bar + 112, pv_done = bar + 128, m_full = bar + 144;  // [2]
  const uint32_t drain = bar + 160;

  if (tid == 0) {
    s_abort = 0;
    s_found[0] = -1;
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(k_full + 8 * i, 128);
      tc::mbar_init(k_free + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(v_full + 8 * i, 128);
      tc::mbar_init(v_free + 8 * i, 1);
      tc::mbar_init(s_full + 8 * i, 1);
      tc::mbar_init(p_full + 8 * i, 128);
      tc::mbar_init(pv_done + 8 * i, 1);
      tc::mbar_init(m_full + 8 * i, 128);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init_fence();
  }
  if (tid < kRows) s_max[tid] = -INFINITY;
  pdl_wait();
  // after the wait: no tensor memory is held while a kernel that may want some is waited for
  if (warp == 0) {
    tc::tmem_alloc(tc::smem_u32(&s_tmem), 512);
    tc::tmem_relinquish();
  }
  const Batch &B = a.B;
  int32_t *err = a.hdr + kHdrError;
  volatile int *abort_flag = &s_abort;

  // ---- which rows: the row tiles of all sequences, the last (in a causal chunk: the longest) first
  auto tiles_of = [&](int b) {
    if (b >= B.batch) return 0;
    const Seq s = load_seq(B, b, a.hdr);
    return (s.n * a.group + P::ROWS - 1) / P::ROWS;
  };
  int total = 0;
  for (int b0 = 0; b0 < B.batch; b0 += P::THREADS) {
    const int n = __reduce_add_sync(~0u, tiles_of(b0 + tid));
    if (lane == 0) s_count[warp] = n;
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) total += s_count[w];
    __syncthreads();
  }
  const int h = blockIdx.x % a.kv_heads, want = total - 1 - (int)(blockIdx.x / a.kv_heads);
  const int split = blockIdx.y;
  int before = 0;
  if (want >= 0) {
    for (int b0 = 0; b0 < B.batch; b0 += P::THREADS) {
      const int n = tiles_of(b0 + tid);
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += up;
      }
      if (lane == 31) s_count[warp] = sum;
      __syncthreads();
      for (int w = 0; w < warp; ++w) sum += s_count[w];
      sum += before;
      if (want < sum && want >= sum - n) {
        s_found[0] = b0 + tid;
        s_found[1] = want - (sum - n);
      }
      for (int w = 0; w < WARPS; ++w) before += s_count[w];
      __syncthreads();
    }
  }
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  PromptItem it = {0, 0, 0, 0, 0, 0};
  const int b_seq = s_found[0];
  if (b_seq >= 0) {
    const Seq s = load_seq(B, b_seq, a.hdr);
    it.row0 = s.row0;
    it.n = s.n;
    it.len = s.len;
    it.rt = s_found[1];
    const int p_first = s.len - s.n + it.rt * P::ROWS / a.group;
    const int p_last = s.len - s.n + min(s.n - 1, (it.rt * P::ROWS + P::ROWS - 1) / a.group);
    it.lo = max(0, first_key(p_first, a.window)) & ~15;
    const int hi = a.causal ? min(p_last + 1, s.len) : s.len;
    it.tiles = max(0, (hi - it.lo + kKeys - 1) / kKeys);
  }
  // row tiles of the block that hold rows
  const int nq = NQ == 2 && it.n * a.group - it.rt * P::ROWS > kRows ? 2 : 1;
  // this split's key tiles
  const int t_begin = (int)((int64_t)it.tiles * split / splits);
  const int tiles = (int)((int64_t)it.tiles * (split + 1) / splits) - t_begin;
  const int key0 = it.lo + t_begin * kKeys, len = it.len;
  const int64_t part = (int64_t)blockIdx.x * splits + split;
  if (splits > 1 && split == 0 && tid == 0)
    a.jobs[blockIdx.x] = make_int4(it.row0, it.n, h, it.rt);
  // page of 16-key group g of this split's tile j (to be checked where it is used)
  auto page_of = [&](int j, int g) {
    const int tok = key0 + j * kKeys + g * 16;
    return j < tiles && tok < len ? raw_page(B, b_seq, tok >> B.page_shift) : kNoPage;
  };

  if (warp < 8) {
    if (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::SOFTMAX_REGS));
    // ======================================================================== softmax
    // Group wg of four warps: head_dim 64, 128: row tile wg, every key tile; head_dim 256: the
    // key tiles of its parity.  Its scores are in S slot wg either way.
    const int wg = warp >> 2, r = tid & 127;
    const int rr = it.rt * P::ROWS + (NQ == 2 ? wg * kRows : 0) + r;
    const int tok = rr / a.group, head = h * a.group + rr - tok * a.group;
    const bool live = tok < it.n;
    const int64_t row = it.row0 + tok;
    float qf = 0.f;
    {
      // a row's words all at once (head_dim 256: half of them in each group, which exchange maxima)
      constexpr int WORDS = NQ == 2 ? D / 8 : D / 16;
      const int c0 = NQ == 2 ? 0 : wg * WORDS;
      const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * a.q_ts + (int64_t)head * a.q_hs) + c0;
      uint4 raw[WORDS];
#pragma unroll
      for (int c = 0; c < WORDS; ++c) raw[c] = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < WORDS; ++c) {
        float f[8];
        if (bf16) unpack8<Bf16>(raw[c], f);
        else unpack8<F16>(raw[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
      }
      if (NQ == 1) {
        s_ml[wg][r].x = top;
        asm volatile("bar.sync 2, 256;" ::: "memory");
        top = fmaxf(top, s_ml[wg ^ 1][r].x);
      }
      const int e = top > 0.f ? min(max(ilogbf(top), -100), 127) : 14;
      const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - e) << 23), a.scale2);
      qf = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * fabsf(a.scale2);
      uint8_t *dst = mem + (NQ == 2 ? wg * P::TILE : 0);
#pragma unroll
      for (int c = 0; c < WORDS; ++c) {
        float f[8];
        if (bf16) unpack8<Bf16>(raw[c], f);
        else unpack8<F16>(raw[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= up;
        *reinterpret_cast<uint4 *>(dst + ((c0 + c) >> 3) * (kRows * 128) + tc::sw128(r, (c0 + c) & 7)) = pack8<F16>(f);
      }
      tc::fence_proxy_async();
    }
    asm volatile("bar.sync 1, 288;" ::: "memory");  // q is there: softmax and issuing warps
    // visible keys of this row, and those that every live row of the warp sees
    const int pos = it.len - it.n + tok;
    const int klo = first_key(pos, a.window), khi = a.causal ? min(pos + 1, len) : len;
    const int all_lo = __reduce_max_sync(~0u, live ? klo : INT_MIN);
    const int all_hi = __reduce_min_sync(~0u, live ? khi : INT_MAX);
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = t_row + 128 * wg, t_o = t_row + 256 + (NQ == 2 ? wg * D : 0);
    const uint32_t s_full_w = s_full + 8 * wg, p_full_w = p_full + 8 * wg;
    // The product of key tile j.  head_dim 256 has a barrier for each parity of j: the last wait
    // may come while the last two products are both under way, and one barrier's parity would
    // take the end of the product before them for that of the last.
    auto wait_pv = [&](int j) {
      return NQ == 2 ? wait_warp(pv_done + 8 * wg, j & 1, abort_flag, err)
                     : wait_warp(pv_done + 8 * (j & 1), (j >> 1) & 1, abort_flag, err);
    };
    constexpr int STEP = NQ == 2 ? 1 : 2;
    const int j_first = NQ == 2 ? 0 : wg, j_end = NQ == 2 && wg >= nq ? 0 : tiles;
    float m = -INFINITY, l = 0.f;
    // a key tile ahead: the magnitudes of this lane's group; two ahead: its page
    auto load_mag = [&](int pg) {
      const int64_t ph = (int64_t)max(pg, 0) * a.kv_heads + h;
      return make_float2(__ldg(a.k_amax + ph), __ldg(a.v_amax + ph));
    };
    int page = check_page(B, page_of(j_first, lane & 7), a.hdr);
    float2 mag = load_mag(page);
    int raw = page_of(j_first + STEP, lane & 7);
    float4 *meta = s_meta[warp];
    bool ok = true;
    for (int j = j_first; j < j_end; j += STEP) {
      const int k0 = key0 + j * kKeys;
      const uint32_t turn = (NQ == 2 ? j : j >> 1) & 1;
      const float va = page < 0 ? 1.f : value_size(mag.y);
      const bool whole = !__any_sync(~0u, page < 0) && k0 >= all_lo && k0 + kKeys <= all_hi;
      // the reciprocal is a number for a magnitude of NaN too: a hidden key's weight of 0 times it is 0, and
      // the rows that see the page have its NaN from the logarithm
      if (lane < 8) meta[lane] = make_float4(page < 0 ? -1.f : mag.x, __log2f(va), fminf(__frcp_rn(va), 2e30f) * sum_scale(kBias), 0.f);
      page = check_page(B, raw, a.hdr);
      mag = load_mag(page);
      raw = page_of(j + 2 * STEP, lane & 7);
      __syncwarp();
      if (!(ok = wait_warp(s_full_w, turn, abort_flag, err))) break;
      tc::tc_fence_after();
      // A tile at the edge of what the rows see: its scores are turned into exponents here, -inf
      // where a key is hidden, and its groups' factors become 1 (a factor of 0 would make NaN of -inf).
      float qe = qf;
      if (!whole) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          float s[16];
          uint32_t u[16];
          tc::tmem_ld16(t_s + 16 * c, s);
          const float4 mt = meta[c];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = k0 + 16 * c + i;
            const float x = fmaf(s[i], mt.x * qf, mt.y);
            u[i] = mt.x < 0.f || key < klo || key >= khi ? 0xFF800000u : __float_as_uint(x);
          }
          tm_st16(t_s + 16 * c, u);
        }
        tm_st_wait();
        __syncwarp();
        if (lane < 8) meta[lane].x = 1.f, meta[lane].y = 0.f;
        __syncwarp();
        qe = 1.f;
      }
      // the maximum of a 16-key group: of its raw scores, then its factor and magnitude
      auto group_top = [&](const uint32_t *s, float4 mt, float &top) {
        float t = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; i += 2) t = max3(t, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        if (t > -INFINITY) top = fmaxf(top, fmaf(t, mt.x * qe, mt.y));
      };
      // its weights, their sum, and what they add to the row's
      auto group_weights = [&](const uint32_t *s, float4 mt, float m0, uint32_t *p, float &l) {
        const float f = mt.x * qe, off = mt.y - m0;
        const uint64_t f2 = pack2(f, f), off2 = pack2(off, off);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 e = unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), f2, off2));
          const float x0 = ex2_approx(e.x), x1 = ex2_approx(e.y);
          sum = add2(sum, pack2(x0, x1));
          p[i] = F16::from_f32x2(x0, x1);
        }
        const float2 both = unpack2(sum);
        l = fmaf(both.x + both.y, mt.z, l);
        return both.x + both.y;
      };
      if (NQ == 2 && whole && j > 0) {
        // One pass: the weights to the reference as it is, in registers.  No weight is more than the sum of
        // its group; only where a row has one above 65504, or has no reference yet, does the warp do
        // the tile again (its scores are still there).
        const float m0 = m == -INFINITY ? 0.f : m;
        uint32_t p[64];
        float sum = 0.f, most = 0.f;
        for_columns<16, 4>(t_s, [&](int c, const uint32_t *s) {
          most = fmaxf(most, group_weights(s, meta[c], m0, p + 8 * c, sum));
        });
        if (!__any_sync(~0u, most > 65504.f || m == -INFINITY)) {
          l += sum;
#pragma unroll
          for (int i = 0; i < 64; i += 8) tm_st8(t_s + i, p + i);
          tm_st_wait();
          tc::tc_fence_before();
          tc::mbar_arrive(p_full_w);
          continue;
        }
      }
      float top = -INFINITY;
      for_columns<P::COLS>(t_s, [&](int c, const uint32_t *s) {
#pragma unroll
        for (int g = 0; g < P::COLS / 16; ++g)
          group_top(s + 16 * g, meta[c * (P::COLS / 16) + g], top);
      });
      // move the reference?  (the first tile sets it: O is not there yet)
      if (NQ == 1) {  // the other group's last tile has decided
        if (j > 0) {
          if (!(ok = wait_warp(m_full + 8 * (wg ^ 1), ((j - 1) >> 1) & 1, abort_flag, err))) break;
          const float held = s_max[r];
          if (held != m) {
            l = m == -INFINITY ? 0.f : Moved(m, held).sum(l);
            m = held;
          }
        }
      }
      const bool move = top > m + P::MOVE || (m == -INFINITY && top > m);
      if (__any_sync(~0u, move)) {
        const float now = move ? top - (float)kBias : m;
        const Moved by(move ? m : 0.f, move ? now : 0.f);
        const float f = by.factor();
        l = by.sum(l);
        m = now;
        if (NQ == 1) s_max[r] = m;
        if (j > 0) {
          // O is only touched between the product of the last tile and that of this one
          if (!(ok = wait_pv(j - 1))) break;
          tc::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tm_ld32(t_o + 32 * c, o);
            uint32_t u[16], w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              u[i] = __float_as_uint(o[i] * f);
              w[i] = __float_as_uint(o[16 + i] * f);
            }
            tm_st16(t_o + 32 * c, u);
            tm_st16(t_o + 32 * c + 16, w);
          }
        }
      }
      if (NQ == 1) tc::mbar_arrive(m_full + 8 * wg);
      const float m0 = m == -INFINITY ? 0.f : m;
      for_columns<P::COLS>(t_s, [&](int c, const uint32_t *s) {
        uint32_t p[P::COLS / 2];
#pragma unroll
        for (int g = 0; g < P::COLS / 16; ++g)
          group_weights(s + 16 * g, meta[c * (P::COLS / 16) + g], m0, p + 8 * g, l);
#pragma unroll
        for (int i = 0; i < P::COLS / 2; i += 8) tm_st8(t_s + c * (P::COLS / 2) + i, p + i);
      });
      tm_st_wait();
      tc::tc_fence_before();
      tc::mbar_arrive(p_full_w);
    }
    if (NQ == 1) {
      // the two groups' sums, to the common maximum
      s_ml[wg][r] = make_float2(m, l);
      asm volatile("bar.sync 2, 256;" ::: "memory");
      const float2 x = s_ml[0][r], y = s_ml[1][r];
      m = fmaxf(x.x, y.x);
      l = (x.x == -INFINITY ? x.y : Moved(x.x, m).sum(x.y)) + (y.x == -INFINITY ? y.y : Moved(y.x, m).sum(y.y));
    }
    if (ok && j_end > 0) ok = wait_pv(j_end - 1);
    tc::tc_fence_after();
    if (ok && it.n > 0 && (NQ == 1 || wg < nq)) {
      // the row saw nothing (O may not exist); a row of NaN has no maximum, but a sum of NaN
      const bool none = tiles == 0 || l == 0.f;
      if (!none && m == -INFINITY) m = 0.f;
      const int c0 = NQ == 2 ? 0 : wg * (D / 64), c1 = NQ == 2 ? D / 32 : c0 + D / 64;
      const bool first = NQ == 2 || wg == 0;
      if (splits > 1) {
        const int64_t at = part * P::ROWS + (NQ == 2 ? wg * kRows : 0) + r;
        float *dst = a.part + at * D;
        if (tiles > 0) {
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float o[32];
            tm_ld32(t_o + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4 *>(dst + 32 * c)[i] =
                  make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (first) a.ml[at] = make_float2(none ? -INFINITY : m, none ? 0.f : l);
      } else {
        const float f = none ? 0.f : out_scale(kBias) / l;
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * a.o_ts + (int64_t)head * a.o_hs);
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float o[32];
          if (tiles > 0) tm_ld32(t_o + 32 * c, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = none ? 0.f : o[8 * i + k] * f;
            if (live) dst[4 * c + i] = bf16 ? pack8<Bf16>(e) : pack8<F16>(e);
          }
        }
        if (a.lse && live && first)
          a.lse[row * a.kv_heads * a.group + head] =
              none ? -INFINITY : row_lse(m, l, kBias);
      }
    }
    tc::tc_fence_before();
  } else if (warp < 8 + P::CW) {
    // ======================================================================== codes -> operands
    const int w = warp & 3;
    // K: this warp's 32 keys; a load covers 8 keys by 64 elements (an atom: 128 bytes of fp16 a key)
    constexpr int ATOMS = D / 64;
    // V: 64 keys by 16 VW elements a unit; lane (tg, dg) holds the VW words of 8 tokens (group tg)
    constexpr int VU = D / (16 * P::VW) * 2 / 4;  // units a warp
    // of elements dg.  Eight lanes load two tokens' 64 bytes; for each 16-byte store of eight tokens
    // they hold the token groups t and t + 4 and the rows 4k + (e ^ dg): the swizzled chunks
    // {t, t + 4} ^ {e ^ dg} are eight different ones.
    const int tg = (lane >> 2 & 1) * 4 + (lane >> 3), dg = lane & 3;
    const uint32_t pair0 = dg | (4 + dg) << 4 | (dg ^ 1) << 8 | (4 + (dg ^ 1)) << 12;  // bytes dg, dg ^ 1
    const uint32_t pair1 = (dg ^ 2) | (4 + (dg ^ 2)) << 4 | (dg ^ 3) << 8 | (4 + (dg ^ 3)) << 12;
    // A page's codes beyond the sequence's end are loaded as they are, and page 0 in the place of one
    // that is not there: their scores are hidden, so their weights are 0.  Nothing is selected after
    // a load, which would wait for it.
    const int8_t *ksrc[2];  // the keys of this warp's two groups in the next tile
    auto find_k = [&](int j, int raw) {
      const int pages = check_page(B, raw, a.hdr);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int pg = max(__shfl_sync(~0u, pages, 2 * w + g), 0);
        const int in_page = (key0 + j * kKeys + 32 * w + 16 * g) & (B.page - 1);
        ksrc[g] = a.k + (((int64_t)pg * a.kv_heads + h) * B.page + in_page + (lane >> 2)) * D + (lane & 3) * 16;
      }
    };
    auto load_k = [&](uint4 (&kr)[4], int atom) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        kr[i] = __ldg(reinterpret_cast<const uint4 *>(ksrc[i >> 1] + (i & 1) * 8 * D + atom * 64));
    };
    auto store_k = [&](const uint4 (&kr)[4], uint8_t *atom) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 32 * w + 8 * i + (lane >> 2), c = 2 * (lane & 3);
        const uint32_t u[4] = {kr[i].x ^ 0x80808080u, kr[i].y ^ 0x80808080u, kr[i].z ^ 0x80808080u,
                               kr[i].w ^ 0x80808080u};
        // 8 lanes: two rows, an even and an odd one, whose four chunks fall into 8 bank groups
        *reinterpret_cast<uint4 *>(atom + tc::sw128(row, c)) =
            make_uint4(codes_f16(u[0], kPickLo), codes_f16(u[0], kPickHi), codes_f16(u[1], kPickLo), codes_f16(u[1], kPickHi));
        *reinterpret_cast<uint4 *>(atom + tc::sw128(row, c + 1)) =
            make_uint4(codes_f16(u[2], kPickLo), codes_f16(u[2], kPickHi), codes_f16(u[3], kPickLo), codes_f16(u[3], kPickHi));
      }
    };
    const int8_t *vsrc[VU];
    auto find_v = [&](int j, int raw) {
      const int pages = check_page(B, raw, a.hdr);
#pragma unroll
      for (int u = 0; u < VU; ++u) {
        const int unit = w * VU + u, half = unit & 1, d0 = (unit >> 1) * 16 * P::VW + dg * 4 * P::VW;
        const int pg = max(__shfl_sync(~0u, pages, half * 4 + (tg >> 1)), 0);
        const int in_page = (key0 + j * kKeys + half * 64 + tg * 8) & (B.page - 1);
        vsrc[u] = a.v + (((int64_t)pg * a.kv_heads + h) * B.page + in_page) * D + d0;
      }
    };
    auto load_v = [&](uint32_t (&vr)[8][P::VW], const int8_t *src) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (P::VW == 4) {
          const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src + i * D));
          vr[i][0] = x.x, vr[i][1] = x.y, vr[i][P::VW - 2] = x.z, vr[i][P::VW - 1] = x.w;
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src + i * D));
          vr[i][0] = x.x, vr[i][1] = x.y;
        }
      }
    };
    auto store_v = [&](const uint32_t (&vr)[8][P::VW], int u, uint8_t *buf) {
      const int unit = w * VU + u, half = unit & 1, d0 = (unit >> 1) * 16 * P::VW + dg * 4 * P::VW;
      uint8_t *atom = buf + half * (D * 128);
#pragma unroll
      for (int k = 0; k < P::VW; ++k) {
        uint32_t z[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e % 2 == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              z[i][e >> 1] = __byte_perm(vr[2 * i][k], vr[2 * i + 1][k], e ? pair1 : pair0) ^ 0x80808080u;
          }
          const uint32_t pick = e & 1 ? kPickHi : kPickLo;
          *reinterpret_cast<uint4 *>(atom + tc::sw128(d0 + 4 * k + (e ^ dg), tg)) =
              make_uint4(codes_f16(z[0][e >> 1], pick), codes_f16(z[1][e >> 1], pick),
                         codes_f16(z[2][e >> 1], pick), codes_f16(z[3][e >> 1], pick));
        }
      }
    };
    // A buffer's n-th contents may be written once the product that read the last ones is done.
    auto free_wait = [&](uint32_t b, int n) {
      return n == 0 || wait_warp(b, (n - 1) & 1, abort_flag, err);
    };
    auto publish = [&](uint32_t b) {
      tc::fence_proxy_async();
      tc::mbar_arrive(b);
    };
    const int page0 = page_of(0, lane & 7);
    int page = page_of(1, lane & 7);
    if constexpr (NQ == 2) {
      // two buffers of whole tiles, the same warps for keys and values
      uint4 kr[ATOMS][4];
      uint32_t vr[VU][8][P::VW];
      find_k(0, page0);
      find_v(0, page0);
#pragma unroll
      for (int i = 0; i < ATOMS; ++i) load_k(kr[i], i);
#pragma unroll
      for (int u = 0; u < VU; ++u) load_v(vr[u], vsrc[u]);
      for (int j = 0; j < tiles; ++j) {
        const int next = page_of(j + 2, lane & 7), b = j & 1;
        find_k(j + 1, page);
        find_v(j + 1, page);
        if (!free_wait(k_free + 8 * b, j >> 1)) break;
#pragma unroll
        for (int i = 0; i < ATOMS; ++i) {
          store_k(kr[i], mem + kAt + b * P::TILE + i * (kKeys * 128));
          load_k(kr[i], i);
        }
        publish(k_full + 8 * b);
        if (!free_wait(v_free + 8 * b, j >> 1)) break;
#pragma unroll
        for (int u = 0; u < VU; ++u) {
          store_v(vr[u], u, mem + vAt + b * P::TILE);
          load_v(vr[u], vsrc[u]);
        }
        publish(v_full + 8 * b);
        page = next;
      }
    } else if (warp < 12) {
      // one buffer of K, whose four atoms come free and are filled one after the other; the next
      // tile's codes are under way
      uint4 kr[ATOMS][4];
      find_k(0, page0);
#pragma unroll
      for (int i = 0; i < ATOMS; ++i) load_k(kr[i], i);
      bool ok = true;
      for (int j = 0; j < tiles && ok; ++j) {
        const int next = page_of(j + 2, lane & 7);
#pragma unroll
        for (int i = 0; i < ATOMS; ++i) {
          ok = ok && free_wait(k_free + 8 * i, j);
          if (!ok) break;
          store_k(kr[i], mem + kAt + i * (kKeys * 128));
          publish(k_full + 8 * i);
          if (i == 0) find_k(j + 1, page);
          load_k(kr[i], i);
        }
        page = next;
      }
    } else {
      // one buffer of V, in halves of 64 keys; the other half's codes are under way
      uint32_t vr[8][P::VW];
      find_v(0, page0);
      load_v(vr, vsrc[0]);
      bool ok = true;
      for (int j = 0; j < tiles && ok; ++j) {
        const int next = page_of(j + 2, lane & 7);
#pragma unroll
        for (int u = 0; u < VU; ++u) {
          ok = ok && free_wait(v_free + 8 * u, j);
          if (!ok) break;
          store_v(vr, u, mem + vAt);
          publish(v_full + 8 * u);
          if (u == VU - 1) find_v(j + 1, page);
          load_v(vr, vsrc[(u + 1) % VU]);
        }
        page = next;
      }
    }
  } else {
    // ======================================================================== products
    // the group of the issuing warp (three of its warps have no work) hands registers to the softmax
    if (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::ISSUE_REGS));
    if (warp == 8 + P::CW) {
      asm volatile("bar.sync 1, 288;" ::: "memory");
      bool ok = true;
      auto wait = [&](uint32_t b, int phase) { ok = ok && wait_warp(b, phase & 1, abort_flag, err); };
      // S slot = Q(q) K^T over the elements [64 first, 64 last) of a K buffer
      auto qk = [&](uint32_t sk, int q, int slot, int first, int last) {
        if (!ok) return;
        tc::tc_fence_after();
        const uint32_t sq = base + q * P::TILE;
#pragma unroll
        for (int ks = 4 * first; ks < 4 * last; ++ks) {
          const uint32_t off = (ks >> 2) * (kKeys * 128) + (ks & 3) * 32;
          tc::mma_bf16_warp(tmem + 128 * slot, tc::desc_k128_sw128(sq + off), tc::desc_k128_sw128(sk + off),
                            idesc_f16(kKeys), ks > 0);
        }
      };
      // O(q) += P slot V over the keys [64 first, 64 last) of a V buffer
      auto pv = [&](uint32_t sv, int q, int slot, int first, int last, bool fresh) {
        if (!ok) return;
        tc::tc_fence_after();
#pragma unroll
        for (int ks = 4 * first; ks < 4 * last; ++ks) {
          const uint32_t off = (ks >> 2) * (D * 128) + (ks & 3) * 32;
          tc::mma_bf16_ts_warp(tmem + 256 + q * D, tmem + 128 * slot + 8 * ks, tc::desc_k128_sw128(sv + off),
                               idesc_f16(D), !fresh || ks > 0);
        }
      };
      auto commit = [&](uint32_t b) {
        if (ok) tc::mma_commit_warp(b);
      };
      if constexpr (NQ == 2) {
        // the two row tiles take turns: while one's weights are computed the other's products run
        if (tiles > 0) {
          wait(k_full, 0);
          for (int q = 0; q < nq; ++q) {
            qk(base + kAt, q, q, 0, D / 64);
            commit(s_full + 8 * q);
          }
          commit(k_free);
        }
        for (int j = 0; j < tiles && ok; ++j) {
          const int b = j & 1;
          wait(v_full + 8 * b, j >> 1);
          for (int q = 0; q < nq; ++q) {
            wait(p_full + 8 * q, j);
            pv(base + vAt + b * P::TILE, q, q, 0, 2, j == 0);
            commit(pv_done + 8 * q);
            if (q == nq - 1) commit(v_free + 8 * b);
            if (j + 1 < tiles) {
              if (q == 0) wait(k_full + 8 * (b ^ 1), (j + 1) >> 1);
              wait(pv_done + 8 * q, j);  // S takes the columns of P
              qk(base + kAt + (b ^ 1) * P::TILE, q, q, 0, D / 64);
              commit(s_full + 8 * q);
              if (q == nq - 1) commit(k_free + 8 * (b ^ 1));
            }
          }
        }
      } else {
        // the next tile's scores are computed under this one's softmax, in the other slot; K's atoms
        // and V's halves are given back as soon as they have been read
        auto scores = [&](int j) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            wait(k_full + 8 * i, j);
            qk(base + kAt, 0, j & 1, i, i + 1);
            commit(k_free + 8 * i);
          }
          commit(s_full + 8 * (j & 1));
        };
        if (tiles > 0) scores(0);
        for (int j = 0; j < tiles && ok; ++j) {
          if (j + 1 < tiles) {
            if (j > 0) wait(pv_done + 8 * ((j - 1) & 1), (j - 1) >> 1);  // that slot's weights have been used
            scores(j + 1);
          }
          wait(p_full + 8 * (j & 1), j >> 1);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            wait(v_full + 8 * u, j);
            pv(base + vAt, 0, j & 1, u, u + 1, j == 0);
            commit(v_free + 8 * u);
          }
          commit(pv_done + 8 * (j & 1));
        }
      }
      // nothing of this warp's products is in flight when the tensor memory is given back
      tc::mma_commit_warp(drain);
      int left = 0;
      tc::wait_bar(drain, 0, &left, err);
      tc::tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------------------- join
// A warp takes a row of a split item: the splits in order.
template <int D>
__global__ void __launch_bounds__(256) kv8_prompt_join_kernel(AttnArgs a, int bf16, int splits) {
  constexpr int ROWS = PromptShape<D>::ROWS;
  pdl_wait();
  const int item = blockIdx.x, r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int4 j = a.jobs[item];
  const int rr = j.w * ROWS + r, tok = rr / a.group;
  if (tok >= j.y) return;
  const int head = j.z * a.group + rr - tok * a.group;
  const int64_t row = j.x + tok;
  float top = -INFINITY, den = 0.f;
  for (int s = 0; s < splits; ++s)
    top = fmaxf(top, a.ml[((int64_t)item * splits + s) * ROWS + r].x);
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  for (int s = 0; s < splits; ++s) {
    const int64_t at = ((int64_t)item * splits + s) * ROWS + r;
    const float2 ml = a.ml[at];
    if (ml.x == -INFINITY) continue;  // its output was not written
    const Moved by(ml.x, top);
    const float f = by.factor();
    den += by.sum(ml.y);
    const float2 *src = reinterpret_cast<const float2 *>(a.part + at * D) + lane;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 u = src[32 * i];
      acc[2 * i] = fmaf(u.x, f, acc[2 * i]);
      acc[2 * i + 1] = fmaf(u.y, f, acc[2 * i + 1]);
    }
  }
  const float f = top == -INFINITY ? 0.f : 1.f / den;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] *= out_scale(kBias);
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + row * a.o_ts + (int64_t)head * a.o_hs) + lane;
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    dst[32 * i] = bf16 ? Bf16::from_f32x2(acc[2 * i] * f, acc[2 * i + 1] * f)
                       : F16::from_f32x2(acc[2 * i] * f, acc[2 * i + 1] * f);
  if (a.lse && lane == 0)
    a.lse[row * a.kv_heads * a.group + head] =
        top == -INFINITY ? -INFINITY : row_lse(top, den, kBias);
}

// ----------------------------------------------------------------------------- launches
PromptPlan prompt_plan(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int q_heads, int window) {
  PromptPlan p = {};
  const int64_t group = q_heads / C.kv_heads, D = C.head_dim;
  const int64_t R = kRows * (D == 256 ? 1 : 2);
  // row tiles: every sequence's last one may be partly filled
  const int64_t rows = std::min<int64_t>(T * group / R + std::min(b.batch, T),
                                         std::min<int64_t>(b.batch, T) * ((b.max_q * group + R - 1) / R));
  const int64_t items = std::max<int64_t>(1, rows) * C.kv_heads;
  if (items > INT32_MAX) return p;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  // key tiles of a row tile, by the host's bounds
  const int64_t all = (b.max_kv + 16LL + kKeys - 1) / kKeys, per_seq = (b.max_q * group + R - 1) / R * C.kv_heads;
  const int64_t tiles = window ? std::min(all, (window + R / group + 17 + kKeys - 1) / kKeys + 1) : all;
  // The keys are split too with few row tiles, so that every SM has a share, of two tiles at least
  // (1568 tokens of one head in a window of 439: 30 us in shares of four tiles or more, 24 of two, 21 of
  // one; 300 tokens of 32 / 8 heads: 17.5 of two, 22 of one); and where one sequence fills the SMs and
  // the last round of blocks would leave most of them idle: 512 row tiles of 256 key tiles are four rounds on 152 SMs, the last a third full, and in halves seven rounds
  // of half the length (2.08 -> 1.95 ms; a share costs its block's start and a write and read of its
  // output, about four key tiles).  Otherwise ragged lengths even themselves out, and more shares
  // than SMs were slower: 9 sequences of 49 tokens after up to 42,909, 5 heads of 128: 66 us with one
  // share an SM, 67, 73 and 86 with two, three and four; 85 of 7 tokens after up to 2576, 32 / 2 heads
  // of 256: 80 whole, 93 in halves.
  // parts in the workspace: more than an SM's each only where the second rule can come to it
  const int64_t most = items < sms || per_seq < sms ? sms : 8 * sms;
  auto time = [&](int64_t n) { return (items * n + sms - 1) / sms * (tiles / (double)n + 4); };
  p.items = (int)items;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(sms / items, tiles / 2));
  if (per_seq >= sms)
    for (int64_t n = 2; n <= tiles / 4 && items * n <= most; ++n)
      if (time(n) < 0.97 * time(p.splits)) p.splits = (int)n;
  // The space is that of the most parts, so that a workspace serves smaller calls too.
  size_t off = kAlign;
  p.off_jobs = off;
  off = align_up(off + most * sizeof(int4));
  p.off_ml = off;
  off = align_up(off + most * R * sizeof(float2));
  p.off_part = off;
  p.total = all >= 4 ? align_up(off + (size_t)most * R * D * sizeof(float)) : kAlign;
  return p;
}

template <int D>
static cudaError_t launch_prompt_dim(const AttnArgs &a, const PromptPlan &p, int bf16, cudaStream_t st) {
  using P = PromptShape<D>;
  static std::atomic<bool> allowed[64];
  cudaError_t e = allow_smem<P::SMEM>(kv8_prompt_kernel<D>, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv8_prompt_kernel<D>, dim3(p.items, p.splits), dim3(P::THREADS), P::SMEM, st, a, bf16, p.splits);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(kv8_prompt_join_kernel<D>, dim3(p.items, P::ROWS / 8), dim3(256), 0, st, a, bf16, p.splits);
}

cudaError_t launch_prompt(const AttnArgs &args, const PromptPlan &p, int D, int bf16, uint8_t *ws,
                          cudaStream_t st) {
  AttnArgs a = args;
  a.jobs = reinterpret_cast<int4 *>(ws + p.off_jobs);
  a.ml = reinterpret_cast<float2 *>(ws + p.off_ml);
  a.part = reinterpret_cast<float *>(ws + p.off_part);
  if (D == 64) return launch_prompt_dim<64>(a, p, bf16, st);
  if (D == 128) return launch_prompt_dim<128>(a, p, bf16, st);
  return launch_prompt_dim<256>(a, p, bf16, st);
}

}  // namespace lq4
