// lily_kv8_attention, the form for many rows a sequence (prompt chunks): tcgen05 tiles.
//
// Bound by the tensor cores (4 * head_dim operations a visible query-key pair).  A block takes 128
// rows -- the group's heads of consecutive tokens of one key/value head, so that every code read
// serves all of them -- and walks its visible keys 128 at a time:
//   S = Q K^T (both in shared memory), P = 2^(S' - m) as fp16 written over S in tensor memory,
//   O += P V (P from tensor memory, V from shared memory), O in tensor memory throughout.
// Warps: 4 of softmax (a thread owns a row: its maximum and sum need no exchange), 4 (head_dim 256:
// 8) that turn codes into fp16 operands, 1 that issues the products.
//
// Operands.  K's codes keep their order; V's are transposed on the way (a lane holds 16 bytes of 8
// consecutive tokens, byte permutes interleave the tokens), so both are K-major tiles with the
// 128-byte swizzle, written without bank conflicts.  Codes of the next tile are in flight in
// registers while the current one is converted.  fp16 holds the codes exactly and q after a scaling
// by a power of two; the weights are rounded to fp16 relative to the largest weight-times-magnitude
// (see kv8_attention.cu for the magnitudes' place in the exponent).
//
// Layouts.  Head_dim 64 and 128: 256 TMEM columns a block (S 128, O 128) and two blocks an SM, whose
// softmax and products fall into each other's gaps.  Head_dim 256: one block an SM, O takes 256
// columns and S is held twice, so the next S is computed under the softmax of the current one.
//
// The running maximum moves only when a row's grows by more than 2^8 (weights up to 256 are as exact
// in fp16), because moving it rescales O in tensor memory.
#include <algorithm>

#include "kv8_device.cuh"
#include "tc_sm100.cuh"

namespace lq4 {

constexpr int kRows = 128, kKeys = 128;

template <int D>
struct PromptShape {
  static constexpr int SB = D == 256 ? 2 : 1;         // S buffers
  static constexpr int CW = D == 256 ? 8 : 4;         // converting warps
  static constexpr int THREADS = 32 * (4 + CW + 1);
  static constexpr int BLOCKS = D == 256 ? 1 : 2;     // of an SM
  static constexpr int COLS = D == 256 ? 512 : 256;   // of tensor memory
  static constexpr int TILE = kKeys * D * 2;          // bytes of a K or V tile (Q's too)
  static constexpr int VW = D == 64 ? 2 : 4;          // words of a token a lane holds of V
  static constexpr int SMEM = 3 * TILE + 1024;
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

// A bounded wait whose answer the whole warp shares: when one lane gives up they all leave together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *err) {
  return __all_sync(~0u, tc::wait_bar(bar, parity, abort_flag, err));
}

struct PromptItem {
  int row0, n, len;  // the sequence
  int h, rt;         // key/value head, row tile
  int lo, tiles;     // first key, key tiles
};

template <int D>
__global__ void __launch_bounds__(PromptShape<D>::THREADS, PromptShape<D>::BLOCKS)
    kv8_prompt_kernel(AttnArgs a, int bf16, int splits) {
  using P = PromptShape<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[8];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_count[P::THREADS / 32], s_found[2];
  __shared__ float4 s_meta[4][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *const mem = smem_raw + (base - tc::smem_u32(smem_raw));
  const uint32_t sq = base, sk = base + P::TILE, sv = base + 2 * P::TILE;
  const uint32_t bar = tc::smem_u32(s_bar);
  const uint32_t k_full = bar, v_full = bar + 8, pv_done = bar + 16, drain = bar + 24;
  const uint32_t s_full = bar + 32, p_full = bar + 48;  // [SB] each

  if (tid == 0) {
    s_abort = 0;
    s_found[0] = -1;
    const int kt = D == 256 ? 128 : 32 * P::CW, vt = kt;
    tc::mbar_init(k_full, kt);
    tc::mbar_init(v_full, vt);
    tc::mbar_init(pv_done, 1);
    tc::mbar_init(drain, 1);
    for (int i = 0; i < P::SB; ++i) {
      tc::mbar_init(s_full + 8 * i, 1);
      tc::mbar_init(p_full + 8 * i, 128);
    }
    tc::mbar_init_fence();
  }
  if (warp == 0) {
    tc::tmem_alloc(tc::smem_u32(&s_tmem), P::COLS);
    tc::tmem_relinquish();
  }
  pdl_wait();
  const Batch &B = a.B;
  int32_t *err = a.hdr + kHdrError;
  volatile int *abort_flag = &s_abort;

  // ---- which rows: the row tiles of all sequences, the last (in a causal chunk: the longest) first
  auto tiles_of = [&](int b) {
    if (b >= B.batch) return 0;
    const Seq s = load_seq(B, b, a.hdr);
    return (s.n * a.group + kRows - 1) / kRows;
  };
  int total = 0;
  for (int b0 = 0; b0 < B.batch; b0 += P::THREADS) {
    const int n = __reduce_add_sync(~0u, tiles_of(b0 + tid));
    if (lane == 0) s_count[warp] = n;
    __syncthreads();
    for (int w = 0; w < P::THREADS / 32; ++w) total += s_count[w];
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
      for (int w = 0; w < P::THREADS / 32; ++w) before += s_count[w];
      __syncthreads();
    }
  }
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  PromptItem it = {0, 0, 0, h, 0, 0, 0};
  if (s_found[0] >= 0) {
    const Seq s = load_seq(B, s_found[0], a.hdr);
    it.row0 = s.row0;
    it.n = s.n;
    it.len = s.len;
    it.rt = s_found[1];
    const int p_first = s.len - s.n + it.rt * kRows / a.group;
    const int p_last = s.len - s.n + min(s.n - 1, (it.rt * kRows + kRows - 1) / a.group);
    it.lo = a.window ? max(0, p_first - a.window + 1) & ~15 : 0;
    const int hi = a.causal ? min(p_last + 1, s.len) : s.len;
    it.tiles = max(0, (hi - it.lo + kKeys - 1) / kKeys);
  }
  const int b_seq = s_found[0];
  // this split's tiles
  const int t_begin = (int)((int64_t)it.tiles * split / splits);
  const int tiles = (int)((int64_t)it.tiles * (split + 1) / splits) - t_begin;
  const int key0 = it.lo + t_begin * kKeys, len = it.len;
  const int64_t part = (int64_t)blockIdx.x * splits + split;
  if (splits > 1 && split == 0 && tid == 0)
    a.jobs[blockIdx.x] = make_int4(it.row0, it.n, h, it.rt);
  // page of 16-key group g of this split's tile j, or -1
  auto page_of = [&](int j, int g) {
    const int tok = key0 + j * kKeys + g * 16;
    return j < tiles && tok < len ? load_page(B, b_seq, tok >> B.page_shift, a.hdr) : -1;
  };

  if (warp < 4) {
    // ======================================================================== softmax
    const int r = tid, rr = it.rt * kRows + r;
    const int tok = rr / a.group, head = h * a.group + rr - tok * a.group;
    const bool live = tok < it.n;
    const int64_t row = it.row0 + tok;
    float qf = 0.f;
    {
      const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * a.q_ts + (int64_t)head * a.q_hs);
      float top = 0.f;
      if (live) {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          float f[8];
          if (bf16) unpack8<Bf16>(src[c], f);
          else unpack8<F16>(src[c], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
        }
      }
      const int e = top > 0.f ? min(max(ilogbf(top), -100), 100) : 14;
      const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - e) << 23), a.scale2);
      qf = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * fabsf(a.scale2);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live) {
          float f[8];
          if (bf16) unpack8<Bf16>(src[c], f);
          else unpack8<F16>(src[c], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= up;
          w = pack8<F16>(f);
        }
        *reinterpret_cast<uint4 *>(mem + (c >> 3) * (kRows * 128) + tc::sw128(r, c & 7)) = w;
      }
      tc::fence_proxy_async();
    }
    asm volatile("bar.sync 1, %0;" ::"n"(160) : "memory");  // q is there: softmax and issuing warps
    // visible keys of this row, and those that every live row of the warp sees
    const int pos = it.len - it.n + tok;
    const int klo = a.window ? pos - a.window + 1 : 0, khi = a.causal ? min(pos + 1, len) : len;
    const int all_lo = __reduce_max_sync(~0u, live ? klo : INT_MIN);
    const int all_hi = __reduce_min_sync(~0u, live ? khi : INT_MAX);
    const uint32_t t_row = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t t_o = t_row + 128 * P::SB;
    float m = -INFINITY, l = 0.f;
    int page = page_of(0, lane & 7);
    auto load_mag = [&](int pg) {
      if (pg < 0) return make_float2(-1.f, 0.f);
      const int64_t ph = (int64_t)pg * a.kv_heads + h;
      return make_float2(__ldg(a.k_amax + ph), __ldg(a.v_amax + ph));
    };
    float2 mag = load_mag(page);
    page = page_of(1, lane & 7);
    bool ok = true;
    for (int j = 0; j < tiles; ++j) {
      const int k0 = key0 + j * kKeys;
      const float va = mag.y < 1e-30f ? 1e-30f : mag.y;
      __syncwarp();
      if (lane < 8) s_meta[warp][lane] = make_float4(mag.x, __log2f(va), __frcp_rn(va), 0.f);
      const bool bad = __any_sync(~0u, mag.x < 0.f);
      const bool whole = !bad && k0 >= all_lo && k0 + kKeys <= all_hi;
      mag = load_mag(page);
      page = page_of(j + 2, lane & 7);
      const int sb = j % P::SB;
      ok = wait_warp(s_full + 8 * sb, (j / P::SB) & 1, abort_flag, err);
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t t_s = t_row + 128 * sb;
      // maximum: of a 16-key group's raw scores, then its factor and magnitude
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float s[32];
        tm_ld32(t_s + 32 * c, s);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float4 mt = s_meta[warp][2 * c + g];
          float t = -INFINITY;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) t = fmaxf(t, s[16 * g + i]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int key = k0 + 32 * c + 16 * g + i;
              if (key >= klo && key < khi && !(mt.x < 0.f)) t = fmaxf(t, s[16 * g + i]);
            }
          }
          if (t > -INFINITY) top = fmaxf(top, fmaf(t, mt.x * qf, mt.y));
        }
      }
      // move the running maximum?  (the first tile sets it: O is not there yet)
      const bool move = top > m + 8.f || (m == -INFINITY && top > m);
      if (__any_sync(~0u, move)) {
        const float now = move ? top : m;
        const float f = move ? ex2_approx(m - now) : 1.f;
        m = now;
        l *= f;
        if (j > 0) {
          if (P::SB > 1) {
            ok = wait_warp(pv_done, (j - 1) & 1, abort_flag, err);
            if (!ok) break;
            tc::tc_fence_after();
          }
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
      const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float s[32];
        uint32_t p[16];
        tm_ld32(t_s + 32 * c, s);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float4 mt = s_meta[warp][2 * c + g];
          const float f = mt.x * qf, off = mt.y - m0;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x = fmaf(s[16 * g + i], f, off);
            if (!whole) {
              const int key = k0 + 32 * c + 16 * g + i;
              if (key < klo || key >= khi || mt.x < 0.f) x = -INFINITY;
            }
            s[16 * g + i] = ex2_approx(x);
            sum += s[16 * g + i];
          }
          l = fmaf(sum, mt.z, l);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            p[8 * g + i] = F16::from_f32x2(s[16 * g + 2 * i], s[16 * g + 2 * i + 1]);
        }
        tm_st16(t_s + 16 * c, p);
      }
      tm_st_wait();
      tc::tc_fence_before();
      tc::mbar_arrive(p_full + 8 * sb);
    }
    if (ok && tiles > 0) ok = wait_warp(pv_done, (tiles - 1) & 1, abort_flag, err);
    tc::tc_fence_after();
    if (ok && it.n > 0) {
      // the row saw nothing (O may not exist); a row of NaN has no maximum, but a sum of NaN
      const bool none = tiles == 0 || l == 0.f;
      if (!none && m == -INFINITY) m = 0.f;
      if (splits > 1) {
        float *dst = a.part + (part * kRows + r) * D;
        if (tiles > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tm_ld32(t_o + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4 *>(dst + 32 * c)[i] =
                  make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        a.ml[part * kRows + r] = make_float2(none ? -INFINITY : m, none ? 0.f : l);
      } else {
        const float f = none ? 0.f : 1.f / (127.f * l);
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * a.o_ts + (int64_t)head * a.o_hs);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
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
        if (a.lse && live)
          a.lse[row * a.kv_heads * a.group + head] =
              none ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
      }
    }
    tc::tc_fence_before();
  } else if (warp < 4 + P::CW) {
    // ======================================================================== codes -> operands
    constexpr bool BOTH = P::CW == 4;
    const int w = (warp - 4) & 3;
    const bool do_k = BOTH || warp < 8, do_v = BOTH || warp >= 8;
    // K: this warp's 32 keys; a load covers 512 bytes of consecutive codes
    constexpr int LPR = D / 16, RPL = 32 / LPR, KL = 32 / RPL;  // lanes a row, rows a load, loads
    // V: 64 keys by 16 VW elements a unit; lane (tg, dg) holds 8 tokens' VW words
    constexpr int VU = D / (16 * P::VW) * 2 / 4;                 // units a warp
    const int tg = lane & 7, dg = lane >> 3;
    uint4 kr[BOTH || D == 256 ? KL : 1];
    uint32_t vr[VU][8][P::VW];
    int page = page_of(0, lane & 7);
    auto load_k = [&](int j, int pages) {
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int row = i * RPL + lane / LPR, key = key0 + j * kKeys + 32 * w + row;
        const int pg = __shfl_sync(~0u, pages, 2 * w + (i * RPL >> 4));
        kr[i] = make_uint4(0, 0, 0, 0);
        if (pg >= 0 && key < len)
          kr[i] = __ldg(reinterpret_cast<const uint4 *>(
              a.k + (((int64_t)pg * a.kv_heads + h) * B.page + (key & (B.page - 1))) * D + (lane % LPR) * 16));
      }
    };
    auto load_v = [&](int j, int pages) {
#pragma unroll
      for (int u = 0; u < VU; ++u) {
        const int unit = w * VU + u, half = unit & 1, d0 = (unit >> 1) * 16 * P::VW + dg * 4 * P::VW;
        const int pg = __shfl_sync(~0u, pages, half * 4 + (tg >> 1));
        const int first = key0 + j * kKeys + half * 64 + tg * 8;
        const int8_t *src = a.v + (((int64_t)max(pg, 0) * a.kv_heads + h) * B.page + (first & (B.page - 1))) * D + d0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = pg >= 0 && first + i < len;
          if (P::VW == 4) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = __ldg(reinterpret_cast<const uint4 *>(src + i * D));
            vr[u][i][0] = x.x, vr[u][i][1] = x.y, vr[u][i][P::VW - 2] = x.z, vr[u][i][P::VW - 1] = x.w;
          } else {
            uint2 x = make_uint2(0, 0);
            if (in) x = __ldg(reinterpret_cast<const uint2 *>(src + i * D));
            vr[u][i][0] = x.x, vr[u][i][1] = x.y;
          }
        }
      }
    };
    if (do_k) load_k(0, page);
    if (do_v) load_v(0, page);
    page = page_of(1, lane & 7);
    for (int j = 0; j < tiles; ++j) {
      if (do_k) {
        if (j > 0 && !wait_warp(s_full + 8 * ((j - 1) % P::SB), ((j - 1) / P::SB) & 1, abort_flag, err))
          break;
#pragma unroll
        for (int i = 0; i < KL; ++i) {
          const int row = 32 * w + i * RPL + lane / LPR, mch = lane % LPR;
          const uint32_t u[4] = {kr[i].x ^ 0x80808080u, kr[i].y ^ 0x80808080u, kr[i].z ^ 0x80808080u,
                                 kr[i].w ^ 0x80808080u};
          const uint4 lo = make_uint4(codes_f16(u[0], kPickLo), codes_f16(u[0], kPickHi),
                                      codes_f16(u[1], kPickLo), codes_f16(u[1], kPickHi));
          const uint4 hi = make_uint4(codes_f16(u[2], kPickLo), codes_f16(u[2], kPickHi),
                                      codes_f16(u[3], kPickLo), codes_f16(u[3], kPickHi));
          // 8 lanes of a row: the second atom's four store their odd chunk first, so that the
          // eight 16-byte stores of a phase meet eight bank groups
          const bool odd = (mch >> 2) & 1;
          uint8_t *atom = mem + P::TILE + (mch >> 2) * (kKeys * 128);
          const int c = 2 * (mch & 3);
          *reinterpret_cast<uint4 *>(atom + tc::sw128(row, c + odd)) = odd ? hi : lo;
          *reinterpret_cast<uint4 *>(atom + tc::sw128(row, c + !odd)) = odd ? lo : hi;
        }
        tc::fence_proxy_async();
        tc::mbar_arrive(k_full);
        load_k(j + 1, page);
      }
      if (do_v) {
        if (j > 0 && !wait_warp(pv_done, (j - 1) & 1, abort_flag, err)) break;
#pragma unroll
        for (int u = 0; u < VU; ++u) {
          const int unit = w * VU + u, half = unit & 1, d0 = (unit >> 1) * 16 * P::VW + dg * 4 * P::VW;
          uint8_t *atom = mem + 2 * P::TILE + half * (D * 128);
#pragma unroll
          for (int k = 0; k < P::VW; ++k) {
            uint32_t z[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = vr[u][2 * i][k] ^ 0x80808080u, y = vr[u][2 * i + 1][k] ^ 0x80808080u;
              z[i][0] = __byte_perm(x, y, 0x5140);
              z[i][1] = __byte_perm(x, y, 0x7362);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t pick = e & 1 ? kPickHi : kPickLo;
              *reinterpret_cast<uint4 *>(atom + tc::sw128(d0 + 4 * k + e, tg)) =
                  make_uint4(codes_f16(z[0][e >> 1], pick), codes_f16(z[1][e >> 1], pick),
                             codes_f16(z[2][e >> 1], pick), codes_f16(z[3][e >> 1], pick));
            }
          }
        }
        tc::fence_proxy_async();
        tc::mbar_arrive(v_full);
        load_v(j + 1, page);
      }
      page = page_of(j + 2, lane & 7);
    }
  } else {
    // ======================================================================== products
    asm volatile("bar.sync 1, %0;" ::"n"(160) : "memory");
    const uint32_t t_o = tmem + 128 * P::SB;
    bool ok = true;
    auto issue_qk = [&](int j) {
      ok = ok && wait_warp(k_full, j & 1, abort_flag, err);
      if (!ok) return;
      tc::tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = (ks >> 2) * (kKeys * 128) + (ks & 3) * 32;
        tc::mma_bf16_warp(tmem + 128 * (j % P::SB), tc::desc_k128_sw128(sq + off),
                          tc::desc_k128_sw128(sk + off), idesc_f16(kKeys), ks > 0);
      }
      tc::mma_commit_warp(s_full + 8 * (j % P::SB));
    };
    if (P::SB > 1 && tiles > 0) issue_qk(0);
    for (int j = 0; j < tiles && ok; ++j) {
      // S(j + SB - 1) takes the columns of P(j - 1): that product has to be done
      if (j > 0) ok = ok && wait_warp(pv_done, (j - 1) & 1, abort_flag, err);
      if (P::SB == 1) issue_qk(j);
      else if (j + 1 < tiles) issue_qk(j + 1);
      ok = ok && wait_warp(v_full, j & 1, abort_flag, err);
      ok = ok && wait_warp(p_full + 8 * (j % P::SB), (j / P::SB) & 1, abort_flag, err);
      if (!ok) break;
      tc::tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < kKeys / 16; ++ks) {
        const uint32_t off = (ks >> 2) * (D * 128) + (ks & 3) * 32;
        tc::mma_bf16_ts_warp(t_o, tmem + 128 * (j % P::SB) + 8 * ks, tc::desc_k128_sw128(sv + off),
                             idesc_f16(D), j > 0 || ks > 0);
      }
      tc::mma_commit_warp(pv_done);
    }
    // nothing of this warp's products is in flight when the tensor memory is given back
    tc::mma_commit_warp(drain);
    int left = 0;
    tc::wait_bar(drain, 0, &left, err);
    tc::tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, P::COLS);
}

// ----------------------------------------------------------------------------- join
// A warp takes a row of a split item: the splits in order.
template <int D>
__global__ void __launch_bounds__(256) kv8_prompt_join_kernel(AttnArgs a, int bf16, int splits) {
  pdl_wait();
  const int item = blockIdx.x, r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int4 j = a.jobs[item];
  const int rr = j.w * kRows + r, tok = rr / a.group;
  if (tok >= j.y) return;
  const int head = j.z * a.group + rr - tok * a.group;
  const int64_t row = j.x + tok;
  float top = -INFINITY, den = 0.f;
  for (int s = 0; s < splits; ++s)
    top = fmaxf(top, a.ml[((int64_t)item * splits + s) * kRows + r].x);
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  for (int s = 0; s < splits; ++s) {
    const int64_t at = ((int64_t)item * splits + s) * kRows + r;
    const float2 ml = a.ml[at];
    if (ml.x == -INFINITY) continue;  // its output was not written
    const float f = ex2_approx(ml.x - top);
    den = fmaf(ml.y, f, den);
    const float2 *src = reinterpret_cast<const float2 *>(a.part + at * D) + lane;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 u = src[32 * i];
      acc[2 * i] = fmaf(u.x, f, acc[2 * i]);
      acc[2 * i + 1] = fmaf(u.y, f, acc[2 * i + 1]);
    }
  }
  const float f = top == -INFINITY ? 0.f : 1.f / (127.f * den);
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + row * a.o_ts + (int64_t)head * a.o_hs) + lane;
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    dst[32 * i] = bf16 ? Bf16::from_f32x2(acc[2 * i] * f, acc[2 * i + 1] * f)
                       : F16::from_f32x2(acc[2 * i] * f, acc[2 * i + 1] * f);
  if (a.lse && lane == 0)
    a.lse[row * a.kv_heads * a.group + head] =
        top == -INFINITY ? -INFINITY : (top + log2f(den)) * 0.69314718056f;
}

// ----------------------------------------------------------------------------- launches
PromptPlan prompt_plan(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int q_heads) {
  PromptPlan p = {};
  const int64_t group = q_heads / C.kv_heads, D = C.head_dim;
  // row tiles: every sequence's last one may be partly filled
  const int64_t rows = std::min<int64_t>(T * group / kRows + std::min(b.batch, T),
                                         std::min<int64_t>(b.batch, T) * ((b.max_q * group + kRows - 1) / kRows));
  const int64_t items = std::max<int64_t>(1, rows) * C.kv_heads;
  if (items > INT32_MAX) return p;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const int64_t slots = sms * (D == 256 ? 1 : 2), tiles = (b.max_kv + 16LL + kKeys - 1) / kKeys;
  // Few row tiles: the keys are split too, so that every SM has a share, of four tiles at least (a
  // share costs its block's start and a write and read of its output).
  p.items = (int)items;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(slots / items, tiles / 4));
  p.total = kAlign;
  if (p.splits > 1) {
    size_t off = kAlign;
    p.off_jobs = off;
    off = align_up(off + items * sizeof(int4));
    p.off_ml = off;
    off = align_up(off + items * p.splits * kRows * sizeof(float2));
    p.off_part = off;
    p.total = align_up(off + (size_t)items * p.splits * kRows * D * sizeof(float));
  }
  return p;
}

template <int D>
static cudaError_t launch_prompt_dim(const AttnArgs &a, const PromptPlan &p, int bf16, cudaStream_t st) {
  using P = PromptShape<D>;
  cudaError_t e = cudaFuncSetAttribute(kv8_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv8_prompt_kernel<D>, dim3(p.items, p.splits), dim3(P::THREADS), P::SMEM, st, a, bf16, p.splits);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(kv8_prompt_join_kernel<D>, dim3(p.items, kRows / 8), dim3(256), 0, st, a, bf16, p.splits);
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
