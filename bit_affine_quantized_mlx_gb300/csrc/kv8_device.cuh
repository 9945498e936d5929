// Device helpers shared by the attention operators: 16-bit types, ragged batches, pages.
#pragma once
#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace lq4 {

// Wait for the kernel before this one on the stream.  (Letting the next kernel's blocks in early was
// tried: they took places from this one's and gained nothing.)
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ----------------------------------------------------------------------------- 16-bit types
struct Bf16 {
  static __device__ __forceinline__ float2 to_f32x2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t from_f32x2(float lo, float hi) {
    __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&r);
  }
};
struct F16 {
  static __device__ __forceinline__ float2 to_f32x2(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2 *>(&v));
  }
  static __device__ __forceinline__ uint32_t from_f32x2(float lo, float hi) {
    __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&r);
  }
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = T::to_f32x2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(T::from_f32x2(f[0], f[1]), T::from_f32x2(f[2], f[3]), T::from_f32x2(f[4], f[5]),
                    T::from_f32x2(f[6], f[7]));
}

// Two fp32 numbers in one instruction: half the issue slots of products and sums.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ----------------------------------------------------------------------------- ragged batches
struct Batch {
  const int32_t *table, *q_start, *kv_len;
  int table_pages, batch, max_q, max_kv, T;
  int page, page_shift, n_pages;
};

struct Seq {
  int row0, n, len;  // first row, rows, cached tokens (the rows' own included); n = 0: nothing to do
};

__device__ __forceinline__ void record_index_error(int32_t *hdr) { hdr[kHdrIndexError] = 1; }

// Lengths and row range of sequence b; one that is out of bounds has no rows and is recorded.
__device__ __forceinline__ Seq load_seq(const Batch &B, int b, int32_t *hdr) {
  const int r0 = __ldg(B.q_start + b), r1 = __ldg(B.q_start + b + 1), len = __ldg(B.kv_len + b);
  Seq s{r0, r1 - r0, len};
  if (r0 < 0 || r1 < r0 || r1 > B.T || r1 - r0 > B.max_q || len < 0 || len > B.max_kv) {
    record_index_error(hdr);
    s = Seq{0, 0, 0};
  }
  return s;
}

// The sequence whose row range holds row t (the last one that starts at or before t and is not
// empty); the caller checks that it does.
__device__ __forceinline__ int find_seq(const Batch &B, int t) {
  int lo = 0, hi = B.batch - 1;  // smallest b with q_start[b + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(B.q_start + mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The first key (or one before key 0) that a row at position p sees in a window, 0 for none.  Positions before
// the first, where there are more rows than tokens, are cut off: less a window near 2^31 they would wrap.
__device__ __forceinline__ int first_key(int p, int window) { return window ? max(p, 0) - window + 1 : 0; }

// Page number of entry i of sequence b, as it stands: checked where it is used (check_page), so that
// a load ahead of its use does not have to be waited for.
__device__ __forceinline__ int raw_page(const Batch &B, int b, int i) {
  return __ldg(B.table + (int64_t)b * B.table_pages + i);
}
constexpr int kNoPage = INT_MIN;  // a place without a token: nothing to record
// The page, or -1 (recorded) when it is none of the cache's.
__device__ __forceinline__ int check_page(const Batch &B, int p, int32_t *hdr) {
  if (p >= 0 && p < B.n_pages) return p;
  if (p != kNoPage) record_index_error(hdr);
  return -1;
}

// Arguments of both forms of lily_kv8_attention.
struct AttnArgs {
  Batch B;
  int32_t *hdr;
  const int8_t *k, *v;
  const float *k_amax, *v_amax;
  const uint16_t *q;
  uint16_t *out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  float *lse;
  int kv_heads, group, causal, window;
  float scale2;  // scale * log2(e) / 127
  int4 *jobs;    // items whose parts are joined by a second launch
  float2 *ml;    // [parts][rows of a tile]: running maximum and sum of a part
  float *part;   // [parts][rows of a tile][D]: unnormalised output
};

struct PromptPlan {
  int items, splits;  // row tiles times key/value heads (a bound), parts of their keys
  size_t off_jobs, off_ml, off_part, total;  // total 0: too many items
};
// The offsets and the total do not depend on the window.
PromptPlan prompt_plan(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int q_heads, int window);
cudaError_t launch_prompt(const AttnArgs &args, const PromptPlan &p, int D, int bf16, uint8_t *ws,
                          cudaStream_t st);

// Softmax weights.  fp16 has 15 octaves above 1 and loses what is below 2^-25, so a weight is
// 2^(x - m) with the reference m `bias` below the largest x seen: the smallest that counts is then
// 2^-(25 + bias) of the largest.  (With m the maximum itself, 262,144 keys 17.5 below one that carries little were
// all lost from the output: 5% of it.)  The sum adds w 2^(6 - bias) / a, a the page's magnitude of values:
// with a from 1e-30 to 3e38 and a million keys it and its reciprocal stay inside fp32's normal numbers.
constexpr float sum_scale(int bias) { return bias > 6 ? 1.f / (1 << (bias - 6)) : 1.f; }
// What turns sums of weights times codes, over the weights' sum, into outputs.
constexpr float out_scale(int bias) { return sum_scale(bias) / 127.f; }
// The log-sum-exp of a row from its reference and sum.
__device__ __forceinline__ float row_lse(float m, float sum, int bias) {
  return (m + (float)(bias - 6) + log2f(sum)) * 0.69314718056f;
}

// The magnitude that a page's values count with in the exponents.  What a page of zeros counts with does
// not matter to the output, but its weights have to stay in the sum: 2^(x - m) is 0 below 2^-126, so beside
// values of 6e4 all weights below 2^-24 of the largest were lost with 1e-30.  With 2^-80 they are there down
// to 2^-36 (prompt chunks; 2^-44 else), and values down to 1e-30 beside such a page still have full weights.
__device__ __forceinline__ float value_size(float a) {
  return a < 1e-30f ? (a == 0.f ? 0x1p-80f : 1e-30f) : a;
}

// A row's sum moved from reference m to now (not below it): half of the way twice, because the sum of
// pages that count as small can be as large as 2^(m - now) is small.
struct Moved {
  float half;
  __device__ __forceinline__ Moved(float m, float now) { asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(half) : "f"(0.5f * (m - now))); }
  __device__ __forceinline__ float factor() const { return half * half; }
  __device__ __forceinline__ float sum(float l) const { return l * half * half; }
};

// Two 8-bit codes of a word whose sign bits are flipped (u = q + 128), as halves: 0x6400 + u is
// the half 1024 + u, and subtracting 1152 leaves q, both exact.
__device__ __forceinline__ uint32_t codes_f16(uint32_t u, uint32_t pick) {
  uint32_t r = __byte_perm(u, 0x64646464u, pick);
  const uint32_t off = 0x64806480u;
  __half2 h = __hsub2(*reinterpret_cast<__half2 *>(&r), *reinterpret_cast<const __half2 *>(&off));
  return *reinterpret_cast<uint32_t *>(&h);
}
constexpr uint32_t kPickLo = 0x4140, kPickHi = 0x4342;  // bytes 0, 1 and bytes 2, 3

}  // namespace lq4
