// lily_add_rms_norm, lily_mx_quantize and lily_mx_read: rows and their microscaled form.
//
// All three are bound by memory: each value is read once and written once in each form asked for.  A
// thread takes eight neighbours (16 bytes of a 16-bit row), so a block of 32 is in four neighbouring
// lanes and its largest magnitude takes two exchanges.
//
// Measured on one GB300: 8192 rows of 2048 with the addition and all outputs 26.0 us (5.8 TB/s, 85% of the measured copy rate);
// without the addition, to 8 bits alone, 18.7 us (2.7 TB/s: bound by the issue of some 30 instructions an element);
// one row 2.0 us (a launch).  151,936 x 2048 of bf16 to 4 bits 126 us (6.2 TB/s), back 114 us (6.9 TB/s).
#include <algorithm>

#include "mx_device.cuh"

namespace lq4 {

// ----------------------------------------------------------------------------- norm
//   s = round16(x + add);   y = round16(s / sqrt(mean(s^2) + eps) * (w + offset));   mx = quantised y
//
// The roundings to 16 bits are those of exact arithmetic: a rounding that falls the other way moves an 8-bit
// element by a whole step, and now and then a block's scale, so results would depend on how a row is
// shared out among threads.  What that takes, in pairs of fp32 numbers (hi + lo) rather than in fp64,
// whose rate here is a 64th:
//  - squares.  A sum T that starts above a thread's largest square takes each square as T' = fma(x, x, T); T' - T is
//    exact (T' <= 2 T), and what T' rounded off, fma(x, x, T - T'), is too, and has a sum of its own.  Four operations an
//    element, and at most 2^-39 of the row's sum lost (that is if all of up to 16 roundings go one way);
//  - the root gets one correction step;
//  - y is s * w * r in plain fp32, twice, a little below and a little above.  Only where these round to different numbers of
//    16 bits is it done again in pairs, hi going to the rounding as an odd number where there is a remainder, so
//    that no tie is made on the way.
struct NormArgs {
  const uint16_t *x, *add, *weight;
  uint16_t *sum, *y;
  uint8_t *codes, *scales;  // the microscaled form, or NULL
  int64_t x_ts, add_ts, sum_ts, y_ts;
  float eps, offset, inv_hi, inv_lo;  // 1 / H as a pair
  int T, H, bits;
};

struct Pair {
  float hi, lo;
};
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  float s, e;
  two_sum(a.hi, b.hi, s, e);
  e = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  Pair r;
  r.hi = __fadd_rn(s, e);
  r.lo = __fsub_rn(e, __fsub_rn(r.hi, s));
  return r;
}
// Sum over a warp, of numbers that are not negative: all in units of 2^-26 of the largest's power of two, as whole numbers of
// these and of 2^-24 of these, which two instructions add up (2^-45 of the sum is lost; pairs would take twelve instructions a
// step of five).
__device__ __forceinline__ Pair warp_total(Pair v) {
  const float hi = __fadd_rn(v.hi, v.lo), lo = __fsub_rn(v.lo, __fsub_rn(hi, v.hi));
  const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(fabsf(hi))) >> 23;
  if (top >= 255) return Pair{NAN, 0.f};
  const uint32_t up = min(279u - top, 253u);  // 2^(up - 127) times the largest is below 2^26
  const float by = __uint_as_float(up << 23), back = __uint_as_float((254 - up) << 23);
  const float h = __fmul_rn(hi, by);
  const int whole = __float2int_rn(h);
  const int part = __float2int_rn(__fmul_rn(__fmaf_rn(lo, by, __fsub_rn(h, __int2float_rn(whole))), 0x1p24f));
  const uint32_t sum = __reduce_add_sync(~0u, (uint32_t)whole);
  const float rest = __fmul_rn(__int2float_rn(__reduce_add_sync(~0u, part)), 0x1p-24f);
  const float most = __uint2float_rz(sum);
  return Pair{__fmul_rn(most, back), __fmul_rn(__fadd_rn(__uint2float_rn(sum - (uint32_t)most), rest), back)};
}
// 1 / sqrt(total / H + eps)
__device__ __forceinline__ Pair pair_rsqrt(Pair total, float eps, const NormArgs &a) {
  Pair m;
  m.hi = __fmul_rn(total.hi, a.inv_hi);
  m.lo = __fmaf_rn(total.hi, a.inv_hi, -m.hi);
  m.lo = __fmaf_rn(total.hi, a.inv_lo, __fmaf_rn(total.lo, a.inv_hi, m.lo));
  m = pair_add(m, Pair{eps, 0.f});
  // an even power of two goes to the end, so that the root's square has a remainder whatever eps is
  const int even = (max(1, (int)(__float_as_uint(m.hi) >> 23)) - 127) & ~1;
  const float by = __uint_as_float((uint32_t)(127 - even) << 23), back = __uint_as_float((uint32_t)(127 - even / 2) << 23);
  m.hi = __fmul_rn(m.hi, by), m.lo = __fmul_rn(m.lo, by);
  // r (1 + e / 2), e = 1 - m r^2: what is left is 3/8 e^2, 2^-43 at the root's accuracy of 2^-22
  const float r = rsqrtf(m.hi), r2 = __fmul_rn(r, r), r2_lo = __fmaf_rn(r, r, -r2);
  float e = __fmaf_rn(-m.hi, r2, 1.f);
  e = __fmaf_rn(-m.hi, r2_lo, __fmaf_rn(-m.lo, r2, e));
  return Pair{__fmul_rn(r, back), __fmul_rn(__fmul_rn(r, back), __fmul_rn(0.5f, e))};
}
// hi + lo as the fp32 number to round further: where hi is even and lo is not 0, hi's odd neighbour on lo's side.
// An odd number is no tie of a shorter format, and lies on the same side of each as hi + lo.
__device__ __forceinline__ float to_odd(float hi, float lo) {
  const uint32_t b = __float_as_uint(hi);
  if ((b & 1) || lo == 0.f) return hi;  // (a zero has no rest)
  return __uint_as_float((__float_as_uint(lo) ^ b) >> 31 ? b - 1 : b + 1);
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) { return fma2(b, pack2(-1.f, -1.f), a); }
// s * (w + offset) * r of eight elements, for a rounding to 16 bits that is the exact product's.
__device__ __forceinline__ void scale_exactly(float (&s)[8], const float (&w)[8], float offset, Pair r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float one, rest;
    two_sum(w[j], offset, one, rest);
    const float p = __fmul_rn(s[j], one);
    const float p_lo = __fmaf_rn(s[j], rest, __fmaf_rn(s[j], one, -p));
    const float hi = __fmul_rn(p, r.hi);
    const float lo = __fmaf_rn(p_lo, r.hi, __fmaf_rn(p, r.lo, __fmaf_rn(p, r.hi, -hi)));
    const float y = __fadd_rn(hi, lo);
    const float odd = to_odd(y, __fsub_rn(lo, __fsub_rn(y, hi)));
    s[j] = __uint_as_float(__float_as_uint(odd) | (__float_as_uint(hi) & 0x80000000u));  // (a sum of zeros loses it)
  }
}
// The same as 16-bit numbers, by plain fp32 products with a root a little smaller and one a little larger: rounding keeps the
// order, so where both round to the same number, all between them does.  With them 2^-22 away the exact product is between
// them: the root, its change and the last product are off by 2^-24 each.  w + offset and its product with s, where they
// are not exact (s * w has 22 bits at most), add as much, and 2^-21 covers that.
template <typename Ty>
__device__ __forceinline__ uint4 scale_eight(const uint4 &s, const uint4 &w, float offset, Pair r) {
  const float root = __fadd_rn(r.hi, r.lo), part = offset == 0.f ? 0x1p-22f : 0x1p-21f;
  const float less = __fmaf_rn(root, -part, root), more = __fmaf_rn(root, part, root);
  const uint64_t off = pack2(offset, offset), low = pack2(less, less), high = pack2(more, more);
  float a[8], b[8], y[8], z[8];
  unpack8<Ty>(s, a);
  unpack8<Ty>(w, b);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t p = mul2(pack2(a[j], a[j + 1]), add2(pack2(b[j], b[j + 1]), off));
    const float2 l = unpack2(mul2(p, low)), h = unpack2(mul2(p, high));
    y[j] = l.x, y[j + 1] = l.y, z[j] = h.x, z[j + 1] = h.y;
  }
  const uint4 one = pack8<Ty>(y), other = pack8<Ty>(z);
  if ((one.x ^ other.x) | (one.y ^ other.y) | (one.z ^ other.z) | (one.w ^ other.w)) {
    scale_exactly(a, b, offset, r);
    return pack8<Ty>(a);
  }
  return one;
}

// Where a sum of squares is out of what the pairs hold, the row is multiplied with a power of two, eps with its square, and
// summed again: the norm is the same, and bf16 holds such rows exactly, but for what is 2^-166 of the largest and less.
// In range nothing counts that fp32 cannot hold: what a square and its remainder lose is 2^-149 at most, of up to 2^15 squares
// 2^-54 of a sum of 2^-80 or, whatever the sum is, 2^-49 of an eps of 2^-100.  (Sums of fp16 squares are 2^-48 to 2^47.)  Large rows go
// to 2^40 instead of 1, so that their small elements do not run out of bits.  (What asking takes: 8192 rows of 2048 with all
// outputs 25.8 -> 26.0 us, to 8 bits alone 18.1 -> 18.7.)
__device__ __forceinline__ bool out_of_range(Pair total, float eps) {
  return !(total.hi < 0x1p100f) || (eps < 0x1p-100f && total.hi < 0x1p-80f);
}

// R threads a row (a warp or more), NV times eight elements each.
template <typename Ty, int NV>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(NormArgs a, int R) {
  constexpr bool kFar = std::is_same<Ty, Bf16>::value;  // rows that can be out_of_range
  __shared__ Pair s_part[32];
  pdl_wait();
  next_may_start();
  const int per = blockDim.x / R, in_row = threadIdx.x % R, which = threadIdx.x / R;
  const int64_t t = (int64_t)blockIdx.x * per + which;
  const bool here = t < a.T;
  const int vecs = a.H >> 3;
  uint4 raw[NV];
  uint32_t most = 0;  // the largest magnitudes, of even and of odd elements
  {
    uint4 more[NV];
    const uint4 *x = reinterpret_cast<const uint4 *>(a.x + (here ? t : 0) * a.x_ts);
    const uint4 *add = reinterpret_cast<const uint4 *>(a.add + (here ? t : 0) * a.add_ts);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = in_row + i * R;
      raw[i] = more[i] = make_uint4(0, 0, 0, 0);
      if (here && v < vecs) {
        raw[i] = x[v];
        if (a.add) more[i] = add[v];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = in_row + i * R;
      if (a.add) {
        float s[8], m[8];
        unpack8<Ty>(raw[i], s);
        unpack8<Ty>(more[i], m);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = __fadd_rn(s[j], m[j]);
        raw[i] = pack8<Ty>(s);
      }
      if (a.sum && here && v < vecs) reinterpret_cast<uint4 *>(a.sum + t * a.sum_ts)[v] = raw[i];
      most = __vmaxu2(most, largest_two(raw[i]));
    }
  }
  Pair total;
  float eps = a.eps;
  for (bool once = true;; once = false) {
    // a power of two, so that taking it off in the end is exact too
    const float top = __uint_as_float((__float_as_uint(largest_of<Ty>(most)) & 0x7F800000u) + 0x800000u), first = __fmul_rn(top, top);
    uint64_t sums = pack2(first, first), rest = 0;  // of even and of odd elements
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s[8];
      unpack8<Ty>(raw[i], s);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint64_t two = pack2(s[j], s[j + 1]), sum = fma2(two, two, sums);
        rest = add2(rest, fma2(two, two, sub2(sums, sum)));
        sums = sum;
      }
    }
    const float2 h = unpack2(sub2(sums, pack2(first, first))), l = unpack2(rest);
    total = warp_total(pair_add(Pair{h.x, l.x}, Pair{h.y, l.y}));
    bool far = kFar && once && out_of_range(total, eps);
    if (R > 32) {
      if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = total;
      if (kFar) far = __syncthreads_or(far);
      else __syncthreads();
      const int warps = R >> 5, places = 1 << (32 - __clz(warps - 1)), place = threadIdx.x & (places - 1);
      total = place < warps ? s_part[which * warps + place] : Pair{0.f, 0.f};
      for (int o = places / 2; o; o >>= 1)
        total = pair_add(total, Pair{__shfl_xor_sync(~0u, total.hi, o), __shfl_xor_sync(~0u, total.lo, o)});
    }
    if (!far) break;
    uint32_t biggest = __reduce_max_sync(~0u, max(most & 0xFFFFu, most >> 16));
    if (R > 32) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5].hi = __uint_as_float(biggest);
      __syncthreads();
      for (int w = 0; w < R >> 5; ++w) biggest = max(biggest, __float_as_uint(s_part[which * (R >> 5) + w].hi));
      __syncthreads();
    }
    // the exponent of the largest magnitude or of eps's root, whichever is larger, to 0 or (see out_of_range) to 40
    const int of_eps = eps > 0.f ? ((int)(__float_as_uint(eps) >> 23) - 126) >> 1 : -127, e = max((int)(biggest >> 7) - 127, of_eps);
    const float by = biggest >= 0x7F80u ? 1.f : __uint_as_float((uint32_t)(127 + (e > 0 ? 40 - e : min(126, -e))) << 23);
    eps = __fmul_rn(__fmul_rn(eps, by), by);
    most = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s[8];
      unpack8<Ty>(raw[i], s);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = __fmul_rn(s[j], by);
      raw[i] = pack8<Ty>(s);
      most = __vmaxu2(most, largest_two(raw[i]));
    }
  }
  const Pair r = pair_rsqrt(total, eps, a);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = in_row + i * R;
    const bool live = here && v < vecs;
    constexpr uint32_t ones = std::is_same<Ty, Bf16>::value ? 0x3F803F80u : 0x3C003C00u;
    const uint4 w = live && a.weight ? reinterpret_cast<const uint4 *>(a.weight)[v] : make_uint4(ones, ones, ones, ones);
    const uint4 y = scale_eight<Ty>(raw[i], w, a.weight ? a.offset : 0.f, r);
    if (a.y && live) reinterpret_cast<uint4 *>(a.y + t * a.y_ts)[v] = y;
    if (a.bits) {
      float s[8];
      unpack8<Ty>(y, s);
      const int64_t at = t * a.H + 8 * v;
      const uint32_t amax = largest8<Ty>(y);
      if (a.bits == 8) mx_store8<8>(s, amax, a.codes + at, a.scales + (at >> 5), live, (v & 3) == 0);
      else mx_store8<4>(s, amax, a.codes + (at >> 1), a.scales + (at >> 5), live, (v & 3) == 0);
    }
  }
}

template <typename Ty>
static cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
  const int vecs = a.H / 8, sms = std::max(1, sm_count());
  // Four vectors a thread where there are rows enough, two or one where there are few: whole warps a row, and whole rows a block
  // of 128 threads or more.  (8192 rows of 4096 with all outputs: 48 us with four vectors a thread, 54 with two;
  // to 8 bits alone 35 and 44: what a thread does once a row, the root and the sums' way to it, is a fifth of its instructions.)
  int nv = 4, R = 0;
  for (; nv >= 1; nv /= 2) {
    R = (vecs + 32 * nv - 1) / (32 * nv) * 32;
    if (nv == 1 || (int64_t)a.T * R >= (int64_t)sms * 1024 || 2 * R > 1024) break;
  }
  const int per = std::max(1, 128 / R);
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(per * R);
  if (nv == 4) return launch_pdl(add_rms_norm_kernel<Ty, 4>, grid, block, 0, st, a, R);
  if (nv == 2) return launch_pdl(add_rms_norm_kernel<Ty, 2>, grid, block, 0, st, a, R);
  return launch_pdl(add_rms_norm_kernel<Ty, 1>, grid, block, 0, st, a, R);
}

int launch_add_rms_norm(const lily_rms_norm &op, int T, const void *x, int64_t x_ts, const void *add,
                        int64_t add_ts, void *sum, int64_t sum_ts, void *y, int64_t y_ts, const lily_mx_mat *mx,
                        cudaStream_t st) {
  NormArgs a = {};
  a.x = static_cast<const uint16_t *>(x), a.x_ts = x_ts;
  a.add = static_cast<const uint16_t *>(add), a.add_ts = add_ts;
  a.sum = static_cast<uint16_t *>(sum), a.sum_ts = sum_ts;
  a.y = static_cast<uint16_t *>(y), a.y_ts = y_ts;
  a.weight = static_cast<const uint16_t *>(op.weight);
  if (mx) a.codes = mx->codes, a.scales = mx->scales, a.bits = mx->bits;
  a.eps = op.eps, a.offset = op.weight_offset;
  const double inv = 1.0 / op.width;
  a.inv_hi = (float)inv, a.inv_lo = (float)(inv - (double)a.inv_hi);
  a.T = T, a.H = op.width;
  const cudaError_t e = op.dtype == LILY_BF16 ? launch_norm<Bf16>(a, st) : launch_norm<F16>(a, st);
  return e == cudaSuccess ? LILY_Q4_OK : (cudaGetLastError(), LILY_Q4_ERR_CUDA);
}

// ----------------------------------------------------------------------------- to and from blocks
struct F32 {};
template <typename Ty>
struct Eight;  // eight neighbours of a row in memory
template <typename Ty>
struct Eight {
  using Elem = uint16_t;
  uint4 v;
  __device__ __forceinline__ void load(const Elem *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void floats(float (&f)[8]) const { unpack8<Ty>(v, f); }
  __device__ __forceinline__ uint32_t largest() const { return largest8<Ty>(v); }
  static __device__ __forceinline__ void store(Elem *p, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(p) = pack8<Ty>(f);
  }
};
template <>
struct Eight<F32> {
  using Elem = float;
  float4 v[2];
  __device__ __forceinline__ void load(const Elem *p) {
    v[0] = __ldcs(reinterpret_cast<const float4 *>(p)), v[1] = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    f[0] = v[0].x, f[1] = v[0].y, f[2] = v[0].z, f[3] = v[0].w;
    f[4] = v[1].x, f[5] = v[1].y, f[6] = v[1].z, f[7] = v[1].w;
  }
  __device__ __forceinline__ uint32_t largest() const {
    float f[8];
    floats(f);
    return largest8(f);
  }
  static __device__ __forceinline__ void store(Elem *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

struct MxArgs {
  void *x;  // rows, dense in themselves, ts elements apart
  int64_t ts, total;  // vectors of eight in all rows
  int vecs;           // and in one
  uint8_t *codes, *scales;
};
constexpr int kMxThreads = 256, kMxAhead = 4;

// Place of vector v in rows that are not dense as a whole.
__device__ __forceinline__ int64_t row_offset(const MxArgs &a, int64_t v) {
  if (a.ts == 8 * (int64_t)a.vecs) return 8 * v;
  const int64_t row = v / a.vecs;
  return row * a.ts + 8 * (v - row * a.vecs);
}

template <typename Ty, int BITS>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(MxArgs a) {
  using E = Eight<Ty>;
  pdl_wait();
  next_may_start();
  const auto *x = static_cast<const typename E::Elem *>(a.x);
  const int64_t base = (int64_t)blockIdx.x * (kMxThreads * kMxAhead) + threadIdx.x;
  E raw[kMxAhead];
#pragma unroll
  for (int i = 0; i < kMxAhead; ++i) {
    const int64_t v = base + i * kMxThreads;
    if (v < a.total) raw[i].load(x + row_offset(a, v));
    else raw[i] = E{};
  }
#pragma unroll
  for (int i = 0; i < kMxAhead; ++i) {
    const int64_t v = base + i * kMxThreads;
    float f[8];
    raw[i].floats(f);
    mx_store8<BITS>(f, raw[i].largest(), a.codes + v * BITS, a.scales + (v >> 2), v < a.total, (v & 3) == 0);
  }
}

template <typename Ty, int BITS>
__global__ void __launch_bounds__(kMxThreads) mx_read_kernel(MxArgs a) {
  using E = Eight<Ty>;
  pdl_wait();
  next_may_start();
  auto *x = static_cast<typename E::Elem *>(a.x);
  const int64_t base = (int64_t)blockIdx.x * (kMxThreads * kMxAhead) + threadIdx.x;
  uint2 raw[kMxAhead];
  uint32_t scale[kMxAhead];
#pragma unroll
  for (int i = 0; i < kMxAhead; ++i) {
    const int64_t v = base + i * kMxThreads;
    raw[i] = make_uint2(0, 0), scale[i] = 0;
    if (v < a.total) {
      if (BITS == 8) raw[i] = __ldcs(reinterpret_cast<const uint2 *>(a.codes) + v);
      else raw[i].x = __ldcs(reinterpret_cast<const uint32_t *>(a.codes) + v);
      scale[i] = __ldg(a.scales + (v >> 2));
    }
  }
#pragma unroll
  for (int i = 0; i < kMxAhead; ++i) {
    const int64_t v = base + i * kMxThreads;
    if (v >= a.total) continue;
    float f[8];
    if (BITS == 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = e4m3x2_floats((j & 2 ? raw[i].y : raw[i].x) >> (16 * (j & 1)) & 0xFFFFu);
        f[2 * j] = p.x, f[2 * j + 1] = p.y;
      }
    } else {
      e2m1x8_floats(raw[i].x, f);
    }
    const float s = mx_power(scale[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= s;
    E::store(x + row_offset(a, v), f);
  }
}

template <typename Ty>
static cudaError_t launch_blocks(const MxArgs &a, int bits, bool read, cudaStream_t st) {
  const int64_t per = kMxThreads * kMxAhead;
  const dim3 grid((unsigned)((a.total + per - 1) / per)), block(kMxThreads);
  if (read)
    return bits == 8 ? launch_pdl(mx_read_kernel<Ty, 8>, grid, block, 0, st, a)
                     : launch_pdl(mx_read_kernel<Ty, 4>, grid, block, 0, st, a);
  return bits == 8 ? launch_pdl(mx_quantize_kernel<Ty, 8>, grid, block, 0, st, a)
                   : launch_pdl(mx_quantize_kernel<Ty, 4>, grid, block, 0, st, a);
}

int launch_mx_blocks(const lily_mx_mat &m, int dtype, void *x, int64_t ts, bool read, cudaStream_t st) {
  const MxArgs a{x, ts, (int64_t)m.rows * (m.cols / 8), m.cols / 8, m.codes, m.scales};
  const cudaError_t e = dtype == LILY_BF16  ? launch_blocks<Bf16>(a, m.bits, read, st)
                        : dtype == LILY_F16 ? launch_blocks<F16>(a, m.bits, read, st)
                                            : launch_blocks<F32>(a, m.bits, read, st);
  return e == cudaSuccess ? LILY_Q4_OK : (cudaGetLastError(), LILY_Q4_ERR_CUDA);
}

}  // namespace lq4
