// lily_sample: a token of each row of logits by temperature, top-k, top-p, min-p and a given number.
//
// In the order (logit descending, index ascending) every filter keeps a beginning of the row, so what is kept is
// (a logit, how many of its equals), and nothing of the vocabulary's size is sorted.  The token is the first in the order
// of indices whose cumulative weight is above u times the total.
//
// Every decision is one between integers: a weight is exp((l - max) / T) as a 64-bit integer, right to 2^-41.5 of itself and
// rounded to a unit that leaves the row's sum its 61 bits (see set_unit), so sums do not depend on their order.  Equal
// logits are all rounded the same way: V of them move a sum by V times half a unit, 2^-61 of the sum, and what weighs nothing
// (below 2^-60 of the largest) by V 2^-60.  A comparison falls otherwise than that of the real numbers only within
// 1e-12 of the sum, then, at the largest V.  Such a weight takes some fifty instructions; where fp32 weights with a
// bound on their error leave the decision in no doubt, they make it instead.
//
// A cluster of blocks holds a row in its shared memory, each block a run of it, and reads it from there for every
// pass; sums, histograms and candidates are exchanged by reading the other blocks' shared memory, all blocks
// deciding the same.  What is exchanged alternates between two buffers, so one cluster barrier an
// exchange is enough.
//
// The ways to a result, the first that is enough:
//  - the short list: the tokens at or above a logit that some threads' largest logits give, ordered by counting;
//  - without a filter, sums of fp32 weights;
//  - the long way: a histogram of the distance from the largest logit, refined inside the bin of the cut until few
//    candidates are left, and sums of exact weights.
//
// Measured on one GB300, fp32 rows of 151,936, one row / 16 / 64: the largest 6.8 / 9.6 / 19.8 us, no filter 11 / 15 to 21 / 30 to 46
// (by how many rows leave fp32 sums in doubt), top_k 20 10.5 / 13.4 / 27.6, top_p 0.9 at T = 0.8 12.3 / 16.4 / 34.6; over a
// flat bulk top_p 0.95 at T = 1.2 (26,634 tokens kept) 47 / 61 / 135, top_k 1000 27 / 34 / 72.  Reading takes 0.1 us a row:
// what bounds one row is the chain of its passes and exchanges (a microsecond a cluster barrier and what goes
// with it; the pass of exact weights over a flat bulk 11), many rows the issue of a pass's instructions and the
// rounds of blocks, two an SM.  (Of a thread's state some 450 bytes are spilled: 64 registers is what two blocks an SM leave.)
#include <algorithm>

#include "mx_device.cuh"

namespace lq4 {

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kBins = kSampleThreads;       // of a histogram: a thread has one
constexpr int kList = kSampleThreads;       // tokens of a list: a thread has one
constexpr int kFewTokens = 80, kManyTokens = 340;  // how many a list is asked for
constexpr int kStep = 128;                  // neighbours that a warp takes at once
constexpr int kMaxSlice = kSampleMaxVocab / 8 + kStep;
constexpr int kMaxSteps = kMaxSlice / kStep;
constexpr int kMaxCluster = 8;
constexpr float kNoWeight = 60.f;           // 2^-60 and less of the largest weighs nothing
constexpr float kBinsAOctave = kBins / 44.5f;  // the last bin takes what is beyond (2^-25 of the sum at most)
constexpr int kFreeBits = 43;               // units of 2^-43 of the largest: any row's sum has room for them
constexpr int kListBits = 52;               // and any list's
constexpr uint32_t kKeyNone = 0x007FFFFFu;  // the key of -infinity

struct SampleArgs {
  const void *logits;
  int64_t ts;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t *top_k;
  int32_t *token, *kept, *hdr;
  float *prob;
  int V, slice, cluster;
  int B;
  bool ordered;  // rows that may take long first
};

// 2^(-i/256) as fp32 pairs.
struct ExpTable {
  float hi[256], lo[256];
};
constexpr ExpTable make_exp_table() {
  ExpTable t = {};
  for (int i = 0; i < 256; ++i) {
    const double a = -0.693147180559945309417232 * i / 256;
    double term = 1, sum = 1;
    for (int n = 1; n < 30; ++n) term *= a / n, sum += term;
    t.hi[i] = (float)sum;
    t.lo[i] = (float)(sum - (double)t.hi[i]);
  }
  return t;
}
__device__ const ExpTable kExpTable = make_exp_table();

// ----------------------------------------------------------------------------- numbers
// Order of fp32 numbers as unsigned integers, and back.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key); }

// What turns a row's logits into weights: x = (max - l) * log2(e) / T, the weight 2^(bits - x).
struct Scale {
  float top, hi, lo;  // the largest logit (finite); log2(e) / T as a pair
  int bits;           // the unit is 2^-bits of the largest weight
};
__device__ __forceinline__ float rough_exponent(const Scale &s, float l) { return __fmul_rn(__fsub_rn(s.top, l), s.hi); }
// 2^(bits - x) to the nearest, 0 from kNoWeight on.  x = n + i/256 + r; 2^-r = 1 - a + a^2 (1/2 - a/6 + a^2/24), a = r ln 2
// below 2^-9.5, whose first term is kept as a pair; the product with the table's pair too.
__device__ __forceinline__ uint64_t weight_of(const Scale &s, float l, const float2 *table) {
  // max - l and what its rounding drops
  const float d = __fsub_rn(s.top, l), b = __fsub_rn(d, s.top);
  const float d_lo = __fsub_rn(__fsub_rn(s.top, __fsub_rn(d, b)), __fadd_rn(l, b));
  const float x = __fmul_rn(d, s.hi);
  if (!(x < kNoWeight)) return 0;
  const float x_lo = __fmaf_rn(d_lo, s.hi, __fmaf_rn(d, s.lo, __fmaf_rn(d, s.hi, -x)));
  constexpr float magic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
  const float rounded = __fmaf_rn(x, 256.f, magic);
  const int k = __float_as_int(rounded) - __float_as_int(magic);
  const float r0 = __fmaf_rn(__fsub_rn(rounded, magic), -1.f / 256, x);
  const float r = __fadd_rn(r0, x_lo), r_lo = __fsub_rn(x_lo, __fsub_rn(r, r0));
  constexpr float ln2 = 0.693147180559945309417f, ln2_lo = (float)(0.693147180559945309417 - (double)ln2);
  const float a = __fmul_rn(r, ln2);
  const float a_lo = __fmaf_rn(r_lo, ln2, __fmaf_rn(r, ln2_lo, __fmaf_rn(r, ln2, -a)));
  const float p = __fmaf_rn(__fmul_rn(a, a), __fmaf_rn(a, __fmaf_rn(a, 1.f / 24, -1.f / 6), 0.5f), -a_lo);
  const float2 t = table[k & 255];
  // t (1 - a + p): hi + lo
  const float m = __fmul_rn(t.x, -a), m_lo = __fmaf_rn(t.x, -a, -m);
  const float hi = __fadd_rn(t.x, m);
  float lo = __fsub_rn(m, __fsub_rn(hi, t.x));
  lo = __fadd_rn(lo, __fmaf_rn(t.x, p, __fmaf_rn(t.y, -a, __fadd_rn(t.y, m_lo))));
  // hi is in (0.49, 1.01): 1 + hi has its bits down to 2^-22 (2^-23 below 2), and what those leave goes to lo
  const float one = __fadd_rn(hi, 1.f), whole = __fsub_rn(one, 1.f);
  lo = __fadd_rn(lo, __fsub_rn(hi, whole));
  const int32_t units = one < 2.f ? __float_as_int(one) - 0x3F800000 : (__float_as_int(one) - 0x40000000 + 0x400000) * 2;
  const uint64_t w = (uint64_t)((int64_t)units * ((int64_t)1 << 37) + (int64_t)__float2int_rn(lo * 0x1p49f) * 2048);  // 2^-60
  const int drop = min(63, 60 - s.bits + (k >> 8));
  return (w + (((uint64_t)1 << drop) >> 1)) >> drop;
}
// The same to 2^-29 and half a unit, for half of the instructions: the table's entry and 2^-r - 1 in one fp32 number.
__device__ __forceinline__ uint64_t near_weight(const Scale &s, float l, const float2 *table) {
  const float d = __fsub_rn(s.top, l), b = __fsub_rn(d, s.top);
  const float d_lo = __fsub_rn(__fsub_rn(s.top, __fsub_rn(d, b)), __fadd_rn(l, b));
  const float x = __fmul_rn(d, s.hi);
  if (!(x < kNoWeight)) return 0;
  const float x_lo = __fmaf_rn(d_lo, s.hi, __fmaf_rn(d, s.lo, __fmaf_rn(d, s.hi, -x)));
  constexpr float magic = 12582912.f, ln2 = 0.693147180559945309417f;
  const float rounded = __fmaf_rn(x, 256.f, magic);
  const int k = __float_as_int(rounded) - __float_as_int(magic);
  const float a = __fmul_rn(__fadd_rn(__fmaf_rn(__fsub_rn(rounded, magic), -1.f / 256, x), x_lo), ln2);
  const float less = __fmul_rn(a, __fmaf_rn(a, __fmaf_rn(a, 1.f / 6, -0.5f), 1.f));  // 1 - 2^-r
  const float2 t = table[k & 255];
  // in units of 2^-31: what the entry's first part has, exactly, and the rest
  const uint32_t first = (uint32_t)((__float_as_int(t.x) & 0x7FFFFF) | 0x800000) << (__float_as_int(t.x) >> 23 == 127 ? 8 : 7);
  const uint32_t w = first + (uint32_t)__float2int_rn(__fmaf_rn(t.x, -less, t.y) * 0x1p31f);
  const int drop = min(63, 61 - s.bits + (k >> 8));
  return (((uint64_t)w << 31 >> drop) + 1) >> 1;
}
// 2^-x in fp32, 0 from kNoWeight on: 2^-22 relative, and what the rounding of max - l does, 2^-24 x ln 2.
__device__ __forceinline__ float fast_weight(const Scale &s, float l) {
  const float d = __fsub_rn(s.top, l), x = __fmul_rn(d, s.hi);
  const float lo = __fmaf_rn(d, s.lo, __fmaf_rn(d, s.hi, -x));
  float w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(-x));
  w = __fmaf_rn(w, lo * -0.693147180559945309f, w);
  return x < kNoWeight ? w : 0.f;
}
// Bin of a logit by its rough exponent, for those below kNoWeight.
__device__ __forceinline__ int bin_of(float x) { return min(kBins - 1, (int)(x * kBinsAOctave)); }
// floor(f * n) for f in [0, 1), or the next integer at or above it
__device__ __forceinline__ uint64_t share_of(float f, uint64_t n, bool up) {
  if (!(f > 0.f)) return 0;
  const uint32_t b = __float_as_uint(f);
  const int e = max(1, (int)(b >> 23));
  const uint64_t m = (b >> 23) ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
  const int shift = 150 - e;  // f = m 2^-shift, shift 24 or more
  const uint64_t lo = m * n, hi = __umul64hi(m, n);
  uint64_t q, rest;
  if (shift < 64) {
    q = (hi << (64 - shift)) | (lo >> shift);
    rest = lo << (64 - shift);
  } else if (shift < 128) {
    q = shift == 64 ? hi : hi >> (shift - 64);
    rest = lo | (shift == 64 ? 0 : hi << (128 - shift));
  } else {
    q = 0, rest = lo | hi;
  }
  return q + (up && rest ? 1 : 0);
}

// ----------------------------------------------------------------------------- exchange
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(const void *p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ uint64_t peer(const uint64_t *p, int rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer_address(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t peer(const uint32_t *p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_address(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void put_peer(uint64_t *p, int rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_address(p, rank)), "l"(v) : "memory");
}
// f(rank, value) for *p of every block of the cluster, in their order; all are read before the first is used.
template <typename T, typename F>
__device__ __forceinline__ void each_peer(const T *p, int cluster, F f) {
  T v[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < cluster) v[r] = peer(p, r);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < cluster) f(r, v[r]);
}

struct SampleShared {
  uint64_t hist[2][kBins];           // of sums; counts take the first half of one
  __device__ uint32_t *counts(int turn) { return reinterpret_cast<uint32_t *>(hist[turn]); }
  uint64_t values[2][4];             // what blocks exchange: sums and extremes
  uint64_t list[2][kList];           // a block's tokens: key, then the complement of the index
  uint64_t all[kList], weight[kList];  // all blocks' tokens
  uint64_t warp_sum[kSampleWarps][4];
  uint64_t step_mass[kMaxSteps];
  uint32_t step_ties[kMaxSteps];
  __align__(8) float tops[kSampleThreads];
  float2 table[256];
  uint64_t found[4];
  uint32_t count;
  float cut;
};

__device__ __forceinline__ uint64_t warp_add(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const T u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// Inclusive sums over the block's threads.
template <typename T>
__device__ __forceinline__ T block_scan(T v, SampleShared &sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_scan(v);
  if (lane == 31) sh.warp_sum[warp][3] = v;
  __syncthreads();
  T before = lane < warp ? (T)sh.warp_sum[lane][3] : 0;  // each warp sums what is before it
#pragma unroll
  for (int o = kSampleWarps / 2; o; o >>= 1) before += __shfl_xor_sync(~0u, before, o);
  return v + __shfl_sync(~0u, before, 0);
}

// A row's cut: keys above it are kept, and `ties` of those equal to it, the ones that come first.
struct Cut {
  uint32_t key;
  uint64_t ties;
};

// What a list is asked for.
constexpr uint64_t kNoRest = ~0ull;
struct ListArgs {
  int k;                // 0 for none
  float top_p;          // 1 for none
  uint32_t least;       // the smallest key that min_p leaves
  int wanted;           // how many tokens the list should have at least; 0: all that min_p leaves
  int bins;             // or the bins that it takes, where they are known to fit; 0: not known
  uint64_t rest;        // how many the row keeps where nothing but top_k ends it (0: not known; kNoRest: what is listed)
  uint64_t total, off;  // what top_p is a share of, to within `off`; 0: the row's sum, found on the way (or that of k tokens)
  int n;                // tokens of the list
  bool all;             // it has all that have a weight and that min_p leaves
};
enum Result { kDone = 0, kNotEnough = 1 };

struct Row {
  SampleShared &sh;
  float *l;  // this block's logits, -infinity beyond the row's end
  Scale scale;
  int rank, cluster, first, padded;  // first: index of l[0]; padded: a multiple of kStep
  int turn, hist_turn;
  uint64_t total, off;  // the row's sum of weights to within `off`, once a list has found it
  bool summed;          // the unit is that of the row's sum

  // f(place, logit) for all of the block's logits
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
    for (int i = threadIdx.x; i < padded / 4; i += kSampleThreads) {
      const float4 v = reinterpret_cast<const float4 *>(l)[i];
      f(4 * i, v.x), f(4 * i + 1, v.y), f(4 * i + 2, v.z), f(4 * i + 3, v.w);
    }
  }
  __device__ __forceinline__ uint64_t weight(float v) const { return weight_of(scale, v, sh.table); }
  // Weights of four neighbours, 0 where not needed.
  __device__ __forceinline__ void weights(const float (&v)[4], const bool (&need)[4], uint64_t (&w)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = need[j] ? weight(v[j]) : 0;
  }
  __device__ __forceinline__ void list(int i, float v) {  // a token to the block's list
    const uint32_t at = atomicAdd(&sh.count, 1u);
    if (at < kList) sh.list[turn][at] = (uint64_t)key_of(v) << 32 | (uint32_t)~(first + i);
  }

  // The unit with which a sum of weights, in largest ones, keeps 61 bits (and below 62, where it is off by less than a half).
  __device__ __forceinline__ void set_unit(float sum) {
    scale.bits = min(60, 187 - (int)(__float_as_uint(sum) >> 23)), summed = true;
  }
  // The same where nothing else gives the sum: from fp32 weights.
  __device__ void find_unit() {
    float sum = 0.f;
    each([&](int, float v) { sum += fast_weight(scale, v); });
    uint64_t all = (uint64_t)(sum * 0x1p43f), none = 0;
    exchange(all, none);
    set_unit((float)all * 0x1p-43f);
  }

  // Sums over the cluster; every thread gets them.
  __device__ void exchange(uint64_t &a, uint64_t &b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_add(a), b = warp_add(b);
    if (lane == 0) sh.warp_sum[warp][0] = a, sh.warp_sum[warp][1] = b;
    __syncthreads();
    if (warp == 0) {
      a = warp_add(lane < kSampleWarps ? sh.warp_sum[lane][0] : 0), b = warp_add(lane < kSampleWarps ? sh.warp_sum[lane][1] : 0);
      if (lane == 0) sh.values[turn][0] = a, sh.values[turn][1] = b;
    }
    cluster_barrier();
    a = b = 0;
    each_peer(&sh.values[turn][0], cluster, [&](int, uint64_t v) { a += v; });
    each_peer(&sh.values[turn][1], cluster, [&](int, uint64_t v) { b += v; });
    turn ^= 1;
  }

  // The cluster's histogram (u32 counts or u64 sums) with the cut in it: the bin where the measure, summed from the
  // first bin, reaches `target`, and the sum before it; false if it does not reach it.  The next histogram is cleared.
  // v: what this thread's bin has.
  template <typename T>
  __device__ bool find_bin(T target, int &bin, T &before, T &v) {
    cluster_barrier();
    v = 0;
    each_peer(reinterpret_cast<T *>(sh.hist[hist_turn]) + threadIdx.x, cluster, [&](int, T x) { v += x; });
    hist_turn ^= 1;
    sh.hist[hist_turn][threadIdx.x] = 0;  // the others are done with it
    const T upto = block_scan(v, sh);
    bin = __syncthreads_count(upto < target);
    if ((int)threadIdx.x == bin) sh.found[0] = upto - v;
    __syncthreads();
    before = (T)sh.found[0];
    __syncthreads();  // found is free again
    return bin < kBins;
  }

  // The blocks' lists (their lengths in values[at][0]) end to end: how long they are together, and the block and place of
  // this thread's entry.
  __device__ uint64_t my_entry(int at, int &from, int &place) {
    uint64_t n = 0;
    from = place = 0;
    each_peer(&sh.values[at][0], cluster, [&](int p, uint64_t v) {
      if (threadIdx.x >= n) from = p, place = (int)(threadIdx.x - n);
      n += v;
    });
    return n;
  }

  // The members of a bin, narrower with every level.
  struct Members {
    int level = 0, bin1 = 0, width = 1, bin2 = 0;  // width: bins of the first histogram from bin1 on
    float finer = kBins;                            // bins of the second in one of the first
    uint32_t lo = 0, hi = 0;
    float least = -INFINITY, most = INFINITY;  // logits beyond these are none of them
    __device__ __forceinline__ void in_bins(int bin, int n, const Scale &s) {
      level = 1, bin1 = bin, width = n, finer = (float)kBins / n;
      least = __fsub_rd(s.top, __fdiv_ru((bin + n) * (1.00001f / kBinsAOctave), s.hi));
      most = fminf(__fsub_ru(s.top, __fdiv_rd(bin * (0.99999f / kBinsAOctave), s.hi)), INFINITY);  // (not NaN)
      if (bin + n == kBins) least = -INFINITY;
    }
    __device__ __forceinline__ bool has(float x, float v) const {
      if (!(x < kNoWeight)) return false;
      if (level == 0) return true;
      if (!(v >= least && v <= most)) return false;
      const float y = x * kBinsAOctave;
      const int at = min(kBins - 1, (int)y);
      if (at < bin1 || at >= bin1 + width) return false;
      if (level == 1) return true;
      if (min(kBins - 1, (int)((y - bin1) * finer)) != bin2) return false;
      if (level == 2) return true;
      const uint32_t k = key_of(v);
      return k >= lo && k <= hi;
    }
    // bin of a member in the next histogram, larger logits first
    __device__ __forceinline__ int next(float x, float v, int shift) const {
      const float y = x * kBinsAOctave;
      if (level == 0) return min(kBins - 1, (int)y);
      if (level == 1) return min(kBins - 1, (int)((y - bin1) * finer));
      return (int)((hi - key_of(v)) >> shift);
    }
  };

  // The shortest beginning whose measure (MASS: weights, else their number) reaches `target`, among logits with a
  // weight; false if all of them do not.  `above` of it lies before the members that `in` starts with, whose histogram
  // is there already where `filled`.
  template <bool MASS>
  __device__ bool select(Members in, uint64_t above, bool filled, uint64_t target, Cut &cut) {
    while (true) {
      int shift = 0;
      if (in.level >= 2) {  // the keys there are
        uint32_t lo = ~0u, hi = 0;
        each([&](int, float v) {
          if (v >= in.least && v <= in.most && in.has(rough_exponent(scale, v), v)) lo = min(lo, key_of(v)), hi = max(hi, key_of(v));
        });
        lo = __reduce_min_sync(~0u, lo), hi = __reduce_max_sync(~0u, hi);
        if (threadIdx.x == 0) sh.found[2] = ~0ull, sh.found[3] = 0;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
          atomicMin(reinterpret_cast<uint32_t *>(&sh.found[2]), lo);
          atomicMax(reinterpret_cast<uint32_t *>(&sh.found[3]), hi);
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.values[turn][0] = (uint32_t)sh.found[2], sh.values[turn][1] = (uint32_t)sh.found[3];
        cluster_barrier();
        in.lo = ~0u, in.hi = 0;
        each_peer(&sh.values[turn][0], cluster, [&](int, uint64_t v) { in.lo = min(in.lo, (uint32_t)v); });
        each_peer(&sh.values[turn][1], cluster, [&](int, uint64_t v) { in.hi = max(in.hi, (uint32_t)v); });
        turn ^= 1;
        in.level = 3;
        if (in.lo == in.hi) {  // equals only
          const uint64_t w = MASS ? weight(logit_of(in.lo)) : 1;
          cut.key = in.lo;
          cut.ties = (target - above + w - 1) / w;
          return true;
        }
        while ((in.hi - in.lo) >> shift >= kBins) ++shift;
      }
      if (!filled)
        each([&](int, float v) {
          const float x = rough_exponent(scale, v);
          if (in.has(x, v)) {
            const int bin = in.next(x, v, shift);
            if (MASS) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.hist[hist_turn][bin]), (unsigned long long)weight(v));
            else atomicAdd(sh.counts(hist_turn) + bin, 1u);
          }
        });
      filled = false;
      int bin;
      if (MASS) {
        uint64_t before, v;
        if (!find_bin<uint64_t>(target - above, bin, before, v)) return false;
        above += before;
      } else {
        uint32_t before, v;
        const bool found = find_bin<uint32_t>((uint32_t)(target - above), bin, before, v);
        if (!summed) {  // every token counts as its bin's largest, a sixteenth more than it weighs at most
          const int t = threadIdx.x;
          const uint64_t sum = block_scan((uint64_t)((float)v * exp2f(20.f - t * (1.f / kBinsAOctave))), sh);
          if (t == kBins - 1) sh.found[0] = sum;
          __syncthreads();
          set_unit((float)sh.found[0] * 0x1p-20f);
          __syncthreads();
        }
        if (!found) return false;
        above += before;
      }
      if (in.level == 0) in.in_bins(bin, 1, scale);
      else if (in.level == 1) in.bin2 = bin, in.level = 2;
      else in.hi -= (uint32_t)bin << shift, in.lo = max(in.lo, in.hi - ((1u << shift) - 1));
      if (candidates<MASS>(in, target - above, cut)) return true;
    }
  }

  // The cut among the members, if they are few; the measure reaches `target` among them.
  template <bool MASS>
  __device__ bool candidates(const Members &in, uint64_t target, Cut &cut) {
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    each([&](int i, float v) {
      if (v >= in.least && v <= in.most && in.has(rough_exponent(scale, v), v)) list(i, v);
    });
    __syncthreads();
    if (threadIdx.x == 0) sh.values[turn][0] = sh.count;
    cluster_barrier();
    int from, place;
    const uint64_t n = my_entry(turn, from, place);
    turn ^= 1;
    if (n > kList) return false;
    // larger is earlier: the key, then the lower index
    if (threadIdx.x < n) {
      const uint64_t mine = peer(&sh.list[turn ^ 1][place], from);
      sh.all[threadIdx.x] = mine;
      sh.weight[threadIdx.x] = MASS ? weight(logit_of((uint32_t)(mine >> 32))) : 1;
    }
    if (threadIdx.x == 0) sh.found[0] = 0;
    __syncthreads();
    // Few: every block orders them all.  Many: each its share, since what takes the time is the comparisons' issue.
    const bool shared = n > 128;
    const int share = shared ? ((int)n + cluster - 1) / cluster : (int)n, begin = shared ? rank * share : 0;
    int group = 1;  // threads an entry
    while (group < 32 && 2 * group * share <= kSampleThreads) group *= 2;
    const int e = begin + threadIdx.x / group;
    const bool entry = (int)threadIdx.x / group < share && e < (int)n;
    const uint64_t mine = entry ? sh.all[e] : ~0ull;
    uint64_t before = 0;
    uint32_t equals = 0;
#pragma unroll 4
    for (int j = threadIdx.x & (group - 1); j < (int)n; j += group) {
      const uint64_t other = sh.all[j];
      if (other > mine) before += sh.weight[j], equals += other >> 32 == mine >> 32;
    }
    for (int o = group / 2; o; o >>= 1) {
      before += __shfl_xor_sync(~0u, before, o);
      equals += __shfl_xor_sync(~0u, equals, o);
    }
    if (entry && (threadIdx.x & (group - 1)) == 0 && before < target && before + sh.weight[e] >= target)
      sh.found[0] = mine >> 32, sh.found[1] = equals + 1;
    __syncthreads();
    if (shared) {
      if (threadIdx.x == 0) sh.values[turn][0] = sh.found[0], sh.values[turn][1] = sh.found[0] ? sh.found[1] : 0;
      cluster_barrier();
      cut = Cut{0, 0};  // one block has it
      each_peer(&sh.values[turn][0], cluster, [&](int, uint64_t v) { cut.key |= (uint32_t)v; });
      each_peer(&sh.values[turn][1], cluster, [&](int, uint64_t v) { cut.ties |= v; });
      turn ^= 1;
    } else {
      cut.key = (uint32_t)sh.found[0], cut.ties = sh.found[1];
    }
    __syncthreads();
    return true;
  }

  // Total weight of what a cut keeps.
  __device__ uint64_t mass(const Cut &cut) {
    uint64_t sum = 0, ties = 0;
    for (int s = threadIdx.x >> 5; s < padded / kStep; s += kSampleWarps) {
      const float4 v4 = reinterpret_cast<const float4 *>(l)[s * (kStep / 4) + (threadIdx.x & 31)];
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
      bool need[4];
      uint64_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) need[j] = key_of(v[j]) > cut.key, ties += key_of(v[j]) == cut.key;
      weights(v, need, w);
      sum += (w[0] + w[1]) + (w[2] + w[3]);
    }
    exchange(sum, ties);
    ties = min(ties, cut.ties);
    if (ties) sum += ties * weight(logit_of(cut.key));
    return sum;
  }

  __device__ bool select_share(float p, uint64_t target, Cut &cut, int &stepped, int &few);
  __device__ int try_list(ListArgs q, const float (&tops)[2], float u, int32_t *token, int32_t *kept, float *prob);
  enum Mode { kFast, kNear, kExact, kStepped };
  template <Mode MODE>
  __device__ bool draw(const SampleArgs &a, int64_t b, const Cut &cut, float u, int k, uint64_t usable_count, int bin);
};

// ----------------------------------------------------------------------------- loading
// A NaN is no token; one zero.
__device__ __forceinline__ float usable(float v) { return v == v ? v + 0.f : -INFINITY; }

struct F32Logits {};
template <typename Ty>
struct Logits {  // eight of 16 bits in 16 bytes
  using Elem = uint16_t;
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(Elem e) { return Ty::to_f32x2(e).x; }
  static __device__ __forceinline__ void many(const uint4 &v, float (&f)[N]) { unpack8<Ty>(v, f); }
};
template <>
struct Logits<F32Logits> {
  using Elem = float;
  static constexpr int N = 4;
  static __device__ __forceinline__ float one(Elem e) { return e; }
  static __device__ __forceinline__ void many(const uint4 &v, float (&f)[N]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
};

// Logits first .. first + padded - 1 of a row to shared memory, -infinity where there are none; their maximum, and how
// many are above -infinity.  `first` is where 16 bytes begin in memory, so it may be before the row; no load
// reaches beyond the row.  fp32 goes straight there, all of it at once.
template <typename Ty>
__device__ __forceinline__ float load_row(const typename Logits<Ty>::Elem *row, int first, int padded, int V, float *to,
                                          uint32_t &drawable) {
  using L = Logits<Ty>;
  constexpr bool COPY = L::N == 4;
  constexpr int AHEAD = 5;
  float top = -INFINITY;
  const int vecs = padded / L::N;
  const auto whole = [&](int v) { return first + v * L::N >= 0 && first + v * L::N + L::N <= V; };
  const auto seen = [&](float v) { top = fmaxf(top, v), drawable += v > -INFINITY; };
  if (COPY) {
    for (int v = threadIdx.x; v < vecs; v += kSampleThreads)
      if (whole(v))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to + 4 * v)),
                     "l"(row + first + 4 * v)
                     : "memory");
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  for (int v0 = threadIdx.x; v0 < vecs; v0 += kSampleThreads * AHEAD) {
    uint4 raw[AHEAD];
    if (!COPY) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int v = v0 + i * kSampleThreads;
        if (v < vecs && whole(v)) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(row + first + v * L::N));
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int v = v0 + i * kSampleThreads, at = first + v * L::N;
      if (v >= vecs) break;
      float f[L::N];
      float4 *out = reinterpret_cast<float4 *>(to + v * L::N);
      const bool in = whole(v);
      if (in && COPY) {
        const float4 w = out[0];
        f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
      } else if (in) {
        L::many(raw[i], f);
      } else {
#pragma unroll
        for (int j = 0; j < L::N; ++j) f[j] = at + j >= 0 && at + j < V ? L::one(row[at + j]) : -INFINITY;
      }
      bool same = in && COPY;  // a NaN and a negative zero are written again
#pragma unroll
      for (int j = 0; j < L::N; ++j) {
        same = same && f[j] == f[j] && __float_as_uint(f[j]) != 0x80000000u;
        seen(f[j] = usable(f[j]));
      }
      if (!same) {
#pragma unroll
        for (int j = 0; j < L::N; j += 4) out[j / 4] = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
      }
    }
  }
  return top;
}

// ----------------------------------------------------------------------------- the long way
// The cut of top_p: the shortest beginning whose weights reach `target`, or, with 0, the share p of the row's sum.  A
// histogram in 32 bits (weights relative to their bin's largest, so that none is lost and none runs over) finds
// the cut's bin; one pass of exact weights then sums what is before it, what is after it, and the bin's own
// histogram.  The sums of what is before it stay in step_mass, and its number in `stepped`; -1 where the histogram leaves the
// bin in doubt and the cut is found by exact weights from the start.  Where the tokens up to the cut's bin are sure to fit a list,
// it stops there, with `few` their bins.
__device__ bool Row::select_share(float p, uint64_t target, Cut &cut, int &stepped, int &few) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  stepped = -1;
  if (few > 0) few = 0;
  each([&](int, float v) {
    const float x = rough_exponent(scale, v);
    if (!(x < kNoWeight)) return;
    const float y = x * kBinsAOctave;
    const int bin = min(kBins - 1, (int)y);
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"((bin - y) * (1.f / kBinsAOctave)));
    atomicAdd(sh.counts(hist_turn) + bin, (uint32_t)__float2int_rn(w * 65536.f));
  });
  cluster_barrier();
  uint64_t v = 0;
  each_peer(sh.counts(hist_turn) + t, cluster, [&](int, uint32_t x) { v += x; });
  hist_turn ^= 1;
  sh.hist[hist_turn][t] = 0;
  const uint64_t rough = block_scan((uint64_t)((float)v * exp2f(scale.bits - 16 - t * (1.f / kBinsAOctave))), sh);
  if (t == kBins - 1) sh.found[0] = rough;
  __syncthreads();
  // Each weight was rounded to 2^-16.9 of it; ex2, its argument and the bin's exponent add 2^-18: 2^-15 covers that for the
  // bins and for what p is a share of.
  const uint64_t whole = sh.found[0], off = whole >> 15;
  const uint64_t near = target ? target : max((uint64_t)1, share_of(p, whole, true));
  const int bin = __syncthreads_count(rough + off < near), high = __syncthreads_count(rough < near + off);
  const int width = high - bin + 1;  // the cut is in one of these
  if (high >= kBins || width > 8) {
    if (target == 0) target = max((uint64_t)1, share_of(p, mass(Cut{kKeyNone, 0}), true));
    return select<true>(Members{}, 0, false, target, cut);
  }
  // a token counts as 61,700 at least: its weight is above 0.9415 of its bin's largest (but in the last bin; a list too long ends)
  const uint64_t tokens = block_scan(t <= high ? v : 0, sh);
  if (t == kBins - 1) sh.found[1] = tokens;
  __syncthreads();
  if (few >= 0 && sh.found[1] <= (uint64_t)kList * 61000) {
    few = high + 1;
    return false;
  }
  few = 0;
  Members in;
  in.in_bins(bin, width, scale);
  uint64_t above = 0, rest = 0;
  for (int s = warp; s < padded / kStep; s += kSampleWarps) {
    const float4 v4 = reinterpret_cast<const float4 *>(l)[s * (kStep / 4) + lane];
    const float f[4] = {v4.x, v4.y, v4.z, v4.w};
    bool need[4];
    uint64_t w[4], m = 0;
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = rough_exponent(scale, f[j]);
      at[j] = x < kNoWeight ? bin_of(x) : kBins;
      need[j] = at[j] <= (target ? high : kBins - 1);  // nothing asks for the sum of those after the bin where the target is known
    }
    weights(f, need, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (at[j] < bin) m += w[j];
      else rest += w[j];
      if (at[j] >= bin && at[j] <= high)
        atomicAdd(reinterpret_cast<unsigned long long *>(&sh.hist[hist_turn][in.next(rough_exponent(scale, f[j]), f[j], 0)]),
                  (unsigned long long)w[j]);
    }
    if (__any_sync(~0u, m != 0)) m = warp_add(m);
    if (lane == 0) sh.step_mass[s] = m, above += m;
  }
  exchange(above, rest);
  if (target == 0) target = max((uint64_t)1, share_of(p, above + rest, true));
  stepped = bin;
  return select<true>(in, above, true, target, cut);
}

// The row's token among what the cut keeps, from sums of every step in the order of indices.  kFast and kNear (without a
// cut): by weights in fp32, or to 2^-29; false where that leaves the token open.  kStepped: what is before `bin` is summed already.
template <Row::Mode MODE>
__device__ bool Row::draw(const SampleArgs &a, int64_t b, const Cut &cut, float u, int k, uint64_t usable_count, int bin) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = padded / kStep;
  uint64_t kept = 0, ties = 0;
#pragma unroll 1
  for (int s = warp; s < steps; s += kSampleWarps) {
    const float4 v4 = reinterpret_cast<const float4 *>(l)[s * (kStep / 4) + lane];
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
    if (MODE == kFast) {
      float m = (fast_weight(scale, v[0]) + fast_weight(scale, v[1])) + (fast_weight(scale, v[2]) + fast_weight(scale, v[3]));
#pragma unroll
      for (int o = 16; o; o >>= 1) m += __shfl_xor_sync(~0u, m, o);
      if (lane == 0) sh.step_mass[s] = (uint64_t)(m * 0x1p43f), sh.step_ties[s] = 0;
      continue;
    }
    if (MODE == kNear) {
      const uint64_t m = warp_add((near_weight(scale, v[0], sh.table) + near_weight(scale, v[1], sh.table)) +
                                  (near_weight(scale, v[2], sh.table) + near_weight(scale, v[3], sh.table)));
      if (lane == 0) sh.step_mass[s] = m;
      continue;
    }
    uint32_t t = 0;
    bool need[4];
    uint64_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t key = key_of(v[j]);
      t += key == cut.key;
      need[j] = key > cut.key, kept += need[j];
      if (MODE == kStepped) need[j] = need[j] && bin_of(fminf(rough_exponent(scale, v[j]), kNoWeight)) >= bin;
    }
    weights(v, need, w);
    uint64_t m = (w[0] + w[1]) + (w[2] + w[3]);
    if (__any_sync(~0u, m != 0)) m = warp_add(m);
    t = __reduce_add_sync(~0u, t);
    if (lane == 0) sh.step_mass[s] = MODE == kStepped ? sh.step_mass[s] + m : m, sh.step_ties[s] = t, ties += t;
  }
  __syncthreads();
  // Every block learns all blocks' totals; the one that holds the place in question looks for it.
  uint64_t block_mass = 0;
  for (int s = threadIdx.x; s < steps; s += kSampleThreads) block_mass += sh.step_mass[s];
  block_mass = warp_add(block_mass);
  constexpr bool SUMS_ONLY = MODE == kFast || MODE == kNear;
  if (!SUMS_ONLY) kept = warp_add(kept), ties = warp_add(ties);
  if (lane == 0) sh.warp_sum[warp][0] = block_mass, sh.warp_sum[warp][1] = kept, sh.warp_sum[warp][2] = ties;
  __syncthreads();
  if (warp < 3) {
    const uint64_t sum = warp_add(lane < kSampleWarps ? sh.warp_sum[lane][warp] : 0);
    if (lane == 0) sh.values[turn][warp] = sum;
  }
  if (threadIdx.x == 0) sh.values[turn][3] = 0;
  cluster_barrier();
  uint64_t all_mass = 0, all_kept = 0, all_ties = 0, mass_before = 0, ties_before = 0;
  each_peer(&sh.values[turn][0], cluster, [&](int p, uint64_t v) {
    if (p == rank) mass_before = all_mass;
    all_mass += v;
  });
  if (!SUMS_ONLY) {
    each_peer(&sh.values[turn][1], cluster, [&](int, uint64_t v) { all_kept += v; });
    each_peer(&sh.values[turn][2], cluster, [&](int p, uint64_t v) {
      if (p == rank) ties_before = all_ties;
      all_ties += v;
    });
  }
  const uint64_t tie_weight = !SUMS_ONLY && cut.ties ? weight(logit_of(cut.key)) : 0;
  const uint64_t total = all_mass + tie_weight * min(all_ties, cut.ties);
  const uint64_t place = share_of(u, total, false);
  // Fast weights are off by 1.1e-6 (see try_list), a step's sum by 9 * 2^-24, its conversion by one: below 2^-19 of the
  // total for a border and for the place each.
  // Near ones are off by 2^-29 and half a unit, equal ones all the same way: each 2^-29 of the total and half a unit a token.
  const uint64_t off = MODE == kFast ? (total >> 18) + 2 * kMaxSteps * kMaxCluster : MODE == kNear ? (total >> 28) + usable_count + 1 : 0;
  auto upto = [&](uint64_t m, uint64_t t) { return m + tie_weight * min(t, cut.ties); };
  const uint64_t my_mass = sh.values[turn][0], my_ties = sh.values[turn][2];
  const bool here = upto(mass_before, ties_before) <= place && place < upto(mass_before + my_mass, ties_before + my_ties);
  if (here && warp == 0) {
    uint64_t m0 = mass_before, t0 = ties_before;
    int s = 0;
    for (int base = 0; base < steps; base += 32) {  // the step that holds it
      const int i = base + lane;
      const uint64_t m = m0 + warp_scan<uint64_t>(i < steps ? sh.step_mass[i] : 0);
      const uint64_t t = t0 + warp_scan<uint32_t>(i < steps ? sh.step_ties[i] : 0);
      const uint32_t past = __ballot_sync(~0u, upto(m, t) > place);
      if (past) {
        const int at = __ffs(past) - 1;
        s = base + at;
        m0 = __shfl_sync(~0u, m, at) - sh.step_mass[s], t0 = __shfl_sync(~0u, t, at) - sh.step_ties[s];
        break;
      }
      m0 = __shfl_sync(~0u, m, 31), t0 = __shfl_sync(~0u, t, 31);
    }
    const float4 v4 = reinterpret_cast<const float4 *>(l)[s * (kStep / 4) + lane];
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
    uint64_t w[4], m = 0;
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t key = key_of(v[j]);
      w[j] = key > cut.key ? weight(v[j]) : 0;
      m += w[j], t += key == cut.key;
    }
    m0 += warp_scan(m) - m, t0 += warp_scan(t) - t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool tie = key_of(v[j]) == cut.key;
      const uint64_t from = upto(m0, t0);
      m0 += w[j], t0 += tie;
      if (from + off <= place && place + off < upto(m0, t0)) {
        sh.values[turn][3] = 1;
        a.token[b] = first + s * kStep + 4 * lane + j;
        if (a.kept)
          a.kept[b] = (int32_t)(SUMS_ONLY ? usable_count : min(all_kept + min(all_ties, cut.ties), k > 0 ? (uint64_t)k : ~(uint64_t)0));
        if (a.prob) a.prob[b] = __fdiv_rn((float)(tie ? tie_weight : w[j]), (float)total);
      }
    }
  }
  cluster_barrier();  // no block leaves while another reads its shared memory
  if (!SUMS_ONLY) return true;
  uint64_t done = 0;
  each_peer(&sh.values[turn][3], cluster, [&](int, uint64_t v) { done += v; });
  if (MODE == kFast) set_unit((float)total * 0x1p-43f);  // (for those that follow)
  turn ^= 1;
  if (done) cluster_barrier();
  return done != 0;
}

// ----------------------------------------------------------------------------- the short list
// Draws the row's token from the list: entry by entry in `mine` (its key, then the complement of its index).  decided(result)
// is called as soon as it is clear whether the list is enough.
template <typename F>
__device__ __forceinline__ void draw_from_list(const Row &row, const ListArgs &q, uint64_t mine, float u, int32_t *token,
                                               int32_t *kept_out, float *prob, F decided) {
  SampleShared &sh = row.sh;
  const int t = threadIdx.x;
  int group = 1;  // threads an entry
  while (group < 32 && 2 * group * q.n <= kSampleThreads) group *= 2;
  if (t < q.n) {
    sh.all[t] = mine;
    sh.weight[t] = row.weight(logit_of((uint32_t)(mine >> 32)));
  }
  if (t < 4) sh.found[t] = 0;
  __syncthreads();
  // `group` threads share the comparisons of entry e, whose first thread speaks for it: how many come before it
  const int e = t / group, part = t & (group - 1);
  const bool entry = e < q.n, first_of = entry && part == 0;
  const uint64_t own_key = entry ? sh.all[e] : 0, own = entry ? sh.weight[e] : 0;
  int place = 0;
#pragma unroll 8
  for (int j = part; j < q.n; j += group) place += sh.all[j] > own_key;
  for (int o = group / 2; o; o >>= 1) place += __shfl_xor_sync(~0u, place, o);
  // and, in that order, their weight
  uint64_t *ordered = sh.list[row.turn];  // (the other one is what peers read)
  __syncthreads();
  if (first_of) ordered[place] = own;
  __syncthreads();
  const uint64_t sums = block_scan(t < q.n ? ordered[t] : 0, sh);
  __syncthreads();
  if (t < q.n) ordered[t] = sums;
  __syncthreads();
  const uint64_t before = first_of ? ordered[place] - own : 0;
  const bool by_count = q.k > 0 && (q.k <= q.n || q.all);
  const int first = by_count ? min(q.k, q.n) : q.n;
  if (first_of && place == q.n - 1) sh.found[0] = before + own;
  if (first_of && place == first - 1) sh.found[1] = before + own;
  __syncthreads();
  uint64_t low = ~0ull, high = ~0ull;  // the cut is between these weights
  bool sure = by_count || q.all;
  if (q.top_p < 1.f) {
    if (by_count || (q.all && q.rest != kNoRest && !q.k)) {  // the list's sum is the row's
      low = high = max((uint64_t)1, share_of(q.top_p, sh.found[1], true));
    } else {
      // the first k, where they are more than are listed, weigh at least what is listed
      low = max((uint64_t)1, share_of(q.top_p, q.k ? sh.found[0] : q.total - q.off, true));
      high = max((uint64_t)1, share_of(q.top_p, q.total + q.off, true));
      sure = (q.all && !q.k) || sh.found[0] >= high;
    }
  }
  const bool in = first_of && place < first && (uint32_t)(own_key >> 32) >= q.least;
  const int kept = __syncthreads_count(in && before < low), kept_high = __syncthreads_count(in && before < high);
  // Where neither top_k, top_p nor min_p ended the list, those without a weight are kept as well.
  const bool open = kept == q.n && low == ~0ull && !(q.k > 0 && q.k <= q.n);
  const bool enough = kept == kept_high && (sure || kept < q.n) && !(open && q.rest == 0);
  decided(enough ? kDone : kNotEnough);
  if (!enough) return;
  const uint64_t said = open && q.rest != kNoRest ? q.rest : (uint64_t)kept;
  const bool stays = entry && place < kept;
  if (first_of && place == kept - 1) sh.found[2] = before + own;
  // What stays, in the order of indices: the first `kept` places of the order hold its indices now (a larger complement is
  // earlier) and weights.
  uint32_t *index = reinterpret_cast<uint32_t *>(sh.all);
  __syncthreads();
  if (first_of && stays) index[place] = (uint32_t)own_key, sh.weight[place] = own;
  __syncthreads();
  int share = 1;  // threads each of them takes
  while (share < 32 && 2 * share * kept <= kSampleThreads) share *= 2;
  const int i = t / share;
  const bool asked = i < kept;
  const uint32_t own_index = asked ? index[i] : 0;
  uint64_t from = 0;
#pragma unroll 4
  for (int j = t & (share - 1); j < kept; j += share)
    if (index[j] > own_index) from += sh.weight[j];
  for (int o = share / 2; o; o >>= 1) from += __shfl_xor_sync(~0u, from, o);
  const uint64_t total = sh.found[2], target = share_of(u, total, false), mass = asked ? sh.weight[i] : 0;
  if (asked && (t & (share - 1)) == 0 && from <= target && target < from + mass) {
    *token = (int32_t)~own_index;
    if (kept_out) *kept_out = (int32_t)said;
    if (prob) *prob = __fdiv_rn((float)mass, (float)total);
  }
}

// A beginning of the order that fits a list, and the result from it.  Where it ends follows from the largest logits of
// the row's parts: the m-th of these has at least m tokens at or above it, and few more.  All blocks gather what is at
// or above it, or what min_p leaves, and the first block draws.  kDone: the cluster is done with the row.
__device__ int Row::try_list(ListArgs q, const float (&tops)[2], float u, int32_t *token, int32_t *kept, float *prob) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  float least = q.k ? -3.402823466e38f : logit_of(q.least);  // what min_p leaves of the first k is found among them
  int bins = q.bins;
  q.all = true;
  if (t == 0) sh.count = 0;
  if (q.wanted && !bins) {
    // every block counts the same largest logits
    uint32_t *counts = sh.counts(hist_turn);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = rough_exponent(scale, tops[i]);
      if (x < kNoWeight) atomicAdd(&counts[bin_of(x)], 1u);
    }
    __syncthreads();
    const uint32_t upto = block_scan(counts[t], sh);
    bins = 1 + __syncthreads_count(upto < (uint32_t)q.wanted);
    counts[t] = 0;
  } else {
    __syncthreads();
  }
  if (bins) {
    // a little below the bins' end, so that rounding leaves none of them out
    q.all = bins >= kBins;
    const float depth = __fdiv_ru(q.all ? kNoWeight * 1.00001f : bins * (1.00001f / kBinsAOctave), scale.hi);
    const float from = __fsub_rd(scale.top, depth);
    if (from > least) least = from;
    else q.all = true;
  }
  float sum = 0.f;
  const bool weigh = q.top_p < 1.f && !(q.k && q.k <= kManyTokens) && q.total == 0;
#pragma unroll 2
  for (int i = t; i < padded / 4; i += kSampleThreads) {
    const float4 v4 = reinterpret_cast<const float4 *>(l)[i];
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
    if (fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) >= least) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v[j] >= least) list(4 * i + j, v[j]);
    }
    if (weigh)
      sum += (fast_weight(scale, v[0]) + fast_weight(scale, v[1])) + (fast_weight(scale, v[2]) + fast_weight(scale, v[3]));
  }
  // the sum of the block's weights, always in the same order
  if (weigh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) sh.warp_sum[warp][0] = __float_as_uint(sum);
  }
  __syncthreads();
  if (warp == 0) {
    float s = weigh && lane < kSampleWarps ? __uint_as_float((uint32_t)sh.warp_sum[lane][0]) : 0.f;
#pragma unroll
    for (int o = kSampleWarps / 2; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0) sh.values[turn][0] = sh.count, sh.values[turn][1] = __float_as_uint(s);
  }
  cluster_barrier();
  int from, place;
  q.n = (int)min((uint64_t)kList + 1, my_entry(turn, from, place));
  const int here = turn;
  turn ^= 1;
  if (weigh) {
    // Weights are off by 1.1e-6 (the distance's rounding times its place, ex2), their sum of up to 24 times four a thread
    // and 31 more by 57 * 2^-24: 4.5e-6 together, below 2^-17.
    float whole = 0.f;
    each_peer(&sh.values[here][1], cluster, [&](int, uint64_t v) { whole += __uint_as_float((uint32_t)v); });
    set_unit(whole);
    total = q.total = (uint64_t)(whole * __uint_as_float((uint32_t)(127 + scale.bits) << 23)), off = q.off = q.total >> 17;
  } else if (!summed) {
    scale.bits = kListBits;
  }
  if (q.n > kList || q.n == 0) return kNotEnough;
  // The other blocks leave, and make room for the next row's, as soon as the first has read their lists or said that they are
  // enough; it says so in their own shared memory, so that nobody reads another block's after that.
  const uint64_t mine = rank == 0 && t < q.n ? peer(&sh.list[here][place], from) : 0;
  const bool always = q.k > 0 && q.k <= q.n;  // enough, whatever it holds
  int result = kDone;
  if (always) cluster_barrier();
  if (rank == 0) {
    draw_from_list(*this, q, mine, u, token, kept, prob, [&](int r) {
      result = r;
      if (always) return;
      if (t < cluster) put_peer(&sh.values[turn][0], t, (uint64_t)r);
      cluster_barrier();
    });
  } else if (!always) {
    cluster_barrier();
    result = (int)sh.values[turn][0];
  }
  turn ^= 1;
  return result;
}

// The row of cluster number n: where not all rows find room at once, in every run of kSampleThreads rows those whose settings may
// need the long way come first, so that the last ones to start are short.  (64 rows of 151,936 with settings of all sorts: 70 -> 57
// us, or 79 -> 67; what it costs a batch whose rows are all alike is a microsecond a round, 64 with top_k 20: 25.8 -> 27.5.)
__device__ __forceinline__ int64_t row_of(const SampleArgs &a, int64_t n, SampleShared &sh) {
  if (!a.ordered) return n;
  const int t = threadIdx.x, at = (int)(n % kSampleThreads);
  const int64_t base = n - at;
  const bool here = base + t < a.B;
  const int k = here && a.top_k ? a.top_k[base + t] : 0;
  const float top_p = here && a.top_p ? a.top_p[base + t] : 1.f;
  const bool by_k = k > 0 && k < a.V;
  const bool slow = here && (top_p < 1.f ? !by_k || k > kManyTokens : by_k && k > kManyTokens);
  const int upto = (int)block_scan((uint32_t)slow, sh), all = __syncthreads_count(slow);
  if (here && (slow ? upto - 1 : all + t - upto) == at) sh.found[0] = t;
  __syncthreads();
  return base + (int64_t)sh.found[0];
}

template <typename Ty>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(SampleArgs a) {
  __shared__ SampleShared sh;
  extern __shared__ __align__(16) float s_logits[];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = blockIdx.x % a.cluster;
  if (t < 256) sh.table[t] = make_float2(kExpTable.hi[t], kExpTable.lo[t]);
  sh.hist[0][t] = 0;
  pdl_wait();
  next_may_start();
  const int64_t b = row_of(a, blockIdx.x / a.cluster, sh);
  // on their way while the row is
  const float temperature = a.temperature ? a.temperature[b] : 1.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float top_p = a.top_p ? a.top_p[b] : 1.f, min_p = a.min_p ? a.min_p[b] : 0.f;
  const float u = fminf(fmaxf(a.u[b], 0.f), 0x1.fffffep-1f);
  using Elem = typename Logits<Ty>::Elem;
  const Elem *logits = static_cast<const Elem *>(a.logits) + b * a.ts;
  // places of 16 bytes in memory, the first of them perhaps before the row
  const int shift = (int)(((uintptr_t)logits & 15) / sizeof(Elem));
  const int first = rank * a.slice - shift, count = max(0, min(a.slice, a.V - first)), padded = (count + kStep - 1) / kStep * kStep;
  uint32_t drawable = 0;
  float top = load_row<Ty>(logits, first, padded, a.V, s_logits, drawable);
  const bool greedy = !(temperature >= 0x1p-100f);
  const bool by_k = k > 0 && k < a.V, by_p = top_p < 1.f, by_min = min_p > 0.f;

  // Every block gets the largest logits of 1024 parts of the row (512 with one block), two a thread, and how many of its
  // logits can be drawn.
  const int lanes = max(1, a.cluster / 2);  // threads a part
  for (int o = 1; o < lanes; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if ((t & (lanes - 1)) == 0) sh.tops[t / lanes] = top;
  drawable = __reduce_add_sync(~0u, drawable);
  if (lane == 0) sh.warp_sum[warp][0] = drawable;
  __syncthreads();
  if (warp == 0) {
    const uint32_t sum = __reduce_add_sync(~0u, lane < kSampleWarps ? (uint32_t)sh.warp_sum[lane][0] : 0);
    if (lane == 0) sh.values[0][0] = sum;
  }
  cluster_barrier();
  float tops[2] = {-INFINITY, -INFINITY};
  {
    const int pairs = kSampleThreads / lanes / 2;  // of a block
    if (t / pairs < a.cluster) {
      const uint64_t two = peer(reinterpret_cast<const uint64_t *>(sh.tops) + t % pairs, t / pairs);
      tops[0] = __uint_as_float((uint32_t)two), tops[1] = __uint_as_float((uint32_t)(two >> 32));
    }
  }
  uint64_t usable_count = 0;
  each_peer(&sh.values[0][0], a.cluster, [&](int, uint64_t v) { usable_count += v; });
  const uint32_t warp_top = __reduce_max_sync(~0u, key_of(fmaxf(tops[0], tops[1])));
  if (lane == 0) sh.warp_sum[warp][1] = warp_top;
  __syncthreads();
  const uint32_t best = __reduce_max_sync(~0u, (uint32_t)sh.warp_sum[lane % kSampleWarps][1]);
  top = logit_of(best);
  Row row{sh, s_logits, Scale{top, 0.f, 0.f, kFreeBits}, rank, a.cluster, first, padded, 1, 0, 0, 0, false};

  if (best == kKeyNone) {
    if (rank == 0 && t == 0) {
      a.token[b] = -1;
      if (a.kept) a.kept[b] = 0;
      if (a.prob) a.prob[b] = 0.f;
      record_index_error(a.hdr);
    }
    cluster_barrier();
    return;
  }
  if (greedy) {
    uint32_t at = ~0u;
    row.each([&](int i, float v) {
      if (v == top) at = min(at, (uint32_t)(first + i));
    });
    at = __reduce_min_sync(~0u, at);
    if (t == 0) sh.found[0] = ~0ull;
    __syncthreads();
    if (lane == 0) atomicMin(reinterpret_cast<uint32_t *>(&sh.found[0]), at);
    __syncthreads();
    if (t == 0) sh.values[1][0] = (uint32_t)sh.found[0];
    cluster_barrier();
    if (rank == 0 && t == 0) {
      uint32_t least = ~0u;
      each_peer(&sh.values[1][0], a.cluster, [&](int, uint64_t v) { least = min(least, (uint32_t)v); });
      a.token[b] = (int32_t)least;
      if (a.kept) a.kept[b] = 1;
      if (a.prob) a.prob[b] = 1.f;
    }
    cluster_barrier();
    return;
  }
  const bool infinite = top == INFINITY;
  if (infinite) {  // beside it nothing counts, and all of them count the same
    uint64_t n = 0, none = 0;
    for (int i = t; i < padded; i += kSampleThreads) {
      const bool is = s_logits[i] == INFINITY;
      s_logits[i] = is ? 0.f : -INFINITY, n += is;
    }
    row.scale.top = top = 0.f;
    for (int i = 0; i < 2; ++i) tops[i] = tops[i] == INFINITY ? 0.f : -INFINITY;
    row.exchange(n, none);
    usable_count = n;
  }
  {
    constexpr float log2e = 1.44269504088896340736f, log2e_lo = (float)(1.44269504088896340736 - (double)log2e);
    row.scale.hi = __fdiv_rn(log2e, temperature);
    row.scale.lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-row.scale.hi, temperature, log2e), log2e_lo), temperature);
    if (temperature == INFINITY) row.scale.hi = row.scale.lo = 0.f;
  }
  uint32_t least = kKeyNone + 1;  // the smallest key there is to keep
  if (by_min) {
    // the smallest logit whose weight is not below: max + T ln(min_p), rounded up
    if (t == 0) sh.cut = __double2float_ru((double)top + (double)temperature * log(fmin((double)min_p, 1.0)));
    __syncthreads();
    least = max(least, key_of(usable(sh.cut)));
  }

  Cut cut{kKeyNone, 0};
  int stepped = -1;
  if (by_k || by_p || by_min) {
    // With a min_p that has a weight, those without a weight are not kept.
    const bool by_weight = min_p >= 0x1p-44f;
    const uint64_t rest = by_weight ? kNoRest : by_min ? 0 : min(usable_count, by_k ? (uint64_t)k : usable_count);
    ListArgs q{by_k ? k : 0, by_p ? top_p : 1.f, least, by_k ? k : by_weight ? 0 : kFewTokens, 0, rest, 0, 0, 0, false};
    const auto enough = [&] {
      return row.try_list(q, tops, u, a.token + b, a.kept ? a.kept + b : nullptr, a.prob ? a.prob + b : nullptr) == kDone;
    };
    if (by_k && k > kManyTokens) {
      // top_p is likely to keep few of so many, whatever they weigh between what is listed and all
      q.wanted = kFewTokens;
      if (by_p && enough()) return;
    } else if (enough()) {
      return;
    }
    if (!row.summed && !by_k) row.find_unit();
    uint64_t target = 0;
    if (by_k) {
      row.select<false>(Row::Members{}, 0, false, (uint64_t)k, cut);
      if (by_p) {
        q.k = 0, q.total = row.mass(cut), q.off = 0, q.wanted = kFewTokens, q.rest = kNoRest;
        if (enough()) return;
        target = max((uint64_t)1, share_of(top_p, q.total, true));
      }
    }
    if (by_p) {
      int few = 0;
      row.select_share(top_p, target, cut, stepped, few);
      if (few) {
        if (!by_k) q.total = row.total, q.off = row.off;
        q.bins = few;
        if (enough()) return;
        few = -1;  // next to a border: exactly, then
        row.select_share(top_p, target, cut, stepped, few);
      }
    }
    if (least > cut.key) cut = Cut{least - 1, 0}, stepped = -1;
  }
  // Without a filter: sums in fp32 first, enough unless u falls next to the border between two tokens.
  if (!(by_k || by_p || by_min)) {
    if (row.draw<Row::kFast>(a, b, cut, u, k, usable_count, 0)) return;
    if (row.draw<Row::kNear>(a, b, cut, u, k, usable_count, 0)) return;
  }
  if (stepped >= 0) row.draw<Row::kStepped>(a, b, cut, u, k, usable_count, stepped);
  else row.draw<Row::kExact>(a, b, cut, u, k, usable_count, 0);
}

template <typename Ty>
static cudaError_t launch_type(SampleArgs a, int B, cudaStream_t st) {
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem<(size_t)kMaxSlice * 4>(sample_kernel<Ty>, done);
  if (e != cudaSuccess) return e;
  const auto slice = [&](int cluster) {  // a place more for what lies before the row in its first 16 bytes
    return ((a.V + 7 + cluster - 1) / cluster + kStep - 1) / kStep * kStep;
  };
  a.cluster = kMaxCluster;
  // Few rows: the most blocks a row.  Many: as few as leave room for two on an SM (200 rows of 50,257: 55 us with 8 a row,
  // 29 with 4 and 29 with 2, where one fits; 200 rows of 8000: 48, 25, 16).
  while (a.cluster > 1 && (int64_t)B * a.cluster > 2 * std::max(1, sm_count()) && slice(a.cluster / 2) * 4 <= 76 * 1024) a.cluster /= 2;
  a.slice = slice(a.cluster);
  a.ordered = (a.top_k || a.top_p) && (int64_t)B * a.cluster > 2 * sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * a.cluster);
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = (size_t)a.slice * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<Ty>, a);
}

int launch_sample(const lily_sampling &op, int B, int V, int dtype, const void *logits, int64_t ts, const float *u,
                  int32_t *token, float *prob, int32_t *kept, void *ws, cudaStream_t st) {
  const SampleArgs a{logits, ts, op.temperature, op.top_p, op.min_p, u, op.top_k, token, kept,
                     static_cast<int32_t *>(ws), prob, V, 0, 0, B, false};
  const cudaError_t e = dtype == LILY_BF16  ? launch_type<Bf16>(a, B, st)
                        : dtype == LILY_F16 ? launch_type<F16>(a, B, st)
                                            : launch_type<F32Logits>(a, B, st);
  return e == cudaSuccess ? LILY_Q4_OK : (cudaGetLastError(), LILY_Q4_ERR_CUDA);
}

}  // namespace lq4
