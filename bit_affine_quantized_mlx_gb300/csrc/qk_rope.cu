// lily_qk_norm_rope: the norm of every query and key head and the position rotation, one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset);   (y_a, y_b) rotated by pos * f
//
// Bound by memory: each head is read and written once (4 bytes an element); at small T by the
// launch.  A warp takes a token and all its heads (a share of them when there are few tokens),
// because the angles are the token's: their sines are computed once, and
// passed through shared memory of the warp's own to the lanes that keep them for all their heads; no
// barrier of the block is needed.  A head is held by 8, 16
// or 32 lanes, 8 elements in each: 8 neighbours, or, where the first R elements turn in half pairs,
// 4 of the lower half and their 4 partners of the upper.  So both elements of a pair are always in
// one lane and only the sum of squares is exchanged.  R / 2 that is not a multiple of 4 breaks the
// half pairs' runs of four: those heads go through shared memory.
//
// Angles: turns[i] is f_i / (2 pi) as a 64-bit fraction of a turn, so pos * turns[i] in wrapping
// 64-bit integers is the angle of any 32-bit position without loss; its top 32 bits, taken as
// signed, are the angle in [-1/2, 1/2) turns, which sincospif takes after a rounding of
// 2^-24 relative.  A 32-bit float product would be off by 0.06 rad at position 10^6.
//
// Measured on one GB300: 8192 tokens, 40 heads of 128 (168 MB): 30 us, 5.6 TB/s, 82% of the copy rate (52 us
// with a block a token and its angles behind a block barrier, 35 with single instead of paired fp32
// instructions: the rest is instruction issue); one token of 18 heads of 256: 2.4 us.
#include <algorithm>
#include <cmath>

#include "kv8_device.cuh"

namespace lq4 {

struct RopeRows {  // q or k
  const uint16_t *in, *weight;
  uint16_t *out;
  int64_t in_ts, in_hs, out_ts, out_hs;
  int heads;
};
struct RopeArgs {
  RopeRows part[2];
  const int32_t *pos;
  const uint64_t *turns;
  float eps, offset, rope_scale;
  int T, D, R, normalize;
};

constexpr int kRopeWarps = 4, kRopeAhead = 4;
enum RopePairs { kPairsNear, kPairsHalf, kPairsHalfOdd };

// LANES a head; kRopeAhead passes (32 / LANES heads each) are loaded together.
template <typename Ty, int PAIRS, int LANES>
__global__ void __launch_bounds__(32 * kRopeWarps, PAIRS == kPairsHalfOdd ? 6 : 7)
    qk_norm_rope_kernel(RopeArgs a, int shares) {
  constexpr int GROUPS = 32 / LANES;
  __shared__ __align__(16) float2 s_cs[kRopeWarps][128];
  __shared__ float s_row[PAIRS == kPairsHalfOdd ? kRopeWarps * 256 : 1];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t task = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int t = (int)(task / shares), share = (int)(task - (int64_t)t * shares);
  if (t >= a.T) return;
  const int c = lane & (LANES - 1), g = lane / LANES;
  const bool live = c * 8 < a.D;
  const int half = a.R >> 1;
  // this lane's elements: e0 .. e0 + 3 and e1 .. e1 + 3
  const bool apart = PAIRS == kPairsHalf && c * 8 < a.R;
  const int e0 = live ? (apart ? 4 * c : 8 * c) : 0, e1 = live ? (apart ? half + 4 * c : 8 * c + 4) : 0;
  // this warp's heads, queries' first
  const int heads = a.part[0].heads + a.part[1].heads, per = (heads + shares - 1) / shares;
  const int from = share * per, to = min(heads, from + per);
  float2 *cs_of = s_cs[warp];
  uint64_t co[2], si[2], no[2];  // cosines, sines and their negatives of the lane's four pairs
  bool angles = false;
  const float inv_d = 1.f / (float)a.D;

#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const RopeRows &p = a.part[w];
    const int skip = w ? a.part[0].heads : 0;
    const int h_begin = max(from - skip, 0), h_end = min(to - skip, p.heads);
    if (h_begin >= h_end) continue;
    const uint16_t *src = p.in + t * p.in_ts + (int64_t)(h_begin + g) * p.in_hs;
    uint16_t *dst = p.out + t * p.out_ts + (int64_t)(h_begin + g) * p.out_hs;
    const int64_t in_step = GROUPS * p.in_hs, out_step = GROUPS * p.out_hs;
    int left = live ? h_end - h_begin - g : 0;  // heads of this lane's group still to do, times GROUPS
    uint2 raw[kRopeAhead][2];
    auto load = [&]() {
#pragma unroll
      for (int i = 0; i < kRopeAhead; ++i) {
        raw[i][0] = raw[i][1] = make_uint2(0, 0);
        if (left > i * GROUPS) {
          raw[i][0] = *reinterpret_cast<const uint2 *>(src + i * in_step + e0);
          raw[i][1] = *reinterpret_cast<const uint2 *>(src + i * in_step + e1);
        }
      }
    };
    load();
    float wt[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[j] = 1.f;
    if (a.normalize && p.weight) {
      const uint2 lo = *reinterpret_cast<const uint2 *>(p.weight + e0), hi = *reinterpret_cast<const uint2 *>(p.weight + e1);
      unpack8<Ty>(make_uint4(lo.x, lo.y, hi.x, hi.y), wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) wt[j] += a.offset;
    }
    // the lane's elements as first and second members of its pairs, two pairs together
    uint64_t w2[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w2[0][j] = PAIRS == kPairsNear ? pack2(wt[4 * j], wt[4 * j + 2]) : pack2(wt[2 * j], wt[2 * j + 1]);
      w2[1][j] = PAIRS == kPairsNear ? pack2(wt[4 * j + 1], wt[4 * j + 3]) : pack2(wt[4 + 2 * j], wt[5 + 2 * j]);
    }
    if (!angles) {  // the loads are under way
      angles = true;
      if (half > 0) {
        const uint64_t pos = (uint64_t)(int64_t)a.pos[t];
        for (int i = lane; i < half; i += 32) {
          float sn, cn;
          sincospif((float)(int32_t)((pos * a.turns[i]) >> 32) * 0x1p-31f, &sn, &cn);
          cs_of[i] = make_float2(cn * a.rope_scale, sn * a.rope_scale);
        }
        __syncwarp();
      }
      // pairs beyond R turn by nothing
      float2 cs[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        cs[j] = PAIRS != kPairsHalfOdd && live && 4 * c + j < half ? cs_of[4 * c + j] : make_float2(1.f, 0.f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        co[j] = pack2(cs[2 * j].x, cs[2 * j + 1].x);
        si[j] = pack2(cs[2 * j].y, cs[2 * j + 1].y);
        no[j] = pack2(-cs[2 * j].y, -cs[2 * j + 1].y);
      }
    }
    for (int base = h_begin; base < h_end; base += kRopeAhead * GROUPS) {
      if (base > h_begin) load();
#pragma unroll
      for (int i = 0; i < kRopeAhead; ++i) {
        if (base + i * GROUPS >= h_end) break;  // the same for every lane
        float y[8];
        unpack8<Ty>(make_uint4(raw[i][0].x, raw[i][0].y, raw[i][1].x, raw[i][1].y), y);
        uint64_t u[2], v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          u[j] = PAIRS == kPairsNear ? pack2(y[4 * j], y[4 * j + 2]) : pack2(y[2 * j], y[2 * j + 1]);
          v[j] = PAIRS == kPairsNear ? pack2(y[4 * j + 1], y[4 * j + 3]) : pack2(y[4 + 2 * j], y[5 + 2 * j]);
        }
        if (a.normalize) {
          uint64_t s2 = mul2(u[0], u[0]);
          s2 = fma2(u[1], u[1], s2);
          s2 = fma2(v[0], v[0], s2);
          s2 = fma2(v[1], v[1], s2);
          const float2 both = unpack2(s2);
          float ss = both.x + both.y;
#pragma unroll
          for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
          const float rs = rsqrtf(fmaf(ss, inv_d, a.eps));
          const uint64_t rs2 = pack2(rs, rs);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            u[j] = mul2(u[j], mul2(rs2, w2[0][j]));
            v[j] = mul2(v[j], mul2(rs2, w2[1][j]));
          }
        }
        if (PAIRS != kPairsHalfOdd) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint64_t x = fma2(u[j], co[j], mul2(v[j], no[j]));
            v[j] = fma2(u[j], si[j], mul2(v[j], co[j]));
            u[j] = x;
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 p = unpack2(u[j]), q = unpack2(v[j]);
          if (PAIRS == kPairsNear) {
            y[4 * j] = p.x, y[4 * j + 2] = p.y, y[4 * j + 1] = q.x, y[4 * j + 3] = q.y;
          } else {
            y[2 * j] = p.x, y[2 * j + 1] = p.y, y[4 + 2 * j] = q.x, y[5 + 2 * j] = q.y;
          }
        }
        if (PAIRS == kPairsHalfOdd) {
          float *row = s_row + warp * 256 + (lane - c) * 8;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) row[c * 8 + j] = y[j];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = c * 8 + j;
            if (e < a.R) {
              const bool low = e < half;
              const float other = row[low ? e + half : e - half];
              const float2 k = cs_of[low ? e : e - half];
              y[j] = low ? y[j] * k.x - other * k.y : other * k.y + y[j] * k.x;
            }
          }
        }
        if (left > i * GROUPS) {
          const uint4 o = pack8<Ty>(y);
          *reinterpret_cast<uint2 *>(dst + i * out_step + e0) = make_uint2(o.x, o.y);
          *reinterpret_cast<uint2 *>(dst + i * out_step + e1) = make_uint2(o.z, o.w);
        }
      }
      src += kRopeAhead * in_step;
      dst += kRopeAhead * out_step;
      left -= kRopeAhead * GROUPS;
    }
  }
}

template <typename Ty, int PAIRS, int LANES>
static cudaError_t launch_lanes(const RopeArgs &a, cudaStream_t st) {
  // A token's heads are shared out until there are about two warps for each that fits on the GPU (28 an
  // SM), down to one pass a warp, at the price of computing the token's sines in each (8192 tokens of
  // 40 heads of 128: 30 us with a warp a token, 32 with two, 37 with four).
  const int passes = (a.part[0].heads + a.part[1].heads + 32 / LANES - 1) / (32 / LANES);
  const int sms = sm_count() > 0 ? sm_count() : 1;
  const int shares = std::max(1, std::min(passes, 54 * sms / a.T));
  const int64_t tasks = (int64_t)a.T * shares;
  return launch_pdl(qk_norm_rope_kernel<Ty, PAIRS, LANES>, dim3((unsigned)((tasks + kRopeWarps - 1) / kRopeWarps)),
                    dim3(32 * kRopeWarps), 0, st, a, shares);
}

template <typename Ty, int PAIRS>
static cudaError_t launch_pairs(const RopeArgs &a, cudaStream_t st) {
  if (a.D <= 64) return launch_lanes<Ty, PAIRS, 8>(a, st);
  if (a.D <= 128) return launch_lanes<Ty, PAIRS, 16>(a, st);
  return launch_lanes<Ty, PAIRS, 32>(a, st);
}

template <typename Ty>
static cudaError_t launch_type(const RopeArgs &a, bool interleaved, cudaStream_t st) {
  if (interleaved) return launch_pairs<Ty, kPairsNear>(a, st);
  if (a.R % 8 == 0) return launch_pairs<Ty, kPairsHalf>(a, st);
  return launch_pairs<Ty, kPairsHalfOdd>(a, st);
}

int launch_qk_norm_rope(const lily_qk_rope &op, int T, int q_heads, int k_heads, const int32_t *pos,
                        const Rows &q, const Rows &q_out, const Rows &k, const Rows &k_out,
                        cudaStream_t st) {
  RopeArgs a = {};
  const Rows *in[2] = {&q, &k}, *out[2] = {&q_out, &k_out};
  const void *weight[2] = {op.q_weight, op.k_weight};
  for (int w = 0; w < 2; ++w)
    a.part[w] = RopeRows{static_cast<const uint16_t *>(in[w]->p), static_cast<const uint16_t *>(weight[w]),
                         static_cast<uint16_t *>(out[w]->p), in[w]->ts, in[w]->hs, out[w]->ts, out[w]->hs,
                         w ? k_heads : q_heads};
  a.pos = pos;
  a.turns = op.turns;
  a.eps = op.eps;
  a.offset = op.weight_offset;
  a.rope_scale = op.rope_scale;
  a.T = T;
  a.D = op.head_dim;
  a.R = op.rotary_dim;
  a.normalize = op.normalize;
  const cudaError_t e = op.dtype == LILY_BF16 ? launch_type<Bf16>(a, op.interleaved, st)
                                              : launch_type<F16>(a, op.interleaved, st);
  return e == cudaSuccess ? LILY_Q4_OK : (cudaGetLastError(), LILY_Q4_ERR_CUDA);
}

int rope_turns(int R, double base, int scaling, double factor, double original_len, double slow,
               double fast, uint64_t *turns) {
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (scaling == LILY_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == LILY_ROPE_YARN) {
      const double n = original_len * f / two_pi;  // turns within the original context
      double keep = (n - slow) / (fast - slow);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      f = f * keep + f / factor * (1 - keep);
    }
    double turn = f / two_pi;
    turn -= std::floor(turn);
    // ldexp(turn, 64) < 2^64 because turn <= 1 - 2^-53
    turns[i] = (uint64_t)std::ldexp(turn, 64);
  }
  return LILY_Q4_OK;
}

}  // namespace lq4
