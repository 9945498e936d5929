// lily_qk_norm_rope: the norm of every query and key head and the position rotation, one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset);   (y_a, y_b) rotated by pos * f
//
// Bound by memory: each head is read and written once (4 bytes an element); at small T by the
// launch.  A block takes tokens and all their heads (or a share of them when there are few
// tokens), because the angles are the token's: their sines are computed once a token into shared
// memory, not once a head, and a lane keeps its own for all its heads.  A head is held by a power of
// two of lanes, 8 elements in each: 8 neighbours, or, where the first R elements turn in half pairs,
// 4 of the lower half and their 4 partners of the upper.  So both elements of a pair are always in
// one lane and only the sum of squares is exchanged.  R / 2 that is not a multiple of 4 breaks the
// half pairs' runs of four: those heads go through shared memory.
//
// Angles: turns[i] is f_i / (2 pi) as a 64-bit fraction of a turn, so pos * turns[i] in wrapping
// 64-bit integers is the angle of any 32-bit position without loss; its top 32 bits, taken as
// signed, are the angle in [-1/2, 1/2) turns, which sincospif takes after a rounding of
// 2^-24 relative.  A 32-bit float product would be off by 0.06 rad at position 10^6.
#include <cmath>

#include "kv8_device.cuh"

namespace lq4 {

struct RopeArgs {
  const int32_t *pos;
  const void *in[2];
  void *out[2];
  const void *weight[2];
  int64_t in_ts[2], in_hs[2], out_ts[2], out_hs[2];
  const uint64_t *turns;
  float eps, offset, rope_scale;
  int T, q_heads, heads, D, R, lanes_shift, normalize;
};

constexpr int kRopeThreads = 256;
enum RopePairs { kPairsNear, kPairsHalf, kPairsHalfOdd };

// PASSES: heads a lane group takes in one go.  A block walks tokens gridDim.x apart; the next
// token's first heads are loaded before the current one's are computed.
template <typename Ty, int PAIRS, int PASSES>
__global__ void __launch_bounds__(kRopeThreads, PAIRS == kPairsHalfOdd ? 3 : 5)
    qk_norm_rope_kernel(RopeArgs a) {
  __shared__ __align__(16) float2 s_cs[2][128];
  __shared__ float s_row[PAIRS == kPairsHalfOdd ? (kRopeThreads / 32) * 256 : 1];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = 1 << a.lanes_shift, c = lane & (lanes - 1);
  const int groups = kRopeThreads >> a.lanes_shift;
  const int g = threadIdx.x >> a.lanes_shift;
  const bool live = c * 8 < a.D;
  const int half = a.R >> 1;
  // this lane's elements: e0 .. e0 + 3 and e1 .. e1 + 3
  const bool split = PAIRS == kPairsHalf && c * 8 < a.R;
  const int e0 = live ? (split ? 4 * c : 8 * c) : 0, e1 = live ? (split ? half + 4 * c : 8 * c + 4) : 0;
  const bool turns = PAIRS != kPairsHalfOdd && live && 4 * c < half;
  // this block's heads
  const int per = (a.heads + gridDim.y - 1) / gridDim.y;
  const int h_begin = blockIdx.y * per, h_end = min(a.heads, h_begin + per);

  uint2 raw[PASSES][2];
  auto load = [&](int t, int base) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int h = base + i * groups + g;
      raw[i][0] = raw[i][1] = make_uint2(0, 0);
      if (t < a.T && h < h_end && live) {
        const int w = h >= a.q_heads;
        const uint16_t *src = static_cast<const uint16_t *>(a.in[w]) + t * a.in_ts[w] +
                              (int64_t)(w ? h - a.q_heads : h) * a.in_hs[w];
        raw[i][0] = *reinterpret_cast<const uint2 *>(src + e0);
        raw[i][1] = *reinterpret_cast<const uint2 *>(src + e1);
      }
    }
  };
  load(blockIdx.x, h_begin);
  auto angles = [&](int t, int buf) {
    if (t < a.T && (int)threadIdx.x < half) {
      const uint64_t turn = (uint64_t)(int64_t)a.pos[t] * a.turns[threadIdx.x];
      float sn, cs;
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
      s_cs[buf][threadIdx.x] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
    }
  };
  angles(blockIdx.x, 0);
  uint2 wraw[2][2] = {};
  if (a.normalize && live) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (!a.weight[w]) continue;
      const uint16_t *src = static_cast<const uint16_t *>(a.weight[w]);
      wraw[w][0] = *reinterpret_cast<const uint2 *>(src + e0);
      wraw[w][1] = *reinterpret_cast<const uint2 *>(src + e1);
    }
  }
  const float inv_d = 1.f / (float)a.D;
  int buf = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
    __syncthreads();  // this token's sines are there, the last one's have been read
    const float2 *cs_of = s_cs[buf];
    float2 cs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[j] = turns && 4 * c + j < half ? cs_of[4 * c + j] : make_float2(1.f, 0.f);
    for (int base = h_begin; base < h_end; base += PASSES * groups) {
      uint2 cur[PASSES][2];
#pragma unroll
      for (int i = 0; i < PASSES; ++i) cur[i][0] = raw[i][0], cur[i][1] = raw[i][1];
      const bool last = base + PASSES * groups >= h_end;
      load(last ? t + gridDim.x : t, last ? h_begin : base + PASSES * groups);
      if (last) angles(t + gridDim.x, buf ^ 1);
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int h = base + i * groups + g;
        if (base + i * groups >= h_end) break;  // the same for every thread of the block
        const int w = h >= a.q_heads;
        float y[8];
        unpack8<Ty>(make_uint4(cur[i][0].x, cur[i][0].y, cur[i][1].x, cur[i][1].y), y);
        if (a.normalize) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
          for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
          const float rs = rsqrtf(fmaf(ss, inv_d, a.eps));
          if (w ? a.weight[1] != nullptr : a.weight[0] != nullptr) {
            float wt[8];
            unpack8<Ty>(w ? make_uint4(wraw[1][0].x, wraw[1][0].y, wraw[1][1].x, wraw[1][1].y)
                          : make_uint4(wraw[0][0].x, wraw[0][0].y, wraw[0][1].x, wraw[0][1].y), wt);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= rs * (wt[j] + a.offset);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= rs;
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
        } else if (turns) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (PAIRS == kPairsNear && 4 * c + j >= half) break;
            float &u = PAIRS == kPairsNear ? y[2 * j] : y[j];
            float &v = PAIRS == kPairsNear ? y[2 * j + 1] : y[4 + j];
            const float x = u * cs[j].x - v * cs[j].y;
            v = u * cs[j].y + v * cs[j].x;
            u = x;
          }
        }
        if (h < h_end && live) {
          uint16_t *dst = static_cast<uint16_t *>(a.out[w]) + t * a.out_ts[w] +
                          (int64_t)(w ? h - a.q_heads : h) * a.out_hs[w];
          const uint4 o = pack8<Ty>(y);
          *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(o.x, o.y);
          *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(o.z, o.w);
        }
      }
    }
  }
}

template <typename Ty, int PAIRS>
static cudaError_t launch_pairs(const RopeArgs &a, cudaStream_t st) {
  const int groups = kRopeThreads >> a.lanes_shift;
  // Enough blocks for every SM: with fewer tokens than that a token's heads are shared out, down
  // to one pass a block, at the price of computing its sines in each.
  const int passes = (a.heads + groups - 1) / groups;
  const int sms = sm_count() > 0 ? sm_count() : 1;
  const int split = max(1, min(passes, 2 * sms / a.T));
  // more tokens than resident blocks: the blocks walk them
  const dim3 grid(min(a.T, 6 * sms), split);
  if ((passes + split - 1) / split <= 1)
    return launch_pdl(qk_norm_rope_kernel<Ty, PAIRS, 1>, grid, dim3(kRopeThreads), 0, st, a);
  return launch_pdl(qk_norm_rope_kernel<Ty, PAIRS, 3>, grid, dim3(kRopeThreads), 0, st, a);
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
  a.pos = pos;
  const Rows *in[2] = {&q, &k}, *out[2] = {&q_out, &k_out};
  for (int w = 0; w < 2; ++w) {
    a.in[w] = in[w]->p;
    a.in_ts[w] = in[w]->ts;
    a.in_hs[w] = in[w]->hs;
    a.out[w] = out[w]->p;
    a.out_ts[w] = out[w]->ts;
    a.out_hs[w] = out[w]->hs;
  }
  a.weight[0] = op.q_weight;
  a.weight[1] = op.k_weight;
  a.turns = op.turns;
  a.eps = op.eps;
  a.offset = op.weight_offset;
  a.rope_scale = op.rope_scale;
  a.T = T;
  a.q_heads = q_heads;
  a.heads = q_heads + k_heads;
  a.D = op.head_dim;
  a.R = op.rotary_dim;
  a.normalize = op.normalize;
  while ((8 << a.lanes_shift) < a.D) ++a.lanes_shift;
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
