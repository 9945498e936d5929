// lily_qk_norm_rope: the norm of every query and key head and the position rotation, one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset);   (y_a, y_b) rotated by pos * f
//
// Bound by memory: each head is read and written once (4 bytes an element); at small T by the
// launch.  A block takes one token and all its heads (or a share of them when there are few
// tokens), because the angles are the token's: their sines are computed once a block into shared
// memory, not once a head.  A head is held by a power of two of lanes, 8 elements (16 bytes) in
// each, so its sum of squares is a few shuffles and its rotation partner sits in the same lane
// (neighbouring pairs) or in one other lane (half pairs with R / 2 a multiple of 8); for other R
// the heads go through shared memory.
//
// Angles: turns[i] is f_i / (2 pi) as a 64-bit fraction of a turn, so pos * turns[i] in wrapping
// 64-bit integers is the angle of any 32-bit position without loss; its top 32 bits, taken as
// signed, are the angle in half-open (-1/2, 1/2] turns, which sincospif takes after a rounding of
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

// PASSES: heads a lane group takes in one go; their loads are all issued before the sines.
template <typename Ty, int PAIRS, int PASSES>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(RopeArgs a) {
  __shared__ float2 s_cs[128];
  __shared__ float s_row[PAIRS == kPairsHalfOdd ? (kRopeThreads / 32) * 256 : 1];
  pdl_wait();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = 1 << a.lanes_shift, c = lane & (lanes - 1);  // chunk of 8 elements
  const int groups = kRopeThreads >> a.lanes_shift;
  const int g = threadIdx.x >> a.lanes_shift;
  const bool live = c * 8 < a.D;
  // this block's heads
  const int per = (a.heads + gridDim.y - 1) / gridDim.y;
  const int h_begin = blockIdx.y * per, h_end = min(a.heads, h_begin + per);

  uint4 raw[PASSES];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int h = base + i * groups + g;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (h < h_end && live) {
        const int w = h >= a.q_heads;
        const int64_t off = t * a.in_ts[w] + (int64_t)(w ? h - a.q_heads : h) * a.in_hs[w] + c * 8;
        raw[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.in[w]) + off);
      }
    }
  };
  load(h_begin);
  const int half = a.R >> 1;
  if ((int)threadIdx.x < half) {
    const uint64_t turn = (uint64_t)(int64_t)a.pos[t] * a.turns[threadIdx.x];
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cs[threadIdx.x] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
  }
  float wt[2][8];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (a.weight[w] && live && a.normalize) {
      unpack8<Ty>(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.weight[w]) + c * 8), wt[w]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) wt[w][i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) wt[w][i] = a.weight[w] ? wt[w][i] + a.offset : 1.f;
  }
  __syncthreads();

  for (int base = h_begin; base < h_end; base += PASSES * groups) {
    if (base != h_begin) load(base);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int h = base + i * groups + g;
      if (base + i * groups >= h_end) break;  // the same for every thread of the block
      const int w = h >= a.q_heads;
      float y[8];
      unpack8<Ty>(raw[i], y);
      if (a.normalize) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
        for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float rs = rsqrtf(ss / (float)a.D + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * rs * (w ? wt[1][j] : wt[0][j]);
      }
      if (PAIRS == kPairsNear) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = c * 4 + j;
          if (p < half) {
            const float2 cs = s_cs[p];
            const float u = y[2 * j], v = y[2 * j + 1];
            y[2 * j] = u * cs.x - v * cs.y;
            y[2 * j + 1] = u * cs.y + v * cs.x;
          }
        }
      } else if (PAIRS == kPairsHalf) {
        // chunk c pairs with chunk c +- R/16, in the same head's lanes
        const int step = a.R >> 4;
        const bool low = c < step, turns = c < 2 * step;
        const int src = (lane - c) + (turns ? (low ? c + step : c - step) : c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float other = __shfl_sync(~0u, y[j], src);
          if (turns) {
            const float2 cs = s_cs[(low ? c : c - step) * 8 + j];
            y[j] = low ? y[j] * cs.x - other * cs.y : other * cs.y + y[j] * cs.x;
          }
        }
      } else {
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
            const float2 cs = s_cs[low ? e : e - half];
            y[j] = low ? y[j] * cs.x - other * cs.y : other * cs.y + y[j] * cs.x;
          }
        }
      }
      if (h < h_end && live) {
        const int64_t off = t * a.out_ts[w] + (int64_t)(w ? h - a.q_heads : h) * a.out_hs[w] + c * 8;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out[w]) + off) = pack8<Ty>(y);
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
  const dim3 grid(a.T, split);
  if ((passes + split - 1) / split <= 1)
    return launch_pdl(qk_norm_rope_kernel<Ty, PAIRS, 1>, grid, dim3(kRopeThreads), 0, st, a);
  return launch_pdl(qk_norm_rope_kernel<Ty, PAIRS, 3>, grid, dim3(kRopeThreads), 0, st, a);
}

template <typename Ty>
static cudaError_t launch_type(const RopeArgs &a, bool interleaved, cudaStream_t st) {
  if (interleaved) return launch_pairs<Ty, kPairsNear>(a, st);
  if (a.R % 16 == 0) return launch_pairs<Ty, kPairsHalf>(a, st);
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
