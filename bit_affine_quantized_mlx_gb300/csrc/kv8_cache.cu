// The paged 8-bit key/value cache: lily_kv8_append and lily_kv8_read.
//
// A page and head has one magnitude amax; a code q stands for q * amax / 127.
//
// Append.  The new tokens of one page ("a run") are quantised with amax' = max(amax, |x|), and
// earlier codes of the page are re-rounded when that grows.  Both roundings are those of exact
// arithmetic, so results do not depend on how the quotient is computed: amax is always a 16-bit
// float (8 or 11 significant bits), so 127 x and q amax are exact in fp32 (at most 18 bits).  Let
// the numerator be an integer times 2^a and amax an integer N < 2^11 times 2^b: a quotient that is
// not an odd multiple of 1/2 differs from every such multiple by at least 2^(a-b) / (2 N), and one
// of 1/2 or more has 2^(a-b) >= 2^-9 or so: by 4e-7 at least.  The product with a rounded
// 127 / amax is off by 2^-22 relative (3e-5 at most), so it decides everything farther than 1e-4
// from a tie; nearer, an IEEE division (3e-8 off at 1/2, 2^-24 relative above) decides, and gives an
// exact tie exactly.
//
// Bound by memory: 2 bytes in and 1 byte out an element; at one token a sequence by the launch
// and one chain of dependent reads (lengths, page number, magnitude).  A run is read once, held
// in registers between finding its magnitude and writing its codes.  Measured on one GB300: 11k
// prompt tokens of 8 heads of 128 (keys and values, 69 MB): 22 us, 3.1 TB/s, half of the copy rate: a
// block's chain of reads before its rows arrive, and about ten instructions an element (36 us with
// one 256-thread block a run and a division an element).  16 sequences of one token: 3 us.
//
// Read, measured: 131,072 tokens of 2 heads of 256 to bf16 (403 MB): 65 us, 6.2 TB/s (91%).
#include <algorithm>
#include <type_traits>

#include "kv8_device.cuh"

namespace lq4 {

struct CacheArgs {
  Batch B;
  int32_t *hdr;
  int8_t *codes[2];
  float *amax[2];
  const void *x[2];   // append: rows in
  void *y[2];         // read: rows out
  int64_t ts[2], hs[2];
  int kv_heads, D, chunk;
};

// 1.5 * 2^23: adding it rounds a number of magnitude below 2^22 to the nearest integer (ties to
// even), which the sum then holds in its low bits, negative ones as two's complement.
constexpr float kRound = 12582912.f;

// The codes rint(x[i] up / den) of exact arithmetic, as bytes; x up and den as described above,
// k = up / den to fp32's precision, or 0 where that is out of fp32's range.
__device__ __forceinline__ uint32_t exact_codes4(const float (&x)[4], float up, float den, float k) {
  float n[4], far = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = x[i] * k;
    n[i] = q + kRound;
    far = fmaxf(far, fabsf(q - (n[i] - kRound)));
  }
  if (far > 0.4999f || k == 0.f) {  // one of them within 1e-4 of a tie
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = __fdiv_rn(x[i] * up, den) + kRound;
  }
  const uint32_t lo = __byte_perm(__float_as_uint(n[0]), __float_as_uint(n[1]), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(n[2]), __float_as_uint(n[3]), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

__device__ __forceinline__ uint32_t umax16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// A position before the first or, which a sequence within its bounds has none of, beyond the table (its
// tokens counted below 2^31).  Without the second half the compiler gives the append of 64-thread teams 88
// registers instead of 80: 11.5k tokens of 8 heads of 128 in pages of 32, repeated, took 20.1 us, not 19.1.
__device__ __forceinline__ bool off_table(const Batch &B, int pos) {
  return pos < 0 || pos >= min(B.table_pages, INT_MAX >> B.page_shift) * B.page;
}

// TEAM threads handle a run; NV chunks of 8 elements a thread hold it (TEAM * NV * 8 >= its size).
// A team walks the runs that start among its `chunk` tokens.  Teams of one warp need no barrier and
// share a block.
template <typename Ty, int TEAM, int TEAMS, int NV>
__global__ void __launch_bounds__(TEAM *TEAMS) kv8_append_kernel(CacheArgs a) {
  static_assert(TEAM == 32 || TEAMS == 1, "a block barrier joins a team");
  __shared__ uint32_t s_max[TEAM / 32];
  pdl_wait();
  const Batch &B = a.B;
  const int tid = threadIdx.x & (TEAM - 1), team = threadIdx.x / TEAM;
  const int h = blockIdx.y, kv = blockIdx.z;
  const int cpr = a.D >> 3;  // chunks of 8 a row
  const int t_first = (blockIdx.x * TEAMS + team) * a.chunk;
  const int t_end = min(B.T, t_first + a.chunk);

  for (int t = t_first; t < t_end;) {
    const int b = find_seq(B, t);
    const Seq s = load_seq(B, b, a.hdr);
    if (t < s.row0 || t >= s.row0 + s.n) {  // a sequence out of bounds: no run starts here
      ++t;
      continue;
    }
    const int pos = s.len - s.n + (t - s.row0);
    if (off_table(B, pos)) {
      record_index_error(a.hdr);
      ++t;
      continue;
    }
    const int in_page = pos & (B.page - 1);
    const int rows = min(B.page - in_page, s.row0 + s.n - t);
    if (t != s.row0 && in_page != 0) {  // the middle of a run that starts earlier
      t += rows;
      continue;
    }
    const int raw = raw_page(B, b, pos >> B.page_shift);  // checked below, the rows under way
    const int t_run = t;
    t += rows;

    // the run's elements and their largest magnitude (as bits: NaN > infinity > finite)
    const uint16_t *x = static_cast<const uint16_t *>(a.x[kv]) + t_run * a.ts[kv] + h * a.hs[kv];
    uint4 v[NV];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TEAM + tid, r = c / cpr;
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) v[i] = *reinterpret_cast<const uint4 *>(x + r * a.ts[kv] + (c - r * cpr) * 8);
    }
    const int page = check_page(B, raw, a.hdr);
    if (page < 0) continue;
    const int64_t ph = (int64_t)page * a.kv_heads + h;
    float *amax = a.amax[kv] + ph;
    const float was = in_page ? *amax : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t m = 0x7FFF7FFFu;
      top = umax16x2(umax16x2(top, umax16x2(v[i].x & m, v[i].y & m)), umax16x2(v[i].z & m, v[i].w & m));
    }
    top = max(top & 0xFFFFu, top >> 16);
    top = __reduce_max_sync(~0u, top);
    if (TEAM > 32) {
      if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TEAM / 32; ++w) top = max(top, s_max[w]);
    }
    const float fresh = Ty::to_f32x2(top).x;
    const float now = __uint_as_float(max(__float_as_uint(fresh), __float_as_uint(was)));
    const bool finite = now < __uint_as_float(0x7F800000u), zero = !(now > 0.f);
    // a power of two that keeps 127 x, q amax and 1 / amax inside fp32's range (exact: whatever
    // underflows by it has code 0)
    const float sc = now > 0x1p60f ? 0x1p-64f : now < 0x1p-60f ? 0x1p64f : 1.f;
    const float den = now * sc, inv = 1.f / den, up = 127.f * sc;

    int8_t *codes = a.codes[kv] + ph * B.page * a.D;
    if (in_page && __float_as_uint(now) != __float_as_uint(was)) {
      // the magnitude grew: re-round the page's earlier codes, 16 at a time
      for (int c = tid; c < in_page * (a.D >> 4); c += TEAM) {
        uint4 w = *reinterpret_cast<uint4 *>(codes + c * 16);
        uint32_t *u = &w.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float num[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) num[e] = (float)(int8_t)(u[j] >> (8 * e));
          const uint32_t r = finite ? exact_codes4(num, was * sc, den, sc == 1.f ? was * inv : 0.f) : 0;
          u[j] = r;
        }
        *reinterpret_cast<uint4 *>(codes + c * 16) = w;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TEAM + tid, r = c / cpr;
      if (r < rows) {
        float f[8];
        unpack8<Ty>(v[i], f);
        uint32_t r2[2] = {0, 0};
        if (finite && !zero) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x4[4] = {f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]};
            r2[e] = exact_codes4(x4, up, den, sc == 1.f ? up * inv : 0.f);
          }
        }
        *reinterpret_cast<uint2 *>(codes + (int64_t)(in_page + r) * a.D + (c - r * cpr) * 8) =
            make_uint2(r2[0], r2[1]);
      }
    }
    __syncwarp();
    if (tid == 0) *amax = now;
    if (TEAM > 32) __syncthreads();  // s_max is written again by the next run
  }
}

// ----------------------------------------------------------------------------- read
// A warp takes up to 8 tokens: as many lanes find their sequences and pages together, then it walks the
// tokens' heads, D / 16 lanes a head and 16 codes a lane, four loads of codes in flight.  Bound by
// memory (1 byte in, 2 or 4 out an element).
constexpr int kReadThreads = 256, kReadAhead = 4;

template <int DT>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(CacheArgs a) {
  const int kReadTokens = a.chunk;
  pdl_wait();
  const Batch &B = a.B;
  const int lane = threadIdx.x & 31;
  const int t0 = (blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5)) * kReadTokens;
  if (t0 >= B.T) return;
  const int kv = blockIdx.y;
  int page = -2, in_page = 0;  // -2: the row is not written, -1: it reads as zero
  if (lane < kReadTokens && t0 + lane < B.T) {
    const int t = t0 + lane, b = find_seq(B, t);
    const Seq s = load_seq(B, b, a.hdr);
    const int pos = s.len - s.n + (t - s.row0);
    if (t >= s.row0 && t < s.row0 + s.n) {
      if (off_table(B, pos)) {
        record_index_error(a.hdr);
      } else {
        page = check_page(B, raw_page(B, b, pos >> B.page_shift), a.hdr);
        in_page = pos & (B.page - 1);
      }
    }
  }
  // heads of 8 tokens in steps of `step` = 512 / D: token i, head h of this lane's next one
  const int step = 512 / a.D, di = step / a.kv_heads, dh = step - di * a.kv_heads;
  const int d = (lane & (a.D / 16 - 1)) * 16;
  int h = lane / (a.D / 16), i = h / a.kv_heads;
  h -= i * a.kv_heads;
  const int8_t *codes = a.codes[kv];
  const float *amax = a.amax[kv];
  const int rounds = (kReadTokens * a.kv_heads + step - 1) / step;
  for (int r0 = 0; r0 < rounds; r0 += kReadAhead) {
    uint4 w[kReadAhead];
    float s[kReadAhead];
    int64_t at[kReadAhead];  // where the values go, or -1
#pragma unroll
    for (int r = 0; r < kReadAhead; ++r) {
      const int src = min(i, kReadTokens - 1);
      const int p = __shfl_sync(~0u, page, src), row = __shfl_sync(~0u, in_page, src);
      at[r] = i < kReadTokens && p != -2 ? (int64_t)(t0 + i) * a.ts[kv] + (int64_t)h * a.hs[kv] + d : -1;
      const int64_t ph = (int64_t)max(p, 0) * a.kv_heads + h;
      w[r] = make_uint4(0, 0, 0, 0);
      s[r] = 0.f;
      if (at[r] >= 0 && p >= 0) {
        w[r] = __ldg(reinterpret_cast<const uint4 *>(codes + (ph * B.page + row) * a.D + d));
        s[r] = __ldg(amax + ph);
      }
      i += di;
      h += dh;
      if (h >= a.kv_heads) {
        h -= a.kv_heads;
        ++i;
      }
    }
#pragma unroll
    for (int r = 0; r < kReadAhead; ++r) {
      if (at[r] < 0) continue;
      float f[16];
      const uint32_t u[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
      // q amax passes fp32's range for magnitudes near the top of it: 2^-8 of it, exactly, does not
      const bool far = s[r] > 0x1p100f;
      const float size = far ? s[r] * 0x1p-8f : s[r], step = far ? 256.f / 127.f : 1.f / 127.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = (float)(int8_t)(u[e >> 2] >> (8 * (e & 3))) * size * step;
      if (DT == LILY_F32) {
        float *o = static_cast<float *>(a.y[kv]) + at[r];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<float4 *>(o + 4 * e) = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
      } else {
        uint16_t *o = static_cast<uint16_t *>(a.y[kv]) + at[r];
        float lo[8], hi[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] = f[e];
          hi[e] = f[8 + e];
        }
        using Ty = typename std::conditional<DT == LILY_BF16, Bf16, F16>::type;
        *reinterpret_cast<uint4 *>(o) = pack8<Ty>(lo);
        *reinterpret_cast<uint4 *>(o + 8) = pack8<Ty>(hi);
      }
    }
  }
}

// ----------------------------------------------------------------------------- launches
Batch make_batch(const lily_kv8_cache &C, const lily_kv8_batch &b, int T) {
  Batch B = {};
  B.table = b.block_table;
  B.q_start = b.q_start;
  B.kv_len = b.kv_len;
  B.table_pages = b.table_pages;
  B.batch = b.batch;
  B.max_q = b.max_q;
  // Below 2^31 by more than the keys that are looked up ahead of a sequence's end (64 turns of 256).
  B.max_kv = (int)std::min<int64_t>(std::min(b.max_kv, INT32_MAX - 65535), (int64_t)b.table_pages * C.page);
  B.T = T;
  B.page = C.page;
  while ((1 << B.page_shift) < C.page) ++B.page_shift;
  B.n_pages = C.n_pages;
  return B;
}

static CacheArgs cache_args(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, void *ws) {
  CacheArgs a = {};
  a.B = make_batch(C, b, T);
  a.hdr = static_cast<int32_t *>(ws);
  a.codes[0] = C.k;
  a.codes[1] = C.v;
  a.amax[0] = C.k_amax;
  a.amax[1] = C.v_amax;
  a.kv_heads = C.kv_heads;
  a.D = C.head_dim;
  return a;
}

template <typename Ty>
static cudaError_t launch_append(CacheArgs &a, cudaStream_t st) {
  const int D = a.D, T = a.B.T;
  const int most = std::min(a.B.max_q, a.B.page);  // rows of the longest run
  const int nv = most * (D / 8);
  // Tokens of a team: about one sequence's or one page's worth, so that it walks one or two runs.
  int chunk = 1;
  while (chunk * 2 <= std::min(most, T / a.B.batch)) chunk *= 2;
  a.chunk = chunk;
  const int walks = (T + chunk - 1) / chunk;
  // The threads that hold a run in 32 registers each.
  if (nv <= 128) return launch_pdl(kv8_append_kernel<Ty, 32, 8, 4>, dim3((walks + 7) / 8, a.kv_heads, 2), dim3(256), 0, st, a);
  if (nv <= 256) return launch_pdl(kv8_append_kernel<Ty, 32, 4, 8>, dim3((walks + 3) / 4, a.kv_heads, 2), dim3(128), 0, st, a);
  const dim3 grid(walks, a.kv_heads, 2);
  if (nv <= 512) return launch_pdl(kv8_append_kernel<Ty, 64, 1, 8>, grid, dim3(64), 0, st, a);
  if (nv <= 1024) return launch_pdl(kv8_append_kernel<Ty, 128, 1, 8>, grid, dim3(128), 0, st, a);
  if (nv <= 2048) return launch_pdl(kv8_append_kernel<Ty, 256, 1, 8>, grid, dim3(256), 0, st, a);
  return launch_pdl(kv8_append_kernel<Ty, 512, 1, 8>, grid, dim3(512), 0, st, a);
}

static int status_of(cudaError_t e) {
  if (e == cudaSuccess) return LILY_Q4_OK;
  cudaGetLastError();
  return LILY_Q4_ERR_CUDA;
}

int launch_kv8_append(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int dtype,
                      const Rows &k, const Rows &v, void *ws, cudaStream_t st) {
  CacheArgs a = cache_args(C, b, T, ws);
  a.x[0] = k.p;
  a.x[1] = v.p;
  a.ts[0] = k.ts;
  a.ts[1] = v.ts;
  a.hs[0] = k.hs;
  a.hs[1] = v.hs;
  return status_of(dtype == LILY_BF16 ? launch_append<Bf16>(a, st) : launch_append<F16>(a, st));
}

int launch_kv8_read(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int dtype, const Rows &k,
                    const Rows &v, void *ws, cudaStream_t st) {
  CacheArgs a = cache_args(C, b, T, ws);
  a.y[0] = k.p;
  a.y[1] = v.p;
  a.ts[0] = k.ts;
  a.ts[1] = v.ts;
  a.hs[0] = k.hs;
  a.hs[1] = v.hs;
  // Tokens of a warp: 8 where that leaves about 64 warps an SM, fewer where there are fewer tokens (16
  // sequences of a page: 9 us with 8, 3 with 1; 13.6k tokens of 8 heads of 128 to fp32: 33 us with 8, 27
  // with 2).
  const int sms = sm_count() > 0 ? sm_count() : 1;
  a.chunk = std::max(1, std::min(8, T / (32 * sms)));
  const int per = kReadThreads / 32 * a.chunk;
  const dim3 grid((T + per - 1) / per, 2), block(kReadThreads);
  if (dtype == LILY_BF16) return status_of(launch_pdl(kv8_read_kernel<LILY_BF16>, grid, block, 0, st, a));
  if (dtype == LILY_F16) return status_of(launch_pdl(kv8_read_kernel<LILY_F16>, grid, block, 0, st, a));
  return status_of(launch_pdl(kv8_read_kernel<LILY_F32>, grid, block, 0, st, a));
}

}  // namespace lq4
