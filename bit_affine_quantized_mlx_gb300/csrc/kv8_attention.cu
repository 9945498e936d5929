// lily_kv8_attention, the form for few rows a sequence (decode, drafts): split over the keys.
//
//   s_j = scale * q . k_j,  out = sum_j 2^(s_j log2 e) v_j / sum_j 2^(s_j log2 e)
//
// Bound by reading the codes once (2 * head_dim bytes a token and key/value head).  The rows of one
// key/value head -- the group's heads times the sequence's new tokens -- share every code read, in
// tiles of 8 * NT rows.
//
// Split.  The work is a list of (sequence, row tile, key/value head) items, each a row of tiles of
// keys; the tiles of all items (and what it costs to begin one, in tiles), laid end to end, are cut into
// equal shares, one a block, whatever the lengths are.  An item that lies within one share is finished by its block; the parts of one
// that crosses shares go to the workspace (running maximum, sum, unnormalised output) and a second
// launch joins them in the order of the keys.  Lengths are read on the device, so a captured graph
// follows them.
//
// Block.  Four warps take the tiles' keys in turns of 4096 bytes of keys and of values each (16 to
// 64 tokens).  Each warp keeps its own ring of two such turns in shared memory, filled by 16-byte
// cp.async of its own, so there is no barrier in the loop; three blocks an SM (head_dim 256: two) keep
// 64 to 96 KB in flight (a third turn in the ring gained nothing).  The codes become fp16 exactly in registers (q + 1152 - 1152, see codes_f16) and meet
// their products as mma.sync m16n8k16 with the KEYS (then the head's elements) as the 16 rows and the
// queries as the 8 columns: at 8 rows a head nothing is padded, and at this shape the tensor pipe is
// far from its limit (the codes arrive at 22 bytes a clock and SM).
//   K: lane (g, t) = (lane / 4, lane % 4) reads 16 bytes of tokens g and g + 8; which element of the
//   head each of the four k-steps sees is any order that q follows.
//   V: the lane reads 16 bytes (its elements of the head) of tokens 2t, 2t+1, 2t+8, 2t+9, and pairs
//   of tokens are interleaved by byte permutes into the transposed operand.
//   Rows in shared memory are rotated so that both reads meet 32 different banks.
// Scores have the layout (token g; queries 2t, 2t+1), which is also the layout of the outputs'
// columns, so the running maximum and the rescaling need no exchange beyond the maximum over g; the
// weights are transposed into the second product's operand by movmatrix.
//
// Page magnitudes.  A page's key magnitude multiplies its scores.  Its value magnitude a enters the
// exponent: x = s log2 e + log2 a, with the running reference m kept 14 below the largest x; 2^(x - m) <= 2^14
// is rounded to fp16 (2^-11 relative down to 2^-28 of the largest, 2^-39 of it absolute below: of the largest
// term that any one key adds to the output) and multiplies the codes; the softmax's sum adds 2^(x - m) / a in
// fp32 (times a power of two, see kv8_device.cuh).
//
// Measured on one GB300: 64 sequences of up to 32,768 tokens (1.12M in all), 32 / 8 heads of 128: 348 us
// (6.6 TB/s of codes, 97% of the measured copy rate); one sequence of 262,144 tokens, 16 / 2 heads of 256:
// 50.2 us with the join (5.3 TB/s, 79%: two blocks an SM, and 8 us of join); one of 777 tokens: 7.3 us, the
// chain of dependent reads (lengths, pages, codes, parts) of two launches.
#include <algorithm>

#include "kv8_device.cuh"
#include "tc_sm100.cuh"

namespace lq4 {

constexpr int kDecThreads = 128, kDecWarps = 4, kDecStages = 2;
// What beginning an item costs a block (its lengths, pages, queries and the join of its warps), in tiles:
// items are that much longer when they are shared out, so that a block with the ends of two has
// fewer tiles.  At 0, 1, 2, 3 and 4: 16 x 3 tokens over 4096 keys, 96 items of 17 tiles: 20.5, 19.3, 19.2, 19.2
// and 21.1 us; one sequence of 777 keys 7.6, 7.7, 7.3, 7.5, 7.6; 64 sequences of up to 32,768: 352, 349, 348, 349, 350.
constexpr int kStart = 2;
constexpr int kTurnBytes = 4096;  // of keys, and of values, a warp and turn
// The reference of a row's weights below its largest exponent: weights up to 2^14, and room for rounding, in fp16.
constexpr int kBias = 14;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Byte offset of 16-byte chunk c of row r in a turn's buffer.  Reads of K (8 lanes: rows 2i, 2i+1,
// chunks 0-3 or 4-7) and of V (8 lanes: rows 0, 2, 4, 6 or 1, 3, 5, 7, chunks 2i, 2i+1) each meet
// eight different 16-byte bank groups.
template <int D>
__device__ __forceinline__ uint32_t turn_addr(int r, int c) {
  if (D == 64) return (r >> 1) * 128 + ((r ^ (r >> 2)) & 1) * 64 + ((c ^ (r & 2)) << 4);
  const int s = (((r ^ (r >> 2)) & 1) << 2) | (r & 2);
  return r * D + ((c ^ s) << 4);
}

// Row r of an item's row tile, or -1: its row among the activations and its query head.
struct RowOf {
  int row, head;
};
__device__ __forceinline__ RowOf row_of(const Seq &s, int rr, int h, int group) {
  const int i = rr / group;
  return RowOf{i < s.n ? s.row0 + i : -1, h * group + rr - i * group};
}

// Bytes of a warp's ring, which holds its outputs (8 NT rows of D + 2 floats) when the warps are joined.
constexpr int ring_bytes(int D, int NT) {
  const int ring = kDecStages * 2 * kTurnBytes, out = 8 * NT * (D + 2) * 4;
  return ring > out ? ring : (out + 127) / 128 * 128;
}

// Bytes of a block's shared memory.
constexpr size_t decode_smem(int D, int NT, int batch) {
  const int RT = 8 * NT, ng = kTurnBytes / D / 16;
  return kDecWarps * ring_bytes(D, NT) + RT * (D * 2 + 16 + 16) +
         4 * (kDecWarps * kDecStages * 2 * ng + RT + 2 * kDecWarps * RT + 4 + batch + 1);
}

// Blocks an SM: three where 168 registers hold a tile of 8 rows (64 sequences up to 32k tokens of 8 heads
// of 128: 383 us with two, 352 with three), else two.
constexpr int decode_blocks(int D, int NT) { return D <= 128 && NT == 1 ? 3 : 2; }

template <int D, int NT>
__global__ void __launch_bounds__(kDecThreads, decode_blocks(D, NT)) kv8_decode_kernel(AttnArgs a, int bf16) {
  constexpr int RT = 8 * NT;             // rows of a tile
  constexpr int WS = kTurnBytes / D;     // tokens of a turn
  constexpr int NG = WS / 16;            // 16-token groups of a turn
  constexpr int TILE = WS * kDecWarps;   // tokens of a tile
  constexpr int MT = D / 16;
  constexpr int QS = D * 2 + 16;         // bytes between rows of q
  constexpr bool QREG = D * NT <= 256;   // q's operands stay in registers
  constexpr int RING = ring_bytes(D, NT);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *s_q = smem + kDecWarps * RING;
  float2 *s_fin = reinterpret_cast<float2 *>(s_q + RT * QS);     // [RT]: maximum and sum of the segment
  int2 *s_row = reinterpret_cast<int2 *>(s_fin + RT);            // [RT]: row (or -1) and query head
  float *s_meta = reinterpret_cast<float *>(s_row + RT);         // [warp][stage][2][NG]
  float *s_qf = s_meta + kDecWarps * kDecStages * 2 * NG;    // [RT]
  float *s_m = s_qf + RT, *s_l = s_m + kDecWarps * RT;       // [warp][RT]
  int *s_scan = reinterpret_cast<int *>(s_l + kDecWarps * RT);  // [4]
  int *s_pre = s_scan + 4;                                   // [batch + 1]

  pdl_wait();
  const Batch &B = a.B;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

  // key range of a sequence (the union of its rows' ranges) and its number of tiles
  auto range_of = [&](const Seq &s, int &lo, int &nt) {
    lo = max(0, first_key(s.len - s.n, a.window)) & ~15;
    nt = max(1, (s.len - lo + TILE - 1) / TILE);
  };
  int base_count = 0;
  for (int b0 = 0; b0 < B.batch; b0 += kDecThreads) {
    int count = 0;
    if (b0 + tid < B.batch) {
      const Seq s = load_seq(B, b0 + tid, a.hdr);
      if (s.n > 0) {
        int lo, nt;
        range_of(s, lo, nt);
        count = (s.n * a.group + RT - 1) / RT * a.kv_heads * (nt + kStart);
      }
    }
    int sum = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) s_scan[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += s_scan[w];
    if (b0 + tid < B.batch) s_pre[b0 + tid + 1] = base_count + sum;
    for (int w = 0; w < kDecWarps; ++w) base_count += s_scan[w];
    __syncthreads();
  }
  if (tid == 0) {
    s_pre[0] = 0;
    a.jobs[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  __syncthreads();
  // equal shares of the work; with less of it than blocks the last blocks have none
  const uint32_t total = s_pre[B.batch], G = min(gridDim.x, total);
  if (blockIdx.x >= G) return;
  // floor(c total / G) in 32 bits: c (total mod G) is below 2^18
  const uint32_t whole_share = total / G, rest = total - whole_share * G;
  const int begin = blockIdx.x * whole_share + blockIdx.x * rest / G;
  const int end = (blockIdx.x + 1) * whole_share + (blockIdx.x + 1) * rest / G;

  uint8_t *ring = smem + warp * RING;
  const uint32_t ring_u32 = tc::smem_u32(ring);
  float *meta = s_meta + warp * kDecStages * 2 * NG;

  for (int cur = begin; cur < end;) {
    int b;
    {
      int lo = 0, hi = B.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid + 1] > cur) hi = mid;
        else lo = mid + 1;
      }
      b = lo;
    }
    const Seq sq = load_seq(B, b, a.hdr);
    int lo, ntile;
    range_of(sq, lo, ntile);
    const int hi = sq.len;
    const int per = ntile + kStart, local = cur - s_pre[b], item = local / per, u0 = local - item * per;
    const int u1 = min(per, u0 + end - cur), t0 = max(u0 - kStart, 0), t1 = max(u1 - kStart, 0);
    if (t0 >= t1) {  // a share that ends before the item's first tile
      cur += u1 - u0;
      continue;
    }
    const int h = item % a.kv_heads, rt = item / a.kv_heads;

    // ---- q's words under way (a warp takes rows warp, warp + 4 ...) before the pages are looked up
    constexpr int E = D / 32, QR = RT / kDecWarps;
    uint32_t qw[QR][E / 2];
#pragma unroll
    for (int k = 0; k < QR; ++k) {
      const RowOf ro = row_of(sq, rt * RT + warp + k * kDecWarps, h, a.group);
      const uint32_t *src = reinterpret_cast<const uint32_t *>(
          a.q + (int64_t)ro.row * a.q_ts + (int64_t)ro.head * a.q_hs + lane * E);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) qw[k][i] = ro.row >= 0 ? __ldg(src + i) : 0;
      if (lane == 0) s_row[warp + k * kDecWarps] = make_int2(ro.row, ro.head);
    }

    // ---- this warp's turns, the first of them under way before q is converted: turn i holds tokens first + i * TILE ...
    const int first = lo + (t0 * kDecWarps + warp) * WS;
    const int turns = min(t1 - t0, max(0, (hi - first + TILE - 1) / TILE));
    auto page_of = [&](int idx) {  // page of 16-token group idx of this warp's turns
      const int i = idx / NG, tok = first + i * TILE + (idx - i * NG) * 16;
      return i < turns && tok < hi ? raw_page(B, b, tok >> B.page_shift) : kNoPage;
    };
    int pages = check_page(B, page_of(lane), a.hdr), pages_next = page_of(32 + lane);
    auto issue = [&](int i) {
      const int idx = i * NG, st = i % kDecStages;
      if (i > 0 && (idx & 31) == 0) {
        pages = check_page(B, pages_next, a.hdr);
        pages_next = page_of(idx + 32 + lane);
      }
      const uint32_t dst = ring_u32 + st * 2 * kTurnBytes;
      const int tok0 = first + i * TILE;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int page = __shfl_sync(~0u, pages, (idx + j) & 31);
        const int64_t ph = (int64_t)page * a.kv_heads + h;
        const int64_t off = page < 0 ? 0 : (ph * B.page + ((tok0 + 16 * j) & (B.page - 1))) * D + lane * 16;
#pragma unroll
        for (int i2 = 0; i2 < D / 32; ++i2) {
          const int e = i2 * 32 + lane, r = e / (D / 16), c = e % (D / 16);
          const bool ok = page >= 0 && tok0 + 16 * j + r < hi;
          const uint32_t to = dst + turn_addr<D>(16 * j + r, c);
          const int64_t from = ok ? off + i2 * 512 : 0;
          tc::cp_async16(to, a.k + from, ok ? 16 : 0);
          tc::cp_async16(to + kTurnBytes, a.v + from, ok ? 16 : 0);
        }
        if (lane == j) {
          float *mp = meta + st * 2 * NG + j;
          if (page >= 0) {
            tc::cp_async4(tc::smem_u32(mp), a.k_amax + ph);
            tc::cp_async4(tc::smem_u32(mp + NG), a.v_amax + ph);
          } else {
            mp[0] = -1.f;  // nothing of this group is seen
            mp[NG] = 0.f;
          }
        }
      }
    };
#pragma unroll
    for (int i = 0; i < kDecStages - 1; ++i) {
      if (i < turns) issue(i);
      tc::cp_async_commit();
    }
    // ---- q, scaled by a power of two for each row so that its largest element is in [2^14, 2^15)
#pragma unroll
    for (int k = 0; k < QR; ++k) {
      const int r = warp + k * kDecWarps;
      float f[E];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 p = bf16 ? Bf16::to_f32x2(qw[k][i]) : F16::to_f32x2(qw[k][i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
        top = fmaxf(top, fmaxf(fabsf(p.x), fabsf(p.y)));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      const int e = top > 0.f ? min(max(ilogbf(top), -100), 127) : 14;
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        reinterpret_cast<uint32_t *>(s_q + r * QS)[lane * (E / 2) + i] =
            F16::from_f32x2(f[2 * i] * up, f[2 * i + 1] * up);
      if (lane == 0) s_qf[r] = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * a.scale2;
    }
    __syncthreads();

    uint32_t bq[QREG ? NT : 1][D / 64][8];
    if (QREG) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 *p = reinterpret_cast<const uint4 *>(s_q + (n * 8 + g) * QS + (c * 64 + t * 16) * 2);
          const uint4 u = p[0], v = p[1];
          bq[n][c][0] = u.x, bq[n][c][1] = u.y, bq[n][c][2] = u.z, bq[n][c][3] = u.w;
          bq[n][c][4] = v.x, bq[n][c][5] = v.y, bq[n][c][6] = v.z, bq[n][c][7] = v.w;
        }
    }
    // this thread's queries (columns 2t, 2t + 1 of each 8): factor and visible keys [klo, khi)
    float qf[NT][2];
    int klo[NT][2], khi[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = n * 8 + 2 * t + e, p = sq.len - sq.n + (rt * RT + r) / a.group;
        qf[n][e] = s_qf[r];
        klo[n][e] = first_key(p, a.window);
        khi[n][e] = a.causal ? min(p + 1, sq.len) : sq.len;
      }
    // keys that every row of the tile sees
    const int p_first = sq.len - sq.n + rt * RT / a.group;
    const int p_last = sq.len - sq.n + min(sq.n - 1, (rt * RT + RT - 1) / a.group);
    const int all_lo = first_key(p_last, a.window);
    const int all_hi = a.causal ? min(p_first + 1, sq.len) : sq.len;

    float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }

    for (int i = 0; i < turns; ++i) {
      if (i + kDecStages - 1 < turns) issue(i + kDecStages - 1);
      tc::cp_async_commit();
      tc::cp_async_wait<kDecStages - 1>();
      __syncwarp();
      const int st = i % kDecStages;
      const uint8_t *bk = ring + st * 2 * kTurnBytes, *bv = bk + kTurnBytes;
      const float *mt = meta + st * 2 * NG;
      const int tok0 = first + i * TILE;

      // scores of the turn, then x = s log2 e + log2 a
      float s[NG][NT][4];
      float top[NT][2], iv[NG];
#pragma unroll
      for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 ka = *reinterpret_cast<const uint4 *>(bk + turn_addr<D>(16 * j + g, c * 4 + t));
          const uint4 kb = *reinterpret_cast<const uint4 *>(bk + turn_addr<D>(16 * j + g + 8, c * 4 + t));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
          uint32_t bs[QREG ? 1 : NT][8];
          if (!QREG) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 *p = reinterpret_cast<const uint4 *>(s_q + (n * 8 + g) * QS + (c * 64 + t * 16) * 2);
              const uint4 u = p[0], v = p[1];
              bs[n][0] = u.x, bs[n][1] = u.y, bs[n][2] = u.z, bs[n][3] = u.w;
              bs[n][4] = v.x, bs[n][5] = v.y, bs[n][6] = v.z, bs[n][7] = v.w;
            }
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t ua = wa[w] ^ 0x80808080u, ub = wb[w] ^ 0x80808080u;
            const uint32_t a0 = codes_f16(ua, kPickLo), a1 = codes_f16(ub, kPickLo);
            const uint32_t a2 = codes_f16(ua, kPickHi), a3 = codes_f16(ub, kPickHi);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t b0 = QREG ? bq[QREG ? n : 0][c][2 * w] : bs[QREG ? 0 : n][2 * w];
              const uint32_t b1 = QREG ? bq[QREG ? n : 0][c][2 * w + 1] : bs[QREG ? 0 : n][2 * w + 1];
              mma_f16(s[j][n], a0, a1, a2, a3, b0, b1);
            }
          }
        }
        const float ka = mt[j];
        const float va = value_size(mt[NG + j]);
        iv[j] = fminf(__frcp_rn(va), 2e30f) * sum_scale(kBias);  // a number for a magnitude of NaN too: 0 times it is 0
        const float lv = __log2f(va);
        const int tk = tok0 + 16 * j;
        const bool whole = ka >= 0.f && tk >= all_lo && tk + 16 <= all_hi;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int qe = e & 1, tok = tk + g + (e >> 1) * 8;
            float x = fmaf(s[j][n][e], ka * qf[n][qe], lv);
            if (!whole && (ka < 0.f || tok < klo[n][qe] || tok >= khi[n][qe])) x = -INFINITY;
            s[j][n][e] = x;
            top[n][qe] = fmaxf(top[n][qe], x);
          }
      }
      // running reference over the turn's tokens (lanes of equal t hold the same queries)
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(~0u, top[n][e], off));
          top[n][e] -= (float)kBias;
          grew |= top[n][e] > m[n][e];
        }
      if (__any_sync(~0u, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float now = fmaxf(m[n][e], top[n][e]);
            const Moved by(m[n][e], now == -INFINITY ? m[n][e] : now);
            const float f = now == -INFINITY ? 1.f : by.factor();
            l[n][e] = now == -INFINITY ? l[n][e] : by.sum(l[n][e]);
            m[n][e] = now;
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              o[k][n][e] *= f;
              o[k][n][e + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
          const float x0 = ex2(s[j][n][0] - m0), x1 = ex2(s[j][n][1] - m1);
          const float x2 = ex2(s[j][n][2] - m0), x3 = ex2(s[j][n][3] - m1);
          l[n][0] = fmaf(x0 + x2, iv[j], l[n][0]);
          l[n][1] = fmaf(x1 + x3, iv[j], l[n][1]);
          p[n][0] = transpose8x8(F16::from_f32x2(x0, x1));
          p[n][1] = transpose8x8(F16::from_f32x2(x2, x3));
        }
        // values: pairs of tokens interleaved, elements 16g + 2i, 16g + 2i + 1 (8g + ... at D = 64)
#pragma unroll
        for (int hf = 0; hf < (D == 256 ? 2 : 1); ++hf) {
          constexpr int NW = D == 64 ? 2 : 4;
          uint32_t w[4][NW];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
            if (D == 64) {
              const uint2 u = *reinterpret_cast<const uint2 *>(bv + turn_addr<D>(row, g >> 1) + (g & 1) * 8);
              w[r][0] = u.x, w[r][1] = u.y;
            } else {
              const uint4 u = *reinterpret_cast<const uint4 *>(bv + turn_addr<D>(row, hf * 8 + g));
              w[r][0] = u.x, w[r][1] = u.y, w[r][NW - 2] = u.z, w[r][NW - 1] = u.w;
            }
          }
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            const uint32_t u0 = w[0][k] ^ 0x80808080u, u1 = w[1][k] ^ 0x80808080u;
            const uint32_t u2 = w[2][k] ^ 0x80808080u, u3 = w[3][k] ^ 0x80808080u;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t lo2 = __byte_perm(u0, u1, z ? 0x7362 : 0x5140);
              const uint32_t hi2 = __byte_perm(u2, u3, z ? 0x7362 : 0x5140);
              const uint32_t a0 = codes_f16(lo2, kPickLo), a1 = codes_f16(lo2, kPickHi);
              const uint32_t a2 = codes_f16(hi2, kPickLo), a3 = codes_f16(hi2, kPickHi);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(o[hf * 8 + 2 * k + z][n], a0, a1, a2, a3, p[n][0], p[n][1]);
            }
          }
        }
      }
      __syncwarp();
    }
    tc::cp_async_wait_all();

    // ---- join the warps: their outputs, scaled to the common maximum, meet in the rings
    constexpr int OS = D + 2;
    float *obuf = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], off);
        if (g == 0) {
          s_m[warp * RT + n * 8 + 2 * t + e] = m[n][e];
          s_l[warp * RT + n * 8 + 2 * t + e] = l[n][e];
        }
      }
    __syncthreads();
    if (tid < RT) {
      float top = s_m[tid], den = 0.f;
#pragma unroll
      for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, s_m[w * RT + tid]);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float mw = s_m[w * RT + tid];
        // without a maximum the sum is 0, or NaN for a row of NaN
        den += mw == -INFINITY ? s_l[w * RT + tid] : Moved(mw, top).sum(s_l[w * RT + tid]);
      }
      s_fin[tid] = make_float2(top, den);
      s_qf[tid] = den == 0.f ? 0.f : 1.f / den;  // q's factors are not needed any more
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = n * 8 + 2 * t + e;
        float top = s_m[r];
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, s_m[w * RT + r]);
        const float f = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - top);
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          const int d = D == 64 ? 8 * g + 2 * k : (k >> 3) * 128 + 16 * g + 2 * (k & 7);
          *reinterpret_cast<float2 *>(obuf + r * OS + d) = make_float2(o[k][n][e] * f, o[k][n][e + 2] * f);
        }
      }
    __syncthreads();
    const bool split = t0 > 0 || t1 < ntile;
    const int slot = 2 * blockIdx.x + (cur == begin ? 0 : 1);
#pragma unroll 8
    for (int e = tid; e < RT * (D / 2); e += kDecThreads) {
      const int r = e / (D / 2), d = (e - r * (D / 2)) * 2;
      const int2 ro = s_row[r];
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 u = *reinterpret_cast<const float2 *>(
            reinterpret_cast<const float *>(smem + w * RING) + r * OS + d);
        sum.x += u.x;
        sum.y += u.y;
      }
      if (ro.x < 0) continue;
      if (split) {
        *reinterpret_cast<float2 *>(a.part + ((int64_t)slot * RT + r) * D + d) = sum;
      } else {
        const float f = s_qf[r];
        sum.x = sum.x * out_scale(kBias) * f;
        sum.y = sum.y * out_scale(kBias) * f;
        const uint32_t w = bf16 ? Bf16::from_f32x2(sum.x, sum.y) : F16::from_f32x2(sum.x, sum.y);
        *reinterpret_cast<uint32_t *>(a.out + (int64_t)ro.x * a.o_ts + (int64_t)ro.y * a.o_hs + d) = w;
      }
    }
    if (tid < RT && s_row[tid].x >= 0) {
      const float2 fin = s_fin[tid];
      if (split)
        a.ml[slot * RT + tid] = fin;
      else if (a.lse)
        a.lse[(int64_t)s_row[tid].x * a.kv_heads * a.group + s_row[tid].y] =
            fin.y == 0.f ? -INFINITY : row_lse(fin.x, fin.y, kBias);
    }
    if (split && t0 == 0 && tid == 0) {
      // the block that holds the item's last tile: the largest c with floor(c total / G) <= it
      const int64_t last = cur - u0 + per - 1;
      const int c_last = (int)(((last + 1) * G - 1) / (int64_t)total);
      a.jobs[2 * blockIdx.x] = make_int4(sq.row0, sq.n, h, rt);
      a.jobs[2 * blockIdx.x + 1] = make_int4(slot, c_last, 0, 0);
    }
    __syncthreads();
    cur += u1 - u0;
  }
}

// ----------------------------------------------------------------------------- join
// Block (c, r): row r of the item that block c of the first launch began and did not finish (blocks of
// kJoinMost threads: of the c-th of these, so that few blocks are launched).  The parts' maxima and sums first (a thread each), then the outputs: a quarter of a head's four-element
// columns take the parts in turns, eight loads in flight a thread.
constexpr int kJoinMost = 512;  // parts of an item

template <int D, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(AttnArgs a, int RT, int bf16, int blocks) {
  constexpr int WARPS = kJoinThreads / 32;
  __shared__ float s_w[kJoinMost], s_red[WARPS], s_den[WARPS];
  __shared__ int s_count[WARPS], s_job;
  __shared__ __align__(16) float s_o[kJoinThreads * 4];
  pdl_wait();
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  int c = blockIdx.x;
  if (kJoinThreads == kJoinMost) {
    // block i takes the i-th of the jobs that there are
    const bool job = tid < blocks && a.jobs[2 * tid].x >= 0;
    const uint32_t some = __ballot_sync(~0u, job);
    if (tid == 0) s_job = -1;
    if (lane == 0) s_count[tid >> 5] = __popc(some);
    __syncthreads();
    int before = __popc(some & ((1u << lane) - 1));
    for (int w = 0; w < tid >> 5; ++w) before += s_count[w];
    if (job && before == (int)blockIdx.x) s_job = tid;
    __syncthreads();
    c = s_job;
    if (c < 0) return;
  }
  const int4 j0 = a.jobs[2 * c], j1 = a.jobs[2 * c + 1];
  if (j0.x < 0) return;
  const RowOf ro = row_of(Seq{j0.x, j0.y, 0}, j0.w * RT + r, j0.z, a.group);
  if (ro.row < 0) return;
  const int parts = j1.y - c + 1;  // at most the first launch's blocks, kJoinMost
  auto slot = [&](int i) { return i == 0 ? j1.x : 2 * (c + i); };

  // the first parts' outputs are under way while their weights are found
  constexpr int COLS = D / 4, GROUPS = kJoinThreads / COLS, AHEAD = 8;
  const int col = tid % COLS, grp = tid / COLS;
  auto part = [&](int i) {
    return *reinterpret_cast<const float4 *>(a.part + ((int64_t)slot(i) * RT + r) * D + col * 4);
  };
  float4 first[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    first[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp + k * GROUPS < parts) first[k] = part(grp + k * GROUPS);
  }
  constexpr int MINE = kJoinMost / kJoinThreads;
  float2 ml[MINE];  // parts tid, tid + kJoinThreads ...
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int i = tid + k * kJoinThreads;
    ml[k] = i < parts ? a.ml[(int64_t)slot(i) * RT + r] : make_float2(-INFINITY, 0.f);
    top = fmaxf(top, ml[k].x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) s_red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_red[w]);
  float den = 0.f;
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const bool none = ml[k].x == -INFINITY;  // sum and output 0, or NaN
    const Moved by(none ? 0.f : ml[k].x, none ? 0.f : top);
    s_w[tid + k * kJoinThreads] = by.factor();
    den += by.sum(ml[k].y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(~0u, den, o);
  if (lane == 0) s_den[tid >> 5] = den;
  __syncthreads();
  den = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) den += s_den[w];

  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4 &u, float w) {
    acc.x = fmaf(u.x, w, acc.x);
    acc.y = fmaf(u.y, w, acc.y);
    acc.z = fmaf(u.z, w, acc.z);
    acc.w = fmaf(u.w, w, acc.w);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (grp + k * GROUPS < parts) add(first[k], s_w[grp + k * GROUPS]);
#pragma unroll 8
  for (int i = grp + AHEAD * GROUPS; i < parts; i += GROUPS) add(part(i), s_w[i]);
  reinterpret_cast<float4 *>(s_o)[tid] = acc;
  __syncthreads();
  if (grp == 0) {
    for (int k = 1; k < GROUPS; ++k) {
      const float4 u = reinterpret_cast<const float4 *>(s_o)[k * COLS + col];
      acc.x += u.x;
      acc.y += u.y;
      acc.z += u.z;
      acc.w += u.w;
    }
    const float g = den == 0.f ? 0.f : 1.f / den;
    acc = make_float4(acc.x * out_scale(kBias), acc.y * out_scale(kBias), acc.z * out_scale(kBias), acc.w * out_scale(kBias));
    uint2 w;
    w.x = bf16 ? Bf16::from_f32x2(acc.x * g, acc.y * g) : F16::from_f32x2(acc.x * g, acc.y * g);
    w.y = bf16 ? Bf16::from_f32x2(acc.z * g, acc.w * g) : F16::from_f32x2(acc.z * g, acc.w * g);
    *reinterpret_cast<uint2 *>(a.out + (int64_t)ro.row * a.o_ts + (int64_t)ro.head * a.o_hs + col * 4) = w;
    if (col == 0 && a.lse)
      a.lse[(int64_t)ro.row * a.kv_heads * a.group + ro.head] =
          den == 0.f ? -INFINITY : row_lse(top, den, kBias);
  }
}

// ----------------------------------------------------------------------------- launches
struct DecodePlan {
  int nt, grid, join;  // 8-row columns of a tile, blocks, threads of a join's block (0: none is needed)
  int rows, items;     // of a tile that can hold something; items, at most the blocks
  size_t smem, off_jobs, off_ml, off_part, total;
};

static DecodePlan decode_plan(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int q_heads) {
  DecodePlan p = {};
  const int group = q_heads / C.kv_heads, D = C.head_dim;
  const int64_t rows = (int64_t)b.max_q * group;
  // rows beyond a tile are further items, which read the keys again: the widest tile that the
  // registers hold (the output takes D * NT / 4 of them)
  p.nt = rows <= 8 ? 1 : rows <= 16 || D == 256 ? 2 : 4;
  const int RT = 8 * p.nt, tile = kTurnBytes / D * kDecWarps;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const int64_t per_seq = (rows + RT - 1) / RT * C.kv_heads, items = std::min<int64_t>(b.batch, T) * per_seq;
  const int64_t tiles = std::max<int64_t>(1, ((int64_t)b.max_kv + 16 + tile - 1) / tile);
  // total 0: the tiles have to be countable in 31 bits, those of all sequences too, because row ranges on the
  // device that go backwards (which is recorded) can give the same rows to many
  if (std::max<int64_t>(1, b.batch) * per_seq > INT32_MAX / (tiles + kStart)) return p;
  p.grid = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(decode_blocks(D, p.nt) * sms, kJoinMost), items * (tiles + kStart)));
  // Few items have many parts each: a large block reads a row's parts together (262,144 tokens, 152
  // parts: 12 us with 256 threads, 8 with 512).  Fewer: small blocks start
  // faster (64 sequences, 512 items: 6 us with 256 threads, 10 with 512).
  p.join = tiles == 1 ? 0 : p.grid / items >= 32 ? kJoinMost : 128;
  p.items = (int)std::min<int64_t>(items, p.grid);
  p.rows = (int)std::min<int64_t>(RT, rows);
  p.smem = decode_smem(D, p.nt, b.batch);
  size_t off = kAlign;
  p.off_jobs = off;
  off = align_up(off + (size_t)p.grid * 2 * sizeof(int4));
  p.off_ml = off;
  off = align_up(off + (size_t)p.grid * 2 * RT * sizeof(float2));
  p.off_part = off;
  p.total = align_up(off + (size_t)p.grid * 2 * RT * D * sizeof(float));
  return p;
}

template <int D, int NT>
static cudaError_t launch_decode_shape(const AttnArgs &a, const DecodePlan &p, int bf16, cudaStream_t st) {
  auto kernel = kv8_decode_kernel<D, NT>;
  static std::atomic<bool> allowed[64];
  cudaError_t e = allow_smem<decode_smem(D, NT, kMaxBatch)>(kernel, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(p.grid), dim3(kDecThreads), p.smem, st, a, bf16);
  if (e != cudaSuccess || !p.join) return e;
  if (p.join == kJoinMost)
    return launch_pdl(kv8_join_kernel<D, kJoinMost>, dim3(p.items, p.rows), dim3(kJoinMost), 0, st, a, 8 * NT, bf16, p.grid);
  return launch_pdl(kv8_join_kernel<D, 128>, dim3(p.grid, p.rows), dim3(128), 0, st, a, 8 * NT, bf16, p.grid);
}

template <int D>
static cudaError_t launch_decode_dim(const AttnArgs &a, const DecodePlan &p, int bf16, cudaStream_t st) {
  if (p.nt == 1) return launch_decode_shape<D, 1>(a, p, bf16, st);
  if (p.nt == 2) return launch_decode_shape<D, 2>(a, p, bf16, st);
  if constexpr (D <= 128) return launch_decode_shape<D, 4>(a, p, bf16, st);
  return cudaErrorInvalidValue;
}

// Rows of a sequence and key/value head from which the tcgen05 form runs.  Measured with both forms
// (us, split / tcgen05): 32 sequences of 4096 keys, 8 heads of 128: 16 rows 71 / 123, 32 rows
// 111 / 123, 48 rows 196 / 124; 4 heads of 64: 16 rows 31 / 45, 32 rows 49 / 46, 64 rows 84 / 46;
// 2 heads of 256: 32 rows 66 / 61, 64 rows 118 / 63; one sequence of 32768 keys, 8 heads of 128:
// 32 rows 33 / 41, 48 rows 56 / 41.  With heads of 256 and so few sequences that the tcgen05 form has to
// split the keys, its parts' outputs (128 rows of 256 each) cost more than reading the codes again:
// one sequence, 2 heads, 32768 keys: 64 rows 36 / 56, 96 rows 51 / 57, 128 rows 62 / 58.
static int prompt_rows(const lily_kv8_cache &C, const lily_kv8_batch &b) {
  const int sms = sm_count() > 0 ? sm_count() : 152;
  return C.head_dim == 256 && (int64_t)b.batch * C.kv_heads * 4 <= sms ? 97 : 33;
}
static bool prompt_form(const lily_kv8_cache &C, const lily_kv8_batch &b, int q_heads) {
  return (int64_t)b.max_q * (q_heads / C.kv_heads) >= prompt_rows(C, b);
}

size_t kv8_attention_ws_bytes(const lily_kv8_cache &C, const lily_kv8_batch &b, int T, int q_heads) {
  if (!prompt_form(C, b, q_heads)) return decode_plan(C, b, T, q_heads).total;
  lily_kv8_batch fewer = b;  // the split form's largest calls, so that the space serves them too
  fewer.max_q = std::max(1, 96 / (q_heads / C.kv_heads));
  return std::max(decode_plan(C, fewer, T, q_heads).total, prompt_plan(C, b, T, q_heads, 0).total);
}

int launch_kv8_attention(const lily_kv8_cache &C, const lily_kv8_batch &b, const AttnShape &s,
                         const Rows &q, const Rows &out, float *lse, void *ws, cudaStream_t st) {
  uint8_t *w = static_cast<uint8_t *>(ws);
  AttnArgs a = {};
  a.B = make_batch(C, b, s.T);
  a.hdr = static_cast<int32_t *>(ws);
  a.k = C.k;
  a.v = C.v;
  a.k_amax = C.k_amax;
  a.v_amax = C.v_amax;
  a.q = static_cast<const uint16_t *>(q.p);
  a.out = static_cast<uint16_t *>(out.p);
  a.q_ts = q.ts;
  a.q_hs = q.hs;
  a.o_ts = out.ts;
  a.o_hs = out.hs;
  a.lse = lse;
  a.kv_heads = C.kv_heads;
  a.group = s.q_heads / C.kv_heads;
  a.causal = s.causal;
  a.window = s.window;
  a.scale2 = s.scale * 1.4426950408889634f / 127.f;
  const int bf16 = s.dtype == LILY_BF16;
  cudaError_t e;
  if (prompt_form(C, b, s.q_heads)) {
    e = launch_prompt(a, prompt_plan(C, b, s.T, s.q_heads, s.window), C.head_dim, bf16, w, st);
    if (e == cudaSuccess) return LILY_Q4_OK;
    cudaGetLastError();
    return LILY_Q4_ERR_CUDA;
  }
  const DecodePlan p = decode_plan(C, b, s.T, s.q_heads);
  a.jobs = reinterpret_cast<int4 *>(w + p.off_jobs);
  a.ml = reinterpret_cast<float2 *>(w + p.off_ml);
  a.part = reinterpret_cast<float *>(w + p.off_part);
  if (C.head_dim == 64) e = launch_decode_dim<64>(a, p, bf16, st);
  else if (C.head_dim == 128) e = launch_decode_dim<128>(a, p, bf16, st);
  else e = launch_decode_dim<256>(a, p, bf16, st);
  if (e == cudaSuccess) return LILY_Q4_OK;
  cudaGetLastError();
  return LILY_Q4_ERR_CUDA;
}

}  // namespace lq4
