// The paged FP4 key/value cache: appending a call's keys and values (with the per-head
// normalization and the position rotation of q and k on the way) and reading rows back.
#include "sharq_common.cuh"
#include "sharq_internal.h"
#include "sharq_kv.h"
#include "sharq_kv_device.cuh"

namespace sharq {
namespace {

__device__ __forceinline__ uint4 ld128(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]) {
  v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&v)[8]) {
  uint4 o;
  uint32_t *w = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return o;
}

// Where a token row of the call lives: its position in its sequence, and its row of the cache.
struct TokenPlace {
  long long group;           // byte of its group of 16 tokens for key head 0; -1: no place in the cache
  int codes[2], scales[2];   // its row's first K and V code and scale byte inside a group
  int pos;                   // may be negative (fewer cached than new tokens)
  int in_use;                // a row of some sequence (rows past the last sequence are not)
};

// The places of `n` consecutive tokens. The block counts the sequences that end at or before the
// first (one pass over cu_q, not a chain of dependent loads); a thread per token searches on.
constexpr int kMaxTokens = 16;
template <int D, bool MX>
__device__ __forceinline__ void find_tokens(const KvBatchView &b, const KvCacheView &c, int token0, int n, TokenPlace *out) {
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  int seq = 0;
  for (int i0 = 0; i0 < b.n_seq; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    seq += __syncthreads_count(i < b.n_seq && __ldg(b.cu_q + i + 1) <= token0);
  }
  if (threadIdx.x < n) {
    const int token = token0 + threadIdx.x;
    int hi = b.n_seq;  // the first sequence that ends behind the token is in [seq, hi]
    while (seq < hi) {
      const int mid = (seq + hi) >> 1;
      if (__ldg(b.cu_q + mid + 1) <= token) seq = mid + 1;
      else hi = mid;
    }
    TokenPlace t{-1, {0, 0}, {0, 0}, 0, 0};
    if (seq < b.n_seq && token >= __ldg(b.cu_q)) {
      t.in_use = 1;
      t.pos = __ldg(b.kv_len + seq) - __ldg(b.cu_q + seq + 1) + token;
      const int col = t.pos >> c.page_shift;
      if (t.pos >= 0 && col < b.max_pages) {
        const int page = __ldg(b.page_table + (size_t)seq * b.max_pages + col);
        const int in_page = t.pos & ((1 << c.page_shift) - 1), r = in_page & 15;
        if (page >= 0 && page < c.num_pages)
          t.group = ((((long long)page * c.kv_heads) << (c.page_shift - 4)) + (in_page >> 4)) * G.bytes;
        t.codes[0] = r * (D / 2), t.codes[1] = G.v_codes + kv_v_place(D, r, 0);
        t.scales[0] = G.k_scales + r * (D / (MX ? 32 : 16)), t.scales[1] = G.v_scales + kv_v_scale_place(r, 0);
      }
    }
    out[threadIdx.x] = t;
  }
  __syncthreads();
}

// What a lane adds to its token's place: element 8 j of a head.
template <int D, bool MX>
struct LanePlace {
  long long head;  // byte of the key head
  int codes, scale, is_v;
  __device__ __forceinline__ LanePlace(const KvCacheView &c, int kh, int v, int j) : is_v(v) {
    constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
    const int run = 8 * j / (D / 8), blk = 8 * j / (MX ? 32 : 16);
    head = ((long long)kh << (c.page_shift - 4)) * G.bytes;
    codes = v ? kv_v_place(D, 0, run) + (D == 128 ? 4 * (j & 1) : 0) : 4 * j;
    scale = v ? kv_v_scale_place(0, blk) : blk;
  }
};

// Append: a block per one to sixteen tokens; D/8 lanes per head, eight elements per lane, a lane
// keeping its head from token to token; partner elements and block maxima come by shuffles. cos and
// sin are formed once per token from the 64-bit angle and rounded once. Bound by its instructions
// near the rate of the bytes (the row read once, q and the codes written once): 6417 rows of 40 heads
// take 30 us bare, 33 us with the rotation and 41 us with both norms, against 19 us of bytes. Blocks fill
// whole waves: five tokens a block in two waves and a bit took 47 us.
template <int D, bool MX>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const AppendParams p, int per_block) {
  constexpr int L = D / 8;  // lanes per head
  // cos and sin of angle f of a token at pair_place(f): the lanes of one load read neighbouring words
  constexpr int NC = D / 16;
  auto pair_place = [](int f) { return ((f & 7) >> 1) * (2 * NC) + (f >> 3) * 2 + (f & 1); };
  __shared__ __align__(16) float2 turns[kMaxTokens][2][D / 2];  // (cos, -sin) for the first of a pair, (cos, sin)
  __shared__ TokenPlace places[kMaxTokens];
  const int token0 = blockIdx.x * per_block, n = min(per_block, p.b.tokens - token0);
  const int kvh = p.c.kv_heads, heads = p.q_heads + 2 * kvh, at_once = blockDim.x / L;
  const int j = threadIdx.x % L, e0 = 8 * j;
  // the rows of two iterations ahead are on their way, the first while the places and sines are found
  int next_head = threadIdx.x / L, next_x = 0;
  const uint16_t *next = p.qkv + (size_t)token0 * p.row_stride + (size_t)next_head * D + e0;
  auto fetch = [&]() {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (next_head < heads) w = ld128(next);
    next += p.row_stride;
    if (++next_x == n) next_x = 0, next_head += at_once, next += (long long)at_once * D - n * p.row_stride;
    return w;
  };
  uint4 ahead1 = fetch(), ahead2 = fetch();
  find_tokens<D, MX>(p.b, p.c, token0, n, places);
  for (int i = threadIdx.x; i < n * p.rot_half; i += blockDim.x) {
    const int x = i / p.rot_half, j = i - x * p.rot_half;
    double s, c;
    sincos((double)places[x].pos * (double)__ldg(p.inv_freq + j), &s, &c);
    const float cf = __double2float_rn(c), sf = __double2float_rn(s);
    turns[x][0][pair_place(j)] = make_float2(cf, -sf), turns[x][1][pair_place(j)] = make_float2(cf, sf);
  }
  __syncthreads();
  // whole warps stay in the loops: the shuffles below name every lane
  for (int h0 = 0; h0 < heads; h0 += at_once) {
    const int head = h0 + threadIdx.x / L;
    const bool live = head < heads, is_q = head < p.q_heads, is_k = !is_q && head < p.q_heads + kvh;
    const int kh = is_q || !live ? 0 : head - p.q_heads - (is_k ? 0 : kvh);
    const LanePlace<D, MX> lp(p.c, kh, is_k ? 0 : 1, j);
    const bool turned = live && (is_q || is_k) && e0 < 2 * p.rot_half;
    const bool first = e0 < p.rot_half;
    const int partner = p.interleaved || !turned ? e0 : first ? e0 + p.rot_half : e0 - p.rot_half;
    const int f0 = p.interleaved ? e0 / 2 : first ? e0 : e0 - p.rot_half;
    const uint16_t *gamma = !live ? nullptr : is_q ? p.q_gamma : is_k ? p.k_gamma : nullptr;
    const bool norm = __any_sync(0xFFFFFFFFu, gamma != nullptr), swaps = __any_sync(0xFFFFFFFFu, partner != e0);
    float g[8];
    unpack8(gamma ? ld128(gamma + e0) : make_uint4(0, 0, 0, 0), g);
    const float *sp = is_k ? p.c.k_scale : p.c.v_scale;
    const float s = MX || !sp ? 1.f : __ldg(sp + kh), gain = __fdiv_rn(1.f, __fmul_rn(6.f, s));
    const int partner_lane = (threadIdx.x & 31) + (partner - e0) / 8;
    uint16_t *q_row = p.q_out + ((size_t)token0 * p.q_heads + head) * D + e0;
    for (int x = 0; x < n; ++x, q_row += (size_t)p.q_heads * D) {
      const uint4 cur = ahead1;
      ahead1 = ahead2;
      ahead2 = fetch();
      float v[8];
      unpack8(cur, v);
      if (norm) {
        // in 64 bits: a rounding of the sum would move codes at the borders between two of them
        double ss = add_squares_exact(cur.x, add_squares_exact(cur.y, add_squares_exact(cur.z, add_squares_exact(cur.w, 0.0))));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float mean = __double2float_rn(ss * (1.0 / D));
        const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, p.eps)));
        if (gamma) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rstd), g[i]);
        }
      }
      // two angles are neighbours, the next two 2 NC on
      const float2 *turn = turns[x][p.interleaved || !first] + pair_place(f0);
      if (swaps) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xFFFFFFFFu, v[i], partner_lane);
        if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = turn[(i >> 1) * 2 * NC + (i & 1)];
            v[i] = __fadd_rn(__fmul_rn(v[i], cs.x), __fmul_rn(y[i], cs.y));
          }
        }
      } else if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 cs = turn[(i >> 1) * 2 * NC + (i & 1)];
          const float a = v[2 * i], b = v[2 * i + 1];
          v[2 * i] = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
          v[2 * i + 1] = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
        }
      }
      const TokenPlace &tp = places[x];
      if (is_q && tp.in_use) *reinterpret_cast<uint4 *>(q_row) = pack8_bf16(v);
      if (__all_sync(0xFFFFFFFFu, is_q || !live)) continue;
      // FP4 codes of the lane's eight elements; the block maximum spans two (four) lanes
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) am = max3abs(am, v[i], v[i + 1]);
      am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      if (MX) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      if (is_q || !live || !tp.in_use || tp.group < 0) continue;
      uint32_t sb;
      float inv;
      if (MX) {
        const int e = (int)(__float_as_uint(am) >> 23) - 2;
        sb = (uint32_t)min(max(e, kKvExpMin), kKvExpMax);
        inv = __uint_as_float((254u - sb) << 23);
      } else {
        sb = cvt_e4m3(__fmul_rn(am, gain));
        const float d = __fmul_rn(e4m3_to_f32(sb), s);
        inv = d == 0.f ? 0.f : __frcp_rn(d);
      }
      uint8_t *grp = p.c.pages + tp.group + lp.head;
      *reinterpret_cast<uint32_t *>(grp + tp.codes[lp.is_v] + lp.codes) =
          cvt_e2m1x8(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv), __fmul_rn(v[2], inv), __fmul_rn(v[3], inv),
                     __fmul_rn(v[4], inv), __fmul_rn(v[5], inv), __fmul_rn(v[6], inv), __fmul_rn(v[7], inv));
      if (e0 % (MX ? 32 : 16) == 0) grp[tp.scales[lp.is_v] + lp.scale] = (uint8_t)sb;
    }
  }
}

// Read: a block per one to sixteen tokens; a lane turns eight codes and their scale into values, the
// same eight elements of four tokens at a time. code * block scale is exact in float16. 32799 tokens
// of eight key heads take 38 us, 4.5 TB/s; 72 us with a token per block, whose instructions to find
// every unit's place were the bound.
template <int D, bool MX>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams p, int per_block) {
  constexpr int L = D / 8, U = 4;
  __shared__ TokenPlace places[kMaxTokens];
  const int token0 = blockIdx.x * per_block, n = min(per_block, p.b.tokens - token0);
  find_tokens<D, MX>(p.b, p.c, token0, n, places);
  const int kvh = p.c.kv_heads;
  for (int in = threadIdx.x; in < 2 * kvh * L; in += blockDim.x) {
    const int j = in % L, is_v = in >= kvh * L, kh = in / L - is_v * kvh;
    const LanePlace<D, MX> lp(p.c, kh, is_v, j);
    const float *sp = is_v ? p.c.v_scale : p.c.k_scale;
    const float s = MX || !sp ? 1.f : __ldg(sp + kh);
    const size_t o0 = ((size_t)token0 * kvh + kh) * D + 8 * j, step = (size_t)kvh * D;
    void *out = is_v ? p.v_out : p.k_out;
    for (int x0 = 0; x0 < n; x0 += U) {
      uint32_t codes[U], sb[U];
#pragma unroll
      for (int y = 0; y < U; ++y) {
        codes[y] = sb[y] = 0u;
        if (x0 + y < n && places[x0 + y].group >= 0) {
          const TokenPlace &tp = places[x0 + y];
          const uint8_t *grp = p.c.pages + tp.group + lp.head;
          codes[y] = *reinterpret_cast<const uint32_t *>(grp + tp.codes[is_v] + lp.codes);
          sb[y] = grp[tp.scales[is_v] + lp.scale];
        }
      }
#pragma unroll
      for (int y = 0; y < U; ++y) {
        if (x0 + y >= n || !places[x0 + y].in_use) continue;
        const uint32_t b = kv_scales2<MX>(sb[y] * 0x101u);
        uint32_t h[4];
        cvt_e2m1x8_to_f16x2(codes[y], h);
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = half2_bits_to_float2(mul2(h[q], b));
          v[2 * q] = __fmul_rn(f.x, s), v[2 * q + 1] = __fmul_rn(f.y, s);
        }
        const size_t o = o0 + (x0 + y) * step;
        if (p.out_f32) {
          float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
          f[0] = make_float4(v[0], v[1], v[2], v[3]);
          f[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + o) = pack8_bf16(v);
        }
      }
    }
  }
}

// Tokens per block: one while every token finds a free slot on the SMs (latency), then as many as
// fill whole waves of resident blocks (1024 threads of an SM: 64 registers each).
int tokens_per_block(int tokens, int threads) {
  const long long slots = (long long)sm_count() * (1024 / threads);
  const long long waves = (tokens + slots * kMaxTokens - 1) / (slots * kMaxTokens);
  return (int)((tokens + slots * waves - 1) / (slots * waves));
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, int d, int fmt, cudaStream_t st) {
  const int lanes = (p.q_heads + 2 * p.c.kv_heads) * (d / 8);
  const int passes = (lanes + 255) / 256;
  const int threads = ((lanes + passes - 1) / passes + 31) / 32 * 32;  // whole warps, even passes
  const int n = tokens_per_block(p.b.tokens, threads), blocks = (p.b.tokens + n - 1) / n;
  if (d == 128) (fmt ? kv_append_kernel<128, true> : kv_append_kernel<128, false>)<<<blocks, threads, 0, st>>>(p, n);
  else (fmt ? kv_append_kernel<64, true> : kv_append_kernel<64, false>)<<<blocks, threads, 0, st>>>(p, n);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const ReadParams &p, int d, int fmt, cudaStream_t st) {
  const int lanes = 2 * p.c.kv_heads * (d / 8);
  const int threads = lanes >= 256 ? 256 : (lanes + 31) / 32 * 32;
  const int n = tokens_per_block(p.b.tokens, threads), blocks = (p.b.tokens + n - 1) / n;
  if (d == 128) (fmt ? kv_read_kernel<128, true> : kv_read_kernel<128, false>)<<<blocks, threads, 0, st>>>(p, n);
  else (fmt ? kv_read_kernel<64, true> : kv_read_kernel<64, false>)<<<blocks, threads, 0, st>>>(p, n);
  return cudaGetLastError();
}

}  // namespace sharq
