// The paged FP4 key/value cache: appending a call's keys and values (with the per-head
// normalization and the position rotation of q and k on the way) and reading rows back.
#include "sharq_common.cuh"
#include "sharq_internal.h"
#include "sharq_kv.h"

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

// Where a token row of the call lives: its position in its sequence, and the row of the cache.
struct TokenPlace {
  int pos;            // may be negative (fewer cached than new tokens)
  int in_use;         // a row of some sequence (rows past the last sequence are not)
  long long page;     // -1: no place in the cache
};

// The places of `n` consecutive tokens. The block counts the sequences that end at or before the
// first (one pass over cu_q, not a chain of dependent loads); a thread per token searches on.
constexpr int kMaxTokens = 8;
__device__ __forceinline__ void find_tokens(const KvBatchView &b, const KvCacheView &c, int token0, int n, TokenPlace *out) {
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
    TokenPlace t{0, 0, -1};
    if (seq < b.n_seq && token >= __ldg(b.cu_q)) {
      t.in_use = 1;
      t.pos = __ldg(b.kv_len + seq) - __ldg(b.cu_q + seq + 1) + token;
      const int col = t.pos >> c.page_shift;
      if (t.pos >= 0 && col < b.max_pages) {
        const int page = __ldg(b.page_table + (size_t)seq * b.max_pages + col);
        if (page >= 0 && page < c.num_pages) t.page = page;
      }
    }
    out[threadIdx.x] = t;
  }
  __syncthreads();
}

// Append: a block per one to eight tokens, D/8 lanes per head, eight elements per lane; the lane of
// the rotation's partner elements loads them itself (they are in L1), so no lane waits for another
// except for the block maxima. cos and sin are formed once per token from the 64-bit angle and
// rounded once. Bound by the bytes of the row (read once, q written once); several tokens per block
// share the latency of finding their places and of the sines.
template <int D, bool MX>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p, int per_block) {
  constexpr int L = D / 8;  // lanes per head
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  constexpr int NB = D / (MX ? 32 : 16);
  __shared__ float2 turns[kMaxTokens][D / 2];
  __shared__ TokenPlace places[kMaxTokens];
  const int token0 = blockIdx.x * per_block, n = min(per_block, p.b.tokens - token0);
  find_tokens(p.b, p.c, token0, n, places);
  for (int i = threadIdx.x; i < n * p.rot_half; i += blockDim.x) {
    const int x = i / p.rot_half, j = i - x * p.rot_half;
    double s, c;
    sincos((double)places[x].pos * (double)__ldg(p.inv_freq + j), &s, &c);
    turns[x][j] = make_float2(__double2float_rn(c), __double2float_rn(s));
  }
  __syncthreads();
  const int kvh = p.c.kv_heads, heads = p.q_heads + 2 * kvh;
  const int j = threadIdx.x % L, e0 = 8 * j;
  // whole warps stay in the loop: the shuffles below name every lane
#pragma unroll 2
  for (int i0 = 0; i0 < n * heads; i0 += blockDim.x / L) {
    const int i = i0 + threadIdx.x / L, x_tok = i / heads, head = i - x_tok * heads, token = token0 + x_tok;
    const TokenPlace tp = places[min(x_tok, n - 1)];
    const bool live = i < n * heads && tp.in_use;
    const uint16_t *row = p.qkv + (size_t)token * p.row_stride;
    const float2 *turn = turns[min(x_tok, n - 1)];
    const bool is_q = live && head < p.q_heads, is_k = live && !is_q && head < p.q_heads + kvh;
    float x[8], y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = ld128(row + (size_t)head * D + e0);
    const bool turned = (is_q || is_k) && e0 < 2 * p.rot_half;
    const int partner = p.interleaved ? e0 : e0 < p.rot_half ? e0 + p.rot_half : e0 - p.rot_half;
    uint4 wp = w;
    if (turned && !p.interleaved) wp = ld128(row + (size_t)head * D + partner);
    unpack8(w, x);
    const uint16_t *gamma = is_q ? p.q_gamma : is_k ? p.k_gamma : nullptr;
    if (p.q_gamma || p.k_gamma) {  // block-uniform
      double ss = 0.0;
      ss = add_squares_exact(w.x, ss), ss = add_squares_exact(w.y, ss);
      ss = add_squares_exact(w.z, ss), ss = add_squares_exact(w.w, ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float mean = __double2float_rn(ss * (1.0 / D));
      const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, p.eps)));
      unpack8(wp, y);
      if (gamma) {
        float g[8], gp[8];
        unpack8(ld128(gamma + e0), g);
        unpack8(ld128(gamma + partner), gp);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = __fmul_rn(__fmul_rn(x[i], rstd), g[i]);
          y[i] = __fmul_rn(__fmul_rn(y[i], rstd), gp[i]);
        }
      }
    } else {
      unpack8(wp, y);
    }
    if (turned) {
      float r[8];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 cs = turn[e0 / 2 + i];
          r[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], cs.x), __fmul_rn(x[2 * i + 1], cs.y));
          r[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], cs.x), __fmul_rn(x[2 * i], cs.y));
        }
      } else {
        const bool first = e0 < p.rot_half;
        const int f0 = first ? e0 : e0 - p.rot_half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 cs = turn[f0 + i];
          const float a = __fmul_rn(x[i], cs.x), b = __fmul_rn(y[i], cs.y);
          r[i] = first ? __fsub_rn(a, b) : __fadd_rn(a, b);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = r[i];
    }
    if (is_q) *reinterpret_cast<uint4 *>(p.q_out + ((size_t)token * p.q_heads + head) * D + e0) = pack8_bf16(x);
    // FP4 codes of the lane's eight elements; the block maximum spans two (four) lanes
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i]));
    am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    if (MX) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    if (is_q || !live || tp.page < 0) continue;
    const int kh = is_k ? head - p.q_heads : head - p.q_heads - kvh;
    uint32_t sb;
    float inv;
    if (MX) {
      const int e = (int)(__float_as_uint(am) >> 23) - 2;
      sb = (uint32_t)min(max(e, kKvExpMin), kKvExpMax);
      inv = __uint_as_float((254u - sb) << 23);
    } else {
      const float *sp = is_k ? p.c.k_scale : p.c.v_scale;
      const float s = sp ? __ldg(sp + kh) : 1.f;
      sb = cvt_e4m3(__fmul_rn(am, __fdiv_rn(1.f, __fmul_rn(6.f, s))));
      const float d = __fmul_rn(e4m3_to_f32(sb), s);
      inv = d == 0.f ? 0.f : __frcp_rn(d);
    }
    const uint32_t codes = cvt_e2m1x8(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv), __fmul_rn(x[2], inv),
                                      __fmul_rn(x[3], inv), __fmul_rn(x[4], inv), __fmul_rn(x[5], inv),
                                      __fmul_rn(x[6], inv), __fmul_rn(x[7], inv));
    const int in_page = tp.pos & ((1 << p.c.page_shift) - 1), r = in_page & 15;
    uint8_t *grp = p.c.pages + ((((size_t)tp.page * kvh + kh) << (p.c.page_shift - 4)) + (in_page >> 4)) * G.bytes;
    const int blk = e0 / (MX ? 32 : 16);
    const bool writes_scale = e0 % (MX ? 32 : 16) == 0;
    if (is_k) {
      *reinterpret_cast<uint32_t *>(grp + r * (D / 2) + 4 * j) = codes;
      if (writes_scale) grp[G.k_scales + r * NB + blk] = (uint8_t)sb;
    } else {
      *reinterpret_cast<uint32_t *>(grp + G.v_codes + kv_v_place(D, r, e0 / (D / 8)) + (D == 128 ? 4 * (j & 1) : 0)) = codes;
      if (writes_scale) grp[G.v_scales + kv_v_scale_place(r, blk)] = (uint8_t)sb;
    }
  }
}

// Read: a block per one to eight tokens; a lane turns eight codes and their scale into values, four
// such units in flight at once.
template <int D, bool MX>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams p, int per_block) {
  constexpr int L = D / 8, U = 4;
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  constexpr int NB = D / (MX ? 32 : 16);
  __shared__ TokenPlace places[kMaxTokens];
  const int token0 = blockIdx.x * per_block, n = min(per_block, p.b.tokens - token0);
  find_tokens(p.b, p.c, token0, n, places);
  const int kvh = p.c.kv_heads, units = 2 * kvh * L;
  for (int i0 = threadIdx.x; i0 < n * units; i0 += U * blockDim.x) {
    uint32_t codes[U], sb[U];
#pragma unroll
    for (int y = 0; y < U; ++y) {
      const int i = i0 + y * blockDim.x;
      codes[y] = sb[y] = 0u;
      if (i >= n * units) continue;
      const int x = i / units, in = i - x * units, j = in % L, is_v = in >= kvh * L, head = in / L - is_v * kvh, e0 = 8 * j;
      const TokenPlace tp = places[x];
      if (tp.page < 0) continue;
      const int in_page = tp.pos & ((1 << p.c.page_shift) - 1), r = in_page & 15, blk = e0 / (MX ? 32 : 16);
      const uint8_t *grp =
          p.c.pages + ((((size_t)tp.page * kvh + head) << (p.c.page_shift - 4)) + (in_page >> 4)) * G.bytes;
      const int at = is_v ? G.v_codes + kv_v_place(D, r, e0 / (D / 8)) + (D == 128 ? 4 * (j & 1) : 0) : r * (D / 2) + 4 * j;
      codes[y] = *reinterpret_cast<const uint32_t *>(grp + at);
      sb[y] = grp[is_v ? G.v_scales + kv_v_scale_place(r, blk) : G.k_scales + r * NB + blk];
    }
#pragma unroll
    for (int y = 0; y < U; ++y) {
      const int i = i0 + y * blockDim.x;
      if (i >= n * units) continue;
      const int x = i / units, in = i - x * units, j = in % L, is_v = in >= kvh * L, head = in / L - is_v * kvh, e0 = 8 * j;
      if (!places[x].in_use) continue;
      const float *sp = is_v ? p.c.v_scale : p.c.k_scale;
      const float s = MX ? 1.f : sp ? __ldg(sp + head) : 1.f, b = MX ? e8m0_to_f32(sb[y]) : e4m3_to_f32(sb[y]);
      uint32_t h[4];
      cvt_e2m1x8_to_f16x2(codes[y], h);
      float v[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = half2_bits_to_float2(h[q]);
        v[2 * q] = __fmul_rn(__fmul_rn(f.x, b), s);
        v[2 * q + 1] = __fmul_rn(__fmul_rn(f.y, b), s);
      }
      const size_t o = ((size_t)(token0 + x) * kvh + head) * D + e0;
      void *out = is_v ? p.v_out : p.k_out;
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

// Tokens per block: one while blocks are few (latency), up to eight once there are several waves.
int tokens_per_block(int tokens) {
  const int waves = tokens / (8 * sm_count());
  return waves < 1 ? 1 : waves < kMaxTokens ? waves : kMaxTokens;
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, int d, int fmt, cudaStream_t st) {
  const int n = tokens_per_block(p.b.tokens), blocks = (p.b.tokens + n - 1) / n;
  const int lanes = (p.q_heads + 2 * p.c.kv_heads) * (d / 8) * n;
  const int passes = (lanes + 255) / 256;
  const int threads = ((lanes + passes - 1) / passes + 31) / 32 * 32;  // whole warps, even passes
  if (d == 128) (fmt ? kv_append_kernel<128, true> : kv_append_kernel<128, false>)<<<blocks, threads, 0, st>>>(p, n);
  else (fmt ? kv_append_kernel<64, true> : kv_append_kernel<64, false>)<<<blocks, threads, 0, st>>>(p, n);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const ReadParams &p, int d, int fmt, cudaStream_t st) {
  const int n = tokens_per_block(p.b.tokens), blocks = (p.b.tokens + n - 1) / n;
  const int lanes = 2 * p.c.kv_heads * (d / 8) * n;
  const int threads = lanes >= 256 ? 256 : (lanes + 31) / 32 * 32;
  if (d == 128) (fmt ? kv_read_kernel<128, true> : kv_read_kernel<128, false>)<<<blocks, threads, 0, st>>>(p, n);
  else (fmt ? kv_read_kernel<64, true> : kv_read_kernel<64, false>)<<<blocks, threads, 0, st>>>(p, n);
  return cudaGetLastError();
}

}  // namespace sharq
