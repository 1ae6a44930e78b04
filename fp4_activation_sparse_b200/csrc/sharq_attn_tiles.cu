// Attention over the paged FP4 cache for many query rows per key head (prompts, pieces of prompts).
//
// One block works on 256 query rows of one key head (the group's heads of consecutive tokens: row
// i * group + g) as two 128-row tiles, and walks the keys in tiles of 128. Both contractions run on
// the tensor cores from float16 operands with float32 accumulators in tensor memory:
//   S_t = Q_t K^T   Q_t and K in shared memory; Q scaled by a power of two per row (exact)
//   O_t += P_t V    P_t in tensor memory (over S_t's columns), V in shared memory as stored
// The cache's codes become float16 on the way into shared memory: code * block scale is exact there
// (2 + 4 significant bits; the E8M0 exponents of the cache are limited to float16's range). The
// second-level scales and the softmax scale are applied in float32.
//   warps 0..3, 4..7  softmax of tile 0 and of tile 1, one row per thread: maximum, exponentials
//                     (float32; rounded to float16 only as the operand P), sum, and the rescaling
//                     of O. O is rescaled only where a row's maximum grew by more than 2^8 since the
//                     last time: exponentials then stay below 2^8, far inside float16's range.
//   warps 8..11       codes and scales from global memory (the next tile's are in flight in
//                     registers), float16 into the shared-memory tiles
//   warp 12           tensor memory, and one thread that issues every MMA
// The two tiles alternate on the tensor pipe: while one tile's exponentials are formed, the other
// tile's products run. Every mbarrier wait is bounded; on expiry the block records a status word,
// stops issuing, waits for what it issued, frees its tensor memory and exits.
#include "sharq_common.cuh"
#include "sharq_kv.h"
#include "sharq_kv_device.cuh"

namespace sharq {

__device__ uint32_t g_attn_status = 0;  // bit 0: a bounded wait gave up

namespace {

constexpr int kRows = 128;  // query rows of a tile
constexpr int kKeys = 128;  // keys of a step
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;  // S0, S1 at 0 and 128; O0, O1 at 256 and 384
constexpr uint64_t kDrainLimitNs = 4000000000ull;
constexpr int kValidRing = 4;

template <int D>
struct TileSmem {
  static constexpr int kSlabs = D / 64;               // 64 elements = one 128-byte swizzled row
  static constexpr int kSlab = 128 * 128;             // bytes of a slab: 128 rows
  static constexpr int kTile = kSlabs * kSlab;        // one operand tile
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kBytes = 6 * kTile;
  static constexpr int kTotal = kBytes + 1024;        // alignment slack
};

struct Bars {
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], drain;
};

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// Gives up after `limit_ns`, or when another role of the block already did.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t *abort_flag) {
  if (mbar_try(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try(bar, parity)) return true;
    if (i == 1 || (i & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer() - t0 > limit_ns) {
        *abort_flag = 1u;
        atomicOr(&g_attn_status, 1u);
        return false;
      }
    }
  }
}
// the same in every lane with a vote, for warps that run aligned instructions afterwards
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                               volatile uint32_t *abort_flag) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit_ns, abort_flag)) != 0;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptors, 128-byte swizzle (layout code 2; bit 46: descriptor version).
// Rows along the outer dimension (Q, K: contraction contiguous): 8-row groups 1024 bytes apart.
// V is stored [key][element], so its contraction runs over the rows: 64-element slabs kSlab bytes
// apart (leading offset), 8-key groups 1024 bytes apart (stride offset).
constexpr uint64_t desc_template(uint32_t lbo, uint32_t sbo) {
  return ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
constexpr uint64_t kDescK = desc_template(16, 1024), kDescV = desc_template(16384, 1024);
__device__ __forceinline__ uint64_t desc(uint64_t tmpl, uint32_t addr) { return tmpl | (uint64_t)((addr >> 4) & 0x3FFFu); }

// kind::f16 instruction descriptor: float16 operands, float32 accumulator, M = 128
constexpr uint32_t idesc_f16(int n, bool b_outer_contiguous) {
  return (1u << 4) | ((b_outer_contiguous ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

#define SHARQ_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define SHARQ_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of the warp's 32 lanes: lane = row, register = column
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SHARQ_R8(v, 0), SHARQ_R8(v, 8), SHARQ_R8(v, 16), SHARQ_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::SHARQ_I8(v, 0),
      SHARQ_I8(v, 8), SHARQ_I8(v, 16), SHARQ_I8(v, 24), "r"(addr)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// What the block works on; every role computes it alike.
struct Work {
  int q0, rows, kh, kv_len, first_pos, row0;
  int lo[2], hi[2];  // key tiles of each row tile; lo >= hi: none
  int begin, end;    // key tiles of the block
};

__device__ __forceinline__ Work block_work(const AttnParams &p) {
  Work w;
  const int per = p.b.n_seq * p.c.kv_heads;
  const int row_tiles = (int)(((long long)p.b.max_q * p.group + 2 * kRows - 1) / (2 * kRows));
  const int rt = row_tiles - 1 - (int)(blockIdx.x / per);  // causal order: the longest first
  const int seq = (blockIdx.x % per) / p.c.kv_heads;
  w.kh = blockIdx.x % p.c.kv_heads;
  const int q1 = __ldg(p.b.cu_q + seq + 1);
  w.q0 = __ldg(p.b.cu_q + seq);
  w.kv_len = __ldg(p.b.kv_len + seq);
  w.row0 = rt * 2 * kRows;
  w.rows = min(min(q1 - w.q0, p.b.max_q) * p.group - w.row0, 2 * kRows);
  w.first_pos = w.kv_len - (q1 - w.q0);
  const int reach = min(w.kv_len, p.b.max_pages << p.c.page_shift);  // no place behind the table
  w.begin = 0x7FFFFFFF, w.end = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    int k_lo = 0, k_hi = reach;
    const int last = min(w.rows, (t + 1) * kRows) - 1;
    if (p.causal) {
      k_hi = min(k_hi, w.first_pos + (w.row0 + max(last, 0)) / p.group + 1);
      if (p.window > 0) k_lo = max(0, w.first_pos + (w.row0 + t * kRows) / p.group - p.window + 1);
    }
    w.lo[t] = k_lo / kKeys;
    w.hi[t] = last >= t * kRows ? (max(k_hi, 0) + kKeys - 1) / kKeys : 0;
    if (w.lo[t] < w.hi[t]) w.begin = min(w.begin, w.lo[t]), w.end = max(w.end, w.hi[t]);
  }
  if (w.end == 0) w.begin = 0;
  return w;
}

// ---------------------------------------------------------------- codes to float16 tiles
// Two groups of 16 tokens per warp and step. K: a 16-byte unit (32 elements of one row) per lane
// and load; V: the 16 bytes of lane 4g + t are four (D = 64) or two (D = 128) rows' runs of D/8
// elements. Stores are 16 bytes to swizzled rows; the lanes of one store cover every bank group
// four times, the least that 512 bytes can take.
template <int D, bool MX>
struct Codes {
  static constexpr int U = D / 64;  // 16-byte units per lane, group and operand
  uint4 u[2][U];
  uint32_t s[2][U];
};

template <int D, bool MX>
__device__ __forceinline__ void load_k(const uint8_t *const (&grp)[2], int lane, Codes<D, MX> &c) {
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  constexpr int NB = D / (MX ? 32 : 16), UR = D / 32;  // scales and units per row
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      c.u[g][x] = make_uint4(0, 0, 0, 0);
      c.s[g][x] = 0;
      if (grp[g]) {
        const int unit = lane + 32 * x;
        c.u[g][x] = __ldg(reinterpret_cast<const uint4 *>(grp[g]) + unit);
        const uint8_t *sp = grp[g] + G.k_scales + (unit / UR) * NB + (unit % UR) * (NB / UR);
        c.s[g][x] = MX ? (uint32_t)__ldg(sp) : (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(sp));
      }
    }
}
template <int D, bool MX>
__device__ __forceinline__ void load_v(const uint8_t *const (&grp)[2], int lane, Codes<D, MX> &c) {
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  constexpr int per_run = (MX ? 32 : 16) / (D / 8);  // runs that share a block
#pragma unroll
  for (int g = 0; g < 2; ++g) {
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      c.u[g][x] = make_uint4(0, 0, 0, 0);
      if (grp[g]) c.u[g][x] = __ldg(reinterpret_cast<const uint4 *>(grp[g] + G.v_codes) + lane + 32 * x);
    }
    c.s[g][0] = 0;
    if (grp[g])
      c.s[g][0] = __ldg(reinterpret_cast<const uint32_t *>(grp[g] + G.v_scales) + (lane >> 2) / per_run * 4 + (lane & 3));
  }
}

// eight codes times one scale pair -> 16 bytes of float16
__device__ __forceinline__ void put8(uint32_t addr, uint32_t codes, uint32_t scale) {
  uint32_t h[4];
  cvt_e2m1x8_to_f16x2(codes, h);
  sts128(addr, mul2(h[0], scale), mul2(h[1], scale), mul2(h[2], scale), mul2(h[3], scale));
}
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int row, int chunk) {
  return base + (chunk >> 3) * (128 * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D, bool MX>
__device__ __forceinline__ void store_k(uint32_t tile, int row0, int lane, const Codes<D, MX> &c) {
  constexpr int UR = D / 32;
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      const int unit = lane + 32 * x, row = row0 + 16 * g + unit / UR, chunk = (unit % UR) * 4;
      const uint32_t two = kv_scales2<MX>(MX ? c.s[g][x] * 0x101u : c.s[g][x]);
      const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
      const uint32_t *w = &c.u[g][x].x;
#pragma unroll
      for (int i = 0; i < 4; ++i) put8(tile_addr(tile, row, chunk + i), w[i], i < 2 ? s0 : s1);
    }
}
// left: keys of each group that exist (the scales of the others may be anything)
template <int D, bool MX>
__device__ __forceinline__ void store_v(uint32_t tile, int row0, int lane, int left, const Codes<D, MX> &c) {
  const int run = lane >> 2, t = lane & 3;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t s = c.s[g][0];
    if (left < 16 * (g + 1)) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (16 * g + 8 * (q >> 1) + 2 * t + (q & 1) >= left) s &= ~(0xFFu << (8 * q));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t two = kv_scales2<MX>(h ? s >> 16 : s & 0xFFFFu);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t sc = __byte_perm(two, 0, j ? 0x3232 : 0x1010);
        const int row = row0 + 16 * g + 8 * h + 2 * t + j;
        if (D == 128) {
          const uint32_t w0 = j ? c.u[g][h % (D / 64)].z : c.u[g][h % (D / 64)].x;
          const uint32_t w1 = j ? c.u[g][h % (D / 64)].w : c.u[g][h % (D / 64)].y;
          const bool swap = run >= 4;  // half the lanes begin with the upper chunk: every bank group in turn
          put8(tile_addr(tile, row, 2 * run + (swap ? 1 : 0)), swap ? w1 : w0, sc);
          put8(tile_addr(tile, row, 2 * run + (swap ? 0 : 1)), swap ? w0 : w1, sc);
        } else {
          const uint4 u = c.u[g][0];
          put8(tile_addr(tile, row, run), h ? (j ? u.w : u.z) : (j ? u.y : u.x), sc);
        }
      }
    }
  }
}

template <int D, bool MX>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const __grid_constant__ AttnParams p) {
  using M = TileSmem<D>;
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;
  __shared__ volatile uint32_t valid[kValidRing];  // a byte per dequantizing warp: two groups' bits

  const Work w = block_work(p);
  if (w.rows <= 0) return;
  const uint32_t base = (kv_smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.limit_ns;
  auto bar = [&](const uint64_t &b) { return kv_smem_u32(&b); };

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.q_full[i]), kRows);
      mbar_init(bar(bars.k_full[i]), 128);
      mbar_init(bar(bars.v_full[i]), 128);
      mbar_init(bar(bars.k_empty[i]), 1);
      mbar_init(bar(bars.v_empty[i]), 1);
      mbar_init(bar(bars.s_full[i]), 1);
      mbar_init(bar(bars.p_full[i]), kRows);
      mbar_init(bar(bars.o_full[i]), 1);
    }
    mbar_init(bar(bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(kv_smem_u32(&tmem_slot)), "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int lo = t ? w.lo[1] : w.lo[0], hi = t ? w.hi[1] : w.hi[0];
    const int row = w.row0 + t * kRows + r;  // row of the sequence's key head
    const bool live = t * kRows + r < w.rows;
    const int token = w.q0 + row / p.group, head = w.kh * p.group + row % p.group;
    const bool real = live && token >= 0 && token < p.b.tokens;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 tensor-memory lanes
    const uint32_t s_tm = tmem + lanes + t * 128, o_tm = tmem + lanes + 256 + t * 128;
    bool ok = true;
    float c;
    {
      // the row's largest value moves to [2^12, 2^13): exact in float16 down to 2^-36 of it
      uint32_t raw[D / 2];
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (real) v = __ldg(reinterpret_cast<const uint4 *>(p.q + (size_t)token * p.q_stride + head * D) + i);
        raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < D / 2; ++i) am = max3abs(am, bf16lo(raw[i]), bf16hi(raw[i]));
      const int e = max((int)(__float_as_uint(am) >> 23) - 127, -100);
      const float factor = (MX || !p.c.k_scale ? 1.f : __ldg(p.c.k_scale + w.kh)) * p.scale_log2;
      // the sign of the score's factor goes into the query, so that maxima stay maxima
      const float up = copysignf(__uint_as_float((uint32_t)(127 + 12 - e) << 23), factor);
      c = __uint_as_float((uint32_t)(127 - 12 + e) << 23) * fabsf(factor);
      if (c < 1e-37f) c = 1e-37f;  // a factor of zero must not meet the masked -inf
      const uint32_t q_tile = base + M::kQ + t * M::kTile;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        uint32_t h[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) h[x] = kv_pack_half2(bf16lo(raw[4 * i + x]) * up, bf16hi(raw[4 * i + x]) * up);
        sts128(tile_addr(q_tile, r, i), h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async();
      mbar_arrive(bar(bars.q_full[t]));
    }
    const int pos = w.first_pos + row / p.group;
    const int see_hi = p.causal ? min(pos, w.kv_len - 1) : w.kv_len - 1;
    const int see_lo = p.causal && p.window > 0 ? pos - p.window : -1;
    const int last = min(w.rows, (t + 1) * kRows) - 1;
    const int tile_lo = w.first_pos + (w.row0 + t * kRows) / p.group, tile_hi = w.first_pos + (w.row0 + max(last, 0)) / p.group;
    float m = -INFINITY, l = 0.f;  // m: reference of the exponentials, in units of log2
    for (int i = lo; i < hi; ++i) {
      const int it = i - lo;
      if (!(ok = mbar_wait_warp(bar(bars.s_full[t]), it & 1, limit, &abort_flag))) break;
      tc_fence_after();
      uint32_t sr[128];
#pragma unroll
      for (int x = 0; x < 4; ++x) tm_ld32(s_tm + 32 * x, sr + 32 * x);
      tc_wait_ld();
      float *s = reinterpret_cast<float *>(sr);
      const int key0 = i * kKeys;
      const uint32_t groups = valid[(i - w.begin) % kValidRing];
      const bool whole = groups == 0x03030303u && key0 + kKeys <= w.kv_len &&
                         (!p.causal || (key0 + kKeys - 1 <= tile_lo && (p.window <= 0 || key0 > tile_hi - p.window)));
      if (!whole) {
        const int top = see_hi - key0, bottom = see_lo - key0;
#pragma unroll
        for (int j = 0; j < 128; ++j)
          if (j > top || j <= bottom || !((groups >> (8 * (j / 32) + (j / 16) % 2)) & 1u)) s[j] = -INFINITY;
      }
      float mx = -INFINITY, mx2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 128; j += 4) mx = max3(mx, s[j], s[j + 1]), mx2 = max3(mx2, s[j + 2], s[j + 3]);
      const float top = fmaxf(mx, mx2) * c;
      const bool grew = top > m + 8.f || (m == -INFINITY && top > m);
      if (__any_sync(0xFFFFFFFFu, grew)) {
        const float next = grew ? top : m;
        const float f = grew ? kv_ex2(m - next) : 1.f;  // 0 where nothing was seen before
        m = next;
        l *= f;
        if (it > 0) {  // the scores' arrival says that the products before them are done
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t ov[32];
            tm_ld32(o_tm + 32 * x, ov);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * f);
            tm_st32(o_tm + 32 * x, ov);
          }
        }
      }
      const float shift = m == -INFINITY ? 0.f : -m;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pr[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float a = kv_ex2(fmaf(s[64 * half + 2 * j], c, shift)), b = kv_ex2(fmaf(s[64 * half + 2 * j + 1], c, shift));
          sum[(2 * j) & 3] += a, sum[(2 * j + 1) & 3] += b;
          pr[j] = kv_pack_half2(a, b);
        }
        tm_st32(s_tm + 32 * half, pr);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(bar(bars.p_full[t]));
    }
    const bool any = lo < hi;
    if (any && ok) ok = mbar_wait_warp(bar(bars.o_full[t]), 0, limit, &abort_flag);
    tc_fence_after();
    if (ok && __any_sync(0xFFFFFFFFu, real)) {
      const float inv = l == 0.f ? 0.f : (MX || !p.c.v_scale ? 1.f : __ldg(p.c.v_scale + w.kh)) / l;
      uint16_t *dst = p.y + ((size_t)token * p.q_heads + head) * D;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        uint32_t ov[32];
        if (any) {
          tm_ld32(o_tm + 32 * x, ov);
          tc_wait_ld();
        }
        uint32_t out[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float a = any ? __uint_as_float(ov[2 * j]) * inv : 0.f, b = any ? __uint_as_float(ov[2 * j + 1]) * inv : 0.f;
          const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
          out[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (real) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            reinterpret_cast<uint4 *>(dst + 32 * x)[j] = make_uint4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
        }
      }
      if (real && p.lse)
        p.lse[(size_t)token * p.q_heads + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
    }
    tc_fence_before();
  } else if (warp < 12) {
    // ------------------------------------------------------------------ codes to float16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int dw = warp - 8, seq_row = (blockIdx.x % (p.b.n_seq * p.c.kv_heads)) / p.c.kv_heads;
    const int *table = p.b.page_table + (size_t)seq_row * p.b.max_pages;
    const int group_mask = (1 << (p.c.page_shift - 4)) - 1;
    auto page_of = [&](int i, int g) -> int {  // page id of the warp's group g of step i; -1: no keys there
      const int gi = i * 8 + 2 * dw + g, col = gi >> (p.c.page_shift - 4);
      if (i >= w.end || 16 * gi >= w.kv_len || col >= p.b.max_pages) return -1;
      const int page = __ldg(table + col);
      return page < p.c.num_pages ? page : -1;
    };
    auto place = [&](int i, int g, int page) -> const uint8_t * {
      if (page < 0) return nullptr;
      const int gi = i * 8 + 2 * dw + g;
      return p.c.pages + ((((size_t)page * p.c.kv_heads + w.kh) << (p.c.page_shift - 4)) + (gi & group_mask)) * G.bytes;
    };
    Codes<D, MX> ck, cv;
    int next0 = page_of(w.begin, 0), next1 = page_of(w.begin, 1);
    const uint8_t *grp[2] = {place(w.begin, 0, next0), place(w.begin, 1, next1)};
    if (w.begin < w.end) {
      load_k<D, MX>(grp, lane, ck);
      load_v<D, MX>(grp, lane, cv);
    }
    next0 = page_of(w.begin + 1, 0), next1 = page_of(w.begin + 1, 1);
    for (int i = w.begin; i < w.end; ++i) {
      const int it = i - w.begin, st = it & 1;
      const uint32_t bits = (grp[0] ? 1u : 0u) | (grp[1] ? 2u : 0u);
      grp[0] = place(i + 1, 0, next0), grp[1] = place(i + 1, 1, next1);
      next0 = page_of(i + 2, 0), next1 = page_of(i + 2, 1);
      if (it >= 2 && !mbar_wait(bar(bars.k_empty[st]), ((it >> 1) - 1) & 1, limit, &abort_flag)) break;
      store_k<D, MX>(base + M::kK + st * M::kTile, 32 * dw, lane, ck);
      if (lane == 0) reinterpret_cast<volatile uint8_t *>(&valid[it % kValidRing])[dw] = (uint8_t)bits;
      fence_proxy_async();
      mbar_arrive(bar(bars.k_full[st]));
      load_k<D, MX>(grp, lane, ck);
      if (it >= 2 && !mbar_wait(bar(bars.v_empty[st]), ((it >> 1) - 1) & 1, limit, &abort_flag)) break;
      store_v<D, MX>(base + M::kV + st * M::kTile, 32 * dw, lane, w.kv_len - (i * kKeys + 32 * dw), cv);
      fence_proxy_async();
      mbar_arrive(bar(bars.v_full[st]));
      load_v<D, MX>(grp, lane, cv);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 12 && lane == 0) {
      // ---------------------------------------------------------------- MMA issue
      constexpr uint32_t id_s = idesc_f16(kKeys, false), id_o = idesc_f16(D, true);
      bool ok = true;
      auto scores = [&](int t, int st) {
        const uint32_t qa = base + M::kQ + t * M::kTile, ka = base + M::kK + st * M::kTile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * M::kSlab + (k & 3) * 32;
          mma_ss(tmem + t * 128, desc(kDescK, qa + off), desc(kDescK, ka + off), id_s, k > 0);
        }
        tc_commit(bar(bars.s_full[t]));
      };
      for (int i = w.begin - 1; ok && i < w.end; ++i) {
        const int it = i - w.begin;
        const bool more = i + 1 < w.end;
        if (more && !(ok = mbar_wait(bar(bars.k_full[(it + 1) & 1]), ((it + 1) >> 1) & 1, limit, &abort_flag))) break;
        if (it >= 0 && !(ok = mbar_wait(bar(bars.v_full[it & 1]), (it >> 1) & 1, limit, &abort_flag))) break;
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok) break;
          if (i >= w.lo[t] && i < w.hi[t]) {
            if (!(ok = mbar_wait(bar(bars.p_full[t]), (i - w.lo[t]) & 1, limit, &abort_flag))) break;
            tc_fence_after();
            const uint32_t va = base + M::kV + (it & 1) * M::kTile;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * k, desc(kDescV, va + k * 2048), id_o, k > 0 || i > w.lo[t]);
            if (i == w.hi[t] - 1) tc_commit(bar(bars.o_full[t]));
          }
          if (i + 1 >= w.lo[t] && i + 1 < w.hi[t]) {
            if (i + 1 == w.lo[t] && !(ok = mbar_wait(bar(bars.q_full[t]), 0, limit, &abort_flag))) break;
            tc_fence_after();
            scores(t, (it + 1) & 1);
          }
        }
        if (it >= 0) tc_commit(bar(bars.v_empty[it & 1]));
        if (more) tc_commit(bar(bars.k_empty[(it + 1) & 1]));
      }
      // everything issued has finished before tensor memory and shared memory go
      tc_commit(bar(bars.drain));
      volatile uint32_t never = 0;
      mbar_wait(bar(bars.drain), 0, kDrainLimitNs, &never);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

template <int D, bool MX>
cudaError_t launch_d(const AttnParams &p, cudaStream_t st) {
  auto kernel = attn_tiles_kernel<D, MX>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TileSmem<D>::kTotal);
  if (e != cudaSuccess) return e;
  const long long row_tiles = ((long long)p.b.max_q * p.group + 2 * kRows - 1) / (2 * kRows);
  const long long blocks = row_tiles * p.c.kv_heads * p.b.n_seq;
  if (blocks > 0x7FFFFFFFll || (long long)p.b.max_q * p.group > 0x7FFF0000ll) return cudaErrorInvalidConfiguration;
  kernel<<<(unsigned)blocks, kThreads, TileSmem<D>::kTotal, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_tiles(const AttnParams &p, int d, int fmt, cudaStream_t st) {
  if (d == 128) return fmt ? launch_d<128, true>(p, st) : launch_d<128, false>(p, st);
  return fmt ? launch_d<64, true>(p, st) : launch_d<64, false>(p, st);
}

cudaError_t read_and_clear_attn_status(uint32_t *status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_attn_status, sizeof *status);
  if (e != cudaSuccess || *status == 0) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_attn_status, &zero, sizeof zero);
}

}  // namespace sharq
