// Device helpers shared by the kernels of the attention side.
#pragma once

#include "sharq_common.cuh"

namespace sharq {

__device__ __forceinline__ uint32_t kv_smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ float kv_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t kv_pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
constexpr uint64_t kKvDrainLimitNs = 4000000000ull;  // own copies and MMAs in flight before a block ends
__device__ __forceinline__ bool kv_mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool kv_mbar_test(uint32_t bar, uint32_t parity) {  // without suspending the thread
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Time since `*t0` (set on the first call) in nanoseconds, at most: SM cycles of at least half a
// nanosecond. (The global timer's steps of a microsecond hide a short wait.)
__device__ __forceinline__ uint64_t kv_waited_ns(uint64_t *t0) {
  const uint64_t t = (uint64_t)clock64();
  if (*t0 == 0) *t0 = t;
  return (t - *t0) >> 1;
}
__device__ __forceinline__ void kv_mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
// two scale codes in the low 16 bits -> half2 (low byte in the low half): exact in the cache's
// range of exponents
template <bool MX>
__device__ __forceinline__ uint32_t kv_scales2(uint32_t two) {
  uint32_t d;
  if (MX) {
    d = kv_pack_half2(__uint_as_float((two & 0xFFu) << 23), __uint_as_float((two & 0xFF00u) << 15));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  }
  return d;
}

// ss + a unit's eight squares, exact products and every addition in float64.
__device__ __forceinline__ double add_squares(const uint4 &v, double ss) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = (double)bf16lo(w[i]), b = (double)bf16hi(w[i]);
    ss = __fma_rn(b, b, __fma_rn(a, a, ss));
  }
  return ss;
}

// Exponents are score * c - m in one rounding, m a rounded reference. Where |m| is beyond 2^24 that rounding of
// m alone is worth powers of two (at 2^28 up to 2^16: past float16, or every key at zero). Such a row's
// product is rounded by itself: the largest is then m exactly, and no other above it.
__device__ __forceinline__ bool kv_is_far(float m) { return fabsf(m) > 0x1p24f && m != -INFINITY; }

// row / group for row < 2^32 / group (the entry point keeps to that)
__device__ __forceinline__ int token_of(int group, uint32_t group_inv, int row) {
  return group == 1 ? row : (int)__umulhi((uint32_t)row, group_inv);
}

// ---------------------------------------------------------------- equal shares of a launch's work
// An item is a block of query rows of one key head; an entry is the items of every head of the same
// rows, which cost the same: their key steps, and ITEM more for what every item costs. The costs
// of all items in a row, entry by entry, are cut into equal shares, one per block. A cut is moved to
// the item's edge where it would leave a piece of `snap` steps or fewer, so that a cut inside an
// item always stands behind its first ITEM units.
struct Share {
  long long total, blocks;  // cost of the launch, blocks that have a share
  long long cut[2];         // begin and end of the share
  long long first;          // where the entry that the share begins in begins
  long long per;            // total = per * blocks + rest
  int rest;
  int entry, snap;
};
// An item's parts: how many, which one a block has, and the block of the first.
struct ItemParts {
  int count, index, owner;
};

// a / b for a quotient below 2^20: float32 finds it to within one. (A 64-bit division takes a few hundred
// cycles; a block makes several in a row before its first load.)
__device__ __forceinline__ int small_quotient(long long a, long long b) {
  int q = (int)__fdividef((float)a, (float)b);
  const long long r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

// block * total / blocks
__device__ __forceinline__ long long raw_cut(const Share &s, long long block) {
  return block >= s.blocks ? s.total : block * s.per + (uint32_t)block * (uint32_t)s.rest / (uint32_t)s.blocks;
}

// All threads: the entries' costs are summed in chunks of the block size, then the entries that
// hold the share's two ends are found (from registers where one chunk holds every entry).
template <int THREADS, int ITEM, class Cost>
__device__ __forceinline__ void find_share(long long entries, int heads, int least, Share *sh, long long *warp_sums,
                                           Cost entry_cost) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long total = 0, before = 0, cost = 0, e = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
    for (long long e0 = 0; e0 < entries; e0 += THREADS) {
      if (pass == 0 || entries > THREADS) {
        e = e0 + threadIdx.x;
        cost = e < entries ? (long long)entry_cost(e) * heads : 0;
        long long inc = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
          if (lane >= o) inc += up;
        }
        __syncthreads();  // the sums of the chunk before have been read
        if (lane == 31) warp_sums[warp] = inc;
        __syncthreads();
        before = base + inc - cost;
        for (int x = 0; x < THREADS / 32; ++x) {
          const long long v = warp_sums[x];
          if (x < warp) before += v;
          base += v;
        }
      }
      if (pass == 1 && cost > 0) {
        const int item = (int)((uint64_t)cost >> 32 ? cost / heads : (uint32_t)cost / (uint32_t)heads);
        for (int i = 0; i < 2; ++i) {
          const long long x = raw_cut(*sh, (long long)blockIdx.x + i);
          if (x < before || x >= before + cost) continue;
          const long long p0 = before + (long long)small_quotient(x - before, item) * item;
          sh->cut[i] = x - p0 <= ITEM + sh->snap ? p0 : p0 + item - x <= sh->snap ? p0 + item : x;
          if (i == 0) sh->entry = (int)e, sh->first = before;
        }
      }
    }
    if (pass == 0) {
      total = base;
      if (threadIdx.x == 0) {
        sh->total = total;
        const uint32_t blocks = total >= (long long)gridDim.x * least ? gridDim.x : max(1u, (uint32_t)total / (uint32_t)least);
        const long long per = (uint64_t)total >> 32 ? total / blocks : (uint32_t)total / blocks;
        sh->blocks = blocks, sh->per = per, sh->rest = (int)(total - per * blocks);
        sh->snap = total >= 8ll * blocks ? 2 : total >= 4ll * blocks ? 1 : 0;
        sh->cut[0] = sh->cut[1] = total;  // ends that no entry holds
        sh->entry = 0, sh->first = 0;
      }
      __syncthreads();
    }
  }
  __syncthreads();
}

// The parts of the item [p0, p1), of which this block has the one that begins at `from`. The cuts
// inside it are those with p0 + ITEM + snap < raw_cut(block) < p1 - snap.
template <int ITEM>
__device__ __forceinline__ ItemParts item_parts(const Share &s, long long p0, long long p1, long long from) {
  const int lo = small_quotient((p0 + ITEM + s.snap + 1) * s.blocks + s.total - 1, s.total);
  const int hi = min(small_quotient((p1 - s.snap) * s.blocks + s.total - 1, s.total) - 1, (int)s.blocks - 1);
  return ItemParts{hi >= lo ? hi - lo + 2 : 1, from == p0 ? 0 : (int)blockIdx.x - lo + 1, lo - 1};
}

}  // namespace sharq
