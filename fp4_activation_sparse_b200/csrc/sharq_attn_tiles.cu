// Attention over the paged FP4 cache for many query rows per key head (prompts, pieces of prompts).
//
// One block works on 256 query rows of one key head (the group's heads of consecutive tokens: row
// i * group + g) as two 128-row tiles, and walks the keys in tiles of 128. Both contractions run on
// the tensor cores from float16 operands with float32 accumulators in tensor memory:
//   S_t = Q_t K^T   Q_t and K in shared memory; Q scaled by a power of two per row
//   O_t += P_t V    P_t in tensor memory (over S_t's columns), V in shared memory as stored
// The cache's codes become float16 on the way into shared memory: code * block scale is exact there
// (2 + 4 significant bits; the E8M0 exponents of the cache are limited to float16's range). The
// second-level scales and the softmax scale are applied in float32.
//   warps 0..3, 4..7  softmax of tile 0 and of tile 1, one row per thread: maximum, exponentials
//                     (float32; rounded to float16 only as the operand P), sum, and the rescaling
//                     of O. O is rescaled only where a row's maximum grew by more than 2^8 since the
//                     last time: exponentials then stay below 2^8, far inside float16's range. They
//                     also bring the queries into shared memory, the next segment's before this
//                     one's output is read, so that its first scores form meanwhile.
//   warps 8..11       codes and scales from global memory (the next tile's are in flight in
//                     registers), float16 into the shared-memory tiles
//   warps 12, 13      one thread each that issues the MMAs of tile 0 and of tile 1 (12: tensor memory)
//   warp 14           the block's work list
// A step's keys come in two halves with a score buffer each, so that the scores of the next half
// form while this half's exponentials do, and the softmax warps never wait for the tensor pipe's
// latency; while one tile's exponentials are formed, the other tile's products run.
//
// The grid is one block per SM, and every block takes an equal, contiguous share of all key steps
// of the launch (found from the device's own lengths), so ragged batches balance and few long
// sequences fill the GPU. Within its share a block goes from segment to segment without draining:
// the queries of the next one load and its first keys are converted while the last step of this
// one is in its softmax. A query block whose steps are cut between blocks leaves its parts (O, m, l
// in float32) in the workspace; the block that arrives last joins them in the order of the keys.
//
// Where a key head has no more than 128 rows (drafted tokens, short prompts) the two tiles are twins: both
// hold the same rows and take every second key step, so that two softmax chains run at once instead of
// one. The first tile's warps join the two outputs as they read them from tensor memory. (Drafted
// tokens, 35 rows: 41.0 us with one tile idle, 39.4 with twins.)
//
// What bounds it. A step (256 rows, 128 keys, 128 elements) takes about 4200 cycles per SM. Its products
// need 2480 on the tensor pipe (the score halves, N = 64, are bound by reading Q and K from shared
// memory: 1540, against 1020 in one piece; the halves pay for that by hiding the latency between
// the roles), its exponentials 2048 on the special-function pipe, and the softmax warps' own chain of
// load, exponentials, store and arrival 1900 per half, of which the special-function pipe is busy
// half the time. Tried without gain: a share of the exponentials by a polynomial, the maximum left
// out, the next scores loaded before the arrival, the two tiles' exponentials kept apart, other
// splits of the registers, the halves unrolled, scores and probabilities in places of their own (the
// wait that this removes is covered by the other tile: 2 % slower).
//
// Measured (NVFP4): one prompt of 8192 tokens, 32 query and 8 key heads of 128, 540 to 560 us with the
// board's power, 980 to 1015 TFLOP/s; 9360 queries over 512 cached keys, 40 heads, 167 us; pieces of four
// prompts in a window of 4096 (64 elements, MXFP4) 89 us; 3 to 5 drafted tokens of 16 contexts, 28 query
// and 4 key heads, 42 us; 256 single tokens beside a prompt of 8192, 741 us.
//
// Every mbarrier wait is bounded; on expiry the block records a status word, stops issuing, waits
// for what it issued, frees its tensor memory and exits.
#include "sharq_common.cuh"
#include "sharq_internal.h"
#include "sharq_kv.h"
#include "sharq_kv_device.cuh"

namespace sharq {

__device__ uint32_t g_attn_status = 0;  // bit 0: a bounded wait gave up

namespace {

constexpr int kRows = 128;  // query rows of a tile
constexpr int kKeys = 128;  // keys of a step
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;  // S of tile t, half h at 128 t + 64 h (P over its first 32); O at 256 + 128 t
constexpr int kValidRing = 4;
// counters, eight (one per softmax warp) each: an item's by its first block, then a group's by the
// block and the slot of its first part
constexpr int kGroupCounter = 256;
static_assert(4 * 8 * (kGroupCounter + 2 * kGroupCounter) <= kAttnCounterBytes, "counters of 256 blocks");

template <int D>
struct TileSmem {
  static constexpr int kSlabs = D / 64;               // 64 elements = one 128-byte swizzled row
  static constexpr int kSlab = 128 * 128;             // bytes of a slab: 128 rows
  static constexpr int kTile = kSlabs * kSlab;        // one operand tile
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kBytes = 6 * kTile;
  static constexpr int kTotal = kBytes + 1024;        // alignment slack
};

struct Bars {
  uint64_t work_full[2], work_empty[2], q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_empty[2], drain[2];  // [row tile][half of a step]
  uint64_t twin_full, twin_empty;  // the second twin's maxima and sums
};
constexpr int kWorkReaders = 8 + 4 + 2;  // warps

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// one arrival for the warp, after all its lanes
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// One thread. Gives up after `limit_ns`, or when another role of the block already did.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t *abort_flag) {
  if (kv_mbar_test(bar, parity)) return true;
  uint64_t t0 = 0;
  kv_waited_ns(&t0);
  bool there;
  do {
    there = kv_mbar_try(bar, parity);
    if (kv_waited_ns(&t0) > limit_ns) {
      *abort_flag = 1u;
      atomicOr(&g_attn_status, 1u);
    }
    if (*abort_flag) return false;
  } while (!there);
  return true;
}
// the same for a whole warp, which leaves the wait together
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                               volatile uint32_t *abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !__all_sync(0xFFFFFFFFu, kv_mbar_try(bar, parity)); ++i) {
    if (i & 31u) continue;
    if (kv_waited_ns(&t0) > limit_ns) {
      *abort_flag = 1u;
      atomicOr(&g_attn_status, 1u);
    }
    if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) return false;
  }
  return true;
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
constexpr uint32_t desc_high(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }
constexpr uint32_t kDescHigh = desc_high(1024);
__device__ __forceinline__ uint32_t desc_low(uint32_t lbo, uint32_t addr) { return (lbo >> 4) << 16 | (addr >> 4); }

// kind::f16 instruction descriptor: float16 operands, float32 accumulator, M = 128
constexpr uint32_t idesc_f16(int n, bool b_outer_contiguous) {
  return (1u << 4) | ((b_outer_contiguous ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// operands by the lower words of their descriptors
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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

// the n lowest bits (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// pairs of float32
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ int token_in(const AttnParams &p, int row) { return token_of(p.group, p.group_inv, row); }

// ---------------------------------------------------------------- what a block works on
// Items are 256 query rows of one key head of one sequence.
// An item costs its key steps and kItemCost more (queries in, output out, the pipeline's start). With
// 2, 3, 4, 6, 8 the prompt of 8192 tokens takes 616, 552, 546, 550, 561 us, the drafted tokens 39.5,
// 40.8, 38.8, 39.3, 39.7, the window 91.1, 88.2, 88.4, 90.2, 90.3; the cross attention does not care.
constexpr int kItemCost = 4;
struct Range {
  int q0, rows, kv_len, first_pos, row0, first_key;  // first_key: no query of the item sees one before it
  int lo[2], hi[2];  // key steps of each row tile; lo >= hi: none
  int begin, end;    // of the item
  __device__ __forceinline__ int cost() const { return rows <= 0 ? 0 : kItemCost + max(1, end - begin); }
};
struct Work {
  Range r;  // lo, hi, begin, end limited to the segment
  int seq, kh;
  ItemParts parts;
};

// A boundary of cu_q as one of the call's rows, so that rows and entries stay what they are for each other.
__device__ __forceinline__ int token_row(const AttnParams &p, int at) { return min(max(at, 0), p.b.tokens); }

// Entries: the row tiles of sequence after sequence. Every sequence has as many places as the longest may need
// where one chunk of the block's threads holds them all. Else sequence b begins at b plus the whole row
// tiles of the rows before it: two places too many at most, so that one long prompt among many single
// tokens, or a loose bound on the rows, costs nothing.
struct Entries {
  int row_tiles;  // of the longest sequence
  bool dense;
  __device__ __forceinline__ Entries(const AttnParams &p, int rt)
      : row_tiles(rt), dense(rt == 1 || (long long)p.b.n_seq * rt <= kThreads) {}
  __device__ __forceinline__ static long long rows_before(const AttnParams &p, int seq) {
    return (long long)token_row(p, __ldg(p.b.cu_q + seq)) * p.group;
  }
  __device__ __forceinline__ int first(const AttnParams &p, int seq) const {
    return seq + (int)(rows_before(p, seq) / (2 * kRows) - rows_before(p, 0) / (2 * kRows));
  }
  __device__ __forceinline__ long long count(const AttnParams &p) const {
    return dense ? (long long)p.b.n_seq * row_tiles : first(p, p.b.n_seq);
  }
  __device__ __forceinline__ void find(const AttnParams &p, int entry, int &seq, int &rt) const {
    if (dense) {
      seq = entry / row_tiles, rt = entry - seq * row_tiles;
      return;
    }
    int lo = 0, hi = p.b.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first(p, mid) <= entry) lo = mid;
      else hi = mid - 1;
    }
    seq = lo, rt = entry - first(p, lo);
  }
};

template <bool TWIN>
__device__ __forceinline__ Range item_range(const AttnParams &p, int seq, int rt) {
  Range w;
  const int q1 = __ldg(p.b.cu_q + seq + 1);
  w.q0 = __ldg(p.b.cu_q + seq);
  w.kv_len = __ldg(p.b.kv_len + seq);
  w.row0 = rt * 2 * kRows;
  w.rows = min(min(token_row(p, q1) - token_row(p, w.q0), p.b.max_q) * p.group - w.row0, 2 * kRows);
  w.first_pos = w.kv_len - (q1 - w.q0);
  const int reach = min(w.kv_len, p.b.max_pages << p.c.page_shift);  // no place behind the table
  w.begin = 0x7FFFFFFF, w.end = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    int k_lo = 0, k_hi = reach;
    const int base = TWIN ? 0 : t * kRows, last = min(w.rows, base + kRows) - 1;
    if (p.causal) {
      k_hi = min(k_hi, w.first_pos + token_in(p, w.row0 + max(last, 0)) + 1);
      const int pos = w.first_pos + token_in(p, w.row0 + base);
      if (p.window > 0 && pos >= p.window) k_lo = pos - p.window + 1;
    }
    if (t == 0) w.first_key = k_lo;
    w.lo[t] = k_lo / kKeys;
    w.hi[t] = last >= base ? (max(k_hi, 0) + kKeys - 1) / kKeys : 0;
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
// [from, left): rows of the two groups that some query sees (the scales of the others may be anything)
template <int D, bool MX>
__device__ __forceinline__ void store_v(uint32_t tile, int row0, int lane, int from, int left, const Codes<D, MX> &c) {
  const int run = lane >> 2, t = lane & 3;
  const bool cut = from > 0 || left < 32;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t s = c.s[g][0];
    if (cut) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 16 * g + 8 * (q >> 1) + 2 * t + (q & 1);
        if (row < from || row >= left) s &= ~(0xFFu << (8 * q));
      }
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

// Entry n of the work list; every warp hands it back when it has read what it needs.
__device__ __forceinline__ bool get_work(Bars &bars, const Work *ring, int n, uint64_t limit, volatile uint32_t *abort_flag) {
  return mbar_wait_warp(kv_smem_u32(&bars.work_full[n & 1]), (n >> 1) & 1, limit, abort_flag) && ring[n & 1].r.rows > 0;
}
__device__ __forceinline__ void done_work(Bars &bars, int n) {
  mbar_arrive_warp(kv_smem_u32(&bars.work_empty[n & 1]));
}

__device__ __forceinline__ void st256(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), SHARQ_I8(v, 0) : "memory");
}

// The work list's warp: where its walk over the share stands, the same in every lane.
struct Walk {
  long long at, end, first;  // the share's next unit of cost and its end; where the costs of (seq, rt) begin
  int seq, rt;
};

// The share's next segment to `out` (rows 0: none is left).
template <bool TWIN>
__device__ __forceinline__ void next_segment(const AttnParams &p, const Share &sh, Walk &walk, Work &out) {
  const int heads = p.c.kv_heads, lane = threadIdx.x & 31;
  Work x;
  int cost = 0;
  x.r.rows = 0;
  while (walk.at < walk.end && walk.seq < p.b.n_seq) {
    x.seq = walk.seq;
    x.r = item_range<TWIN>(p, walk.seq, walk.rt);
    cost = x.r.cost();
    if (walk.at < walk.first + (long long)cost * heads) break;
    walk.first += (long long)cost * heads;
    const int rows = x.r.rows;
    x.r.rows = 0;
    ++walk.rt;
    if (rows == 2 * kRows) continue;
    // the next sequence with new tokens, 32 at a time
    walk.rt = 0;
    uint32_t some = 0;
    for (++walk.seq; walk.seq < p.b.n_seq; walk.seq += 32) {
      const int i = walk.seq + lane;
      some = __ballot_sync(0xFFFFFFFFu, i < p.b.n_seq && __ldg(p.b.cu_q + i + 1) > __ldg(p.b.cu_q + i));
      if (some) break;
    }
    if (some) walk.seq += __ffs(some) - 1;
  }
  if (x.r.rows > 0) {
    x.kh = small_quotient(walk.at - walk.first, cost);
    const long long p0 = walk.first + (long long)x.kh * cost, p1 = p0 + cost;
    const long long to = min(walk.end, p1);
    x.parts = item_parts<kItemCost>(sh, p0, p1, walk.at);
    if (x.r.begin < x.r.end) {
      const int from = walk.at == p0 ? x.r.begin : x.r.begin + (int)(walk.at - p0) - kItemCost;
      const int until = x.r.begin + (int)(to - p0) - kItemCost;
      x.r.begin = from, x.r.end = until;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        x.r.lo[t] = max(x.r.lo[t], from), x.r.hi[t] = min(x.r.hi[t], until);
        if (TWIN) x.r.lo[t] += (x.r.lo[t] ^ t) & 1, x.r.hi[t] -= ((x.r.hi[t] - 1) ^ t) & 1;
      }
    }
    walk.at = to;
  }
  if (lane == 0) out = x;
}

// A warp's 32 query rows of a segment to the shared-memory tile, D/16 lanes (32 bytes each) per row,
// all loads in flight at once. The row's largest value moves to [2^12, 2^13): eight significant bits
// are exact in float16 from 2^-17 on, 2^-29 of the largest, and an element below that is rounded by at most
// 2^-25, 2^-37 of the largest. The sign of the score's factor goes into the query, so that maxima stay maxima.
template <int D, bool MX>
__device__ __forceinline__ void load_queries(const AttnParams &p, const Work &w, int first, int row_base, int lane, uint32_t q_tile,
                                             float *coef) {
  constexpr int L = D / 16, RW = 32 / L, N = 32 / RW;
  const int sub = lane / L, chunk = lane % L * 2;
  const float factor = (MX || !p.c.k_scale ? 1.f : __ldg(p.c.k_scale + w.kh)) * p.scale_log2;
  uint4 v[N][2];
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const int r = first + row_base + x * RW + sub, row = w.r.row0 + r;
    const int at = token_in(p, row), token = w.r.q0 + at, head = w.kh * p.group + row - at * p.group;
    v[x][0] = v[x][1] = make_uint4(0, 0, 0, 0);
    if (r < w.r.rows && token >= 0 && token < p.b.tokens) {
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t)token * p.q_stride + head * D) + chunk;
      v[x][0] = __ldg(src), v[x][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int x = 0; x < N; ++x) {
    float am = 0.f;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      am = max3abs(max3abs(am, bf16lo(v[x][y].x), bf16hi(v[x][y].x)), bf16lo(v[x][y].y), bf16hi(v[x][y].y));
      am = max3abs(max3abs(am, bf16lo(v[x][y].z), bf16hi(v[x][y].z)), bf16lo(v[x][y].w), bf16hi(v[x][y].w));
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
    const int e = max((int)(__float_as_uint(am) >> 23) - 127, -100);
    const float up = copysignf(__uint_as_float((uint32_t)(127 + 12 - e) << 23), factor);
    const int r = row_base + x * RW + sub;
#pragma unroll
    for (int y = 0; y < 2; ++y)
      sts128(tile_addr(q_tile, r, chunk + y), kv_pack_half2(bf16lo(v[x][y].x) * up, bf16hi(v[x][y].x) * up),
             kv_pack_half2(bf16lo(v[x][y].y) * up, bf16hi(v[x][y].y) * up),
             kv_pack_half2(bf16lo(v[x][y].z) * up, bf16hi(v[x][y].z) * up),
             kv_pack_half2(bf16lo(v[x][y].w) * up, bf16hi(v[x][y].w) * up));
    const float c = __uint_as_float((uint32_t)(127 - 12 + e) << 23) * fabsf(factor);
    if (chunk == 0) coef[r] = c < 1e-37f ? 1e-37f : c;  // 0 must not meet the masked -inf
  }
  fence_proxy_async();
  __syncwarp();
}

template <int D, bool MX, bool TWIN>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const __grid_constant__ AttnParams p, int row_tiles) {
  using M = TileSmem<D>;
  constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ Share share;
  __shared__ Work ring[2];
  __shared__ long long warp_sums[kThreads / 32];
  __shared__ float2 twin_ml[TWIN ? kRows : 1];  // the second twin's maxima and sums
  __shared__ float row_coef[2 * kRows];  // score factor of each row of the segment
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;
  __shared__ volatile uint32_t valid[kValidRing];  // a byte per dequantizing warp: two groups' bits

  const uint32_t base = (kv_smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const uint64_t limit = p.limit_ns;
  auto bar = [&](const uint64_t &b) { return kv_smem_u32(&b); };

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      kv_mbar_init(bar(bars.work_full[i]), 1);
      kv_mbar_init(bar(bars.work_empty[i]), kWorkReaders);
      kv_mbar_init(bar(bars.q_full[i]), 4);
      kv_mbar_init(bar(bars.k_full[i]), 4);
      kv_mbar_init(bar(bars.v_full[i]), 4);
      kv_mbar_init(bar(bars.k_empty[i]), 2);
      kv_mbar_init(bar(bars.v_empty[i]), 2);
      for (int h = 0; h < 2; ++h) {
        kv_mbar_init(bar(bars.s_full[i][h]), 1);
        kv_mbar_init(bar(bars.p_full[i][h]), 4);
        kv_mbar_init(bar(bars.pv_done[i][h]), 1);
      }
      kv_mbar_init(bar(bars.o_empty[i]), 4);
      kv_mbar_init(bar(bars.drain[i]), 1);
    }
    kv_mbar_init(bar(bars.twin_full), 4);
    kv_mbar_init(bar(bars.twin_empty), 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const Entries entries(p, row_tiles);
  find_share<kThreads, kItemCost>(entries.count(p), p.c.kv_heads, kItemCost + 2, &share, warp_sums, [&](long long e) {
    int seq, rt;
    entries.find(p, (int)e, seq, rt);
    return rt < row_tiles ? item_range<TWIN>(p, seq, rt).cost() : 0;
  });
  if (share.cut[0] >= share.cut[1]) return;
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(kv_smem_u32(&tmem_slot)), "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_slot, 0);  // uniform

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 tensor-memory lanes
    const uint32_t s_tm = tmem + lanes + t * 128, o_tm = tmem + lanes + 256 + t * 128;
    const int first = TWIN ? 0 : t * kRows, stride = TWIN ? 2 : 1;  // this tile's rows and key steps
    int n = 0, steps = 0;  // steps of this row tile, key steps of all segments so far
    auto queries = [&](int seg) {
      const Work &x = ring[seg & 1];
      if ((t ? x.r.lo[1] : x.r.lo[0]) >= (t ? x.r.hi[1] : x.r.hi[0])) return;
      load_queries<D, MX>(p, x, first, 32 * (warp & 3), lane, base + M::kQ + t * M::kTile, row_coef + t * kRows);
      mbar_arrive_warp(bar(bars.q_full[t]));
    };
    bool more = get_work(bars, ring, 0, limit, &abort_flag);
    if (more) queries(0);
    for (int seg = 0; more; done_work(bars, seg), ++seg) {
      const Work &w = ring[seg & 1];
      const int lo = t ? w.r.lo[1] : w.r.lo[0], hi = t ? w.r.hi[1] : w.r.hi[0];
      const int step0 = steps - w.r.begin;
      steps += w.r.end - w.r.begin;
      const int kv_len = w.r.kv_len, pos = w.r.first_pos + token_in(p, w.r.row0 + first + r);
      const int see_hi = p.causal ? min(pos, kv_len - 1) : kv_len - 1;
      const int see_lo = p.causal && p.window > 0 && pos >= p.window ? pos - p.window : -1;
      const int last = max(min(w.r.rows, first + kRows) - 1, 0);
      const int tile_lo = w.r.first_pos + token_in(p, w.r.row0 + first), tile_hi = w.r.first_pos + token_in(p, w.r.row0 + last);
      const float c = row_coef[t * kRows + r];  // of this warp's making; unused without steps
      float m = -INFINITY, l = 0.f;  // m: reference of the exponentials, in units of log2
      bool ok = true;
      for (int i = lo; i < hi && ok; i += stride, ++n) {
        const int key0 = i * kKeys;
        uint32_t groups = 0x03030303u;
        bool whole = true;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!(ok = mbar_wait_warp(bar(bars.s_full[t][h]), n & 1, limit, &abort_flag))) break;
          tc_fence_after();
          uint32_t sr[64];
          tm_ld32(s_tm + 64 * h, sr), tm_ld32(s_tm + 64 * h + 32, sr + 32);
          if (h == 0) {
            groups = valid[(step0 + i) % kValidRing];
            whole = groups == 0x03030303u && key0 + kKeys <= kv_len &&
                    (!p.causal || (key0 + kKeys - 1 <= tile_lo && (p.window <= 0 || tile_hi - key0 < p.window)));
          }
          tc_wait_ld();
          float *s = reinterpret_cast<float *>(sr);
          float by = c;  // what the scores are still to be multiplied by
          const bool far = __any_sync(0xFFFFFFFFu, kv_is_far(m));
          if (!whole || far) {
            const int top = see_hi - key0 - 64 * h, bottom = see_lo - key0 - 64 * h;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t g = groups >> (16 * h + 8 * x);
              const uint32_t there = (g & 1u ? 0xFFFFu : 0u) | (g & 2u ? 0xFFFF0000u : 0u);
              const uint32_t see = there & bits_below(top + 1 - 32 * x) & ~bits_below(bottom + 1 - 32 * x);
#pragma unroll
              for (int j = 0; j < 32; ++j) s[32 * x + j] = see & (1u << j) ? s[32 * x + j] : -INFINITY;
            }
            if (far) {
              const float first = kv_is_far(m) ? c : 1.f;
#pragma unroll
              for (int j = 0; j < 64; ++j) s[j] = __fmul_rn(s[j], first);
              by = kv_is_far(m) ? 1.f : c;
            }
          }
          // The exponentials are formed against the reference at hand while the maximum is taken, and
          // once more in the rare half whose maximum is too far above it.
          const uint64_t c2 = pack2(by, by);
          uint32_t pr[32];
          float sum;
          auto exponentials = [&]() {
            const float shift = m == -INFINITY ? 0.f : -m;
            const uint64_t shift2 = pack2(shift, shift);
            uint64_t sums[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float a, b;
              unpack2(fma2(pack2(s[2 * j], s[2 * j + 1]), c2, shift2), a, b);
              a = kv_ex2(a), b = kv_ex2(b);
              sums[j & 1] = add2(sums[j & 1], pack2(a, b));
              pr[j] = kv_pack_half2(a, b);
            }
            float a, b;
            unpack2(add2(sums[0], sums[1]), a, b);
            sum = a + b;
          };
          exponentials();
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 8)
#pragma unroll
            for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], s[j + 2 * x], s[j + 2 * x + 1]);
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * by;
          const bool grew = top > m + 8.f;
          if (__any_sync(0xFFFFFFFFu, grew)) {
            const float next = grew ? top : m;
            const float f = grew ? kv_ex2(m - next) : 1.f;  // 0 where nothing was seen before
            const bool turned = __any_sync(0xFFFFFFFFu, kv_is_far(next) != kv_is_far(m));
            m = next;
            l *= f;
            exponentials();
            if (i > lo || h > 0) {
              // the products of the half before must be in O
              if (!(ok = mbar_wait_warp(bar(bars.pv_done[t][h ^ 1]), (h ? n : n - 1) & 1, limit, &abort_flag))) break;
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < D / 32; ++x) {
                uint32_t ov[32];
                tm_ld32(o_tm + 32 * x, ov);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * f);
                tm_st32(o_tm + 32 * x, ov);
              }
            }
            if (__builtin_expect(turned, 0)) {  // the half once more, with these rows' scores multiplied first
              --h;
              continue;
            }
          }
          tm_st32(s_tm + 64 * h, pr);
          l += sum;
          tc_wait_st();
          tc_fence_before();
          mbar_arrive_warp(bar(bars.p_full[t][h]));
        }
      }
      if (!ok) break;
      if (m == INFINITY) l = NAN;  // an infinite score has no softmax
      // every score product of this segment has arrived: its queries may go
      more = get_work(bars, ring, seg + 1, limit, &abort_flag);
      if (more) queries(seg + 1);
      if (first >= w.r.rows) continue;
      const bool any = lo < hi;
      if (any) {
        if (!mbar_wait_warp(bar(bars.pv_done[t][1]), (n - 1) & 1, limit, &abort_flag)) break;
        tc_fence_after();
      }
      // The second twin hands maxima and sums over; its O is read where it lies, by the warp whose
      // tensor-memory lanes, and so whose rows, are the same.
      float f0 = 1.f, f1 = 0.f;
      bool other = false;
      if (TWIN) {
        if (t) {
          if (seg && !mbar_wait_warp(bar(bars.twin_empty), (seg - 1) & 1, limit, &abort_flag)) break;
          twin_ml[r] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive_warp(bar(bars.twin_full));
          continue;
        }
        other = w.r.lo[1] < w.r.hi[1];
        if (!mbar_wait_warp(bar(bars.twin_full), seg & 1, limit, &abort_flag)) break;
        tc_fence_after();
        const float2 ml = twin_ml[r];
        mbar_arrive_warp(bar(bars.twin_empty));
        const float both = fmaxf(m, ml.x), ref = both == -INFINITY ? 0.f : both;
        f0 = kv_ex2(m - ref), f1 = kv_ex2(ml.x - ref);
        l = l * f0 + ml.y * f1, m = both;
      }
      const int row = w.r.row0 + first + r;  // row of the sequence's key head
      const bool live = first + r < w.r.rows;
      const int at = token_in(p, row), token = w.r.q0 + at, head = w.kh * p.group + row - at * p.group;
      const bool real = live && token >= 0 && token < p.b.tokens;
      const float v_scale = MX || !p.c.v_scale ? 1.f : __ldg(p.c.v_scale + w.kh);
      uint16_t *dst = p.y + ((size_t)token * p.q_heads + head) * D;
      const bool wide = ((uintptr_t)p.y & 31u) == 0;  // whole 32-byte sectors at once
      auto put = [&](int x, const float *o, float f) {  // 32 elements of the row
        uint32_t out[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * j] * f, o[2 * j + 1] * f);
          out[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (!real) return;
        if (wide) {
          st256(dst + 32 * x, out), st256(dst + 32 * x + 16, out + 8);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            reinterpret_cast<uint4 *>(dst + 32 * x)[j] = make_uint4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
        }
      };
      auto put_lse = [&](float mm, float ll) {
        if (real && p.lse)
          p.lse[(size_t)token * p.q_heads + head] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * 0.69314718055994531f;
      };
      const float inv = l == 0.f ? 0.f : v_scale / l;
      // parts: [block][first or not][row tile]: O as [4 elements][row], then m and l by row
      const int tiles = TWIN ? 1 : 2;
      float *const parts = reinterpret_cast<float *>(p.workspace + kAttnCounterBytes);
      auto part_at = [&](int j) {
        return parts + (((size_t)(w.parts.owner + j) * 2 + (j == 0 ? 1 : 0)) * tiles + t) * kRows * (D + 2);
      };
      float *mine = part_at(w.parts.index);
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t ov[32];
        if (any) {
          tm_ld32(o_tm + 32 * x, ov);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
        float *o = reinterpret_cast<float *>(ov);
        if (TWIN) {
          uint32_t tv[32];
          if (other) {
            tm_ld32(o_tm + 128 + 32 * x, tv);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) tv[j] = 0u;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = fmaf(o[j], f0, __uint_as_float(tv[j]) * f1);
        }
        if (w.parts.count == 1) put(x, o, inv);
        else if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            __stcg(reinterpret_cast<float4 *>(mine) + (8 * x + j) * kRows + r,
                   make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
        }
      }
      if (any) {
        tc_fence_before();
        mbar_arrive_warp(bar(bars.o_empty[t]));
      }
      if (other) {
        tc_fence_before();
        mbar_arrive_warp(bar(bars.o_empty[1]));
      }
      if (w.parts.count == 1) {
        put_lse(m, l);
        continue;
      }
      if (live) __stcg(reinterpret_cast<float2 *>(mine + D * kRows) + r, make_float2(m, l));
      // Each warp joins its own 32 rows with the same warp of the item's other parts (a barrier among the
      // four would wait without limit for a warp that gave up), the last one to arrive all of them.
      // More than eight parts (few long contexts) join in two levels, each group into its first part's
      // place: one warp alone would take longer than all blocks' keys.
      auto arrive_last = [&](int counter, int members) {
        __threadfence();
        __syncwarp();
        uint32_t is_last = 0;
        if (lane == 0) {
          uint32_t *c = reinterpret_cast<uint32_t *>(p.workspace) + 8 * counter + warp;
          is_last = atomicAdd(c, 1u) + 1 == (uint32_t)members;
          if (is_last) *c = 0;  // ready for the next call
        }
        is_last = __shfl_sync(0xFFFFFFFFu, is_last, 0);
        if (is_last) __threadfence();
        return is_last != 0;
      };
      const int count = w.parts.count, owner = w.parts.owner;
      int size = 4;  // parts of a group: about as many as groups
      while (size * size < count) ++size;
      bool whole = count <= 8;
      int j0 = whole ? 0 : w.parts.index / size * size, step = 1, n_join = whole ? count : min(size, count - j0);
      bool joins = whole ? arrive_last(owner, count) : arrive_last(kGroupCounter + 2 * (owner + j0) + (j0 == 0 ? 1 : 0), n_join);
      while (joins) {
        auto joined = [&](int j) { return part_at(j0 + j * step); };
        auto ml_at = [&](int j) { return __ldcg(reinterpret_cast<const float2 *>(joined(j) + D * kRows) + r); };
        if (live) {
          // Latency is most of the joining: the first four parts' m and l are loaded at once, O by four parts
          // between twins, by two else (four take registers that the prompt's loop misses: 1 % there).
          constexpr int kAtOnce = TWIN ? 4 : 2;
          float2 ml[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) ml[j] = j < n_join ? ml_at(j) : make_float2(-INFINITY, 0.f);
          float mm = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), ll = 0.f;
#pragma unroll 4
          for (int j = 4; j < n_join; ++j) mm = fmaxf(mm, ml_at(j).x);
          const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int j = 0; j < 4; ++j) ml[j].x = kv_ex2(ml[j].x - ref), ll += ml[j].y * ml[j].x;
#pragma unroll 4
          for (int j = 4; j < n_join; ++j) {
            const float2 v = ml_at(j);
            ll += v.y * kv_ex2(v.x - ref);
          }
          const float inv_all = ll == 0.f ? 0.f : v_scale / ll;
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            float o[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0.f;
#pragma unroll 1
            for (int j = 0; j < n_join; j += kAtOnce) {
              float4 v[kAtOnce][8];
              float f[kAtOnce];
#pragma unroll
              for (int y = 0; y < kAtOnce; ++y) {
                const bool some = j + y < n_join;
                const float4 *src = reinterpret_cast<const float4 *>(joined(j + (some ? y : 0))) + 8 * x * kRows + r;
                f[y] = !some ? 0.f : j == 0 ? ml[y].x : j == 2 ? ml[(2 + y) & 3].x : kv_ex2(ml_at(j + y).x - ref);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[y][e] = some ? __ldcg(src + e * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int y = 0; y < kAtOnce; ++y)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  o[4 * e] = fmaf(v[y][e].x, f[y], o[4 * e]), o[4 * e + 1] = fmaf(v[y][e].y, f[y], o[4 * e + 1]);
                  o[4 * e + 2] = fmaf(v[y][e].z, f[y], o[4 * e + 2]), o[4 * e + 3] = fmaf(v[y][e].w, f[y], o[4 * e + 3]);
                }
            }
            if (whole) {
              put(x, o, inv_all);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                __stcg(reinterpret_cast<float4 *>(joined(0)) + (8 * x + e) * kRows + r,
                       make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            }
          }
          if (whole) put_lse(mm, ll);
          else __stcg(reinterpret_cast<float2 *>(joined(0) + D * kRows) + r, make_float2(mm, ll));
        }
        if (whole) break;
        __syncwarp();
        joins = arrive_last(owner, (count + size - 1) / size);
        whole = true, j0 = 0, step = size, n_join = (count + size - 1) / size;
      }
    }
    tc_fence_before();
  } else if (warp < 12) {
    // ------------------------------------------------------------------ codes to float16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int dw = warp - 8, group_mask = (1 << (p.c.page_shift - 4)) - 1;
    int n = 0;  // key steps of all segments
    bool ok = true;
    // the lanes go on or give up together: those left behind would wait for the others without limit
    auto wait = [&](const uint64_t &b, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar(b), parity, limit, &abort_flag));
    };
    for (int seg = 0; ok && get_work(bars, ring, seg, limit, &abort_flag); ++seg) {
      const int begin = ring[seg & 1].r.begin, end = ring[seg & 1].r.end, kv_len = ring[seg & 1].r.kv_len, first_key = ring[seg & 1].r.first_key,
                kh = ring[seg & 1].kh;
      const int *table = p.b.page_table + (size_t)ring[seg & 1].seq * p.b.max_pages;
      done_work(bars, seg);
      auto page_of = [&](int i, int g) -> int {  // page id of the warp's group g of step i; -1: no keys there
        const int gi = i * 8 + 2 * dw + g, col = gi >> (p.c.page_shift - 4);
        if (i >= end || 16 * gi >= kv_len || col >= p.b.max_pages) return -1;
        const int page = __ldg(table + col);
        return page < p.c.num_pages ? page : -1;
      };
      auto place = [&](int i, int g, int page) -> const uint8_t * {
        if (page < 0) return nullptr;
        const int gi = i * 8 + 2 * dw + g;
        return p.c.pages + ((((size_t)page * p.c.kv_heads + kh) << (p.c.page_shift - 4)) + (gi & group_mask)) * G.bytes;
      };
      // K runs one step ahead of V, as the products do
      Codes<D, MX> ck, cv;
      int next0 = page_of(begin, 0), next1 = page_of(begin, 1);
      const uint8_t *k_grp[2] = {place(begin, 0, next0), place(begin, 1, next1)};
      load_k<D, MX>(k_grp, lane, ck);
      load_v<D, MX>(k_grp, lane, cv);
      next0 = page_of(begin + 1, 0), next1 = page_of(begin + 1, 1);
      for (int i = begin - 1; i < end; ++i) {
        if (i + 1 < end) {
          const int nk = n + 1 + i - begin, st = nk & 1;
          const uint32_t bits = (k_grp[0] ? 1u : 0u) | (k_grp[1] ? 2u : 0u);
          if (nk >= 2 && !(ok = wait(bars.k_empty[st], ((nk >> 1) - 1) & 1))) break;
          store_k<D, MX>(base + M::kK + st * M::kTile, 32 * dw, lane, ck);
          if (lane == 0) reinterpret_cast<volatile uint8_t *>(&valid[nk % kValidRing])[dw] = (uint8_t)bits;
          fence_proxy_async();
          mbar_arrive_warp(bar(bars.k_full[st]));
        }
        const uint8_t *v_grp[2] = {k_grp[0], k_grp[1]};
        k_grp[0] = place(i + 2, 0, next0), k_grp[1] = place(i + 2, 1, next1);
        next0 = page_of(i + 3, 0), next1 = page_of(i + 3, 1);
        load_k<D, MX>(k_grp, lane, ck);
        if (i < begin) continue;
        const int nv = n + i - begin, st = nv & 1;
        if (nv >= 2 && !(ok = wait(bars.v_empty[st], ((nv >> 1) - 1) & 1))) break;
        store_v<D, MX>(base + M::kV + st * M::kTile, 32 * dw, lane, first_key - (i * kKeys + 32 * dw), kv_len - (i * kKeys + 32 * dw), cv);
        fence_proxy_async();
        mbar_arrive_warp(bar(bars.v_full[st]));
        load_v<D, MX>(v_grp, lane, cv);
      }
      n += end - begin;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");  // all four warps of the group at one instruction
    if (warp < 14) {
      // ------------------------------------------------------------------ MMA issue
      // One warp per row tile: a single one, waiting for one tile's operands and then the other's, left
      // the tensor pipe idle a third of the time. The whole warp takes every step, so that the elected
      // thread's operands stay uniform.
      constexpr uint32_t id_s = idesc_f16(kKeys / 2, false), id_o = idesc_f16(D, true);
      const int t = warp - 12;
      const bool lead = elect_one();
      bool ok = true;
      auto wait = [&](const uint64_t &b, uint32_t parity) {
        ok = ok && mbar_wait_warp(bar(b), parity, limit, &abort_flag);
        tc_fence_after();
      };
      const uint32_t qd = desc_low(16, base + M::kQ + t * M::kTile), o_tm = tmem + 256 + t * 128, s_tm = tmem + t * 128;
      const int skip = TWIN ? 1 : 0;  // every second step is the other tile's
      uint32_t q_n = 0, p_n = 0, items = 0;  // parities of the queries and of the products; there was an item
      int n0 = 0;                            // key steps of all segments
      for (int seg = 0; ok && get_work(bars, ring, seg, limit, &abort_flag); ++seg) {
        const Range &r = ring[seg & 1].r;
        auto uniform = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
        const int begin = uniform(r.begin), end = uniform(r.end), lo = uniform(t ? r.lo[1] : r.lo[0]), hi = uniform(t ? r.hi[1] : r.hi[0]);
        done_work(bars, seg);
        for (int i = begin - 1; ok && i < end; ++i) {
          const int n = n0 + i - begin;
          const bool more = i + 1 < end, products = i >= lo && i < hi && !((i ^ t) & skip),
                     scores = i + 1 >= lo && i + 1 < hi && !((i + 1 ^ t) & skip);
          // a tile without keys here waits too: both warps hand every operand tile back, once a step
          if (more) wait(bars.k_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
          if (i >= begin) wait(bars.v_full[n & 1], (n >> 1) & 1);
          const uint32_t vd = desc_low(16384, base + M::kV + (n & 1) * M::kTile);
          const uint32_t kd = desc_low(16, base + M::kK + ((n + 1) & 1) * M::kTile);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (products) {
              // O is written anew with the first product: the segment before must have read it
              if (h == 0 && i == lo && items) wait(bars.o_empty[t], q_n);
              wait(bars.p_full[t][h], p_n);
              if (ok && lead) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_ts(o_tm, s_tm + 64 * h + 8 * k, vd + h * 512 + k * 128, id_o, k > 0 || h > 0 || i > lo);
                tc_commit(bar(bars.pv_done[t][h]));
              }
              __syncwarp();
            }
            if (scores) {
              if (h == 0 && i + 1 == lo) {
                wait(bars.q_full[t], q_n);
                q_n ^= 1;
              }
              if (ok && lead) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint32_t off = ((k >> 2) * M::kSlab + (k & 3) * 32) >> 4;
                  mma_ss(s_tm + 64 * h, qd + off, kd + h * 512 + off, id_s, k > 0);
                }
                tc_commit(bar(bars.s_full[t][h]));
              }
              __syncwarp();
            }
          }
          if (products) p_n ^= 1, items |= i == hi - 1;
          if (lead) {
            if (i >= begin) tc_commit(bar(bars.v_empty[n & 1]));
            if (more) tc_commit(bar(bars.k_empty[(n + 1) & 1]));
          }
          __syncwarp();
        }
        n0 += end - begin;
      }
      // everything issued has finished before tensor memory and shared memory go
      if (lead) {
        tc_commit(bar(bars.drain[t]));
        volatile uint32_t never = 0;
        mbar_wait(bar(bars.drain[t]), 0, kKvDrainLimitNs, &never);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ work list
      if (warp == 14) {
        Walk walk{share.cut[0], share.cut[1], share.first, 0, 0};
        entries.find(p, share.entry, walk.seq, walk.rt);
        for (int seg = 0;; ++seg) {
          if (seg >= 2 && !mbar_wait_warp(bar(bars.work_empty[seg & 1]), ((seg >> 1) - 1) & 1, limit, &abort_flag)) break;
          next_segment<TWIN>(p, share, walk, ring[seg & 1]);
          __syncwarp();
          const bool end = ring[seg & 1].r.rows <= 0;
          mbar_arrive_warp(bar(bars.work_full[seg & 1]));
          if (end) break;
        }
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

int row_tiles(const AttnParams &p) {
  return (int)(((long long)p.b.max_q * p.group + 2 * kRows - 1) / (2 * kRows));
}

template <int D, bool MX, bool TWIN>
cudaError_t launch_t(const AttnParams &p, cudaStream_t st) {
  auto kernel = attn_tiles_kernel<D, MX, TWIN>;
  static SmemOnce once;
  if (cudaError_t e = once.set(kernel, TileSmem<D>::kTotal)) return e;
  kernel<<<sm_count(), kThreads, TileSmem<D>::kTotal, st>>>(p, row_tiles(p));
  return cudaGetLastError();
}

bool is_twin(const AttnParams &p) { return (long long)p.b.max_q * p.group <= kRows; }

template <int D, bool MX>
cudaError_t launch_d(const AttnParams &p, cudaStream_t st) {
  return is_twin(p) ? launch_t<D, MX, true>(p, st) : launch_t<D, MX, false>(p, st);
}

}  // namespace

size_t attention_tiles_workspace(const AttnParams &p, int d) {
  const int tiles = is_twin(p) ? 1 : 2;  // row tiles that a part can have
  return kAttnCounterBytes + (size_t)sm_count() * 2 * tiles * kRows * (d + 2) * sizeof(float);
}

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
