// Attention over the paged FP4 cache for few query rows per key head (decode, drafted tokens).
//
// For one key head the query rows are the group's heads of the call's new tokens: row
// i * group + g. Scores and outputs are formed transposed, S^T = K Q^T and O^T = V^T P^T, so the
// 16-row side of the matrix instruction holds keys and value elements and the 8-column side the
// few query rows. Codes become float16 in registers: code * block scale is exact there (2 + 4
// significant bits; the cache's E8M0 exponents are limited to float16's range), the second-level
// scales and the softmax scale are applied in float32. Queries are scaled by a power of two per row and
// are exact in float16 down to 2^-29 of the row's largest. Probabilities are rounded to float16 (11 bits, against the
// 8 of the bfloat16 output); their sum, the maxima and both accumulators are float32.
//
// Bound by the cache's bytes (144 or 136 per key and key head at 128 elements). Every block takes an
// equal, contiguous share of all key steps of the launch, found from the device's own lengths, so
// that ragged batches balance and a few long sequences fill the GPU; its eight warps walk a
// segment's 32-key tiles in turn, each with copies of its own in flight, and join at its end. The
// parts of an item that is cut between blocks go through the workspace; the block that arrives last
// joins them in the order of the keys. Bulk copies (one per group of 16 tokens, issued by the lane that
// looked up its page) keep the copying out of the instruction stream: about 640 instructions per 32 keys and
// warp, half of them turning codes into float16. No unit is full (issue 0.6 per cycle, the busiest pipe half the
// time): with 3.8 warps per scheduler their latencies are not hidden.
//
// Measured (32 query and 8 key heads of 128): 64 contexts of 33 to 8191 tokens 74 us, 4.2 TB/s; two of
// 120 to 131 thousand 66 us, 4.1 TB/s; one of 777 tokens 9 us, which is latency. Tried without gain: more
// warps (ten or twelve of them spill: 90 and 116 us for the 64 contexts), a third tile in the ring,
// the score products split into two chains.
#include "sharq_common.cuh"
#include "sharq_internal.h"
#include "sharq_kv.h"
#include "sharq_kv_device.cuh"

namespace sharq {

__device__ uint32_t g_attn_rows_status = 0;  // bit 0: a bounded wait gave up

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 32;   // keys per step of a warp: two groups of the cache
constexpr int kStagesA = 2;  // tiles of a warp's ring: the next one loads while one is used (a third gained nothing)
// What an item costs besides its tiles (queries, joining eight warps), in tiles. With 8, 12, 16, 20, 32:
// 64 uneven contexts 78.4, 73.5, 72.6, 73.0, 74.8 us, two of 128K tokens 66.1, 65.4, 64.8, 64.8, 65.0,
// 128 of 200 to 1500 tokens 51.8, 46.5, 46.8, 48.0, 48.5.
constexpr int kItemCost = 16;
constexpr int kJoin = 16;  // parts that one block joins
// counters: an item's by its first block, then a group's by the block and the slot of its first part
constexpr int kGroupCounter = 512;
static_assert(4 * (kGroupCounter + 2 * kGroupCounter) <= kAttnCounterBytes, "counters of 512 blocks");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// The warp waits for a stage's copies. A wait longer than `limit_ns` sets the status word and goes
// on, bounded again, so that no copy is in flight when the block ends.
__device__ __forceinline__ void wait_copies(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (bool there = kv_mbar_test(bar, parity); !there;) {
    const uint64_t waited = kv_waited_ns(&t0);
    if (waited > limit_ns) atomicOr(&g_attn_rows_status, 1u);
    if (waited > limit_ns + kKvDrainLimitNs) break;
    there = kv_mbar_try(bar, parity);
    if (there && kv_waited_ns(&t0) > limit_ns) atomicOr(&g_attn_rows_status, 1u);
  }
  __syncwarp();
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t *v) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t *v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// byte i (0..3, constant) of a word of codes -> half2 of its two values
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(d) : "r"(w), "n"(I));
  return d;
}

template <int D, bool MX, int NT>
struct RowsKernel {
  static constexpr KvLayout G = kv_group(D, MX ? 1 : 0);
  static constexpr int R = 8 * NT;  // query rows of a block
  static constexpr int KS = D / 16;  // matrix steps over D, and 16-row tiles of O^T
  static constexpr int kStageBytes = 2 * G.bytes;
  static constexpr int kRing = kWarps * kStagesA * kStageBytes;
  static constexpr int kMerge = kWarps * R * D * 4;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
};

// One sequence's query rows (all of them: the launch has at most R per key head) and key tiles.
struct RowsRange {
  int q0, rows, kv_len, first_pos, first_key, lo, hi;  // first_key: no query sees one before it
  __device__ __forceinline__ int cost() const { return rows <= 0 ? 0 : kItemCost + max(1, hi - lo); }
};
__device__ __forceinline__ RowsRange rows_range(const AttnParams &p, int seq) {
  RowsRange r;
  const int q1 = __ldg(p.b.cu_q + seq + 1);
  r.q0 = __ldg(p.b.cu_q + seq);
  r.kv_len = __ldg(p.b.kv_len + seq);
  const int q_len = min(q1 - r.q0, p.b.max_q);
  r.rows = q_len * p.group;
  r.first_pos = r.kv_len - (q1 - r.q0);  // position of the sequence's first new token
  int k_lo = 0, k_hi = min(r.kv_len, p.b.max_pages << p.c.page_shift);  // no place behind the table
  if (p.causal) {
    k_hi = min(k_hi, r.first_pos + q_len);
    if (p.window > 0 && r.first_pos >= p.window) k_lo = r.first_pos - p.window + 1;
  }
  r.first_key = k_lo;
  r.lo = k_lo / kTile;
  r.hi = (max(k_hi, 0) + kTile - 1) / kTile;
  return r;
}

template <int D, bool MX, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 2 : 1) attn_rows_kernel(const AttnParams p) {
  using C = RowsKernel<D, MX, NT>;
  constexpr KvLayout G = C::G;
  constexpr int KS = C::KS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sh_m[kWarps][C::R], sh_l[kWarps][C::R];
  __shared__ uint64_t bars[kWarps][kStagesA];
  __shared__ uint32_t last_part;
  __shared__ Share share;
  __shared__ long long warp_sums[kWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < kStagesA; ++i) kv_mbar_init(kv_smem_u32(&bars[warp][i]), 2);  // a lane per group
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  find_share<kWarps * 32, kItemCost>(p.b.n_seq, p.c.kv_heads, kWarps, &share, warp_sums,
                                     [&](long long e) { return rows_range(p, (int)e).cost(); });
  const uint32_t ring = kv_smem_u32(smem) + warp * kStagesA * C::kStageBytes, bar0 = kv_smem_u32(&bars[warp][0]);
  int load_stage = 0, use_stage = 0;  // the ring runs on from segment to segment
  uint32_t use_parity = 0;
  int seq = share.entry;
  long long first = share.first;
  for (long long at = share.cut[0]; at < share.cut[1];) {
    // ---- the next segment of the share
    RowsRange w;
    int cost;
    for (;; ++seq) {  // sequences without new tokens have no items
      w = rows_range(p, seq);
      cost = w.cost();
      if (at < first + (long long)cost * p.c.kv_heads) break;
      first += (long long)cost * p.c.kv_heads;
    }
    const int kh = small_quotient(at - first, cost);
    const long long p0 = first + (long long)kh * cost, p1 = p0 + cost, to = min(share.cut[1], p1);
    const ItemParts parts = item_parts<kItemCost>(share, p0, p1, at);
    int t_lo = w.lo, t_hi = w.hi;
    if (t_lo < t_hi) {
      t_hi = w.lo + (int)(to - p0) - kItemCost;
      if (at != p0) t_lo = w.lo + (int)(at - p0) - kItemCost;
    }
    at = to;
    const int q0 = w.q0, rows = w.rows, kv_len = w.kv_len, first_pos = w.first_pos, first_key = w.first_key;
    const int pos_lo = first_pos, pos_hi = first_pos + token_of(p.group, p.group_inv, rows - 1);

    // ---- copies: 32 keys a stage, one bulk copy per group of 16
    const int page_groups = 1 << (p.c.page_shift - 4);
    const int *table = p.b.page_table + (size_t)seq * p.b.max_pages;
    // page id of the group `gi` of the sequence, -1 where it holds no keys
    auto page_of = [&](int gi) -> int {
      const int col = gi >> (p.c.page_shift - 4);
      if (16 * gi >= kv_len || col >= p.b.max_pages) return -1;
      const int page = __ldg(table + col);
      return page < p.c.num_pages ? page : -1;
    };
    // Lane 2i + h has group h of the warp's tile base + i, its place in memory and the page id of the
    // group 16 tiles on, and issues its copy itself.
    auto page_ahead = [&](int i) { return page_of(2 * (t_lo + warp + kWarps * (i + (lane >> 1))) + (lane & 1)); };
    auto place = [&](int i, int id) {
      const int in_page = (2 * (t_lo + warp + kWarps * (i + (lane >> 1))) + (lane & 1)) & (page_groups - 1);
      return p.c.pages + ((((size_t)max(id, 0) * p.c.kv_heads + kh) << (p.c.page_shift - 4)) + in_page) * G.bytes;
    };
    int base = 0, id = page_ahead(0), id_next = page_ahead(16);
    const uint8_t *grp = place(0, id);
    uint32_t there = __ballot_sync(0xFFFFFFFFu, id >= 0);
    const int my_tiles = t_hi - t_lo > warp ? (t_hi - t_lo - warp + kWarps - 1) / kWarps : 0;
    uint32_t valid_bits = 0;  // bits 2s, 2s+1: the groups of ring stage s hold keys
    auto load = [&](int i) {
      if (i >= my_tiles) return;
      if (i - base >= 16) {
        base += 16;
        id = id_next;
        id_next = page_ahead(base + 16);
        grp = place(base, id);
        there = __ballot_sync(0xFFFFFFFFu, id >= 0);
      }
      const int pair = i - base;
      valid_bits = (valid_bits & ~(3u << (2 * load_stage))) | (((there >> (2 * pair)) & 3u) << (2 * load_stage));
      if (lane >> 1 == pair) {
        const uint32_t bar = bar0 + 8 * load_stage;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(id >= 0 ? G.bytes : 0) : "memory");
        if (id >= 0) bulk_load(ring + load_stage * C::kStageBytes + (lane & 1) * G.bytes, grp, G.bytes, bar);
      }
      load_stage = load_stage == kStagesA - 1 ? 0 : load_stage + 1;
    };
    for (int i = 0; i < kStagesA - 1; ++i) load(i);

    // ---- query fragments: lane (g, t) holds elements [D/4 * t, D/4 * (t + 1)) of row g of each n tile
    uint32_t qf[NT][KS][2];
    float coef[NT][2];  // score factor of columns 2t, 2t+1: softmax scale, key scale, the row's power of two
    const float factor = (MX || !p.c.k_scale ? 1.f : __ldg(p.c.k_scale + kh)) * p.scale_log2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 8 + g, tok = token_of(p.group, p.group_inv, r);
      const int token = q0 + tok, head = kh * p.group + r - tok * p.group;
      uint32_t raw[KS * 2];
      if (r < rows && token >= 0 && token < p.b.tokens) {
        const uint16_t *src = p.q + (size_t)token * p.q_stride + head * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
          raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) raw[i] = 0u;
      }
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < KS * 2; ++i) am = max3abs(am, bf16lo(raw[i]), bf16hi(raw[i]));
      am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      // the row's largest value moves to [2^12, 2^13). Float16's last step there is 2^-24, so that eight
      // significant bits are exact from 2^-17 on, 2^-29 of the largest; below that an element is rounded, by
      // at most 2^-25: 2^-37 of the largest. The sign of the score's factor goes into the query, so that
      // maxima stay maxima
      const int e = max((int)(__float_as_uint(am) >> 23) - 127, -100);
      const float up = copysignf(__uint_as_float((uint32_t)(127 + 12 - e) << 23), factor);
#pragma unroll
      for (int i = 0; i < KS * 2; ++i) qf[n][i >> 1][i & 1] = kv_pack_half2(bf16lo(raw[i]) * up, bf16hi(raw[i]) * up);
      float down = __uint_as_float((uint32_t)(127 - 12 + e) << 23) * fabsf(factor);
      if (down < 1e-37f) down = 1e-37f;  // 0 must not meet the masked -inf
      coef[n][0] = __shfl_sync(0xFFFFFFFFu, down, 8 * t);
      coef[n][1] = __shfl_sync(0xFFFFFFFFu, down, 8 * t + 4);
    }

    float o[KS][NT][4], m[NT][2], l[NT][2];  // m: reference of the exponentials, in units of log2
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[i][n][q] = 0.f;
    }

    for (int it = 0; it < my_tiles; ++it) {
      __syncwarp();  // every lane has left the stage that the next load overwrites
      load(it + kStagesA - 1);
      wait_copies(bar0 + 8 * use_stage, use_parity, p.limit_ns);
      const uint32_t st = ring + use_stage * C::kStageBytes;
      const int key0 = (t_lo + warp + kWarps * it) * kTile;
      const uint32_t valid = (valid_bits >> (2 * use_stage)) & 3u;
      use_stage = use_stage == kStagesA - 1 ? 0 : use_stage + 1;
      if (use_stage == 0) use_parity ^= 1u;

      // ---- S^T: two 16-key tiles
      float sc[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) sc[h][n][q] = 0.f;
        uint32_t ca[KS / 2], cb[KS / 2];  // codes of rows g and g + 8: D/8 bytes from element D/4 * t
        const uint32_t kc = st + h * G.bytes;
        if (D == 128) {
          lds128(kc + g * 64 + t * 16, ca);
          lds128(kc + (g + 8) * 64 + t * 16, cb);
        } else {
          lds64(kc + g * 32 + t * 8, ca);
          lds64(kc + (g + 8) * 32 + t * 8, cb);
        }
        // scales of the lane's elements: blocks of the first and second half of its matrix steps
        uint32_t sa[2], sb[2];
        const uint32_t kscale = kc + G.k_scales;
        if (!MX && D == 128) {
          const uint32_t a2 = kv_scales2<MX>(lds16(kscale + g * 8 + 2 * t)), b2 = kv_scales2<MX>(lds16(kscale + (g + 8) * 8 + 2 * t));
          sa[0] = __byte_perm(a2, 0, 0x1010), sa[1] = __byte_perm(a2, 0, 0x3232);
          sb[0] = __byte_perm(b2, 0, 0x1010), sb[1] = __byte_perm(b2, 0, 0x3232);
        } else {
          constexpr int NB = D / (MX ? 32 : 16);
          const int blk = NB == 4 ? t : t >> 1;
          const uint32_t two = kv_scales2<MX>(lds8(kscale + g * NB + blk) | (lds8(kscale + (g + 8) * NB + blk) << 8));
          sa[0] = sa[1] = __byte_perm(two, 0, 0x1010);
          sb[0] = sb[1] = __byte_perm(two, 0, 0x3232);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint32_t wa = ca[k >> 1], wb = cb[k >> 1];
          const uint32_t fa = sa[2 * k / KS], fb = sb[2 * k / KS];
          uint32_t a[4];
          if (k & 1) a[0] = code_pair<2>(wa), a[1] = code_pair<2>(wb), a[2] = code_pair<3>(wa), a[3] = code_pair<3>(wb);
          else a[0] = code_pair<0>(wa), a[1] = code_pair<0>(wb), a[2] = code_pair<1>(wa), a[3] = code_pair<1>(wb);
          a[0] = mul2(a[0], fa), a[1] = mul2(a[1], fb), a[2] = mul2(a[2], fa), a[3] = mul2(a[3], fb);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(sc[h][n], a, qf[n][k][0], qf[n][k][1]);
        }
      }
      // ---- masks
      const bool whole = valid == 3u && key0 + kTile <= kv_len &&
                         (!p.causal || (key0 + kTile - 1 <= pos_lo && (p.window <= 0 || pos_hi - key0 < p.window)));
      uint32_t keep[2] = {~0u, ~0u};  // the lane's value scales of keys that some query sees
      if (!whole) {
        // the others may be anything: zero keeps 0 * v from NaN
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int key = key0 + 16 * h + 8 * (q >> 1) + 2 * t + (q & 1);
            if (key < first_key || key >= kv_len) keep[h] &= ~(0xFFu << (8 * q));
          }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int pos = first_pos + token_of(p.group, p.group_inv, n * 8 + 2 * t + c);
            const int hi = p.causal ? min(pos, kv_len - 1) : kv_len - 1;
            const int lo = p.causal && p.window > 0 && pos >= p.window ? pos - p.window : -1;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int key = key0 + 16 * h + g + 8 * q;
                if (!((valid >> h) & 1u) || key > hi || key <= lo) sc[h][n][2 * q + c] = -INFINITY;
              }
          }
      }
      // ---- exponentials against the reference at hand. It moves (and O and l are rescaled) only where
      // a column's maximum is more than 2^8 above it: exponentials then stay far inside float16's range
      float top[NT][2];
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[n][c] = fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), fmaxf(sc[1][n][c], sc[1][n][2 + c])) * coef[n][c];
          grew = grew || top[n][c] > m[n][c] + 8.f;
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = top[n][c];
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            const float next = fmaxf(m[n][c], mx), f = next == -INFINITY ? 1.f : kv_ex2(m[n][c] - next);
            m[n][c] = next;
            l[n][c] *= f;
#pragma unroll
            for (int i = 0; i < KS; ++i) o[i][n][c] *= f, o[i][n][2 + c] *= f;
          }
      }
      float most = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) most = max3abs(most, m[n][0], m[n][1]);
      if (!__any_sync(0xFFFFFFFFu, most > 0x1p24f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float shift = m[n][c] == -INFINITY ? 0.f : -m[n][c];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const float e = kv_ex2(fmaf(sc[h][n][2 * q + c], coef[n][c], shift));
                sc[h][n][2 * q + c] = e;
                l[n][c] += e;
              }
          }
      } else {  // a column is far (see kv_is_far), or has seen nothing yet
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float shift = m[n][c] == -INFINITY ? 0.f : -m[n][c];
              float &v = sc[x >> 1][n][2 * (x & 1) + c];
              v = kv_ex2(kv_is_far(m[n][c]) ? __fadd_rn(__fmul_rn(v, coef[n][c]), shift) : fmaf(v, coef[n][c], shift));
              l[n][c] += v;
            }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!((valid >> h) & 1u)) continue;  // warp-uniform; its probabilities are zero
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          pf[n][0] = trans8x8(kv_pack_half2(sc[h][n][0], sc[h][n][1]));
          pf[n][1] = trans8x8(kv_pack_half2(sc[h][n][2], sc[h][n][3]));
        }
        const uint32_t vc = st + h * G.bytes + G.v_codes;
        uint32_t v[2][4];  // [slot half][words]: D = 128: key 2t {lo, hi}, key 2t+1 {lo, hi}
        lds128(vc + lane * 16, v[0]);
        if (D == 128) lds128(vc + 512 + lane * 16, v[1]);
        constexpr int per_run = (MX ? 32 : 16) / (D / 8);  // runs that share a block: 1, 2 or 4
        const uint32_t vs = lds32(st + h * G.bytes + G.v_scales + (g / per_run * 4 + t) * 4) & keep[h];
        const uint32_t s0 = kv_scales2<MX>(vs & 0xFFFFu), s1 = kv_scales2<MX>(vs >> 16);
        uint32_t even[2][2], odd[2][2];  // [word][slot half]: nibbles of two keys of one element per byte
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t a = D == 128 ? v[hh][x] : v[0][2 * hh], b = D == 128 ? v[hh][2 + x] : v[0][2 * hh + 1];
            even[x][hh] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
            odd[x][hh] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
          }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint32_t a[4];
          const uint32_t e0 = even[i >> 2][0], e1 = even[i >> 2][1], o0 = odd[i >> 2][0], o1 = odd[i >> 2][1];
          switch (i & 3) {
            case 0: a[0] = code_pair<0>(e0), a[1] = code_pair<0>(o0), a[2] = code_pair<0>(e1), a[3] = code_pair<0>(o1); break;
            case 1: a[0] = code_pair<1>(e0), a[1] = code_pair<1>(o0), a[2] = code_pair<1>(e1), a[3] = code_pair<1>(o1); break;
            case 2: a[0] = code_pair<2>(e0), a[1] = code_pair<2>(o0), a[2] = code_pair<2>(e1), a[3] = code_pair<2>(o1); break;
            default: a[0] = code_pair<3>(e0), a[1] = code_pair<3>(o0), a[2] = code_pair<3>(e1), a[3] = code_pair<3>(o1);
          }
          a[0] = mul2(a[0], s0), a[1] = mul2(a[1], s0), a[2] = mul2(a[2], s1), a[3] = mul2(a[3], s1);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[i][n], a, pf[n][0], pf[n][1]);
        }
      }
    }

    // ---- join the warps: common maximum, every warp's O to shared memory, summed by all threads in
    // the warps' order. Sixteen-byte units of a row are swapped by the row, so that a store's eight
    // lanes (two runs of four rows) cover every bank.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (m[n][c] == INFINITY) l[n][c] = NAN;  // an infinite score has no softmax
        l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 4);
        l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 8);
        l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 16);
        if (g == 0) sh_m[warp][n * 8 + 2 * t + c] = m[n][c], sh_l[warp][n * 8 + 2 * t + c] = l[n][c];
      }
    __syncthreads();
    auto swap4 = [](int row) { return D == 128 ? (row >> 1) & 3 : ((row >> 1) & 1) | (((row >> 1) & 2) << 1); };
    float4 *slots = reinterpret_cast<float4 *>(smem);
    constexpr int F4 = D / 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = n * 8 + 2 * t + c;
        float mm = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, sh_m[x][row]);
        const float f = kv_ex2(m[n][c] - (mm == -INFINITY ? 0.f : mm));
#pragma unroll
        for (int j = 0; j < KS / 2; ++j)
          slots[(warp * C::R + row) * F4 + ((g * (KS / 2) + j) ^ swap4(row))] =
              make_float4(o[2 * j][n][c] * f, o[2 * j][n][2 + c] * f, o[2 * j + 1][n][c] * f, o[2 * j + 1][n][2 + c] * f);
      }
    __syncthreads();
    const float v_scale = MX || !p.c.v_scale ? 1.f : __ldg(p.c.v_scale + kh);
    // parts: [block][first or not]: O by row, then m and l
    float *const all = reinterpret_cast<float *>(p.workspace + kAttnCounterBytes);
    auto part_at = [&](int j) { return all + ((size_t)(parts.owner + j) * 2 + (j == 0 ? 1 : 0)) * C::R * (D + 2); };
    auto put = [&](int row, int i4, float4 v, float mm, float ll) {
      const int tok = token_of(p.group, p.group_inv, row), token = q0 + tok, head = kh * p.group + row - tok * p.group;
      if (token < 0 || token >= p.b.tokens) return;
      const float inv = ll == 0.f ? 0.f : v_scale / ll;  // a NaN query stays NaN
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * inv, v.y * inv), b = __floats2bfloat162_rn(v.z * inv, v.w * inv);
      uint2 h;
      h.x = *reinterpret_cast<const uint32_t *>(&a), h.y = *reinterpret_cast<const uint32_t *>(&b);
      const size_t at_row = (size_t)token * p.q_heads + head;
      *reinterpret_cast<uint2 *>(p.y + at_row * D + 4 * i4) = h;
      if (i4 == 0 && p.lse) p.lse[at_row] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * 0.69314718055994531f;
    };
    for (int idx = threadIdx.x; idx < rows * F4; idx += kWarps * 32) {
      const int row = idx / F4, i4 = idx % F4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, sh_m[x][row]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        ll += sh_l[x][row] * kv_ex2(sh_m[x][row] - (mm == -INFINITY ? 0.f : mm));
        const float4 u = slots[(x * C::R + row) * F4 + (i4 ^ swap4(row))];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      if (parts.count == 1) {
        put(row, i4, v, mm, ll);
      } else {
        float *mine = part_at(parts.index);
        __stcg(reinterpret_cast<float4 *>(mine) + idx, v);
        if (i4 == 0) __stcg(reinterpret_cast<float2 *>(mine + C::R * D) + row, make_float2(mm, ll));
      }
    }
    if (parts.count > 1) {
      // The last block to arrive joins. More than two groups of kJoin parts (a few long contexts) join
      // in two levels, each group into its first part's place: one block alone would read up to 148
      // or 296 parts, and took longer than all blocks' keys.
      auto arrive_last = [&](int counter, int members) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
          uint32_t *c = reinterpret_cast<uint32_t *>(p.workspace) + counter;
          last_part = atomicAdd(c, 1u) + 1 == (uint32_t)members;
          if (last_part) *c = 0;  // ready for the next call
        }
        __syncthreads();
        const bool last = last_part != 0;
        if (last) __threadfence();
        return last;
      };
      // parts j0, j0 + step, ... below `end`, in the order of the keys
      bool whole = parts.count <= 2 * kJoin;
      int j0 = whole ? 0 : parts.index / kJoin * kJoin, step = 1, end = whole ? parts.count : min(j0 + kJoin, parts.count);
      bool last = whole ? arrive_last(parts.owner, parts.count)
                        : arrive_last(kGroupCounter + 2 * (parts.owner + j0) + (j0 == 0 ? 1 : 0), end - j0);
      while (last) {
        // eight parts' loads are in flight at once, references move from eight to eight
        for (int base = 0; base < rows * F4; base += kWarps * 32) {  // whole rows at a time
          const int idx = base + threadIdx.x, row = idx / F4, i4 = idx % F4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          float mm = -INFINITY, ll = 0.f;
          for (int ja = j0; ja < end && row < rows; ja += 8 * step) {
            float2 ml[8];
            float4 u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const bool some = ja + j * step < end;
              const float *src = part_at(some ? ja + j * step : ja);
              ml[j] = some ? __ldcg(reinterpret_cast<const float2 *>(src + C::R * D) + row) : make_float2(-INFINITY, 0.f);
              u[j] = some ? __ldcg(reinterpret_cast<const float4 *>(src) + idx) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = mm;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, ml[j].x);
            const float ref = top == -INFINITY ? 0.f : top, keep = kv_ex2(mm - ref);
            mm = top;
            ll *= keep, v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float f = kv_ex2(ml[j].x - ref);
              ll += ml[j].y * f;
              v.x = fmaf(u[j].x, f, v.x), v.y = fmaf(u[j].y, f, v.y), v.z = fmaf(u[j].z, f, v.z), v.w = fmaf(u[j].w, f, v.w);
            }
          }
          if (whole) {
            if (row < rows) put(row, i4, v, mm, ll);
            continue;
          }
          __syncthreads();  // every thread of a row has read the m and l that are overwritten
          if (row >= rows) continue;
          __stcg(reinterpret_cast<float4 *>(part_at(j0)) + idx, v);
          if (i4 == 0) __stcg(reinterpret_cast<float2 *>(part_at(j0) + C::R * D) + row, make_float2(mm, ll));
        }
        if (whole) break;
        last = arrive_last(parts.owner, (parts.count + kJoin - 1) / kJoin);
        whole = true, j0 = 0, step = kJoin, end = parts.count;
      }
    }
    // the next segment's copies overwrite what was just read
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
}

// tiles of 8 query rows: 1, 2 or 4; one of them leaves registers for two blocks per SM
int row_tiles(const AttnParams &p) {
  const long long rows = (long long)p.b.max_q * p.group;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}
int blocks_of(int nt) { return sm_count() * (nt == 1 ? 2 : 1); }

template <int D, bool MX, int NT>
cudaError_t launch_rows(const AttnParams &p, cudaStream_t st) {
  using C = RowsKernel<D, MX, NT>;
  auto kernel = attn_rows_kernel<D, MX, NT>;
  static SmemOnce once;
  if (cudaError_t e = once.set(kernel, C::kSmem)) return e;
  kernel<<<blocks_of(NT), kWarps * 32, C::kSmem, st>>>(p);
  return cudaGetLastError();
}

template <int D, bool MX>
cudaError_t launch_d(const AttnParams &p, cudaStream_t st) {
  const int nt = row_tiles(p);
  return nt == 1 ? launch_rows<D, MX, 1>(p, st) : nt == 2 ? launch_rows<D, MX, 2>(p, st) : launch_rows<D, MX, 4>(p, st);
}

}  // namespace

namespace {
// Up to 16 rows the kernel above holds everything in registers; its form for 17 to 32 spills at 128 elements
// (372 bytes of stores) and pads to 32. For 16 contexts of 1500 to 6000 tokens it takes 22, 35, 37 us at 14,
// 21, 28 rows (4 key heads) where the 128-row tiles take 40, and 34, 57, 60 us at 16, 24, 32 rows (8 key
// heads) where they take 58; for one context of 50000 tokens and one key head 17, 25, 28 us at 12, 24, 32
// rows where they take 45 to 49.
bool use_tiles(const AttnParams &p) { return (long long)p.b.max_q * p.group > 32; }
}  // namespace

size_t attention_workspace(const AttnParams &p, int d) {
  if (use_tiles(p)) return attention_tiles_workspace(p, d);
  const int nt = row_tiles(p);
  return kAttnCounterBytes + (size_t)blocks_of(nt) * 2 * 8 * nt * (d + 2) * sizeof(float);
}

cudaError_t launch_attention(const AttnParams &p, int d, int fmt, cudaStream_t st) {
  if (use_tiles(p)) return launch_attention_tiles(p, d, fmt, st);
  if (d == 128) return fmt ? launch_d<128, true>(p, st) : launch_d<128, false>(p, st);
  return fmt ? launch_d<64, true>(p, st) : launch_d<64, false>(p, st);
}

cudaError_t read_and_clear_attn_rows_status(uint32_t *status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_attn_rows_status, sizeof *status);
  if (e != cudaSuccess || *status == 0) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_attn_rows_status, &zero, sizeof zero);
}

}  // namespace sharq
