// Norms before and after a block, fused with the block's gate and the scaled residual stream:
//   z  = y * rstd(y) * post_gamma          (or y)
//   r' = bf16(alpha * r + gate * z)        (gate 1 without one)
//   h  = bf16(r' * rstd(r') * pre_gamma)   (optional; rstd of r' as stored)
// Bound by its bytes: y and r read once, r' and h written once, 8 bytes per element. One block
// per row keeps the row in registers between the two reductions, so nothing is read twice.
// Measured: 32760 x 5120 with a gate and both norms 216 us (6.2 TB/s). The squares are added in float64 one
// by one, as the stand-alone norm does, so that a row's rstd is the same to the bit: 2 us of the 216 (with eight
// squares in float32 first, off by up to 4e-7, it took 214). A conversion per element is cheaper than
// building the double from the bits (226), and the division by k is a product with the host's 1/k (a step of
// float64 apart; 222 with it in every warp). Loading the next row ahead in a persistent block gained nothing.
// Few rows take a unit per thread (16 x 4096: 3.1 us, against 5.1 with four).
#include "sharq_common.cuh"
#include "sharq_internal.h"
#include "sharq_kv.h"
#include "sharq_kv_device.cuh"

namespace sharq {
namespace {

__device__ __forceinline__ uint4 ld128(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// rstd of a row from every thread's sum; every warp adds the warps' sums itself, so one barrier is
// enough. red: this norm's own.
__device__ __forceinline__ float block_rstd(double ss, double inv_k, float eps, double *red) {
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += red[i];
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__double2float_rn(t * inv_k), eps)));
}

// One row from its y and r in registers, U 16-byte units (8 bf16) per thread.
template <int U>
__device__ __forceinline__ void norm_row(const NormResidualParams &p, size_t row, uint4 (&y)[U], uint4 (&r)[U],
                                         double (&red)[2][32]) {
  const int units = p.k / 8;
  const uint32_t gate_row = p.gate && p.rows_per_gate ? (uint32_t)row / (uint32_t)p.rows_per_gate : 0u;
  const uint16_t *gate = p.gate ? p.gate + (size_t)gate_row * p.k : nullptr;
  double ss = 0.0;
  float rs = 1.f;
  if (p.post_gamma) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (threadIdx.x + i * blockDim.x < units) ss = add_squares(y[i], ss);
    rs = block_rstd(ss, p.inv_k, p.eps, red[0]);
  }
  ss = 0.0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      uint4 g, t;
      if (p.post_gamma) g = __ldg(reinterpret_cast<const uint4 *>(p.post_gamma) + u);
      if (gate) t = __ldg(reinterpret_cast<const uint4 *>(gate) + u);
      uint32_t *rw = &r[i].x;
      const uint32_t *yw = &y[i].x, *gw = &g.x, *tw = &t.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a = bf16lo(yw[j]), b = bf16hi(yw[j]);
        if (p.post_gamma) {
          a = __fmul_rn(__fmul_rn(a, rs), bf16lo(gw[j]));
          b = __fmul_rn(__fmul_rn(b, rs), bf16hi(gw[j]));
        }
        if (gate) {
          a = __fmul_rn(a, bf16lo(tw[j]));
          b = __fmul_rn(b, bf16hi(tw[j]));
        }
        a = __fadd_rn(__fmul_rn(p.alpha, bf16lo(rw[j])), a);
        b = __fadd_rn(__fmul_rn(p.alpha, bf16hi(rw[j])), b);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        rw[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
      if (p.pre_gamma) ss = add_squares(r[i], ss);
      __stcs(reinterpret_cast<uint4 *>(p.residual_out + row * p.k) + u, r[i]);
    }
  }
  if (!p.pre_gamma) return;
  rs = block_rstd(ss, p.inv_k, p.eps, red[1]);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      const uint4 g = __ldg(reinterpret_cast<const uint4 *>(p.pre_gamma) + u);
      const uint32_t *gw = &g.x, *rw = &r[i].x;
      uint4 o;
      uint32_t *ow = &o.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h =
            __floats2bfloat162_rn(__fmul_rn(__fmul_rn(bf16lo(rw[j]), rs), bf16lo(gw[j])),
                                  __fmul_rn(__fmul_rn(bf16hi(rw[j]), rs), bf16hi(gw[j])));
        ow[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
      __stcs(reinterpret_cast<uint4 *>(p.h_out + row * p.k) + u, o);
    }
  }
}

// A block per row, k <= 8192 U.
template <int U>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const NormResidualParams p) {
  __shared__ double red[2][32];
  const size_t row = blockIdx.x;
  const int units = p.k / 8;
  uint4 y[U], r[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      y[i] = ld128(p.y + row * p.k + (size_t)u * 8);
      r[i] = ld128(p.residual + row * p.k + (size_t)u * 8);
    }
  }
  norm_row<U>(p, row, y, r, red);
}

}  // namespace

cudaError_t launch_norm_residual(const NormResidualParams &p, cudaStream_t st) {
  const int units = p.k / 8, four = ((units + 3) / 4 + 31) / 32 * 32;
  if (four > 1024) return cudaErrorInvalidValue;
  if (p.tokens <= 2 * sm_count() && units <= 1024)
    norm_residual_kernel<1><<<p.tokens, (units + 31) / 32 * 32, 0, st>>>(p);
  else
    norm_residual_kernel<4><<<p.tokens, four, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sharq
