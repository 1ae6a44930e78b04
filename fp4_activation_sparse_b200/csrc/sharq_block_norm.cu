// Norms before and after a block, fused with the block's gate and the scaled residual stream:
//   z  = y * rstd(y) * post_gamma          (or y)
//   r' = bf16(alpha * r + gate * z)        (gate 1 without one)
//   h  = bf16(r' * rstd(r') * pre_gamma)   (optional; rstd of r' as stored)
// Bound by its bytes: y and r read once, r' and h written once, 8 bytes per element. One block
// per row keeps the row in registers between the two reductions, so nothing is read twice.
#include "sharq_common.cuh"
#include "sharq_kv.h"

namespace sharq {
namespace {

constexpr int kUnits = 4;  // 16-byte units (8 bf16) per thread: k <= 32768 with 1024 threads

__device__ __forceinline__ uint4 ld128(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// rstd of a row from every thread's 64-bit sum of squares (float64: the order of the partial
// sums does not reach the float32 result)
__device__ __forceinline__ float block_rstd(double ss, int k, float eps, double *red, float *out) {
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += red[i];
    *out = __frcp_rn(__fsqrt_rn(__fadd_rn(__double2float_rn(__ddiv_rn(t, (double)k)), eps)));
  }
  __syncthreads();
  return *out;
}

__global__ void __launch_bounds__(1024) norm_residual_kernel(const NormResidualParams p) {
  __shared__ double red[2][32];
  __shared__ float rstd[2];
  const size_t row = blockIdx.x;
  const int units = p.k / 8;
  const uint16_t *gate = p.gate ? p.gate + (p.rows_per_gate ? row / p.rows_per_gate : 0) * p.k : nullptr;
  uint4 y[kUnits], r[kUnits];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      y[i] = ld128(p.y + row * p.k + (size_t)u * 8);
      r[i] = ld128(p.residual + row * p.k + (size_t)u * 8);
      const uint32_t *w = &y[i].x;
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = add_squares_exact(w[j], ss);
    }
  }
  float rs = 1.f;
  if (p.post_gamma) rs = block_rstd(ss, p.k, p.eps, red[0], &rstd[0]);
  ss = 0.0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      uint4 g, t;
      if (p.post_gamma) g = ld128(p.post_gamma + (size_t)u * 8);
      if (gate) t = ld128(gate + (size_t)u * 8);
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
        ss = add_squares_exact(rw[j], ss);
      }
      *reinterpret_cast<uint4 *>(p.residual_out + row * p.k + (size_t)u * 8) = r[i];
    }
  }
  if (!p.pre_gamma) return;
  rs = block_rstd(ss, p.k, p.eps, red[1], &rstd[1]);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = threadIdx.x + i * blockDim.x;
    if (u < units) {
      const uint4 g = ld128(p.pre_gamma + (size_t)u * 8);
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
      *reinterpret_cast<uint4 *>(p.h_out + row * p.k + (size_t)u * 8) = o;
    }
  }
}

}  // namespace

cudaError_t launch_norm_residual(const NormResidualParams &p, cudaStream_t st) {
  const int units = p.k / 8;
  int threads = (units + kUnits - 1) / kUnits;
  threads = (threads + 31) / 32 * 32;
  if (threads > 1024) return cudaErrorInvalidValue;
  norm_residual_kernel<<<p.tokens, threads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sharq
