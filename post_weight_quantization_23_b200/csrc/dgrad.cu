// The gradient of the inference product with respect to its input
// (gptq_gemm_dgrad), read straight from the packed codes:
//   dX[t, c] = sum_j dY[t, j] scale[j, g(c)] (code[j, c] - zero[j, g(c)]).
// The reduction runs over the rows of W, the output over its columns: the other
// way round than gptq_gemm over the same packed words.
#include "common.cuh"

namespace gptq {

namespace {

template <typename T> __device__ __forceinline__ T dg_out(float v);
template <> __device__ __forceinline__ __half dg_out<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 dg_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// General kernel: any bit width, g_idx, group size and alignment.  64 tokens x 64
// columns per CTA, 32 rows of W at a time: the weights are formed in fp32 in
// shared memory, each thread sums a 4 x 4 block in fp32.  A g_idx entry outside
// [0, ngroups) is not read through: its column's weights become NaN.
constexpr int DG_T = 64, DG_C = 64, DG_K = 32;

template <typename T>
__global__ void __launch_bounds__(256)
dgrad_general_kernel(const T* __restrict__ dY, int64_t lddy, int m, int n,
                     const int32_t* __restrict__ qw, int bits, const float* __restrict__ scales,
                     const int32_t* __restrict__ zeros, const int32_t* __restrict__ g_idx, int G,
                     int ngroups, int k, T* __restrict__ dX, int64_t lddx) {
  __shared__ float sy[DG_K][DG_T + 4];
  __shared__ float sw[DG_K][DG_C + 4];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int c0 = blockIdx.x * DG_C, t0 = blockIdx.y * DG_T;
  const int64_t wpr = (int64_t)k * bits / 32;
  const uint32_t mask = (1u << bits) - 1u;
  float acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int j0 = 0; j0 < n; j0 += DG_K) {
    __syncthreads();
    for (int e = tid; e < DG_K * DG_T; e += 256) {
      const int j = j0 + e % DG_K, t = t0 + e / DG_K;
      sy[e % DG_K][e / DG_K] = (j < n && t < m) ? to_f32(dY[(int64_t)t * lddy + j]) : 0.f;
    }
    for (int e = tid; e < DG_K * DG_C; e += 256) {
      const int c = c0 + e % DG_C, j = j0 + e / DG_C;
      float w = 0.f;
      if (j < n && c < k) {
        const int g = g_idx != nullptr ? g_idx[c] : c / G;
        if (g < 0 || g >= ngroups) {
          w = __int_as_float(0x7fc00000);
        } else {
          const int64_t bit = (int64_t)c * bits;
          const uint32_t* wr = reinterpret_cast<const uint32_t*>(qw) + (int64_t)j * wpr;
          const int sh = (int)(bit & 31);
          uint32_t v = wr[bit >> 5] >> sh;
          if (sh + bits > 32) v |= wr[(bit >> 5) + 1] << (32 - sh);
          w = scales[(int64_t)j * ngroups + g] *
              (float)((int)(v & mask) - zeros[(int64_t)j * ngroups + g]);
        }
      }
      sw[e / DG_C][e % DG_C] = w;
    }
    __syncthreads();
#pragma unroll 8
    for (int j = 0; j < DG_K; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(&sy[j][4 * ty]);
      const float4 w = *reinterpret_cast<const float4*>(&sw[j][4 * tx]);
      const float yv[4] = {y.x, y.y, y.z, y.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(yv[i], wv[q], acc[i][q]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = t0 + 4 * ty + i, c = c0 + 4 * tx + q;
      if (t < m && c < k) dX[(int64_t)t * lddx + c] = dg_out<T>(acc[i][q]);
    }
}

}  // namespace

gptq_status dgrad_impl(const void* dY, gptq_dtype dt, int64_t m, int64_t n, int64_t lddy,
                       const int32_t* qw, const float* scales, const int32_t* zeros,
                       const int32_t* g_idx, int64_t k, int bits, int group_size, int64_t ngroups,
                       void* dX, int64_t lddx, cudaStream_t s) {
  const int G = group_size == -1 ? (int)k : group_size;
  const dim3 grid((unsigned)cdiv(k, DG_C), (unsigned)cdiv(m, DG_T));
  if (dt == GPTQ_F16)
    launch_pdl(dgrad_general_kernel<__half>, grid, dim3(256), 0, s, (const __half*)dY, lddy, (int)m,
               (int)n, qw, bits, scales, zeros, g_idx, G, (int)ngroups, (int)k, (__half*)dX, lddx);
  else
    launch_pdl(dgrad_general_kernel<__nv_bfloat16>, grid, dim3(256), 0, s,
               (const __nv_bfloat16*)dY, lddy, (int)m, (int)n, qw, bits, scales, zeros, g_idx, G,
               (int)ngroups, (int)k, (__nv_bfloat16*)dX, lddx);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace gptq
