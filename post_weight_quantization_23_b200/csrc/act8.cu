// Activation checkpoints in 8 bits (gptq_act_checkpoint, gptq_act_restore).
//
// A row is cut into blocks of 128 columns.  Per block, with top = max |x|:
//   scale = fl32(top / 127),  inv = fl32(127 / top),
//   code[c] = the integer nearest to x[c] * inv, halves to even,
//   restored x[c] = code[c] * scale.
// x * inv is never rounded before the integer is taken: one fused multiply-add
// with 1.5 * 2^23 rounds the exact product at the integers (|x * inv| <= 127 +
// 2^-16, so the sum stays in the binade whose spacing is 1), and the code is the
// sum's low bits.  The halves matter: x = top / 2 sits on 63.5 in every block.
//
// Bound by HBM: 2 bytes in and 1 + 4/128 out per element (16-bit X), the other
// way round for the restore.  One thread owns 8 columns (a 16-byte load, an
// 8-byte store), 16 neighbouring lanes a block, so every access of a warp is
// contiguous and the maximum takes four shuffles; four vectors per thread are
// requested before the first is used.  8192 x 11008 bf16
// saved and restored: 94 us in a replayed graph (547 MB, 5.8 TB/s, 0.90 of measured HBM; 101 us
// through the two Python calls); with scalar maxima and both divisions in every lane the save
// alone took 91 us, its instructions the bound.
#include "common.cuh"

#include <algorithm>

namespace gptq {

namespace {

constexpr int A8_BLOCK = 128;      // columns per scale
constexpr int A8_VEC = 8;          // columns per thread
constexpr int A8_THREADS = 256;
constexpr int A8_UNROLL = 4;       // vectors in flight per thread
// a block whose largest magnitude is below this is stored as zeros (127 / top
// must stay finite)
constexpr float A8_TINY = 7.8886090522101181e-31f;  // 2^-100

// Division by a fixed number below 2^31 as a multiplication, n / d for n < 2^31 (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994).
struct A8Div {
  uint32_t mul, shift;
};
A8Div a8_div(uint32_t d) {
  A8Div r;
  r.shift = 0;
  while (((uint64_t)1 << r.shift) < d) ++r.shift;
  r.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << r.shift) - d)) / d + 1);
  return r;
}
__device__ __forceinline__ uint32_t a8_quot(uint32_t n, A8Div d) {
  return (__umulhi(d.mul, n) + n) >> d.shift;
}

// Eight columns as they lie in memory; columns past `have` are zeros.
template <typename T> struct A8Raw { uint32_t w[sizeof(T) * 2]; };

template <typename T>
__device__ __forceinline__ A8Raw<T> a8_load(const T* __restrict__ p, int have, bool vec) {
  A8Raw<T> r;
  if (vec && have == A8_VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(r.w)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < have ? p[i] : T(0.f);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * 2; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(v)[i];
  }
  return r;
}

// The bits of the largest |x| of 128 columns (16 lanes), as fp32; a NaN is above infinity.
// 16-bit types are compared two at a time as integers, which order like the magnitudes.
template <typename T>
__device__ __forceinline__ uint32_t a8_top(const A8Raw<T>& r) {
  if (sizeof(T) == 4) {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, r.w[i] & 0x7fffffffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
    return t;
  }
  uint32_t t = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __vmaxu2(t, r.w[i] & 0x7fff7fffu);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
  const unsigned short h = (unsigned short)max(t & 0xffffu, t >> 16);
  return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&h)));
}

template <typename T>
__device__ __forceinline__ float a8_value(const A8Raw<T>& r, int i) {
  if (sizeof(T) == 4) return __uint_as_float(r.w[i]);
  const unsigned short h = (unsigned short)(r.w[i / 2] >> (16 * (i % 2)));
  return to_f32(*reinterpret_cast<const T*>(&h));
}

template <typename T> __device__ __forceinline__ T a8_out(float v);
template <> __device__ __forceinline__ float a8_out<float>(float v) { return v; }
template <> __device__ __forceinline__ __half a8_out<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 a8_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// rows of X from row 0; nvp = vectors per row rounded up to whole blocks.  The two
// divisions of a block are done once: of a thread's four vectors, lane l takes those of
// vector l % 4 and hands the factor round.
template <typename T>
__global__ void __launch_bounds__(A8_THREADS)
act_checkpoint_kernel(const T* __restrict__ X, int64_t ldx, uint32_t total, uint32_t nvp, A8Div div,
                      int k, int nb, int xvec, int cvec, int8_t* __restrict__ codes, int64_t ldc,
                      float* __restrict__ scales) {
  static_assert(A8_UNROLL == 4, "a lane per vector");
  pdl_wait();
  pdl_trigger();
  const uint32_t base = blockIdx.x * (A8_THREADS * A8_UNROLL) + threadIdx.x;
  const int lane = threadIdx.x & 31;
  A8Raw<T> x[A8_UNROLL];
  uint32_t row[A8_UNROLL], top[A8_UNROLL];
  int col[A8_UNROLL], have[A8_UNROLL];
#pragma unroll
  for (int u = 0; u < A8_UNROLL; ++u) {
    const uint32_t e = base + u * A8_THREADS;
    row[u] = a8_quot(e, div);
    col[u] = (int)(e - row[u] * nvp) * A8_VEC;
    have[u] = e < total ? min(max(k - col[u], 0), A8_VEC) : 0;
    x[u] = a8_load(X + (int64_t)row[u] * ldx + col[u], have[u], xvec != 0);
  }
#pragma unroll
  for (int u = 0; u < A8_UNROLL; ++u) top[u] = a8_top(x[u]);
  float inv;
  {
    const int u = lane & 3;
    const uint32_t t = u == 0 ? top[0] : u == 1 ? top[1] : u == 2 ? top[2] : top[3];
    const uint32_t r = u == 0 ? row[0] : u == 1 ? row[1] : u == 2 ? row[2] : row[3];
    const int c = u == 0 ? col[0] : u == 1 ? col[1] : u == 2 ? col[2] : col[3];
    const float f = __uint_as_float(t);
    const bool bad = t >= 0x7f800000u, tiny = f < A8_TINY;  // bad: NaN or infinity in the block
    inv = (bad || tiny) ? 0.f : __fdiv_rn(127.f, f);
    const float scale = bad ? __uint_as_float(0x7fc00000u) : tiny ? 0.f : __fdiv_rn(f, 127.f);
    if ((lane & 15) < 4 && base + u * A8_THREADS < total)
      scales[(int64_t)r * nb + c / A8_BLOCK] = scale;
  }
#pragma unroll
  for (int u = 0; u < A8_UNROLL; ++u) {
    const float f = __shfl_sync(0xffffffffu, inv, (lane & ~3) | u);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __float_as_uint(__fmaf_rn(a8_value(x[u], i), f, 12582912.f));
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)  // the low bytes
      w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040),
                         __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
    if (top[u] >= 0x7f800000u) w[0] = w[1] = 0u;
    int8_t* dst = codes + (int64_t)row[u] * ldc + col[u];
    if (cvec && have[u] == A8_VEC) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
      for (int i = 0; i < have[u]; ++i) dst[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(A8_THREADS)
act_restore_kernel(const int8_t* __restrict__ codes, int64_t ldc, const float* __restrict__ scales,
                   uint32_t total, uint32_t nvp, A8Div div, int k, int nb, int cvec, int ovec,
                   T* __restrict__ out, int64_t ldo) {
  pdl_wait();
  pdl_trigger();
  const uint32_t base = blockIdx.x * (A8_THREADS * A8_UNROLL) + threadIdx.x;
  uint2 w[A8_UNROLL];
  float s[A8_UNROLL];
  uint32_t row[A8_UNROLL];
  int col[A8_UNROLL];
#pragma unroll
  for (int u = 0; u < A8_UNROLL; ++u) {
    const uint32_t e = base + u * A8_THREADS;
    row[u] = a8_quot(e, div);
    col[u] = (int)(e - row[u] * nvp) * A8_VEC;
    const int have = e < total ? min(max(k - col[u], 0), A8_VEC) : 0;
    const int8_t* p = codes + (int64_t)row[u] * ldc + col[u];
    w[u] = make_uint2(0u, 0u);
    s[u] = 0.f;
    if (have > 0) s[u] = scales[(int64_t)row[u] * nb + col[u] / A8_BLOCK];
    if (cvec && have == A8_VEC) {
      w[u] = *reinterpret_cast<const uint2*>(p);
    } else {
      uint32_t b[2] = {0u, 0u};
      for (int i = 0; i < have; ++i) b[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i % 4));
      w[u] = make_uint2(b[0], b[1]);
    }
  }
#pragma unroll
  for (int u = 0; u < A8_UNROLL; ++u) {
    const uint32_t e = base + u * A8_THREADS;
    if (e >= total) continue;
    const int have = min(max(k - col[u], 0), A8_VEC);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = i < 4 ? w[u].x : w[u].y;
      v[i] = (float)(int)(int8_t)(word >> (8 * (i % 4))) * s[u];
      // 127 * fl(top / 127) may round past the largest fp32 value: that value then
      if (sizeof(T) == 4 && isinf(v[i]) && isfinite(s[u])) v[i] = copysignf(3.402823466e38f, v[i]);
    }
    T* dst = out + (int64_t)row[u] * ldo + col[u];
    if (ovec && have == A8_VEC) {
      if (sizeof(T) == 2) {
        uint4 o;
        T* h = reinterpret_cast<T*>(&o);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = a8_out<T>(v[i]);
        *reinterpret_cast<uint4*>(dst) = o;
      } else {
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
      for (int i = 0; i < have; ++i) dst[i] = a8_out<T>(v[i]);
    }
  }
}

// Rows per launch: the flat vector index stays below 2^31.
int64_t a8_rows_per_launch(int64_t nvp) {
  return std::max<int64_t>(1, (((int64_t)1 << 31) - 4 * A8_THREADS * A8_UNROLL) / nvp);
}

template <typename T>
gptq_status checkpoint_typed(const T* X, int64_t m, int64_t k, int64_t ldx, int8_t* codes,
                             int64_t ldc, float* scales, cudaStream_t s) {
  const int64_t nb = cdiv(k, A8_BLOCK), nvp = nb * (A8_BLOCK / A8_VEC);
  const int xvec = (uintptr_t)X % 16 == 0 && (ldx * (int64_t)sizeof(T)) % 16 == 0;
  const int cvec = (uintptr_t)codes % 8 == 0 && ldc % 8 == 0;
  const int64_t step = a8_rows_per_launch(nvp);
  for (int64_t r0 = 0; r0 < m; r0 += step) {
    const int64_t rows = std::min(step, m - r0), total = rows * nvp;
    launch_pdl(act_checkpoint_kernel<T>, dim3((unsigned)cdiv(total, A8_THREADS * A8_UNROLL)),
               dim3(A8_THREADS), 0, s, X + r0 * ldx, ldx, (uint32_t)total, (uint32_t)nvp,
               a8_div((uint32_t)nvp), (int)k, (int)nb, xvec, cvec, codes + r0 * ldc, ldc, scales + r0 * nb);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

template <typename T>
gptq_status restore_typed(const int8_t* codes, int64_t ldc, const float* scales, int64_t m,
                          int64_t k, T* out, int64_t ldo, cudaStream_t s) {
  const int64_t nb = cdiv(k, A8_BLOCK), nvp = nb * (A8_BLOCK / A8_VEC);
  const int cvec = (uintptr_t)codes % 8 == 0 && ldc % 8 == 0;
  const int ovec = (uintptr_t)out % 16 == 0 && (ldo * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t step = a8_rows_per_launch(nvp);
  for (int64_t r0 = 0; r0 < m; r0 += step) {
    const int64_t rows = std::min(step, m - r0), total = rows * nvp;
    launch_pdl(act_restore_kernel<T>, dim3((unsigned)cdiv(total, A8_THREADS * A8_UNROLL)),
               dim3(A8_THREADS), 0, s, codes + r0 * ldc, ldc, scales + r0 * nb, (uint32_t)total,
               (uint32_t)nvp, a8_div((uint32_t)nvp), (int)k, (int)nb, cvec, ovec, out + r0 * ldo, ldo);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

}  // namespace

gptq_status act_checkpoint_impl(const void* X, gptq_dtype dt, int64_t m, int64_t k, int64_t ldx,
                                int8_t* codes, int64_t ldc, float* scales, cudaStream_t s) {
  if (dt == GPTQ_F32) return checkpoint_typed((const float*)X, m, k, ldx, codes, ldc, scales, s);
  if (dt == GPTQ_F16) return checkpoint_typed((const __half*)X, m, k, ldx, codes, ldc, scales, s);
  return checkpoint_typed((const __nv_bfloat16*)X, m, k, ldx, codes, ldc, scales, s);
}

gptq_status act_restore_impl(const int8_t* codes, int64_t ldc, const float* scales, int64_t m,
                             int64_t k, gptq_dtype dt, void* out, int64_t ldo, cudaStream_t s) {
  if (dt == GPTQ_F32) return restore_typed(codes, ldc, scales, m, k, (float*)out, ldo, s);
  if (dt == GPTQ_F16) return restore_typed(codes, ldc, scales, m, k, (__half*)out, ldo, s);
  return restore_typed(codes, ldc, scales, m, k, (__nv_bfloat16*)out, ldo, s);
}

}  // namespace gptq
