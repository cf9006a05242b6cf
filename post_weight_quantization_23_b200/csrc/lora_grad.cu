// Gradients of the adapters (gptq_lora_backward): with U = scaling B^T dY of the
// tensor-core pass over dY and V = scaling A x kept from the forward pass,
//   dA_a = sum_t U[t] x_t^T,   dB_a = sum_t dY[t] V[t]^T,
// t over the rows of adapter a's requests.  Both are sums over tokens of a wide
// row (x or dY, `S` below) times a narrow fp32 row (U or V, `W` below).
#include "lora.cuh"

namespace gptq {

gptq_status lora_low_impl(LoraArgs a, bool bf16, cudaStream_t s);

// One of the two gradients.
struct LoraGradArgs {
  const void* S;         // (m, C) wide rows: 16-bit values or int8 codes
  int64_t lds;
  const float* s_scales; // codes: (m, ceil(C / 128)) scales, else NULL
  const float* W;        // (m, r) narrow rows
  void* out;             // adapter a, column c, rank row p at a r C + c col_stride + p rank_stride
  int64_t col_stride, rank_stride;
  int C;
};

struct LoraGradCommon {
  const int32_t* starts;
  const int32_t* adapter;
  int m, r, na, nreq;
  uint32_t spin;
};

namespace {

// General kernel: 32 columns x the whole rank of one adapter per CTA, any
// alignment; 32 tokens at a time through shared memory.
constexpr int LG_COLS = 32, LG_TOK = 32;

template <bool BF16>
__global__ void __launch_bounds__(256)
lora_grad_general_kernel(LoraGradArgs a, LoraGradCommon c) {
  using Ty = LoraType<BF16>;
  using T = typename Ty::T;
  __shared__ float sw[LG_TOK][LORA_MAX_RANK];
  __shared__ float ss[LG_TOK][LG_COLS];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, x = tid % LG_COLS, y = tid / LG_COLS;
  const int col0 = blockIdx.x * LG_COLS, ad = blockIdx.y;
  const int nb = (a.C + 127) / 128;
  float acc[LORA_MAX_RANK / 8];
#pragma unroll
  for (int i = 0; i < LORA_MAX_RANK / 8; ++i) acc[i] = 0.f;
  for (int q = 0; q < c.nreq; ++q) {
    if (c.adapter[q] != ad) continue;
    const int b = lora_clamp(c.starts[q], c.m), e = lora_clamp(c.starts[q + 1], c.m);
    for (int t0 = b; t0 < e; t0 += LG_TOK) {
      __syncthreads();
      for (int i = tid; i < LG_TOK * c.r; i += 256) {
        const int tt = i / c.r, p = i % c.r;
        sw[tt][p] = t0 + tt < e ? a.W[(int64_t)(t0 + tt) * c.r + p] : 0.f;
      }
      for (int i = tid; i < LG_TOK * LG_COLS; i += 256) {
        const int tt = i / LG_COLS, cc = col0 + i % LG_COLS;
        float v = 0.f;
        if (t0 + tt < e && cc < a.C) {
          const int64_t row = t0 + tt;
          v = a.s_scales != nullptr
                  ? (float)((const int8_t*)a.S)[row * a.lds + cc] * a.s_scales[row * nb + cc / 128]
                  : to_f32(((const T*)a.S)[row * a.lds + cc]);
        }
        ss[tt][i % LG_COLS] = v;
      }
      __syncthreads();
      for (int tt = 0; tt < LG_TOK; ++tt) {
        const float v = ss[tt][x];
#pragma unroll
        for (int i = 0; i < LORA_MAX_RANK / 8; ++i)
          if (y + 8 * i < c.r) acc[i] = fmaf(sw[tt][y + 8 * i], v, acc[i]);
      }
    }
  }
  if (col0 + x < a.C) {
    T* o = (T*)a.out + (int64_t)ad * c.r * a.C + (col0 + x) * a.col_stride;
#pragma unroll
    for (int i = 0; i < LORA_MAX_RANK / 8; ++i)
      if (y + 8 * i < c.r) o[(y + 8 * i) * a.rank_stride] = Ty::cvt(acc[i]);
  }
}

gptq_status grad_general(const LoraGradArgs& a, const LoraGradCommon& c, bool bf16,
                         cudaStream_t s) {
  const dim3 grid((unsigned)cdiv(a.C, LG_COLS), (unsigned)c.na);
  if (bf16)
    launch_pdl(lora_grad_general_kernel<true>, grid, dim3(256), 0, s, a, c);
  else
    launch_pdl(lora_grad_general_kernel<false>, grid, dim3(256), 0, s, a, c);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace

// dA (na, r, k) and dB (na, n, r) from U, V (m, r).
gptq_status lora_grads_impl(const LoraGradArgs& ga, const LoraGradArgs& gb,
                            const LoraGradCommon& c, bool bf16, cudaStream_t s) {
  gptq_status st = grad_general(ga, c, bf16, s);
  if (st != GPTQ_OK) return st;
  return grad_general(gb, c, bf16, s);
}

gptq_status lora_backward_impl(LoraArgs low, const void* X, int64_t ldx, const float* x_scales,
                               const float* V, void* dA, void* dB, bool bf16, cudaStream_t s) {
  if (low.nreq > 0) {
    const gptq_status st = lora_low_impl(low, bf16, s);
    if (st != GPTQ_OK) return st;
  }
  const int k = low.N, n = low.K, r = low.r;
  LoraGradCommon c;
  c.starts = low.starts, c.adapter = low.adapter;
  c.m = low.m, c.r = r, c.na = low.na, c.nreq = low.nreq, c.spin = low.spin;
  LoraGradArgs ga, gb;
  ga.S = X, ga.lds = ldx, ga.s_scales = x_scales, ga.W = low.V, ga.out = dA;
  ga.col_stride = 1, ga.rank_stride = k, ga.C = k;
  gb.S = low.X, gb.lds = low.ldx, gb.s_scales = nullptr, gb.W = V, gb.out = dB;
  gb.col_stride = r, gb.rank_stride = 1, gb.C = n;
  return lora_grads_impl(ga, gb, c, bf16, s);
}

}  // namespace gptq
