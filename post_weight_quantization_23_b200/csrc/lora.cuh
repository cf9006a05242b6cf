// Shared pieces of the adapter kernels (lora.cu, lora_tc.cu, lora_grad.cu).
//
// Requests are rows [starts[q], starts[q + 1]) of the batch, each with one
// adapter (an index outside [0, na) means none).  The kernels never trust the
// device arrays: starts are clamped to [0, m], a request whose end is not above
// its start is empty, so no access leaves the batch whatever they hold.
#pragma once

#include "cluster.cuh"

namespace gptq {

constexpr int LORA_MAX_RANK = 128;
constexpr int LORA_CLUSTER = 8;  // CTAs that share one piece of a request

struct LoraPiece {
  int t0 = 0;    // first row
  int cnt = 0;   // rows (0: no such piece)
  int a = -1;    // adapter, -1 = none
};

__device__ __forceinline__ int lora_clamp(int v, int m) { return min(max(v, 0), m); }

// Pieces of TT rows of one request that this launch takes (lengths in
// [min_len, max_len]).
__device__ __forceinline__ int lora_pieces(const int32_t* starts, int q, int m, int TT, int min_len,
                                           int max_len) {
  const int len = lora_clamp(starts[q + 1], m) - lora_clamp(starts[q], m);
  return (len < min_len || len > max_len || len <= 0) ? 0 : (len + TT - 1) / TT;
}

// ---- 16-bit types ------------------------------------------------------------

template <bool BF16> struct LoraType;
template <> struct LoraType<false> {
  using T = __half;
  __device__ static T cvt(float v) { return __float2half_rn(v); }
  __device__ static uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
};
template <> struct LoraType<true> {
  using T = __nv_bfloat16;
  __device__ static T cvt(float v) { return __float2bfloat16_rn(v); }
  __device__ static uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static float2 unpack(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
  }
};

// Two 32-bit values as the sum of two 16-bit pairs, hi + lo (2 x 8 significant
// bits for bf16, 2 x 11 for f16).  A value whose hi part is not finite has no lo.
template <bool BF16>
__device__ __forceinline__ void lora_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  using Ty = LoraType<BF16>;
  hi = Ty::pack(a, b);
  const float2 h = Ty::unpack(hi);
  const float la = isfinite(h.x) ? a - h.x : 0.f, lb = isfinite(h.y) ? b - h.y : 0.f;
  lo = Ty::pack(la, lb);
}

// The same for bf16 without the look at hi: a value that is not finite in bf16 gives NaN.
__device__ __forceinline__ void lora_split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = LoraType<true>::pack(a, b);
  lo = LoraType<true>::pack(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

// f16 only: the power of two that brings a row whose largest magnitude is `top`
// to [2^7, 2^8), where neither half of the split leaves f16's range; 1 for a
// zero or non-finite row.  Exact to apply and to take back.
__device__ __forceinline__ float lora_row_factor(float top) {
  if (!(top > 0.f) || !isfinite(top)) return 1.f;
  int e = (int)((__float_as_uint(top) >> 23) & 0xFFu) - 127;
  e = min(max(e, -100), 120);
  return __uint_as_float((uint32_t)(127 + 7 - e) << 23);
}

// The requests of a batch, and the arguments that the adapter kernels share.  Forward (add): reduction over
// K = k with P = A (na, r, k), output over N = n with Q = B (na, n, r).
// Backward: K = n with P = B, N = k with Q = A.
struct LoraRequests {
  const int32_t* starts;
  const int32_t* adapter;
  int m, na, nreq;
  int min_len, max_len;  // request lengths that this launch takes
};

struct LoraArgs : LoraRequests {
  const void* X;  // (m, K) the rows that are reduced
  int64_t ldx;
  const void* P;
  const void* Q;
  const float* scaling;
  const void* Y;  // (m, N) added to, or NULL
  int64_t ldy;
  void* out;      // (m, N), or NULL: V alone
  int64_t ldo;
  float* V;       // (m, r) or NULL
  int K, N, r;
  uint32_t spin;
};

constexpr int LORA_ANY = -1;

// Pieces first, first + stride, .. (at most `cap`, from the `skip`-th of them) of
// TT rows, of one adapter's requests (only >= 0) or of all that have an adapter
// (LORA_ANY), into `table`, by the whole CTA; their number.  Each thread counts the
// pieces of a run of requests, a scan locates them, and each thread writes those
// of its run that are asked for.  `sm` holds NT / 32 + 1 ints.
template <int NT>
__device__ __forceinline__ int lora_find_pieces(const LoraRequests& a, int TT, int first,
                                                int stride, int skip, LoraPiece* table, int cap,
                                                int* sm, int only) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.nreq + NT - 1) / NT;
  const int q0 = min(a.nreq, tid * per), q1 = min(a.nreq, q0 + per);
  int own = 0;
  // the thread's first request; mostly its only one, and its three loads are in flight together
  int b0 = 0, e0 = 0, ad0 = -1;
  if (q0 < q1) b0 = a.starts[q0], e0 = a.starts[q0 + 1], ad0 = a.adapter[q0];
  auto pieces = [&](int q, int& b, int& e, int& ad) {
    b = lora_clamp(q == q0 ? b0 : a.starts[q], a.m);
    e = lora_clamp(q == q0 ? e0 : a.starts[q + 1], a.m);
    ad = q == q0 ? ad0 : a.adapter[q];
    if (only >= 0 ? ad != only : ad < 0 || ad >= a.na) return 0;
    return e - b < a.min_len || e - b > a.max_len ? 0 : (e - b + TT - 1) / TT;
  };
  int b, e, ad;
  for (int q = q0; q < q1; ++q) own += pieces(q, b, e, ad);
  int inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  __syncthreads();  // the last use of sm and table is over
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  int at = inc - own, total = 0;  // pieces before this thread's run, of all
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) at += sm[w];
    total += sm[w];
  }
  // the i-th entry is piece first + (skip + i) * stride
  const int64_t p0 = first + (int64_t)skip * stride;
  const int n = total > p0 ? (int)min((uint32_t)cap, ((uint32_t)(total - p0) + stride - 1) / stride) : 0;
  for (int q = q0; q < q1 && n > 0; ++q) {
    const int c = pieces(q, b, e, ad);
    if (c > 0) {
      uint32_t i = at <= p0 ? 0 : ((uint32_t)(at - p0) + stride - 1) / stride;
      for (; i < (uint32_t)n && p0 + (int64_t)i * stride < at + c; ++i) {
        LoraPiece r;
        r.t0 = b + (int)(p0 + (int64_t)i * stride - at) * TT;
        r.cnt = min(TT, e - r.t0);
        r.a = ad;
        table[i] = r;
      }
    }
    at += c;
  }
  __syncthreads();
  return n;
}

// Columns [j0, j1) of a row from y (zeros if NULL) to o by one warp; eight vectors are
// loaded before the first is stored (the two might be the same memory, so the compiler
// keeps loads behind stores: one vector at a time waits for HBM each time).
template <typename T>
__device__ __forceinline__ void lora_copy_row(const T* y, T* o, int j0, int j1, int vec) {
  const int lane = threadIdx.x & 31;
  if (vec) {
    for (int b = j0; b < j1; b += 8 * 256) {
      uint4 w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int j = b + 256 * q + 8 * lane;
        w[q] = y != nullptr && j + 8 <= j1 ? __ldcg(reinterpret_cast<const uint4*>(y + j))
                                           : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int j = b + 256 * q + 8 * lane;
        if (j + 8 <= j1) *reinterpret_cast<uint4*>(o + j) = w[q];
      }
    }
    j0 = j1 - j1 % 8;  // j0 and vectors are multiples of 8
  }
  for (int j = j0 + lane; j < j1; j += 32)
    reinterpret_cast<unsigned short*>(o)[j] =
        y != nullptr ? __ldcg(reinterpret_cast<const unsigned short*>(y) + j) : (unsigned short)0;
}

// Rows without an adapter: out = Y (0 without Y) unless they are the same, V = 0, over
// the whole batch, for a launch whose pieces have adapters only: part
// `part` of `nparts` takes every nparts-th row of every such request; `nthreads` (a
// multiple of 32) threads of the CTA call it, thread `tid` of them.
template <typename T>
__device__ __forceinline__ void lora_copy_bare(const LoraArgs& a, int part, int nparts, int tid,
                                               int nthreads, int vec) {
  const bool rows = a.out != nullptr && a.Y != a.out;
  if (!rows && a.V == nullptr) return;
  const int lane = threadIdx.x & 31;
  for (int q0 = 0; q0 < a.nreq; q0 += 32) {
    const int q = q0 + lane;
    bool bare = false;
    if (q < a.nreq) {
      const int ad = a.adapter[q];
      bare = (ad < 0 || ad >= a.na) && lora_pieces(a.starts, q, a.m, 1, a.min_len, a.max_len) > 0;
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, bare); left != 0; left &= left - 1) {
      const int r = q0 + __ffs(left) - 1;
      const int b = lora_clamp(a.starts[r], a.m), e = lora_clamp(a.starts[r + 1], a.m);
      const int mine = (e - b - part + nparts - 1) / nparts;  // rows b + part, + nparts, ..
      if (mine <= 0) continue;
      if (rows) {
        for (int i = tid / 32; i < mine; i += nthreads / 32) {  // a row per warp
          const int64_t row = b + part + (int64_t)i * nparts;
          lora_copy_row<T>(a.Y != nullptr ? (const T*)a.Y + row * a.ldy : nullptr,
                           (T*)a.out + row * a.ldo, 0, a.N, vec);
        }
      }
      if (a.V != nullptr)
        for (int x = tid; x < mine * a.r; x += nthreads)
          a.V[(int64_t)(b + part + (x / a.r) * nparts) * a.r + x % a.r] = 0.f;
    }
  }
}

}  // namespace gptq
