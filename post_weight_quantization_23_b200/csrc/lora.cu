// The adapters of many requests beside a shared projection (gptq_lora_add):
//   V[t] = scaling_a (A_a x_t),   out[t] = Y[t] + B_a V[t],
// a = the adapter of the request that holds row t.  V stays in fp32; the sum
// with Y is rounded once.
//
// Kernels:
//   lora_decode_kernel   short requests and small batches: one launch, a cluster of
//                        8 CTAs per piece of 8 rows of one adapter;
//   lora_tc_kernel       (lora_tc.cu) long requests and the backward pass: the same
//                        cluster on the 5th-generation tensor cores;
//   lora_general_kernel  operands whose rows the wide loads cannot take.
#include "lora.cuh"

#include <algorithm>

namespace gptq {

bool lora_tc_supported(const LoraArgs& a, bool backward);
gptq_status lora_tc(const LoraArgs& a, bool bf16, bool backward, cudaStream_t s);

namespace {

// ---- general kernel ------------------------------------------------------------

// One CTA per row, any alignment and strides.
template <bool BF16>
__global__ void __launch_bounds__(256)
lora_general_kernel(LoraArgs a, int backward) {
  using Ty = LoraType<BF16>;
  using T = typename Ty::T;
  __shared__ float v[LORA_MAX_RANK];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int lo = 0, hi = a.nreq;  // the last request that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.starts[mid] <= t) lo = mid; else hi = mid;
  }
  if (t < a.starts[lo] || t >= a.starts[lo + 1]) return;
  const int len = lora_clamp(a.starts[lo + 1], a.m) - lora_clamp(a.starts[lo], a.m);
  if (len < a.min_len || len > a.max_len) return;
  const int ad = a.adapter[lo];
  const bool none = ad < 0 || ad >= a.na;
  const T* x = (const T*)a.X + (int64_t)t * a.ldx;
  const T* P = (const T*)a.P + (none ? 0 : (int64_t)ad * a.r * a.K);
  const T* Q = (const T*)a.Q + (none ? 0 : (int64_t)ad * a.r * a.N);
  const int64_t prs = backward ? 1 : a.K, pcs = backward ? a.r : 1;
  const int64_t qrs = backward ? a.N : 1, qcs = backward ? 1 : a.r;
  const float sc = none ? 0.f : a.scaling[ad];
  for (int p = warp; p < a.r; p += 8) {
    float s = 0.f;
    if (!none)
      for (int c = lane; c < a.K; c += 32) s = fmaf(to_f32(x[c]), to_f32(P[p * prs + c * pcs]), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      v[p] = none ? 0.f : s * sc;
      if (a.V != nullptr) a.V[(int64_t)t * a.r + p] = v[p];
    }
  }
  __syncthreads();
  if (a.out == nullptr) return;
  const T* y = (const T*)a.Y + (int64_t)t * a.ldy;
  T* o = (T*)a.out + (int64_t)t * a.ldo;
  if (none) {
    if (a.Y != a.out)
      for (int j = threadIdx.x; j < a.N; j += 256) o[j] = a.Y != nullptr ? y[j] : Ty::cvt(0.f);
    return;
  }
  for (int j = threadIdx.x; j < a.N; j += 256) {
    float s = 0.f;
    for (int p = 0; p < a.r; ++p) s = fmaf(v[p], to_f32(Q[p * qrs + j * qcs]), s);
    o[j] = Ty::cvt(a.Y != nullptr ? to_f32(y[j]) + s : s);
  }
}

// ---- decode kernel --------------------------------------------------------------

constexpr int LD_THREADS = 256;
constexpr int LD_WARPS = LD_THREADS / 32;
constexpr int LD_TT = 8;  // rows per piece: the n of mma.sync m16n8k16

template <bool BF16>
__device__ __forceinline__ void ld_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Every load of this kernel goes to L2 (cache-global): beside the tensor-core kernel it
// starts without waiting for it (see `late`), so no L1 line of an earlier kernel may serve.
__device__ __forceinline__ uint4 ld_u4(const void* p) {
  return __ldcg(reinterpret_cast<const uint4*>(p));
}

// A piece is up to 8 rows of one adapter, of one request or of several (a batch of single
// tokens often shares adapters, and the adapter's matrices are what a piece costs).  In
// windows of 256 requests, one per thread, each thread counts the rows that earlier
// requests of the window give the same adapter; rows of rank 8 i .. 8 i + 7 are a piece.
struct LdWindow {
  int start, len, a, before;  // this thread's request: rows, adapter (-1: none), rank of its first row
  int at, own, total;         // pieces before its own, its own, of the window
};

struct LdShared {
  int ad[LD_THREADS], len[LD_THREADS];
  int scan[LD_WARPS];
  int piece[2];        // adapter and first rank of the piece looked up
  int row[LD_TT];
};

__device__ __forceinline__ LdWindow ld_window(const LoraArgs& a, int q0, LdShared& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = q0 + tid;
  LdWindow w = {0, 0, -1, 0, 0, 0, 0};
  if (q < a.nreq) {
    const int b = __ldcg(a.starts + q), e = __ldcg(a.starts + q + 1), ad = __ldcg(a.adapter + q);
    w.start = lora_clamp(b, a.m);
    w.len = lora_clamp(e, a.m) - w.start;
    if (w.len < a.min_len || w.len > a.max_len) w.len = 0;
    w.a = ad < 0 || ad >= a.na ? -1 : ad;
  }
  __syncthreads();  // the last window is done
  sm.ad[tid] = w.a;
  sm.len[tid] = w.len;
  __syncthreads();
  const int n = min(a.nreq - q0, LD_THREADS);
  for (int i = 0; i < n; i += 4) {
    const int4 x = *reinterpret_cast<const int4*>(sm.ad + i);
    const int4 l = *reinterpret_cast<const int4*>(sm.len + i);
    w.before += (i < tid && x.x == w.a ? l.x : 0) + (i + 1 < tid && x.y == w.a ? l.y : 0) +
                (i + 2 < tid && x.z == w.a ? l.z : 0) + (i + 3 < tid && x.w == w.a ? l.w : 0);
  }
  w.own = w.len > 0 ? (w.before + w.len + LD_TT - 1) / LD_TT - (w.before + LD_TT - 1) / LD_TT : 0;
  int inc = w.own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sm.scan[warp] = inc;
  __syncthreads();
  w.at = inc - w.own;
#pragma unroll
  for (int i = 0; i < LD_WARPS; ++i) {
    const int v = sm.scan[i];
    if (i < warp) w.at += v;
    w.total += v;
  }
  return w;
}

// The window's p-th piece: its adapter; its rows in sm.row (-1 behind the last).
__device__ __forceinline__ int ld_piece(const LdWindow& w, int p, LdShared& sm) {
  __syncthreads();  // the last piece's rows are read
  if (threadIdx.x < LD_TT) sm.row[threadIdx.x] = -1;
  if (p >= w.at && p < w.at + w.own) {  // the request that holds the piece's first row
    sm.piece[0] = w.a;
    sm.piece[1] = ((w.before + LD_TT - 1) / LD_TT + p - w.at) * LD_TT;
  }
  __syncthreads();
  const int ad = sm.piece[0], first = sm.piece[1];
  if (w.len > 0 && w.a == ad)
    for (int r = max(w.before, first); r < min(w.before + w.len, first + LD_TT); ++r)
      sm.row[r - first] = w.start + (r - w.before);
  __syncthreads();
  return ad;
}

// A cluster of 8 CTAs takes one piece after another.  The
// adapter's matrices are what it has to read ((k + n) r elements, the rows are few),
// so both products take them straight from global memory as the 16-row operand of
// mma.sync m16n8k16 with the 8 tokens as its columns: the order of a reduction is
// free, so lane (g, t) takes 8 consecutive columns of row g in one 16-byte load where
// the fragment layout would want four 4-byte ones, and the activations' fragments take
// the same columns in the same lanes.
//   1. V^T = A x: the cluster's 64 warps share the columns in runs of 64; the
//      warps of a CTA add up in shared memory, and each CTA hands its sums to all
//      eight through distributed shared memory (one cluster barrier).
//   2. out^T = B V: the 64 warps share the n output rows, 16 at a time; V is the
//      other operand, each value as hi + lo of the 16-bit type (f16: each row
//      first scaled by a power of two, so that neither leaves the type's range).
// Latency is what it spends its time on, so the tiles of B and Y are requested several at a
// time, the first of them before the barrier.  One launch, no workspace, sums in a fixed order.
// In a replayed graph: one token, rank 16, 4096 -> 4096 4.4 us (look-up 1.2, loads of A 1.0, sums
// and exchange 1.2, output 0.6; the rest launch); 64 tokens over 16 adapters, 4096 -> 12288 9.4 us
// (half as long again with a piece per token, each adapter read four times; a sixth more with
// three CTAs an SM, fewer tiles of B in flight and more clusters that find no piece).
template <bool BF16, int RP>
__global__ void __launch_bounds__(LD_THREADS, RP <= 64 ? 2 : 1)
lora_decode_kernel(LoraArgs a, int yvec, int late) {
  using Ty = LoraType<BF16>;
  using T = typename Ty::T;
  constexpr int MT = RP / 16;                  // 16-row tiles of the rank
  constexpr int KC = RP >= 32 ? RP / 32 : 1;   // 32-wide chunks of the rank in product 2
  constexpr int NS = RP >= 32 ? 2 : 1;         // 16-wide steps per chunk
  constexpr int U = RP == 16 ? 6 : RP == 32 ? 4 : RP == 64 ? 2 : 1;  // tiles of B in flight
  extern __shared__ __align__(16) float ld_smem[];
  constexpr int PS = RP * LD_TT;               // values of one partial sum
  float* red = ld_smem;                        // [LD_WARPS][PS] per-warp sums, then V
  constexpr int RED = PS > LD_TT * 20 ? LD_WARPS * PS : LD_WARPS * LD_TT * 20;
  float* parts = ld_smem + RED;                // [2][LORA_CLUSTER][PS], piece by piece in turn
  __shared__ float fac[LD_TT];
  __shared__ __align__(16) LdShared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = (int)cluster_rank();
  const int stride = (int)gridDim.x / LORA_CLUSTER, cid = (int)blockIdx.x / LORA_CLUSTER;
  const T* Y = (const T*)a.Y;
  T* out = (T*)a.out;
  const int gw = rank * LD_WARPS + warp;
  constexpr int NW = LORA_CLUSTER * LD_WARPS;
  const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
  cluster_arrive();  // this CTA runs: peers may write to its shared memory
  // late: the kernel before this one is the tensor-core kernel of the same call, on other
  // rows.  All of its CTAs had waited for the kernels before the call when this one could
  // start, so this one runs beside it and waits for it before it ends: whatever follows
  // then finds both done.
  if (!late) pdl_wait();
  pdl_trigger();
  bool waited = false;
  int turn = 0;
  int64_t next = cid;  // of this cluster's pieces, counted over all windows
  int64_t base = 0;
  for (int q0 = 0; q0 < a.nreq; q0 += LD_THREADS) {
    const LdWindow win = ld_window(a, q0, sm);
    for (; next < base + win.total; next += stride) {
      const int ad = ld_piece(win, (int)(next - base), sm);
      const int64_t row_g = sm.row[g];  // of token g
      const bool tok = row_g >= 0;
      if (ad < 0) {
        // no adapter: the rows are copied, each CTA its share of the columns, a row per warp
        const int64_t r = sm.row[warp];
        const int per = (a.N + 8 * LORA_CLUSTER - 1) / (8 * LORA_CLUSTER) * 8;
        const int c0 = min(a.N, rank * per), c1 = min(a.N, c0 + per);
        if (r >= 0 && out != nullptr && a.Y != a.out)
          lora_copy_row<T>(Y != nullptr ? Y + r * a.ldy : nullptr, out + r * a.ldo, c0, c1,
                           yvec == 2);
        if (r >= 0 && a.V != nullptr && rank == 0)
          for (int p = lane; p < a.r; p += 32) a.V[r * a.r + p] = 0.f;
        continue;
      }
      const T* A = (const T*)a.P + (int64_t)ad * a.r * a.K;
      const T* B = (const T*)a.Q + (int64_t)ad * a.r * a.N;
      const int64_t row = tok ? row_g : 0;
      const T* xrow = (const T*)a.X + row * a.ldx;
      float* part = parts + (turn & 1) * (LORA_CLUSTER * PS);

      // 1. per-warp sums of A x over this warp's columns
      float acc[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll 2
      for (int c0 = gw * 64; c0 < a.K; c0 += NW * 64) {
        const int ca = c0 + 8 * t, cb = ca + 32;
        const bool oka = ca < a.K, okb = cb < a.K;
        const uint4 xa = tok && oka ? ld_u4(xrow + ca) : zero4;
        const uint4 xb = tok && okb ? ld_u4(xrow + cb) : zero4;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int p0 = 16 * i + g, p1 = p0 + 8;
          const T* r0 = A + (int64_t)p0 * a.K;
          const T* r1 = A + (int64_t)p1 * a.K;
          const uint4 a0 = p0 < a.r && oka ? ld_u4(r0 + ca) : zero4;
          const uint4 a1 = p1 < a.r && oka ? ld_u4(r1 + ca) : zero4;
          const uint4 b0 = p0 < a.r && okb ? ld_u4(r0 + cb) : zero4;
          const uint4 b1 = p1 < a.r && okb ? ld_u4(r1 + cb) : zero4;
          ld_mma<BF16>(acc[i], a0.x, a1.x, a0.y, a1.y, xa.x, xa.y);
          ld_mma<BF16>(acc[i], a0.z, a1.z, a0.w, a1.w, xa.z, xa.w);
          ld_mma<BF16>(acc[i], b0.x, b1.x, b0.y, b1.y, xb.x, xb.y);
          ld_mma<BF16>(acc[i], b0.z, b1.z, b0.w, b1.w, xb.z, xb.w);
        }
      }
      // tiles j0, j0 + 16 NW, .. of B (rows of this warp, the lane's columns of the rank) and,
      // as lane (token g, output columns 4 t ..), of Y
      uint4 w0[U][KC], w1[U][KC];
      uint2 yv[U];
      auto request = [&](int j0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int ju = j0 + u * NW * 16;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const int p = RP >= 32 ? 32 * c + 8 * t : 4 * t;
            const bool ok0 = p < a.r && ju + g < a.N, ok1 = p < a.r && ju + g + 8 < a.N;
            const T* q0 = B + (int64_t)(ju + g) * a.r + p;
            const T* q1 = q0 + (int64_t)8 * a.r;
            if (RP >= 32) {
              w0[u][c] = ok0 ? ld_u4(q0) : zero4;
              w1[u][c] = ok1 ? ld_u4(q1) : zero4;
            } else {
              const uint2 u0 = ok0 ? __ldcg((const uint2*)q0) : make_uint2(0u, 0u);
              const uint2 u1 = ok1 ? __ldcg((const uint2*)q1) : make_uint2(0u, 0u);
              w0[u][c] = make_uint4(u0.x, u0.y, 0u, 0u);
              w1[u][c] = make_uint4(u1.x, u1.y, 0u, 0u);
            }
          }
          const int j = ju + 4 * t;
          yv[u] = tok && yvec && a.Y != nullptr && j + 4 <= a.N
                      ? __ldcg(reinterpret_cast<const uint2*>(Y + row * a.ldy + j))
                      : make_uint2(0u, 0u);
        }
      };
      if (out != nullptr) request(gw * 16);
      __syncthreads();  // the last piece is done with red
      // lane (g, t) holds (rank row 16 i + g | + 8, token 2 t | + 1); laid out by token
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float* rw = red + warp * PS + 16 * i + g;
        rw[(2 * t) * RP] = acc[i][0];
        rw[(2 * t + 1) * RP] = acc[i][1];
        rw[(2 * t) * RP + 8] = acc[i][2];
        rw[(2 * t + 1) * RP + 8] = acc[i][3];
      }
      __syncthreads();
      if (!waited) {
        cluster_wait();  // every CTA of the cluster runs
        waited = true;
      }
      for (int e = tid; e < PS / 4; e += LD_THREADS) {
        float4 s = reinterpret_cast<const float4*>(red)[e];
#pragma unroll
        for (int w = 1; w < LD_WARPS; ++w) {
          const float4 v = reinterpret_cast<const float4*>(red + w * PS)[e];
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(part + rank * PS + 4 * e);
#pragma unroll
        for (int c = 0; c < LORA_CLUSTER; ++c) cluster_st_f4(cluster_map(dst, c), s);
      }
      cluster_arrive();
      cluster_wait();
      // (a peer writes to this half of parts again only after the next piece's barrier)
      const float sc = __ldcg(a.scaling + ad);
      float* vs = red;  // V of the piece, [token][RP]
      for (int e = tid; e < PS; e += LD_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < LORA_CLUSTER; ++c) s += part[c * PS + e];
        // columns that only pad the rank stay 0 where an infinity met their zeros
        const int tk = e / RP, p = e % RP;
        s = p < a.r ? s * sc : 0.f;
        vs[e] = s;
        if (a.V != nullptr && rank == 0 && sm.row[tk] >= 0 && p < a.r)
          a.V[(int64_t)sm.row[tk] * a.r + p] = s;
      }
      ++turn;
      __syncthreads();
      if (out == nullptr) continue;
      if (!BF16) {
        float top = 0.f;
        for (int p = lane; p < RP; p += 32) top = fmaxf(top, fabsf(vs[warp * RP + p]));
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) fac[warp] = lora_row_factor(top);
        __syncthreads();
      }
      uint32_t vh[KC * NS][2], vl[KC * NS][2];
      {
        const float f = BF16 ? 1.f : fac[g];
        const float* vr = vs + g * RP;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int h = 0; h < NS; ++h) {
            const int p = RP >= 32 ? 32 * c + 8 * t + 4 * h : 4 * t;
            const float4 v = *reinterpret_cast<const float4*>(vr + p);
            lora_split<BF16>(v.x * f, v.y * f, vh[c * NS + h][0], vl[c * NS + h][0]);
            lora_split<BF16>(v.z * f, v.w * f, vh[c * NS + h][1], vl[c * NS + h][1]);
          }
      }
      const float if0 = BF16 ? 1.f : __fdiv_rn(1.f, fac[2 * t]);  // powers of two: exact
      const float if1 = BF16 ? 1.f : __fdiv_rn(1.f, fac[2 * t + 1]);
      __syncthreads();  // red is reused as the warps' transposing buffers
      float* tile = red + warp * (LD_TT * 20);  // [token][16 + 4]
      for (int j0 = gw * 16; j0 < a.N; j0 += U * NW * 16) {
        if (j0 != gw * 16) request(j0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int ju = j0 + u * NW * 16;
          if (ju >= a.N) break;
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint4 x = w0[u][c], y = w1[u][c];
            ld_mma<BF16>(d, x.x, y.x, x.y, y.y, vl[c * NS][0], vl[c * NS][1]);
            ld_mma<BF16>(d, x.x, y.x, x.y, y.y, vh[c * NS][0], vh[c * NS][1]);
            if (NS == 2) {
              ld_mma<BF16>(d, x.z, y.z, x.w, y.w, vl[c * NS + NS - 1][0], vl[c * NS + NS - 1][1]);
              ld_mma<BF16>(d, x.z, y.z, x.w, y.w, vh[c * NS + NS - 1][0], vh[c * NS + NS - 1][1]);
            }
          }
          tile[(2 * t) * 20 + g] = d[0] * if0;
          tile[(2 * t + 1) * 20 + g] = d[1] * if1;
          tile[(2 * t) * 20 + g + 8] = d[2] * if0;
          tile[(2 * t + 1) * 20 + g + 8] = d[3] * if1;
          __syncwarp();
          // lane = (token g, four output columns 4 t)
          const int j = ju + 4 * t;
          if (tok && j < a.N) {
            const float4 v = *reinterpret_cast<const float4*>(tile + g * 20 + 4 * t);
            T* op = out + row * a.ldo + j;
            if (yvec && j + 4 <= a.N) {
              const float2 y0 = Ty::unpack(yv[u].x), y1 = Ty::unpack(yv[u].y);
              *reinterpret_cast<uint2*>(op) =
                  make_uint2(Ty::pack(y0.x + v.x, y0.y + v.y), Ty::pack(y1.x + v.z, y1.y + v.w));
            } else {
              const T* yp = Y + row * a.ldy + j;
              const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (j + i < a.N)
                  op[i] = Ty::cvt((a.Y != nullptr ? to_f32(__ldcg(yp + i)) : 0.f) + e[i]);
            }
          }
          __syncwarp();
        }
      }
    }
    base += win.total;
  }
  if (!waited) cluster_wait();
  if (late) pdl_wait();
}

template <bool BF16, int RP>
gptq_status launch_decode(const LoraArgs& a, int64_t pieces, bool late, cudaStream_t s) {
  // rows of Y and out on 16-byte (2) or 8-byte (1) boundaries
  auto on = [&](int bytes) {
    return (uintptr_t)a.Y % bytes == 0 && (uintptr_t)a.out % bytes == 0 &&
           (a.Y == nullptr || a.ldy * 2 % bytes == 0) && a.ldo * 2 % bytes == 0;
  };
  const int yvec = on(16) ? 2 : on(8) ? 1 : 0;
  // a warp's transposing buffer may reach past its sums at rank 16
  constexpr size_t smem =
      sizeof(float) * (std::max(LD_WARPS * RP * LD_TT, LD_WARPS * LD_TT * 20) +
                       2 * LORA_CLUSTER * RP * LD_TT);
  if (smem_optin((const void*)lora_decode_kernel<BF16, RP>, smem) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  // as many clusters as fit the device at once; each takes piece after piece
  pieces = std::min<int64_t>(pieces, resident_clusters((const void*)lora_decode_kernel<BF16, RP>,
                                                       LORA_CLUSTER, LD_THREADS, smem));
  launch_cluster_pdl(lora_decode_kernel<BF16, RP>, dim3((unsigned)(pieces * LORA_CLUSTER)),
                     dim3(LD_THREADS), smem, LORA_CLUSTER, s, a, yvec, (int)late);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <bool BF16>
gptq_status decode_ranks(const LoraArgs& a, int64_t pieces, bool late, cudaStream_t s) {
  if (a.r <= 16) return launch_decode<BF16, 16>(a, pieces, late, s);
  if (a.r <= 32) return launch_decode<BF16, 32>(a, pieces, late, s);
  if (a.r <= 64) return launch_decode<BF16, 64>(a, pieces, late, s);
  return launch_decode<BF16, 128>(a, pieces, late, s);
}

bool rows16(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }

gptq_status lora_general(const LoraArgs& a, bool bf16, bool backward, cudaStream_t s) {
  if (bf16)
    launch_pdl(lora_general_kernel<true>, dim3((unsigned)a.m), dim3(256), 0, s, a, (int)backward);
  else
    launch_pdl(lora_general_kernel<false>, dim3((unsigned)a.m), dim3(256), 0, s, a, (int)backward);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace

// Batches of up to this many rows go to the decode kernel whole; in larger ones it
// takes the requests of up to LORA_SHORT rows.  (A tensor-core piece costs its 128 rows
// whatever it holds, 10 us and more through the exchange; three pieces of 8 rows less.)
// The tensor-core kernel's time hardly depends on the rows; the decode kernel's grows with the
// rank and by a step wherever its pieces need another CTA per SM (33 pieces of 8 rows each), and
// that step, not the layer's width or the number of adapters, is where the two meet.  Decode
// against tensor cores in us, 4096 -> 4096 and 4096 -> 11008, one request:
//   rank 16   512 rows 11.0 : 12.8 and 16.7 : 20.5,   536 rows 13.7 : 12.9 and 22.5 : 20.7
//   rank 32   512 rows 13.9 : 13.9 and 20.4 : 21.8,   544 rows 17.3 : 14.0 and 26.7 : 22.0
//   rank 64   256 rows 11.1 : 15.0 and 15.8 : 22.6,   288 rows 16.5 : 15.0 and 24.9 : 22.7
//   rank 128  192 rows 18.1 : 20.9 and 26.6 : 31.5,   256 rows 25.4 : 20.9 and 39.8 : 31.7
// Four requests on four adapters: within 0.5 of these, but for 4096 -> 11008 at rank 64, 256 rows
// 19.5 : 22.6, and at rank 128, 192 rows 36.1 : 33.6.  2048 -> 2048: within 1 us of each other
// at the rule's edges but for rank 128 (192 rows 14.5 : 17.0).
// Several requests may all be short, and then both kernels run, the one for nothing: at rank 16
// and 4096 -> 4096 the decode kernel alone against the two takes 16.1 : 20.7 us for 40 requests
// of 15 rows, 29.4 : 44.2 for 600 of one, 15.8 : 13.4 for 6 of 100 (the host does not know).
constexpr int lora_decode_rows(int r, int nreq) {
  return r <= 16 ? (nreq > 1 ? 704 : 512) : r <= 32 ? 512 : r <= 64 ? 256 : 192;
}
constexpr int LORA_SHORT = 24;

gptq_status lora_add_impl(LoraArgs a, bool bf16, cudaStream_t s) {
  a.min_len = 1;
  a.max_len = a.m;
  // the decode kernel reads rows of X, A and B in 16-byte pieces
  if (!rows16(a.X, a.ldx) || !rows16(a.P, a.K) || !rows16(a.Q, a.r))
    return lora_general(a, bf16, false, s);
  const bool tc = a.m > lora_decode_rows(a.r, a.nreq) && lora_tc_supported(a, false);
  if (tc) {
    // the long requests first, the short ones beside them on the SMs that are left (the lengths
    // are on the device: with several requests both kernels are launched, whatever they find)
    if (a.nreq > 1) a.min_len = LORA_SHORT + 1;
    const gptq_status st = lora_tc(a, bf16, false, s);
    if (st != GPTQ_OK || a.nreq == 1) return st;
    a.min_len = 1;
    a.max_len = LORA_SHORT;
  }
  // a piece that is not full is the last of its adapter (or of none) in its window
  const int64_t last = cdiv(a.nreq, LD_THREADS) * std::min(a.na + 1, LD_THREADS);
  const int64_t pieces =
      std::min<int64_t>(std::min<int64_t>(a.m, (int64_t)a.m / LD_TT + std::min<int64_t>(a.nreq, last)),
                        a.nreq * cdiv(std::min(a.max_len, a.m), LD_TT));
  return bf16 ? decode_ranks<true>(a, pieces, tc, s) : decode_ranks<false>(a, pieces, tc, s);
}

// U = scaling B^T dY and, where a.out is set, out = Y + A^T U.
gptq_status lora_low_impl(LoraArgs a, bool bf16, cudaStream_t s) {
  a.min_len = 1;
  a.max_len = a.m;
  if (lora_tc_supported(a, true)) return lora_tc(a, bf16, true, s);
  return lora_general(a, bf16, true, s);
}

}  // namespace gptq
