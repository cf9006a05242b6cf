// The gradient of the inference product with respect to its input
// (gptq_gemm_dgrad), read straight from the packed codes:
//   dX[t, c] = sum_j dY[t, j] scale[j, g(c)] (code[j, c] - zero[j, g(c)]).
// The reduction runs over the rows of W, the output over its columns: the other
// way round than gptq_gemm over the same packed words.
//
// Bound by the tensor cores from a few hundred tokens on (2 m n k flops against
// n k / 2 + 2 m (n + k) bytes).  Tensor-core kernel: one CTA per MT * 128 columns x N
// tokens, the rows of W in stages of 64:
//   warp 0       TMA: the packed words of the 64 rows (MT * 64 bytes each, swizzled
//                so that 8 rows read without bank conflicts) and the N x 64 box of dY;
//   warps 2..    groups of four, one per stage of the ring (a slot belongs to one group,
//                which sees every phase of its barrier): a thread turns runs of 32 codes
//                of a row into weights, two at a time.  A byte permute and a mask
//                put codes c_2i, c_2i+1 into the mantissas of a pair M + c (M = 1024
//                for f16, 128 for bf16), M + zero is subtracted: c - zero, exactly.
//                The fp32 scale is split into two 16-bit parts, and
//                w = fl(d * s_hi + fl(d * s_lo)): the product with the fp32 scale
//                rounded once (f16 2^-11, bf16 2^-8), where a scale rounded first
//                would add its own error.  The codes of a word are neighbours along
//                the output axis, so the weights are written as an MN-major operand,
//                16 bytes per word;
//   warp 1       kind::f16 MMAs D[128 x N] += W^T dY^T per 128 columns, fp32 in TMEM.
// The same warps are the epilogue (TMEM lane = column, TMEM column = token).
// The weights' rounding is the operator's largest error, about that of the rounded result;
// two MMAs on a weight of two parts would take it away and double the tensor work.
// f16's range: all weights of a group's column carry one power of two, taken back in the
// epilogue (it has to be common to everything that is summed).  2^8 suits groups whose
// largest scale is 6.1e-5 to 1.8; the dequantizing warps note the largest scale on the way,
// and a CTA that finds another kind goes over its rows again with the power that brings it
// to [2^7, 2^8) (no lower part of a scale, and with |code - zero| <= 142 no weight, leaves
// the type).  A pass over the scales first would cost every call some 2 us at 4096 rows (a line
// each, and the L1 looks up one a cycle).  So |w error| <= u |w| + (|code - zero| + 2) 2^-19 of the group's
// largest scale, u = 2^-11, whatever the sizes of the scales.
// MT = 2 halves the stages' dY traffic, and where the tiles leave SMs idle the CTAs of a
// cluster share a tile's rows of W (every split-th stage each) and add up through
// distributed shared memory in a fixed order; launch_shape picks MT, N and the split.
// Every wait is bounded; a CTA that gives up drains its copies and MMAs, frees TMEM and
// writes NaN over its outputs.
// 22016 x 4096, 4096 tokens, bf16: 605 us, 1220 TFLOP/s, 0.71 of the measured bf16 burst (690 us
// in a long run, under the power cap), f16 625; 4096 x 4096, 512 tokens: 30 us (f16 30.5, and
// 64 with scales of 1e-6, which take the second pass).
#include "cluster.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

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

// ---- tensor-core kernel ------------------------------------------------------------

constexpr int DT_K = 64;                    // rows of W per stage
constexpr int DT_GROUP = 4;                 // warps of a dequantizing group
constexpr int DT_NMAX = 256;
constexpr int DT_LD = 132;                  // floats of a token's row of staged sums
// zeros up to this magnitude are exact in 128 + zero and code - zero of bf16; a group that holds
// another one becomes NaN
constexpr int DT_ZERO = 127;
// f16: the power of two that weights carry, and the largest scales of a group that it suits
constexpr float DT_FACTOR = 256.f, DT_TOP_MIN = 0x1p-14f, DT_TOP_MAX = 1.8f;  // 1.8 142 256 < 65504

template <int MT>
struct DtShape {
  static constexpr int A = MT * 128 * DT_K * 2;   // weights
  static constexpr int B = DT_NMAX * DT_K * 2;    // dY
  static constexpr int P = MT * 128 * DT_K / 2;   // packed words
  static constexpr int STAGE = A + B + P;
  static constexpr int S = MT == 2 ? 3 : 4;     // stages, and dequantizing groups
  static constexpr int THREADS = 64 + 32 * DT_GROUP * S;
  // the grids of a group's stage: 64 rows x up to one group per 32 columns
  static constexpr int GRID = MT * 4 * DT_K * 6;
  static constexpr size_t SMEM = (size_t)S * (STAGE + GRID) + 256;
  static_assert(SMEM <= 232448 && STAGE % 1024 == 0, "shared memory of a CTA");
};

struct DtArgs {
  const float* scales;
  const int32_t* zeros;
  void* dX;
  int64_t lddx;
  int n, m, k, G, ngroups;
  int N;          // tokens of a tile
  int split;      // CTAs that share a tile (MT = 1)
  uint32_t spin;  // polls before a pipeline wait gives up
};

template <bool BF16> struct DtType;
template <> struct DtType<false> {
  using T = __half;
  using T2 = __half2;
  static constexpr uint32_t MAGIC = 0x64006400u;  // 1024 in both halves: ulp 1 on [1024, 2048)
  static constexpr float BASE = 1024.f;
  __device__ static T one(float v) { return __float2half_rn(v); }
  __device__ static T2 both(T v) { return __half2half2(v); }
  __device__ static T2 pair(float v) { return __float2half2_rn(v); }
  __device__ static float back(T2 v) { return __low2float(v); }
};
template <> struct DtType<true> {
  using T = __nv_bfloat16;
  using T2 = __nv_bfloat162;
  static constexpr uint32_t MAGIC = 0x43004300u;  // 128 in both halves: ulp 1 on [128, 256)
  static constexpr float BASE = 128.f;
  __device__ static T one(float v) { return __float2bfloat16_rn(v); }
  __device__ static T2 both(T v) { return __bfloat162bfloat162(v); }
  __device__ static T2 pair(float v) { return __float2bfloat162_rn(v); }
  __device__ static float back(T2 v) { return __low2float(v); }
};

// The power of two that brings a group's largest scale to [2^7, 2^8); it and its inverse are
// normal numbers.
__device__ __forceinline__ float dt_factor(float top) {
  const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -119), 126);
  return __uint_as_float((uint32_t)(127 + 7 - e) << 23);
}

// 1 / f of a power of two: the exponents add up to 254.
__device__ __forceinline__ float dt_inverse(float f) {
  return __uint_as_float((254u << 23) - __float_as_uint(f));
}

template <bool BF16, int MT, bool SPLIT>
__global__ void __launch_bounds__(DtShape<MT>::THREADS, 1)
dgrad_tc_kernel(const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap pmap,
                DtArgs a) {
  using Ty = DtType<BF16>;
  using T2 = typename Ty::T2;
  using Sh = DtShape<MT>;
  constexpr int S = Sh::S;
  extern __shared__ __align__(1024) uint8_t dt_smem[];
  uint8_t* grids = dt_smem + S * Sh::STAGE;
  uint64_t* bars = (uint64_t*)(grids + S * Sh::GRID);
  uint64_t* full = bars;            // [S] packed words and dY landed
  uint64_t* ready = bars + S;       // [S] the weights are written
  uint64_t* empty = bars + 2 * S;   // [S] the stage's MMAs are done
  uint64_t* done = bars + 3 * S;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;
  // f16, per group of the tile: the largest finite scale (its bits), the factor
  uint32_t* tops = (uint32_t*)(bars + 16);
  float* facs = (float*)(tops + 4 * MT);
  static_assert((3 * S + 1) * 8 + 12 <= 128 && 128 + 8 * 4 * MT <= 256, "fits");

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = SPLIT ? a.split : 1, part = SPLIT ? (int)blockIdx.x % split : 0;
  const int c0 = (int)blockIdx.x / split * (MT * 128), t0 = blockIdx.y * a.N;
  // stages of this CTA: part, part + split, ..
  const int ns = ((a.n + DT_K - 1) / DT_K - part + split - 1) / split;
  auto first_row = [&](int i) { return (part + i * split) * DT_K; };
  const int g0 = c0 / a.G, ng = (min(c0 + MT * 128, a.k) - 1) / a.G - g0 + 1;  // groups of the tile
  auto stage = [&](int it) { return dt_smem + (size_t)(it % S) * Sh::STAGE; };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&ready[s], DT_GROUP);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    *issued = 0;
    for (int g = 0; g < 4 * MT; ++g) tops[g] = 0u, facs[g] = BF16 ? 1.f : DT_FACTOR;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&ymap);
    tc::prefetch_tensormap(&pmap);
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 1) tc::tmem_alloc(tmem_slot, MT * 256);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // stages of earlier passes: a second one follows where the factors did not suit (f16)
  int base = 0;
  for (;;) {
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t bytes = Sh::P + (uint32_t)a.N * DT_K * 2;
        for (int i = 0; i < ns; ++i) {
          const int it = base + i, s = it % S;
          if (it >= S && !tc::mbar_wait(&empty[s], (uint32_t)(it / S - 1) & 1u, abort_flag, a.spin))
            break;
          uint8_t* sb = stage(it);
          tc::mbar_arrive_expect_tx(&full[s], bytes);
          tc::tma_load_2d(sb + Sh::A + Sh::B, &pmap, &full[s], c0 / 8, first_row(i));
          tc::tma_load_2d(sb + Sh::A, &ymap, &full[s], first_row(i), t0);
          *issued = it + 1;
        }
      }
    } else if (warp == 1) {
      if (tc::elect_one()) {
        const uint32_t id = tc::instr_desc(BF16 ? 1 : 0, 128, a.N, 1, 0);  // W MN-major, dY K-major
        const uint32_t s0 = tc::smem_u32(dt_smem);
        const uint64_t dw = tc::smem_desc_sw128(s0, 8192, 1024);
        const uint64_t dy = tc::smem_desc_sw128(s0 + Sh::A, 16, 1024);
        int s = base % S;
        uint32_t ph = (uint32_t)(base / S) & 1u;
        for (int i = 0; i < ns; ++i) {
          // the dequantizing warps waited for the copies before they arrived
          if (!tc::mbar_wait(&ready[s], ph, abort_flag, a.spin)) break;
          tc::tc_fence_after();
          const uint64_t w = tc::desc_add(dw, (uint32_t)s * Sh::STAGE);
          const uint64_t y = tc::desc_add(dy, (uint32_t)s * Sh::STAGE);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int kk = 0; kk < DT_K / 16; ++kk)
              tc::mma_f16_ss(tmem + 256 * mt, tc::desc_add(w, mt * 16384 + kk * 2048),
                             tc::desc_add(y, kk * 32), id, kk > 0 ? 1u : (uint32_t)(i > 0));
          tc::mma_commit(&empty[s]);
          if (++s == S) s = 0, ph ^= 1u;
        }
      }
    } else {
      const int grp = (warp - 2) / DT_GROUP, gw = (warp - 2) % DT_GROUP;
      // quads (32 columns) MT gw .. of rows lane and lane + 32; neighbouring lanes are
      // neighbouring rows
      constexpr int R = 2 * MT;
      // The grids: thread = (row, every second group of the tile) of the group's next stage,
      // requested a stage of the group ahead and handed round through shared memory.  (Each
      // thread fetching those of its own runs cost four times the scattered loads: 32 rows
      // are 32 lines, and the L1 looks up one a cycle.)
      const int gt = gw * 32 + lane, grow = gt % DT_K, ghalf = gt / DT_K;
      float* gsc = (float*)(grids + grp * Sh::GRID);                              // [4 MT][64]
      typename Ty::T* gze = (typename Ty::T*)(grids + grp * Sh::GRID + MT * 4 * DT_K * 4);
      float fs[R];
      int fz[R];
      float fac[R];
      uint32_t top[R];
#pragma unroll
      for (int i = 0; i < R; ++i) fac[i] = facs[ghalf + 2 * i], top[i] = 0u;
      auto fetch = [&](int st) {
        const int j = first_row(st) + grow;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const bool ok = ghalf + 2 * i < ng && st < ns && j < a.n;
          const int64_t at = (int64_t)j * a.ngroups + g0 + ghalf + 2 * i;
          fs[i] = ok ? __ldg(a.scales + at) : 0.f;
          fz[i] = ok ? __ldg(a.zeros + at) : 0;
        }
      };
      int gq[MT];  // the group slot of each quad
#pragma unroll
      for (int q = 0; q < MT; ++q) gq[q] = min(c0 + 32 * (MT * gw + q), a.k - 1) / a.G - g0;
      int st = (grp - base % S + S) % S;  // the group's stages of this pass
      fetch(st);
      bool gave_up = false;
      for (; st < ns; st += S) {
        const int it = base + st, s = it % S;
        // the last stage's grids are read; a give-up ends the loop of the whole group
        if (tc::named_bar_any(1 + grp, 32 * DT_GROUP, gave_up)) break;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (ghalf + 2 * i < ng) {
            if (!BF16) {
              const uint32_t t = __float_as_uint(fs[i]) & 0x7fffffffu;
              if (t < 0x7f800000u) top[i] = max(top[i], t);
            }
            const bool fits = fz[i] >= -DT_ZERO && fz[i] <= DT_ZERO;
            gsc[(ghalf + 2 * i) * DT_K + grow] =
                !fits ? __int_as_float(0x7fc00000) : BF16 ? fs[i] : fs[i] * fac[i];
            gze[(ghalf + 2 * i) * DT_K + grow] = Ty::one(Ty::BASE + (float)fz[i]);  // exact where it fits
          }
        tc::named_bar_sync(1 + grp, 32 * DT_GROUP);
        fetch(st + S);
        T2 hi[R], lo[R], zz[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int at = gq[r / 2] * DT_K + lane + 32 * (r & 1);
          const float sc = gsc[at];
          hi[r] = Ty::pair(sc);
          const float h = Ty::back(hi[r]);
          lo[r] = Ty::pair(isfinite(h) ? sc - h : 0.f);  // an infinity stays one
          zz[r] = Ty::both(gze[at]);
        }
        if (!tc::mbar_wait_warp(&full[s], (uint32_t)(it / S) & 1u, abort_flag, a.spin)) {
          gave_up = true;
          continue;
        }
        uint8_t* sb = stage(it);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int j = lane + 32 * (r & 1), quad = MT * gw + r / 2;
          const int pos = MT == 2 ? j * 128 + ((quad ^ (j & 7)) << 4)          // 128-byte swizzle
                                  : j * 64 + ((quad ^ ((j >> 1) & 3)) << 4);   // 64-byte swizzle
          const uint4 pw = *reinterpret_cast<const uint4*>(sb + Sh::A + Sh::B + pos);
          const uint32_t words[4] = {pw.x, pw.y, pw.z, pw.w};
          uint8_t* row = sb + (quad / 2) * 8192 + j * 128;  // 64-column atoms
#pragma unroll
          for (int wi = 0; wi < 4; ++wi) {
            const uint32_t w = words[wi], w4 = w >> 4;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // byte i of w (c_2i low) into half 0, byte i of w >> 4 (c_2i+1 low) into half 1
              const uint32_t v =
                  __byte_perm(w, w4, (uint32_t)(i | (i << 4) | ((4 + i) << 8) | (i << 12)));
              const uint32_t h = (v & 0x000F000Fu) | Ty::MAGIC;               // M + c, exact
              const T2 d = __hsub2(*reinterpret_cast<const T2*>(&h), zz[r]);  // c - zero, exact
              const T2 x = __hfma2(d, hi[r], __hmul2(d, lo[r]));
              o[i] = *reinterpret_cast<const uint32_t*>(&x);
            }
            *reinterpret_cast<uint4*>(row + ((((quad % 2) * 4 + wi) ^ (j & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        tc::fence_proxy_async_smem();  // the MMA reads what this thread wrote
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ready[s]);
      }
      if (!BF16) {
#pragma unroll
        for (int i = 0; i < R; ++i) {  // ghalf is the warp's
          const uint32_t t = __reduce_max_sync(0xffffffffu, top[i]);
          if (lane == 0 && t != 0u) atomicMax(&tops[ghalf + 2 * i], t);
        }
      }
    }
    __syncthreads();
    if (BF16 || base > 0 || *abort_flag) break;
    bool again = false;
    for (int g = 0; g < ng; ++g) {
      const float t = __uint_as_float(tops[g]);
      again |= t > 0.f && !(t >= DT_TOP_MIN && t <= DT_TOP_MAX);
    }
    if (!again) break;
    if (threadIdx.x < ng && tops[threadIdx.x] != 0u)
      facs[threadIdx.x] = dt_factor(__uint_as_float(tops[threadIdx.x]));
    __syncthreads();
    base = ns;
  }
  if (warp == 1) {
    if (tc::elect_one()) tc::mma_commit(done);  // the lane that issued them: fires when all are over
  }
  // (the barrier comes before this wait: the idle lanes of the copying and the issuing warp,
  // polling beside their one busy lane, slowed the kernel by a seventh)
  // all MMAs done (shared memory is free for the sums), all copies landed
  const bool finished = tc::mbar_wait_warp(done, 0, abort_flag, tc::kSpinLimit);
  if (*abort_flag && threadIdx.x == 0)
    for (int p = max(0, *issued - S); p < *issued; ++p)
      for (uint32_t i = 0; i < tc::kSpinLimit; ++i)
        if (tc::mbar_try_wait(&full[p % S], (uint32_t)(p / S) & 1u)) break;
  __syncthreads();
  tc::tc_fence_after();
  const bool ok = finished && !*abort_flag;
  float* sums = (float*)dt_smem;  // [N][DT_LD], split > 1
  if (warp >= 2) {
    // epilogue: this warp's lane quarter of the 128-column tiles, its share of the tokens
    const int quarter = warp & 3, nch = (a.N + 31) / 32;  // 32-token chunks of a tile
    for (int x = (warp - 2) / 4; x < MT * nch; x += S) {
      const int mt = x / nch, q = x % nch * 32;
      const int c = c0 + mt * 128 + quarter * 32 + lane;
      typename Ty::T* out = reinterpret_cast<typename Ty::T*>(a.dX) + c;
      // one over the power of two that this column's weights carry
      const float inv = BF16 ? 1.f : dt_inverse(facs[min(c - lane, a.k - 1) / a.G - g0]);
      float v[32];
      tc::tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(256 * mt + q), v);
      tc::tmem_ld_wait();
      if (!SPLIT) {
#pragma unroll
        for (int t = 0; t < 32; ++t)
          if (c < a.k && q + t < a.N && t0 + q + t < a.m)
            out[(int64_t)(t0 + q + t) * a.lddx] =
                dg_out<typename Ty::T>(ok ? v[t] * inv : __int_as_float(0x7fc00000));
      } else {
#pragma unroll
        for (int t = 0; t < 32; ++t)
          if (q + t < a.N)
            sums[(q + t) * DT_LD + quarter * 32 + lane] =
                ok ? v[t] * inv : __int_as_float(0x7fc00000);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (SPLIT) {
    cluster_arrive();
    cluster_wait();
    // this CTA's share of the tokens, summed over the cluster
    const int per = (a.N + split - 1) / split;
    for (int e = threadIdx.x; e < per * 32; e += Sh::THREADS) {
      const int t = part * per + e / 32, c4 = e % 32;
      if (t >= a.N || t0 + t >= a.m) continue;
      const uint32_t at = tc::smem_u32(sums + t * DT_LD + 4 * c4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < split; ++q) {
        const float4 w = cluster_ld_f4(cluster_map(at, (uint32_t)q));
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      const float f[4] = {v.x, v.y, v.z, v.w};
      typename Ty::T* out = reinterpret_cast<typename Ty::T*>(a.dX) + (int64_t)(t0 + t) * a.lddx;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + 4 * c4 + i < a.k) out[c0 + 4 * c4 + i] = dg_out<typename Ty::T>(f[i]);
    }
    cluster_arrive();  // no CTA leaves while another reads its sums
    cluster_wait();
  }
  if (warp == 1) tc::tmem_dealloc(tmem, MT * 256);
}

bool dgrad_tc_supported(const void* dY, int64_t lddy, const int32_t* qw, int bits, int64_t k,
                        int64_t n, int G, bool has_gidx) {
  return bits == 4 && !has_gidx && n > 0 && (G >= k || G % 32 == 0) && (uintptr_t)dY % 16 == 0 &&
         lddy % 8 == 0 && (uintptr_t)qw % 16 == 0 && tensormap_encoder() != nullptr;
}

// Columns (MT * 128) and tokens (N, a multiple of 16) of a tile: the pair whose waves
// over the SMs cost least.  A stage costs its MMAs (2 MT N cycles) or, more often, its
// shared-memory traffic at 128 bytes a cycle: copies N 128 + MT 4096, weights MT (4096 +
// 16384) read and written, operands MT (16384 + N 128) read by the MMAs.  Measured
// (22016 x 4096, 4096 tokens): 2 x 128 columns with 240 tokens 659 us, 256 tokens 678,
// 128 columns with 240 tokens 746.
// The join of a split tile is counted as 8000 + 24 N cycles.
void launch_shape(int64_t m, int64_t n, int64_t k, int& MT, int& N, int& split) {
  const int64_t sms = sm_count(), ns = cdiv(n, DT_K);
  int64_t best = 0;
  for (int mt = 1; mt <= 2; ++mt)
    for (int nn = 16; nn <= DT_NMAX; nn += 16) {
      const int64_t tiles = cdiv(k, mt * 128) * cdiv(m, nn);
      const int64_t stage = std::max(2 * mt * nn, nn * (1 + mt) + 320 * mt);
      for (int sp = 1; sp <= (mt == 1 ? 8 : 1) && sp * 4 <= std::max<int64_t>(ns, 4); sp *= 2) {
        if (sp > 1 && tiles * sp > sms) break;
        const int64_t cost = cdiv(tiles * sp, sms) * cdiv(ns, sp) * stage + (sp > 1 ? 8000 + 24 * nn : 0);
        if (best == 0 || cost < best) best = cost, MT = mt, N = nn, split = sp;
      }
    }
}

template <bool BF16, int MT, bool SPLIT>
gptq_status launch_dgrad(const void* dY, int64_t lddy, const int32_t* qw, DtArgs a, cudaStream_t s) {
  using Sh = DtShape<MT>;
  EncodeTiledFn enc = tensormap_encoder();
  CUtensorMap ymap, pmap;
  cuuint32_t es[2] = {1, 1};
  {
    cuuint64_t gdim[2] = {(cuuint64_t)a.n, (cuuint64_t)a.m};
    cuuint64_t gstride[1] = {(cuuint64_t)lddy * 2};
    cuuint32_t box[2] = {DT_K, (cuuint32_t)a.N};
    if (enc(&ymap, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(dY), gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return GPTQ_ERR_CUDA;
  }
  {
    cuuint64_t gdim[2] = {(cuuint64_t)(a.k / 8), (cuuint64_t)a.n};
    cuuint64_t gstride[1] = {(cuuint64_t)(a.k / 8) * 4};
    cuuint32_t box[2] = {MT * 16, DT_K};
    if (enc(&pmap, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<int32_t*>(qw), gdim, gstride, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            MT == 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return GPTQ_ERR_CUDA;
  }
  if (smem_optin((const void*)dgrad_tc_kernel<BF16, MT, SPLIT>, Sh::SMEM) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  static_assert(MT == 2 || DT_NMAX * DT_LD * 4 <= Sh::S * Sh::STAGE, "a split tile's sums fit");
  const dim3 grid((unsigned)(cdiv(a.k, MT * 128) * a.split), (unsigned)cdiv(a.m, a.N));
  if (!SPLIT)
    launch_pdl(dgrad_tc_kernel<BF16, MT, SPLIT>, grid, dim3(Sh::THREADS), Sh::SMEM, s, ymap, pmap, a);
  else
    launch_cluster_pdl(dgrad_tc_kernel<BF16, MT, SPLIT>, grid, dim3(Sh::THREADS), Sh::SMEM, a.split, s, ymap,
                       pmap, a);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace

gptq_status dgrad_impl(const void* dY, gptq_dtype dt, int64_t m, int64_t n, int64_t lddy,
                       const int32_t* qw, const float* scales, const int32_t* zeros,
                       const int32_t* g_idx, int64_t k, int bits, int group_size, int64_t ngroups,
                       void* dX, int64_t lddx, cudaStream_t s) {
  const int G = group_size == -1 ? (int)k : group_size;
  if (dgrad_tc_supported(dY, lddy, qw, bits, k, n, G, g_idx != nullptr)) {
    DtArgs a;
    a.scales = scales, a.zeros = zeros, a.dX = dX, a.lddx = lddx;
    a.n = (int)n, a.m = (int)m, a.k = (int)k, a.G = G, a.ngroups = (int)ngroups;
    a.spin = wait_limit();
    int MT = 1;
    launch_shape(m, n, k, MT, a.N, a.split);
    if (dt == GPTQ_BF16)
      return MT == 2       ? launch_dgrad<true, 2, false>(dY, lddy, qw, a, s)
             : a.split > 1 ? launch_dgrad<true, 1, true>(dY, lddy, qw, a, s)
                           : launch_dgrad<true, 1, false>(dY, lddy, qw, a, s);
    return MT == 2       ? launch_dgrad<false, 2, false>(dY, lddy, qw, a, s)
           : a.split > 1 ? launch_dgrad<false, 1, true>(dY, lddy, qw, a, s)
                         : launch_dgrad<false, 1, false>(dY, lddy, qw, a, s);
  }
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
