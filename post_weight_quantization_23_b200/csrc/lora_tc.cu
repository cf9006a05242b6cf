// The adapters on the 5th-generation tensor cores: the forward call for long
// requests and the pass of the backward call over dY (lora.cuh: LoraArgs).
//   forward:  V = s X A^T (reduction over k),   out = Y + V B^T;
//   backward: U = s dY B  (reduction over n),   out = dX + U A.
// One kernel for both: P is the operand of the reduction, Q of the expansion, and
// they only differ in which of their axes is contiguous (forward K-major, backward
// MN-major tiles of the same row-major A and B; no transposed copy is kept).
//
// Bound by HBM at common ranks (per row 2 (K + 2 N) bytes against 2 r (K + N)
// flops), so V never leaves the chip between the two products, and both run in one
// launch: a cluster of 8 CTAs takes 128 rows of one request.
//   1. CTA q reduces its eighth of K: TMA brings 128 x 64 tiles of X and P,
//      one thread issues kind::f16 MMAs D1[128 x RP] into TMEM.
//   2. Exchange through distributed shared memory: each CTA hands its partial sums
//      to the CTA that owns the row (16 rows each); the owner adds the eight, scales,
//      and hands V to all eight.  The sums run in a fixed order.  Two mbarriers with
//      cluster scope order it, so the producer warp runs on: the first tiles of
//      step 3 are in shared memory before V is.
//   3. CTA q takes every eighth 64-column tile of the output: V as hi + lo of the
//      16-bit type (f16: each row scaled by a power of two, taken back exactly) is
//      the A operand, D2[128 x 64] double-buffered in TMEM, the tile of Y arrives
//      by TMA beside Q, the sum is rounded once and stored row by row (a TMA
//      store would also write rows of the next request).
// Warps: 0 TMA, 1 MMA, 2..9 epilogue and exchange (two per TMEM lane quarter).
// Every wait is bounded; a CTA that gives up drains its copies and MMAs, frees
// TMEM and writes NaN over its part of out and V.
#include "lora.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

namespace gptq {

namespace {

constexpr int LT_M = 128, LT_K = 64, LT_N = 64;
constexpr int LT_EPI = 8;
constexpr int LT_THREADS = 64 + 32 * LT_EPI;
constexpr int LT_ROWS_OWNED = LT_M / LORA_CLUSTER;  // 16
constexpr int LT_TILE = LT_M * LT_K * 2;            // 16 KB of X or Y
constexpr int LT_TMEM = 256;                        // D1 in columns 0..127, D2 in 128..255

template <int RP>
struct LtShape {
  static constexpr int PQ = (RP > 64 ? RP : 64) * 128;  // bytes of a P or Q tile
  static constexpr int STAGE = LT_TILE + PQ;
  static constexpr int OPND = (RP > 32 ? RP : 32) * 512;  // V as hi | lo, 64-column atoms
  static constexpr int VBUF = RP * 512;                  // fp32 V of the 128 rows
  // stages: two CTAs per SM up to rank 32, one beyond
  static constexpr int S = RP <= 16 ? 3 : RP == 32 ? 3 : RP == 64 ? 6 : 3;
  static constexpr size_t SMEM = (size_t)S * STAGE + OPND + VBUF + 1024 + 512;
};

// float4 slot of columns 4 c4.. of a row of V (conflict-free for 8 rows at a time)
template <int RP>
__device__ __forceinline__ int lt_vslot(int row, int c4) {
  return row * (RP / 4) + (RP == 16 ? c4 ^ ((row >> 1) & 3) : c4 ^ (row & 7));
}

template <bool BF16, int RP, bool BWD>
__global__ void __launch_bounds__(LT_THREADS, RP <= 32 ? 2 : 1)
lora_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap pmap,
               const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap ymap,
               LoraArgs a, int ovec) {
  using Ty = LoraType<BF16>;
  using T = typename Ty::T;
  using Sh = LtShape<RP>;
  constexpr int S = Sh::S;
  extern __shared__ uint8_t lt_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)lt_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* opnd = smem + S * Sh::STAGE;
  float* red = (float*)opnd;                     // [8][16][RP] partial sums of this CTA's rows
  float* vbuf = (float*)(opnd + Sh::OPND);       // [128][RP]
  uint64_t* bars = (uint64_t*)(opnd + Sh::OPND + Sh::VBUF);
  uint64_t* full = bars;              // [S] tiles landed
  uint64_t* empty1 = bars + S;        // [S] reduction MMAs done with the slot
  uint64_t* empty2 = bars + 2 * S;    // [S] epilogue done with the slot
  uint64_t* d1_full = bars + 3 * S;
  uint64_t* x1 = d1_full + 1;         // partial sums of this CTA's rows arrived
  uint64_t* x2 = d1_full + 2;         // V of all rows arrived
  uint64_t* v_full = d1_full + 3;     // the V operand is written
  uint64_t* d2_full = d1_full + 4;    // [2]
  uint64_t* d2_empty = d1_full + 6;   // [2]
  uint64_t* done = d1_full + 8;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;  // copies that the producer started
  int* scan = (int*)(tmem_slot + 3);      // LT_THREADS / 32 + 3 ints

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty1[s], 1);
      tc::mbar_init(&empty2[s], LT_EPI);
    }
    tc::mbar_init(d1_full, 1);
    tc::mbar_init(x1, LORA_CLUSTER * 2);        // two warps of each CTA hold a row
    tc::mbar_init(x2, LORA_CLUSTER * LT_EPI);
    tc::mbar_init(v_full, LT_EPI);
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&d2_full[b], 1);
      tc::mbar_init(&d2_empty[b], LT_EPI);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&xmap);
    tc::prefetch_tensormap(&pmap);
    tc::prefetch_tensormap(&qmap);
    tc::prefetch_tensormap(&ymap);
  }
  pdl_wait();
  pdl_trigger();
  const LoraPiece pc =
      lora_find_piece<LT_THREADS>(a.starts, a.adapter, a.nreq, a.m, a.na, LT_M, a.min_len,
                                  a.max_len, (int)blockIdx.x / LORA_CLUSTER, scan);
  if (pc.cnt == 0) return;  // the same for the whole cluster
  T* out = (T*)a.out;
  const int n2 = (a.N + LT_N - 1) / LT_N;                    // output tiles
  const int nt = a.out == nullptr || n2 <= rank ? 0 : (n2 - rank + LORA_CLUSTER - 1) / LORA_CLUSTER;
  if (pc.a < 0) {
    for (int i = warp; i < pc.cnt; i += LT_THREADS / 32) {
      const int64_t row = pc.t0 + i;
      if (out != nullptr && a.Y != a.out)
        for (int j = rank * 32 + lane; j < a.N; j += LORA_CLUSTER * 32)
          out[row * a.ldo + j] = a.Y != nullptr ? ((const T*)a.Y)[row * a.ldy + j] : Ty::cvt(0.f);
      if (a.V != nullptr && i % LORA_CLUSTER == rank)
        for (int p = lane; p < a.r; p += 32) a.V[row * a.r + p] = 0.f;
    }
    return;
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, LT_TMEM);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  cluster_arrive();  // every CTA of the cluster runs and its barriers are set up
  cluster_wait();
  const uint32_t tmem = *tmem_slot;
  const int nk = (a.K + LT_K - 1) / LT_K;
  const int k0 = (int)((int64_t)nk * rank / LORA_CLUSTER);
  const int n1 = (int)((int64_t)nk * (rank + 1) / LORA_CLUSTER) - k0;  // reduction stages
  auto slot = [&](int s) { return smem + (size_t)s * Sh::STAGE; };
  constexpr uint32_t P_BYTES = BWD ? Sh::PQ : RP * 128;   // TMA boxes per stage
  constexpr uint32_t Q_BYTES = BWD ? RP * 128 : Sh::PQ;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (; it < n1 + nt; ++it) {
        const int s = it % S;
        if (it >= S) {  // the slot's last tenant: a reduction stage, or an output tile
          const int pr = it - S;
          if (pr < n1) {
            ok = tc::mbar_wait(&empty1[s], (uint32_t)(pr / S) & 1u, abort_flag, a.spin);
          } else {
            const int first = n1 > s ? (n1 - s + S - 1) / S : 0;  // round of the first output tile
            ok = tc::mbar_wait(&empty2[s], (uint32_t)(pr / S - first) & 1u, abort_flag, a.spin);
          }
          if (!ok) break;
        }
        uint8_t* sb = slot(s);
        if (it < n1) {
          const int c = (k0 + it) * LT_K;
          tc::mbar_arrive_expect_tx(&full[s], LT_TILE + P_BYTES);
          tc::tma_load_2d(sb, &xmap, &full[s], c, pc.t0);
          if (!BWD) {
            tc::tma_load_3d(sb + LT_TILE, &pmap, &full[s], c, 0, pc.a);
          } else {
#pragma unroll
            for (int p = 0; p < Sh::PQ / 8192; ++p)
              tc::tma_load_3d(sb + LT_TILE + p * 8192, &pmap, &full[s], p * 64, c, pc.a);
          }
        } else {
          const int j = (rank + LORA_CLUSTER * (it - n1)) * LT_N;
          tc::mbar_arrive_expect_tx(&full[s], (a.Y != nullptr ? LT_TILE : 0) + Q_BYTES);
          if (!BWD) {
#pragma unroll
            for (int p = 0; p < Sh::PQ / 8192; ++p)
              tc::tma_load_3d(sb + LT_TILE + p * 8192, &qmap, &full[s], p * 64, j, pc.a);
          } else {
            tc::tma_load_3d(sb + LT_TILE, &qmap, &full[s], j, 0, pc.a);
          }
          if (a.Y != nullptr) tc::tma_load_2d(sb, &ymap, &full[s], j, pc.t0);
        }
      }
      *issued = it;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id1 = tc::instr_desc(BF16 ? 1 : 0, LT_M, RP, 0, BWD ? 1 : 0);
      const uint32_t id2 = tc::instr_desc(BF16 ? 1 : 0, LT_M, LT_N, 0, BWD ? 1 : 0);
      const int steps = (a.r + 15) / 16;  // 16-wide steps of the rank that hold values
      bool ok = true;
      for (int it = 0; it < n1; ++it) {
        const int s = it % S;
        if (!tc::mbar_wait(&full[s], (uint32_t)(it / S) & 1u, abort_flag, a.spin)) { ok = false; break; }
        tc::tc_fence_after();
        const uint32_t sx = tc::smem_u32(slot(s)), sp = sx + LT_TILE;
#pragma unroll
        for (int kk = 0; kk < LT_K / 16; ++kk)
          tc::mma_f16_ss(tmem, tc::smem_desc_sw128(sx + kk * 32, 16, 1024),
                         BWD ? tc::smem_desc_sw128(sp + kk * 2048, 8192, 1024)
                             : tc::smem_desc_sw128(sp + kk * 32, 16, 1024),
                         id1, (it > 0 || kk > 0) ? 1u : 0u);
        tc::mma_commit(&empty1[s]);
      }
      tc::mma_commit(d1_full);
      if (ok && nt > 0 && tc::mbar_wait(v_full, 0, abort_flag, a.spin)) {
        tc::tc_fence_after();
        const uint32_t sv = tc::smem_u32(opnd);
        for (int i = 0; i < nt; ++i) {
          const int it = n1 + i, s = it % S, b = i & 1;
          if (i >= 2 && !tc::mbar_wait(&d2_empty[b], (uint32_t)(i / 2 - 1) & 1u, abort_flag, a.spin)) break;
          if (!tc::mbar_wait(&full[s], (uint32_t)(it / S) & 1u, abort_flag, a.spin)) break;
          tc::tc_fence_after();
          const uint32_t sq = tc::smem_u32(slot(s)) + LT_TILE;
          const uint32_t d2 = tmem + 128 + 64 * b;
          for (int h = 1; h >= 0; --h)  // the low halves first
            for (int p = 0; p < steps; ++p) {
              const int kc = h * RP + p * 16;
              tc::mma_f16_ss(
                  d2, tc::smem_desc_sw128(sv + (kc / 64) * LT_TILE + (kc % 64) * 2, 16, 1024),
                  BWD ? tc::smem_desc_sw128(sq + p * 2048, 8192, 1024)
                      : tc::smem_desc_sw128(sq + (p / 4) * 8192 + (p % 4) * 32, 16, 1024),
                  id2, (h == 0 || p > 0) ? 1u : 0u);
            }
          tc::mma_commit(&d2_full[b]);
        }
      }
      tc::mma_commit(done);  // fires once every MMA issued above has finished
      for (uint32_t i = 0; i < tc::kSpinLimit; ++i)
        if (tc::mbar_try_wait(done, 0)) break;
    }
  } else {
    const int ew = warp - 2, etid = threadIdx.x - 64;
    const int quarter = warp & 3, hf = ew >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    bool ok = tc::mbar_wait_warp(d1_full, 0, abort_flag, a.spin);
    if (ok) {
      // this CTA's partial sums of the row to the CTA that owns it
      tc::tc_fence_after();
      constexpr int HC = RP / 2, CW = HC < 32 ? HC : 32;  // columns of this warp, per load
      const uint32_t dst = cluster_map(
          tc::smem_u32(red) + (uint32_t)(((rank * LT_ROWS_OWNED) + row % LT_ROWS_OWNED) * RP) * 4,
          (uint32_t)(row / LT_ROWS_OWNED));
#pragma unroll
      for (int c = 0; c < HC; c += CW) {
        float v[CW];
        const uint32_t ta = tmem + lanes + (uint32_t)(hf * HC + c);
        if (CW == 8) tc::tmem_ld_32x32b_x8(ta, v);
        else if (CW == 16) tc::tmem_ld_32x32b_x16(ta, v);
        else tc::tmem_ld_32x32b_x32(ta, v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < CW; e += 4)
          cluster_st_f4(dst + (uint32_t)(hf * HC + c + e) * 4,
                        n1 > 0 ? make_float4(v[e], v[e + 1], v[e + 2], v[e + 3])
                               : make_float4(0.f, 0.f, 0.f, 0.f));
      }
      __syncwarp();
      if (lane < 2) cluster_mbar_arrive(cluster_map(tc::smem_u32(x1), (uint32_t)(2 * quarter + lane)));
      ok = cluster_mbar_wait_warp(x1, 0, abort_flag, a.spin);
    }
    if (ok) {
      // the rows that this CTA owns: add the eight parts, scale, hand V to all
      const float sc = a.scaling[pc.a];
      for (int e = etid; e < LT_ROWS_OWNED * RP / 4; e += 32 * LT_EPI) {
        float4 v = reinterpret_cast<const float4*>(red)[e];
#pragma unroll
        for (int c = 1; c < LORA_CLUSTER; ++c) {
          const float4 w = reinterpret_cast<const float4*>(red)[c * (LT_ROWS_OWNED * RP / 4) + e];
          v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        v.x *= sc, v.y *= sc, v.z *= sc, v.w *= sc;
        const int r = rank * LT_ROWS_OWNED + e / (RP / 4), c4 = e % (RP / 4);
        const uint32_t va = tc::smem_u32(vbuf) + 16u * (uint32_t)lt_vslot<RP>(r, c4);
#pragma unroll
        for (int c = 0; c < LORA_CLUSTER; ++c) cluster_st_f4(cluster_map(va, (uint32_t)c), v);
        if (a.V != nullptr && r < pc.cnt && 4 * c4 < a.r) {  // r % 8 == 0
          float* o = a.V + (int64_t)(pc.t0 + r) * a.r + 4 * c4;
          o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
        }
      }
      __syncwarp();
      if (lane < LORA_CLUSTER) cluster_mbar_arrive(cluster_map(tc::smem_u32(x2), (uint32_t)lane));
      ok = cluster_mbar_wait_warp(x2, 0, abort_flag, a.spin);
    }
    float back = 1.f;
    if (ok && nt > 0) {
      // V as the A operand: columns 0.. hold hi, RP.. hold lo (red is free now)
      const float4* vr = reinterpret_cast<const float4*>(vbuf);
      float f = 1.f;
      if (!BF16) {
        float top = 0.f;
#pragma unroll 8
        for (int c4 = 0; c4 < RP / 4; ++c4) {
          const float4 v = vr[lt_vslot<RP>(row, c4)];
          top = fmaxf(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))), top);
        }
        f = lora_row_factor(top);
        back = __fdiv_rn(1.f, f);  // a power of two: exact
      }
#pragma unroll
      for (int c8 = hf * (RP / 16); c8 < (hf + 1) * (RP / 16); ++c8) {
        const float4 v0 = vr[lt_vslot<RP>(row, 2 * c8)], v1 = vr[lt_vslot<RP>(row, 2 * c8 + 1)];
        uint4 hi, lo;
        lora_split<BF16>(v0.x * f, v0.y * f, hi.x, lo.x);
        lora_split<BF16>(v0.z * f, v0.w * f, hi.y, lo.y);
        lora_split<BF16>(v1.x * f, v1.y * f, hi.z, lo.z);
        lora_split<BF16>(v1.z * f, v1.w * f, hi.w, lo.w);
        const int kh = c8, kl = RP / 8 + c8;  // 16-byte chunks of the row
        *reinterpret_cast<uint4*>(opnd + (kh / 8) * LT_TILE + row * 128 +
                                  (((kh % 8) ^ (row & 7)) << 4)) = hi;
        *reinterpret_cast<uint4*>(opnd + (kl / 8) * LT_TILE + row * 128 +
                                  (((kl % 8) ^ (row & 7)) << 4)) = lo;
      }
      tc::fence_proxy_async_smem();  // the MMA reads what this thread wrote
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(v_full);
      for (int i = 0; i < nt; ++i) {
        const int it = n1 + i, s = it % S, b = i & 1;
        const int j0 = (rank + LORA_CLUSTER * i) * LT_N;
        if (!tc::mbar_wait_warp(&d2_full[b], (uint32_t)(i / 2) & 1u, abort_flag, a.spin)) break;
        tc::tc_fence_after();
        float v[32];
        tc::tmem_ld_32x32b_x32(tmem + lanes + (uint32_t)(128 + 64 * b + 32 * hf), v);
        tc::tmem_ld_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&d2_empty[b]);
        // the copies of the slot have landed (the MMA that read it waited for them); this
        // wait makes the tile of Y visible to this thread
        if (!tc::mbar_wait_warp(&full[s], (uint32_t)(it / S) & 1u, abort_flag, a.spin)) break;
        uint8_t* ys = slot(s);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4* p = reinterpret_cast<uint4*>(ys + row * 128 + (((4 * hf + c) ^ (row & 7)) << 4));
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          if (a.Y != nullptr) {
            const uint4 y = *p;
            w[0] = y.x, w[1] = y.y, w[2] = y.z, w[3] = y.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = a.Y != nullptr ? Ty::unpack(w[e]) : make_float2(0.f, 0.f);
            w[e] = Ty::pack(fmaf(v[8 * c + 2 * e], back, y.x), fmaf(v[8 * c + 2 * e + 1], back, y.y));
          }
          *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        // this warp's 32 rows x 32 columns, 64 contiguous bytes per row
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = quarter * 32 + 8 * q + lane / 4, c = 4 * hf + lane % 4;
          const int j = j0 + 8 * c;
          if (r >= pc.cnt || j >= a.N) continue;
          const uint4 w = *reinterpret_cast<const uint4*>(ys + r * 128 + ((c ^ (r & 7)) << 4));
          T* o = out + (int64_t)(pc.t0 + r) * a.ldo + j;
          if (ovec && j + 8 <= a.N) {
            *reinterpret_cast<uint4*>(o) = w;
          } else {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (j + e < a.N) {
                const unsigned short h = (unsigned short)(u[e / 2] >> (16 * (e % 2)));
                reinterpret_cast<unsigned short*>(o)[e] = h;
              }
          }
        }
        tc::fence_proxy_async_smem();  // the next copy into the slot comes after these accesses
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty2[s]);
      }
    }
  }
  __syncthreads();
  if (*abort_flag) {  // a wait gave up: this CTA's part of the outputs becomes NaN
    if (threadIdx.x == 0)  // the copies in flight land before the CTA exits
      for (int p = max(0, *issued - S); p < *issued; ++p)
        for (uint32_t i = 0; i < tc::kSpinLimit; ++i)
          if (tc::mbar_try_wait(&full[p % S], (uint32_t)(p / S) & 1u)) break;
    const T bad = Ty::cvt(__int_as_float(0x7fc00000));
    for (int i = warp; i < pc.cnt; i += LT_THREADS / 32) {
      const int64_t row = pc.t0 + i;
      for (int q = 0; q < nt; ++q)
        for (int j = (rank + LORA_CLUSTER * q) * LT_N + lane;
             j < min(a.N, (rank + LORA_CLUSTER * q + 1) * LT_N); j += 32)
          out[row * a.ldo + j] = bad;
      if (a.V != nullptr && i / LT_ROWS_OWNED == rank)
        for (int p = lane; p < a.r; p += 32) a.V[row * a.r + p] = __int_as_float(0x7fc00000);
    }
  }
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, LT_TMEM);
  cluster_arrive();  // no CTA leaves while another may still write to its shared memory
  cluster_wait();
}

// A tensor map over 16-bit values, 128-byte swizzle, 64 x rows boxes.
bool lt_map(CUtensorMap* map, bool bf16, int dims, const void* p, int64_t d0, int64_t d1,
            int64_t d2, int64_t ld1, int64_t ld2, int rows) {
  cuuint64_t gdim[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  cuuint64_t gstride[2] = {(cuuint64_t)ld1 * 2, (cuuint64_t)ld2 * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return tensormap_encoder()(
             map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims,
             const_cast<void*>(p), gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int RP, bool BWD>
gptq_status launch_tc(const LoraArgs& a, int64_t pieces, cudaStream_t s) {
  using Sh = LtShape<RP>;
  static_assert(Sh::SMEM <= 232448, "shared memory of a CTA");
  CUtensorMap xm, pm, qm, ym;
  const int64_t r = a.r, K = a.K, N = a.N, na = a.na;
  bool ok = lt_map(&xm, BF16, 2, a.X, K, a.m, 1, a.ldx, 0, LT_M);
  if (!BWD)
    ok = ok && lt_map(&pm, BF16, 3, a.P, K, r, na, K, r * K, RP) &&
         lt_map(&qm, BF16, 3, a.Q, r, N, na, r, r * N, LT_N);
  else
    ok = ok && lt_map(&pm, BF16, 3, a.P, r, K, na, r, r * K, LT_K) &&
         lt_map(&qm, BF16, 3, a.Q, N, r, na, N, r * N, RP);
  if (a.Y != nullptr && a.out != nullptr)
    ok = ok && lt_map(&ym, BF16, 2, a.Y, N, a.m, 1, a.ldy, 0, LT_M);
  else
    ym = xm;  // not read
  if (!ok || smem_optin((const void*)lora_tc_kernel<BF16, RP, BWD>, Sh::SMEM) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  const int ovec = (uintptr_t)a.out % 16 == 0 && a.ldo % 8 == 0;
  launch_cluster_pdl(lora_tc_kernel<BF16, RP, BWD>, dim3((unsigned)(pieces * LORA_CLUSTER)),
                     dim3(LT_THREADS), Sh::SMEM, LORA_CLUSTER, s, xm, pm, qm, ym, a, ovec);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <bool BF16, bool BWD>
gptq_status tc_ranks(const LoraArgs& a, int64_t pieces, cudaStream_t s) {
  if (a.r <= 16) return launch_tc<BF16, 16, BWD>(a, pieces, s);
  if (a.r <= 32) return launch_tc<BF16, 32, BWD>(a, pieces, s);
  if (a.r <= 64) return launch_tc<BF16, 64, BWD>(a, pieces, s);
  return launch_tc<BF16, 128, BWD>(a, pieces, s);
}

bool rows16(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }

}  // namespace

// Rows on 16-byte boundaries for everything that TMA reads.  A matrix of one
// rank row needs no wider box than TMA's rules allow: r, K and N only have to be
// multiples of 8 where they are a leading dimension.
bool lora_tc_supported(const LoraArgs& a, bool backward) {
  return rows16(a.X, a.ldx) && (a.Y == nullptr || a.out == nullptr || rows16(a.Y, a.ldy)) &&
         rows16(a.P, backward ? a.r : a.K) && rows16(a.Q, backward ? a.N : a.r) &&
         tensormap_encoder() != nullptr;
}

gptq_status lora_tc(const LoraArgs& a, bool bf16, bool backward, cudaStream_t s) {
  // pieces of the requests that are long enough: each fills its last piece at most partly
  const int64_t pieces =
      std::min<int64_t>(a.m, (int64_t)a.m / LT_M + std::min<int64_t>(a.nreq, a.m / a.min_len));
  if (bf16) return backward ? tc_ranks<true, true>(a, pieces, s) : tc_ranks<true, false>(a, pieces, s);
  return backward ? tc_ranks<false, true>(a, pieces, s) : tc_ranks<false, false>(a, pieces, s);
}

}  // namespace gptq
