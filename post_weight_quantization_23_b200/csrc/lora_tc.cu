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
// launch: a cluster of CS CTAs takes 128 rows of one request (a piece) after another.
//   1. CTA q reduces every CS-th 64-column tile of K (together the cluster reads
//      whole runs of a row): TMA brings 128 x 64 tiles of X and P, one thread
//      issues kind::f16 MMAs D1[128 x RP] into TMEM.
//   2. Exchange through distributed shared memory: each CTA hands its partial sums
//      to the CTA that owns the row (128 / CS rows each, in eights); the owner adds them in a
//      fixed order, scales, and hands V to all.  V as hi + lo of the 16-bit type
//      (f16: each row scaled by a power of two, taken back exactly; the MMA takes A and B of
//      one type, and two parts leave u^2 of V, far below the u of the rounded result, where
//      one would add u) becomes the A operand of
//   3. CTA q takes every CS-th 64-column tile of the output, D2[128 x 64] in a TMEM
//      buffer per epilogue group; the tile of Y arrives by TMA beside Q, the sum is rounded once
//      and stored row by row (a TMA store would also write rows of the next request).
// A CTA has an SM to itself (every kernel that uses tcgen05 gets one CTA per SM on
// this driver, whatever its registers and shared memory), so the overlap is inside:
// one ring of stages feeds both products, step 1 of the next piece runs ahead of step
// 3 of this one, and the exchange has warps of its own (up to rank 64; rank 128
// leaves no shared memory for the second operand and takes the steps in turn).
// Warps: 0 TMA, 1 MMA, 2..5 exchange, 6..17 epilogue (three groups of four, tile by tile
// in turn, a TMEM buffer each).
// 8192 tokens, rank 64, 4096 -> 11008: 89 us in a replayed graph, the caller's zero-fill of V
// included (432 MB, 4.8 TB/s, 0.75 of measured HBM; 96 us through the Python call): its
// two rounds of output tiles run at 5.8 TB/s, the first reduction and exchange (22 us) before
// them are half covered by the second reduction.  Two epilogue groups instead of three: 83
// -> 87 us for 3001 ragged f16 tokens at rank 8; asking for tiles in L2 ahead changed nothing.
// Every wait is bounded; a cluster in which one gives up drains its copies
// and MMAs, frees TMEM and writes NaN over its part of out and V.
#include "lora.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

namespace gptq {

namespace {

constexpr int LT_M = 128, LT_K = 64, LT_N = 64;
constexpr int LT_XCH = 4, LT_GROUPS = 3;        // exchange warps, epilogue groups of four
constexpr int LT_EPI = 4 * LT_GROUPS;
constexpr int LT_THREADS = 64 + 32 * (LT_XCH + LT_EPI);
constexpr int LT_TILE = LT_M * LT_K * 2;        // 16 KB of X or Y
constexpr int LT_TMEM = 512;                    // D1: 2 x 128 columns, D2: a group each 64 from 256
constexpr int LT_TABLE = 32;                    // pieces of a cluster looked up at a time

template <int RP, int CS>
struct LtShape {
  // rows whose sums a CTA forms, in whole swizzle periods: the last owner may have fewer
  static constexpr int OWNED = (LT_M / 8 + CS - 1) / CS * 8;
  static constexpr bool PIPE = RP <= 64;                // step 1 runs a piece ahead
  static constexpr int PQ = (RP > 64 ? RP : 64) * 128;  // bytes of a P or Q tile
  static constexpr int STAGE = LT_TILE + PQ;
  static constexpr int OPND = (RP > 32 ? RP : 32) * 512;  // V as hi | lo, 64-column atoms
  static constexpr int VBUF = RP * 512;                  // fp32, 128 rows
  static constexpr int RED = PIPE ? CS * OWNED * RP * 4 : 0;  // else in the operand's place
  static_assert(PIPE || CS * OWNED * RP * 4 <= OPND, "fits");
  static constexpr int S = RP == 16 ? (RED > VBUF ? 7 : 8) : RP == 32 ? 7 : RP == 64 ? 5 : 3;
  static constexpr size_t SMEM = (size_t)S * STAGE + OPND + VBUF + RED + 2304;
};

// float4 slot of columns 4 c4.. of a row of V (conflict-free for 8 rows at a time)
template <int RP>
__device__ __forceinline__ int lt_vslot(int row, int c4) {
  return row * (RP / 4) + (RP == 16 ? c4 ^ ((row >> 1) & 3) : c4 ^ (row & 7));
}

template <bool BF16, int RP, bool BWD, int CS>
__global__ void __launch_bounds__(LT_THREADS, 1)
lora_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap pmap,
               const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap ymap,
               LoraArgs a, int ovec) {
  using Ty = LoraType<BF16>;
  using T = typename Ty::T;
  using Sh = LtShape<RP, CS>;
  constexpr int S = Sh::S;
  constexpr int OWNED = Sh::OWNED;
  constexpr int OWN4 = OWNED * RP / 4;          // their float4s
  extern __shared__ __align__(1024) uint8_t lt_smem[];  // the swizzle atoms need 1024
  uint8_t* opnd = lt_smem + S * Sh::STAGE;
  float* vbuf = (float*)(opnd + Sh::OPND);      // [128][RP]
  float* red = Sh::PIPE ? vbuf + Sh::VBUF / 4 : (float*)opnd;  // [CS][OWNED][RP]
  uint64_t* bars = (uint64_t*)(opnd + Sh::OPND + Sh::VBUF + Sh::RED);
  uint64_t* full = bars;              // [S] tiles landed
  uint64_t* empty1 = bars + S;        // [S] the reduction's MMAs are done with the slot
  uint64_t* empty2 = bars + 2 * S;    // [S] the epilogue is
  uint64_t* d1_full = bars + 3 * S;   // [2]
  uint64_t* d1_empty = d1_full + 2;   // [2]
  uint64_t* x1 = d1_full + 4;         // partial sums of this CTA's rows arrived
  uint64_t* x2 = d1_full + 5;         // V of all rows arrived
  uint64_t* v_full = d1_full + 6;     // the V operand is written
  uint64_t* v_empty = d1_full + 7;    // the MMAs that read it are done
  uint64_t* p_seen = d1_full + 8;     // the epilogue has begun the piece
  uint64_t* d2_full = d1_full + 9;    // [4]
  uint64_t* d2_empty = d1_full + 13;  // [4]
  uint64_t* done = d1_full + 17;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;  // copies that the producer started
  int* scan = (int*)(tmem_slot + 3);      // LT_THREADS / 32 + 1 ints
  LoraPiece* table = (LoraPiece*)(scan + 20);
  float* rowback = (float*)(table + LT_TABLE);  // f16: [2][128] factors to take back
  static_assert((3 * S + 18) * 8 + 12 + 80 + LT_TABLE * sizeof(LoraPiece) + 1024 <= 2304, "fits");

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty1[s], 1);
      tc::mbar_init(&empty2[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&d1_full[b], 1);
      tc::mbar_init(&d1_empty[b], LT_XCH);
    }
    tc::mbar_init(x1, CS * LT_XCH);
    tc::mbar_init(x2, CS * LT_XCH);
    tc::mbar_init(v_full, LT_XCH);
    tc::mbar_init(v_empty, 1);
    tc::mbar_init(p_seen, LT_EPI);
    for (int b = 0; b < LT_GROUPS; ++b) {
      tc::mbar_init(&d2_full[b], 1);
      tc::mbar_init(&d2_empty[b], 4);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    *issued = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&xmap);
    tc::prefetch_tensormap(&pmap);
    tc::prefetch_tensormap(&qmap);
    tc::prefetch_tensormap(&ymap);
  }
  __syncthreads();
  cluster_arrive();  // this CTA runs and its barriers are set up
  pdl_wait();
  pdl_trigger();
  T* out = (T*)a.out;
  const int stride = (int)gridDim.x / CS, cid = (int)blockIdx.x / CS;
  const int n2 = (a.N + LT_N - 1) / LT_N;                  // output tiles
  const int nt = out == nullptr || n2 <= rank ? 0 : (n2 - rank + CS - 1) / CS;
  const int nk = (a.K + LT_K - 1) / LT_K;                  // reduction tiles
  const int n1 = nk <= rank ? 0 : (nk - rank + CS - 1) / CS;
  constexpr uint32_t P_BYTES = BWD ? Sh::PQ : RP * 128;    // TMA boxes per stage
  constexpr uint32_t Q_BYTES = BWD ? RP * 128 : Sh::PQ;
  // without the pipeline the partial sums come where the operand is: one piece at a time,
  // a cluster barrier between two
  constexpr int CAP = Sh::PIPE ? LT_TABLE : 1;
  int np = lora_find_pieces<LT_THREADS>(a, LT_M, cid, stride, 0, table, CAP, scan, LORA_ANY);
  if (np == 0) {  // the same for the whole cluster
    lora_copy_bare<T>(a, (int)blockIdx.x, (int)gridDim.x, threadIdx.x, LT_THREADS, ovec);
    cluster_wait();
    return;
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, LT_TMEM);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  cluster_wait();
  const uint32_t tmem = *tmem_slot;
  auto slot = [&](int s) { return lt_smem + (size_t)s * Sh::STAGE; };
  // ring index of the first output tile of the i-th of n pieces, counted from the first
  // stage of this table; the pieces of earlier tables came before
  int base_it = 0, base_g = 0, base_p = 0;  // ring stages, output tiles, pieces so far
  uint32_t tenant = 0, phase1 = 0, phase2 = 0;  // the producer's view of the slots
  auto first_tile = [&](int i, int n) {
    return base_it + n1 * (Sh::PIPE ? min(i + 2, n) : i + 1) + nt * i;
  };
  for (int chunk = 0;; ++chunk) {
    int n = np;
    if (warp == 0) {
      if (tc::elect_one()) {
        int it = base_it;
        bool ok = true;
        auto take = [&](uint32_t kind) {  // the next slot of the ring, empty; kind 1: output tile
          const int s = it % S;
          const uint32_t bit = 1u << s;
          if (it >= S) {  // who had it last says on which barrier to wait
            if (tenant & bit) {
              ok = tc::mbar_wait(&empty2[s], (phase2 & bit) != 0, abort_flag, a.spin);
              phase2 ^= bit;
            } else {
              ok = tc::mbar_wait(&empty1[s], (phase1 & bit) != 0, abort_flag, a.spin);
              phase1 ^= bit;
            }
          }
          tenant = kind ? tenant | bit : tenant & ~bit;
          return s;
        };
        auto reduce_tiles = [&](const LoraPiece pc) {
          for (int i = 0; i < n1 && ok; ++i) {
            const int s = take(0);
            if (!ok) break;
            uint8_t* sb = slot(s);
            const int c = (rank + CS * i) * LT_K;
            tc::mbar_arrive_expect_tx(&full[s], LT_TILE + P_BYTES);
            tc::tma_load_2d(sb, &xmap, &full[s], c, pc.t0);
            if (!BWD) {
              tc::tma_load_3d(sb + LT_TILE, &pmap, &full[s], c, 0, pc.a);
            } else {
#pragma unroll
              for (int p = 0; p < Sh::PQ / 8192; ++p)
                tc::tma_load_3d(sb + LT_TILE + p * 8192, &pmap, &full[s], p * 64, c, pc.a);
            }
            *issued = ++it;
          }
        };
        auto output_tiles = [&](const LoraPiece pc) {
          for (int i = 0; i < nt && ok; ++i) {
            const int s = take(1);
            if (!ok) break;
            uint8_t* sb = slot(s);
            const int j = (rank + CS * i) * LT_N;
            tc::mbar_arrive_expect_tx(&full[s], (a.Y != nullptr ? LT_TILE : 0) + Q_BYTES);
            if (a.Y != nullptr) tc::tma_load_2d(sb, &ymap, &full[s], j, pc.t0);
            if (!BWD) {
#pragma unroll
              for (int p = 0; p < Sh::PQ / 8192; ++p)
                tc::tma_load_3d(sb + LT_TILE + p * 8192, &qmap, &full[s], p * 64, j, pc.a);
            } else {
              tc::tma_load_3d(sb + LT_TILE, &qmap, &full[s], j, 0, pc.a);
            }
            *issued = ++it;
          }
        };
        for (int i = 0; i < n && ok; ++i) {
          reduce_tiles(table[i]);
          if (!Sh::PIPE) output_tiles(table[i]);
          else if (i > 0) output_tiles(table[i - 1]);
        }
        if (Sh::PIPE && n > 0) output_tiles(table[n - 1]);
      }
    } else if (warp == 1) {
      if (tc::elect_one()) {
        const uint32_t id1 = tc::instr_desc(BF16 ? 1 : 0, LT_M, RP, 0, BWD ? 1 : 0);
        const uint32_t id2 = tc::instr_desc(BF16 ? 1 : 0, LT_M, LT_N, 0, BWD ? 1 : 0);
        // descriptors of slot 0 and of the V operand
        const uint32_t s0 = tc::smem_u32(lt_smem);
        const uint64_t dx = tc::smem_desc_sw128(s0, 16, 1024);
        const uint64_t dp = BWD ? tc::smem_desc_sw128(s0 + LT_TILE, 8192, 1024)
                                : tc::smem_desc_sw128(s0 + LT_TILE, 16, 1024);
        const uint64_t dv = tc::smem_desc_sw128(tc::smem_u32(opnd), 16, 1024);
        int g = base_g, s = base_it % S;
        uint32_t ph = (uint32_t)(base_it / S) & 1u;  // of the ring's current round
        bool ok = true;
        auto advance = [&]() {
          if (++s == S) s = 0, ph ^= 1u;
        };
        auto reduce_mma = [&](int pi) {  // pi: running number of the piece
          const int b = pi & 1;
          const uint32_t d1 = tmem + 128 * b;
          if (pi >= 2)
            ok = ok && tc::mbar_wait(&d1_empty[b], (uint32_t)(pi / 2 - 1) & 1u, abort_flag, a.spin);
          tc::tc_fence_after();
          for (int i = 0; i < n1 && ok; ++i) {
            ok = tc::mbar_wait(&full[s], ph, abort_flag, a.spin);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t so = (uint32_t)s * Sh::STAGE;
            const uint64_t x = tc::desc_add(dx, so), p = tc::desc_add(dp, so);
#pragma unroll
            for (int kk = 0; kk < LT_K / 16; ++kk)
              tc::mma_f16_ss(d1, tc::desc_add(x, kk * 32), tc::desc_add(p, kk * (BWD ? 2048 : 32)),
                             id1, kk > 0 ? 1u : (uint32_t)(i > 0));
            tc::mma_commit(&empty1[s]);
            advance();
          }
          if (ok) tc::mma_commit(&d1_full[b]);
        };
        auto output_mma = [&](int pi) {
          ok = ok && tc::mbar_wait(v_full, (uint32_t)pi & 1u, abort_flag, a.spin);
          tc::tc_fence_after();
          for (int i = 0; i < nt && ok; ++i, ++g) {
            const int b = g % LT_GROUPS;
            const uint32_t d2 = tmem + 256 + 64 * b;
            if (g >= LT_GROUPS)
              ok = tc::mbar_wait(&d2_empty[b], (uint32_t)(g / LT_GROUPS - 1) & 1u, abort_flag, a.spin);
            ok = ok && tc::mbar_wait(&full[s], ph, abort_flag, a.spin);
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t q = tc::desc_add(dp, (uint32_t)s * Sh::STAGE);
#pragma unroll
            for (int h = 1; h >= 0; --h)  // the low halves first; columns past r are zeros
#pragma unroll
              for (int p = 0; p < RP / 16; ++p) {
                const int kc = h * RP + p * 16;
                tc::mma_f16_ss(d2, tc::desc_add(dv, (kc / 64) * LT_TILE + (kc % 64) * 2),
                               tc::desc_add(q, BWD ? p * 2048 : (p / 4) * 8192 + (p % 4) * 32), id2,
                               (h == 0 || p > 0) ? 1u : 0u);
              }
            tc::mma_commit(&d2_full[b]);
            advance();
          }
          if (ok) tc::mma_commit(v_empty);
        };
        for (int i = 0; i < n && ok; ++i) {
          reduce_mma(base_p + i);
          if (!Sh::PIPE) output_mma(base_p + i);
          else if (i > 0) output_mma(base_p + i - 1);
        }
        if (Sh::PIPE && n > 0 && ok) output_mma(base_p + n - 1);
      }
    } else if (warp < 2 + LT_XCH) {
      // ---- exchange: thread = row of the piece ----
      // A give-up ends the loop; the flag goes to the other CTAs, whose waits look at it.
      const int xt = threadIdx.x - 64;
      const int quarter = warp & 3, row = quarter * 32 + lane;
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      for (int i = 0; i < n; ++i) {
        const int pi = base_p + i, b = pi & 1;
        const uint32_t ph = (uint32_t)pi & 1u;
        const LoraPiece pc = table[i];
        const float sc = a.scaling[pc.a];
        const int live4 = (pc.cnt + 7) / 8 * 8 * (RP / 4);  // float4s of the rows that are used
        bool ok = tc::mbar_wait_warp(&d1_full[b], (uint32_t)(pi / 2) & 1u, abort_flag, a.spin);
        if (ok) {  // this CTA's partial sums, to shared memory
          tc::tc_fence_after();
          constexpr int CW = RP < 32 ? RP : 32;  // columns per load
#pragma unroll
          for (int c = 0; c < RP; c += CW) {
            float v[CW];
            const uint32_t ta = tmem + lanes + (uint32_t)(128 * b + c);
            if (CW == 16) tc::tmem_ld_32x32b_x16(ta, v);
            else tc::tmem_ld_32x32b_x32(ta, v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < CW; e += 4)
              reinterpret_cast<float4*>(vbuf)[lt_vslot<RP>(row, (c + e) / 4)] =
                  n1 > 0 ? make_float4(v[e], v[e + 1], v[e + 2], v[e + 3])
                         : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&d1_empty[b]);
        }
        // the exchange warps go on, or give up, together
        if (tc::named_bar_any(1, 32 * LT_XCH, !ok)) break;
        {
          // each owner's rows to it, consecutive lanes to consecutive addresses
          const uint32_t dst = tc::smem_u32(red) + 16u * (uint32_t)(rank * OWN4);
#pragma unroll 4
          for (int e = xt; e < live4; e += 32 * LT_XCH)
            cluster_st_f4(cluster_map(dst + 16u * (uint32_t)(e % OWN4), (uint32_t)(e / OWN4)),
                          reinterpret_cast<const float4*>(vbuf)[e]);
          __syncwarp();
          if (lane < CS) cluster_mbar_arrive(cluster_map(tc::smem_u32(x1), (uint32_t)lane));
          ok = cluster_mbar_wait_warp(x1, ph, abort_flag, a.spin);
        }
        if (ok) {
          // the rows that this CTA owns: add the parts, scale, hand V to all.  (A peer writes
          // V over the block of vbuf that went to it, which has arrived there by now.)
          const float4* part = reinterpret_cast<const float4*>(red);
          for (int e = xt; e < min(OWN4, live4 - rank * OWN4); e += 32 * LT_XCH) {
            float4 v = part[e];
#pragma unroll
            for (int c = 1; c < CS; ++c) {
              const float4 w = part[c * OWN4 + e];
              v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
            }
            const int r = e / (RP / 4);
            const int c4 = RP == 16 ? (e % (RP / 4)) ^ ((r >> 1) & 3) : (e % (RP / 4)) ^ (r & 7);
            v.x *= sc, v.y *= sc, v.z *= sc, v.w *= sc;
            // columns that only pad the rank stay 0 where an infinity met their zeros
            if (4 * c4 >= a.r) v = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t va = tc::smem_u32(vbuf) + 16u * (uint32_t)(rank * OWN4 + e);
#pragma unroll
            for (int c = 0; c < CS; ++c) cluster_st_f4(cluster_map(va, (uint32_t)c), v);
            if (a.V != nullptr && rank * OWNED + r < pc.cnt && 4 * c4 < a.r) {  // r % 8 == 0
              float* o = a.V + (int64_t)(pc.t0 + rank * OWNED + r) * a.r + 4 * c4;
              o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
            }
          }
          __syncwarp();
          if (lane < CS) cluster_mbar_arrive(cluster_map(tc::smem_u32(x2), (uint32_t)lane));
          ok = cluster_mbar_wait_warp(x2, ph, abort_flag, a.spin);
        }
        // the operand is free, and the epilogue has begun the piece before (it holds that
        // piece's factors, and is at most one phase of v_full behind)
        if (ok && pi >= 1)
          ok = tc::mbar_wait_warp(v_empty, (uint32_t)(pi - 1) & 1u, abort_flag, a.spin);
        if (ok && pi >= 1)
          ok = tc::mbar_wait_warp(p_seen, (uint32_t)(pi - 1) & 1u, abort_flag, a.spin);
        if (tc::named_bar_any(1, 32 * LT_XCH, !ok)) break;
        // V as the A operand: columns 0.. hold hi, RP.. hold lo
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
          rowback[128 * b + row] = __fdiv_rn(1.f, f);  // a power of two: exact
        }
#pragma unroll 4
        for (int c8 = 0; c8 < RP / 8; ++c8) {
          const float4 v0 = vr[lt_vslot<RP>(row, 2 * c8)], v1 = vr[lt_vslot<RP>(row, 2 * c8 + 1)];
          uint4 hi, lo;
          lora_split<BF16>(v0.x * f, v0.y * f, hi.x, lo.x);
          lora_split<BF16>(v0.z * f, v0.w * f, hi.y, lo.y);
          lora_split<BF16>(v1.x * f, v1.y * f, hi.z, lo.z);
          lora_split<BF16>(v1.z * f, v1.w * f, hi.w, lo.w);
          const int kl = RP / 8 + c8;  // 16-byte chunks of the row
          *reinterpret_cast<uint4*>(opnd + (c8 / 8) * LT_TILE + row * 128 +
                                    (((c8 % 8) ^ (row & 7)) << 4)) = hi;
          *reinterpret_cast<uint4*>(opnd + (kl / 8) * LT_TILE + row * 128 +
                                    (((kl % 8) ^ (row & 7)) << 4)) = lo;
        }
        tc::fence_proxy_async_smem();  // the MMA reads what this thread wrote
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(v_full);
      }
      if (lane < CS && *abort_flag)
        cluster_st_u32(cluster_map(tc::smem_u32((const void*)abort_flag), (uint32_t)lane), 1u);
    } else {
      // ---- epilogue: group `grp` takes every third output tile ----
      const int grp = (warp - 2 - LT_XCH) / 4;
      const int quarter = warp & 3, row = quarter * 32 + lane;
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      // rows without an adapter are copied while the first piece is reduced
      if (chunk == 0)
        lora_copy_bare<T>(a, (int)blockIdx.x, (int)gridDim.x, threadIdx.x - 64 - 32 * LT_XCH,
                          32 * LT_EPI, ovec);
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int pi = base_p + i;
        const LoraPiece pc = table[i];
        ok = tc::mbar_wait_warp(v_full, (uint32_t)pi & 1u, abort_flag, a.spin);
        if (!ok) break;
        const float back = BF16 ? 1.f : rowback[128 * (pi & 1) + row];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_seen);
        const int it0 = first_tile(i, n), g0 = base_g + nt * i;
        for (int q = 0; q < nt; ++q) {
          const int g = g0 + q, it = it0 + q;
          if (g % LT_GROUPS != grp) continue;
          const int s = it % S, b = grp;
          const int j0 = (rank + CS * q) * LT_N;
          ok = tc::mbar_wait_warp(&d2_full[b], (uint32_t)(g / LT_GROUPS) & 1u, abort_flag, a.spin);
          if (!ok) break;
          // the MMA waited for the slot's copies, so this phase is over; the wait makes the
          // tile of Y visible here.  (Before the MMA the slot might still be a phase behind,
          // which the parity cannot tell from this one.)
          ok = tc::mbar_wait_warp(&full[s], (uint32_t)(it / S) & 1u, abort_flag, a.spin);
          if (!ok) break;
          uint8_t* ys = slot(s);
          tc::tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 32 columns at a time
            float v[32];
            tc::tmem_ld_32x32b_x32(tmem + lanes + (uint32_t)(256 + 64 * b + 32 * h), v);
            uint4 yv[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              yv[c] = a.Y != nullptr ? *reinterpret_cast<const uint4*>(
                                           ys + row * 128 + (((4 * h + c) ^ (row & 7)) << 4))
                                     : make_uint4(0u, 0u, 0u, 0u);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4] = {yv[c].x, yv[c].y, yv[c].z, yv[c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 y = Ty::unpack(w[e]);
                w[e] = Ty::pack(fmaf(v[8 * c + 2 * e], back, y.x),
                                fmaf(v[8 * c + 2 * e + 1], back, y.y));
              }
              *reinterpret_cast<uint4*>(ys + row * 128 + (((4 * h + c) ^ (row & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&d2_empty[b]);
          // this warp's 32 rows, 128 contiguous bytes per row; the slot goes back before the
          // stores, whose way to L2 it would wait for
          const int c = lane % 8, j = j0 + 8 * c, r0 = quarter * 32 + lane / 8;
          uint4 w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = *reinterpret_cast<const uint4*>(ys + (r0 + 4 * e) * 128 +
                                                   ((c ^ ((r0 + 4 * e) & 7)) << 4));
          tc::fence_proxy_async_smem();  // the next copy into the slot comes after these accesses
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&empty2[s]);
          T* o = out + (int64_t)(pc.t0 + r0) * a.ldo + j;
          if (ovec && j + 8 <= a.N) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (r0 + 4 * e < pc.cnt) *reinterpret_cast<uint4*>(o + (int64_t)(4 * e) * a.ldo) = w[e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (r0 + 4 * e >= pc.cnt) continue;
              const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (j + x < a.N)
                  reinterpret_cast<unsigned short*>(o + (int64_t)(4 * e) * a.ldo)[x] =
                      (unsigned short)(u[x / 2] >> (16 * (x % 2)));
            }
          }
        }
      }
    }
    __syncthreads();
    // every CTA is done with these pieces: no write or arrival into another CTA is under way,
    // and a give-up in one of them is known to all
    if (threadIdx.x < CS && *abort_flag)
      cluster_st_u32(cluster_map(tc::smem_u32((const void*)abort_flag), threadIdx.x), 1u);
    tc::tc_fence_before();
    cluster_arrive();
    cluster_wait();
    tc::tc_fence_after();
    if (*abort_flag) {  // the outputs of what this cluster had left become NaN
      if (warp == 1) {  // every MMA issued above finishes before TMEM goes
        if (tc::elect_one()) {  // the lane that issued them
          tc::mma_commit(done);
          for (uint32_t i = 0; i < tc::kSpinLimit; ++i)
            if (tc::mbar_try_wait(done, 0)) break;
        }
        __syncwarp();
      }
      if (threadIdx.x == 0)  // the copies in flight land before the shared memory goes
        for (int p = max(0, *issued - S); p < *issued; ++p)
          for (uint32_t i = 0; i < tc::kSpinLimit; ++i)
            if (tc::mbar_try_wait(&full[p % S], (uint32_t)(p / S) & 1u)) break;
      const T bad = Ty::cvt(__int_as_float(0x7fc00000));
      for (;;) {
        for (int i = 0; i < n; ++i) {
          const LoraPiece pc = table[i];
          for (int e = warp; e < pc.cnt; e += LT_THREADS / 32) {
            const int64_t r = pc.t0 + e;
            for (int q = 0; q < nt; ++q)
              for (int j = (rank + CS * q) * LT_N + lane;
                   j < min(a.N, (rank + CS * q + 1) * LT_N); j += 32)
                out[r * a.ldo + j] = bad;
            if (a.V != nullptr && e / OWNED == rank)
              for (int p = lane; p < a.r; p += 32) a.V[r * a.r + p] = __int_as_float(0x7fc00000);
          }
        }
        ++chunk;
        __syncthreads();
        n = lora_find_pieces<LT_THREADS>(a, LT_M, cid, stride, chunk * CAP, table, CAP, scan, LORA_ANY);
        if (n == 0) break;
      }
      break;
    }
    base_it += n * (n1 + nt);
    base_g += n * nt;
    base_p += n;
    if (np < CAP) break;
    np = lora_find_pieces<LT_THREADS>(a, LT_M, cid, stride, (chunk + 1) * CAP, table, CAP,
                                      scan, LORA_ANY);
    if (np == 0) break;
  }
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, LT_TMEM);
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

// Clusters that are resident at once (0: the shared memory is refused).
template <bool BF16, int RP, bool BWD, int CS>
int tc_fit() {
  if (smem_optin((const void*)lora_tc_kernel<BF16, RP, BWD, CS>, LtShape<RP, CS>::SMEM) != cudaSuccess)
    return 0;
  return resident_clusters((const void*)lora_tc_kernel<BF16, RP, BWD, CS>, CS, LT_THREADS,
                           LtShape<RP, CS>::SMEM);
}


template <bool BF16, int RP, bool BWD, int CS>
gptq_status launch_tc(const LoraArgs& a, int64_t pieces, cudaStream_t s) {
  using Sh = LtShape<RP, CS>;
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
  if (!ok) return GPTQ_ERR_CUDA;
  const int ovec = (uintptr_t)a.out % 16 == 0 && a.ldo % 8 == 0;
  // as many clusters as fit the device at once; each takes piece after piece
  const int fit = tc_fit<BF16, RP, BWD, CS>();
  if (fit == 0) return GPTQ_ERR_CUDA;
  pieces = std::min<int64_t>(pieces, fit);
  launch_cluster_pdl(lora_tc_kernel<BF16, RP, BWD, CS>, dim3((unsigned)(pieces * CS)),
                     dim3(LT_THREADS), Sh::SMEM, CS, s, xm, pm, qm, ym, a, ovec);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

// The size of the clusters.  A piece takes a cluster the longer the fewer CTAs it has, but
// larger clusters fit the device less often (the GPCs' 16 to 18 free SMs: 15 of 8, 22 of 6,
// 26 of 5, 33 of 4, 45 of 3): the size whose rounds over the pieces, by its CTAs, are fewest.
// Measured (4096 -> 11008, rank 64), clusters of 8, 6, 4, 3: 600 tokens 28, 33, 42, 51 us;
// 2000 tokens 48, 38, 45, 53; 5000 tokens 72, 66, 82, 64; 8192 tokens 110, 94, 93, 105.
// The lengths are on the device.  Of several requests one in 512 rows is taken to be long,
// with a last piece half full, and the others to be single rows; a wrong guess costs time.
template <bool BF16, int RP, bool BWD>
gptq_status tc_cluster(const LoraArgs& a, int64_t pieces, cudaStream_t s) {
  const int64_t longer = std::min<int64_t>(a.nreq, std::max(1, a.m / 512));
  const int64_t rows = a.m - (a.nreq - longer);
  const int64_t guess = a.nreq == 1 ? cdiv(a.m, LT_M)
                                    : std::max<int64_t>(1, (rows + longer * (LT_M / 2)) / LT_M);
  int size = 0;
  int64_t rounds = 0;
  auto weigh = [&](int cs, int fit) {
    const int64_t n = fit > 0 ? cdiv(guess, fit) : INT32_MAX;
    if (size == 0 || n * size < rounds * cs || (n * size == rounds * cs && n < rounds))
      size = cs, rounds = n;
  };
  weigh(8, tc_fit<BF16, RP, BWD, 8>());
  weigh(4, tc_fit<BF16, RP, BWD, 4>());
  if constexpr (RP <= 64) {
    weigh(6, tc_fit<BF16, RP, BWD, 6>());
    weigh(5, tc_fit<BF16, RP, BWD, 5>());
    weigh(3, tc_fit<BF16, RP, BWD, 3>());
    if (size == 3) return launch_tc<BF16, RP, BWD, 3>(a, pieces, s);
    if (size == 5) return launch_tc<BF16, RP, BWD, 5>(a, pieces, s);
    if (size == 6) return launch_tc<BF16, RP, BWD, 6>(a, pieces, s);
  }
  if (size == 4) return launch_tc<BF16, RP, BWD, 4>(a, pieces, s);
  return launch_tc<BF16, RP, BWD, 8>(a, pieces, s);
}

template <bool BF16, bool BWD>
gptq_status tc_ranks(const LoraArgs& a, int64_t pieces, cudaStream_t s) {
  if (a.r <= 16) return tc_cluster<BF16, 16, BWD>(a, pieces, s);
  if (a.r <= 32) return tc_cluster<BF16, 32, BWD>(a, pieces, s);
  if (a.r <= 64) return tc_cluster<BF16, 64, BWD>(a, pieces, s);
  return tc_cluster<BF16, 128, BWD>(a, pieces, s);
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
