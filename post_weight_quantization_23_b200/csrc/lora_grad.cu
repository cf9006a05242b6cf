// Gradients of the adapters (gptq_lora_backward): with U = scaling B^T dY of the
// tensor-core pass over dY and V = scaling A x kept from the forward pass,
//   dA_a = sum_t U[t] x_t^T,   dB_a = sum_t dY[t] V[t]^T,
// t over the rows of adapter a's requests.  Both are sums over tokens of a wide
// row (x or dY, `S` below) times a narrow fp32 row (U or V, `W` below).
//
// Bound by HBM: the wide rows are read once (2 bytes or, from an 8-bit checkpoint,
// 1 + 4/128 per element) against 2 r flops per element.  Tensor-core kernel: a CTA
// sums 128 columns of one gradient over the adapter's tokens (or over every SPLIT-th
// 64-token tile of them; the SPLIT CTAs of a cluster then add up through distributed
// shared memory in a fixed order), D[128 x RP] fp32 in TMEM, tokens as the MMA's K.
// Both operands are MN-major: rows of S as TMA brings them, and rows of W.
//   W is split into two bf16 parts, hi + lo (16 significant bits; bf16 for its range:
//     gradients are small, f16 would lose them among its subnormals), side by side as one
//     operand of 2 RP columns: S is read from shared memory, whose bandwidth sets the
//     pace, once for both, and the two halves of D are added at the end.  What the split
//     leaves, 2^-17 of W, is far below the result's rounding (2^-9, f16 2^-12).
//   S in bf16 is used as it is.  S in f16 is split into two bf16 parts as well (exactly),
//     three products: lo x lo, 2^-17 of a product at most, is not worth a fourth MMA.
//   S in 8-bit codes becomes bf16 exactly (|code| <= 127), and its scales, one per token
//     and 128-column block, multiply the rows of W: the checkpoint is never restored.
// Tiles to be converted land in a ring of their own, deeper than the operands' (a tile of
// codes is 8 KB, and the way from its copy to its MMA is twice as long as a bf16 tile's).
// Rows behind a request's end in its last tile belong to others (or hold anything):
// both operands are zeroed there.
// Warps: 0 TMA, 1 MMA, then the operand warps (groups of four, tile by tile in turn),
// which are the epilogue too.  The number of stages is a multiple of the groups, so a
// slot belongs to one group, which sees every phase of its barrier (a wait that skips
// phases cannot tell the one before from the one it wants).
// Every wait is bounded; a CTA that gives up writes NaN.
// 4096 tokens, rank 64, 4096 x 11008 from codes: 52 us alone, 46 with X in bf16; 8192 tokens
// 92 and 82.  So a 64-token tile takes 1100 cycles where there are columns of codes (conversion
// of codes and W, some 2000 warp instructions) and 980 in bf16 (copies' latency), and what does
// not grow with the tokens is 12 us (64 tokens alone: 14; launch, look-up, TMEM, first copies,
// sums, stores).  At HBM's rate the 108 MB of 4096 tokens take 17 us.
#include "lora.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

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

struct LoraGradCommon : LoraRequests {
  int r;
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

// ---- tensor-core kernel ------------------------------------------------------------

constexpr int GT_C = 128, GT_T = 64;         // columns and tokens of a tile
constexpr int GT_ATOM = GT_T * 128;          // 64 tokens x 64 16-bit columns, 8 KB
constexpr int GT_TABLE = 128;                // tiles looked up at a time
constexpr int GT_LD = GT_C + 1;              // row stride of the staged sums (no bank conflicts)
constexpr int GT_BARS = 384;                 // bytes of barriers and small words

// A slot of the operand ring: S hi (and lo), W hi | lo.  Tiles to be converted (f16,
// codes) land in RAW bytes behind the slots.
template <int RP, bool F16>
struct GtShape {
  static constexpr int HI = 0, LO = 2 * GT_ATOM;
  static constexpr int W = (F16 ? 4 : 2) * GT_ATOM;  // 2 RP columns in atoms of 64
  static constexpr int STAGE = W + (2 * RP + 63) / 64 * GT_ATOM;
  static constexpr int S = F16 ? (RP > 64 ? 2 : 3) : 4;
  // groups of operand warps: as many as slots, where their registers allow it
  static constexpr int NG = RP <= 64 ? S : 2;
  static constexpr int RAW = (RP > 64 ? 4 : F16 ? 6 : 8) * GT_ATOM;
  static constexpr int R_CODES = RAW / GT_ATOM, R_F16 = RAW / (2 * GT_ATOM);
  // a bf16 S needs no raw ring: its place holds more slots, for fewer groups (their work
  // is half of that on codes, the copies' latency is what is left to cover)
  static constexpr int S_DIRECT = RP <= 64 ? 6 : 4, NG_DIRECT = RP <= 64 ? 3 : 2;
  static constexpr int THREADS = 64 + 128 * NG;
  static_assert(S % NG == 0 && R_CODES % NG == 0 && (!F16 || R_F16 % NG == 0) &&
                    S_DIRECT % NG_DIRECT == 0 && (F16 || NG_DIRECT <= NG),
                "a slot belongs to one group");
  static_assert(F16 || S_DIRECT * STAGE <= S * STAGE + RAW, "the slots of bf16 tiles fit");
  static constexpr int SUMS = RP * GT_LD * 4;
  static constexpr size_t SMEM =
      (size_t)S * STAGE + RAW + GT_BARS + GT_TABLE * sizeof(LoraPiece);
  static_assert(SUMS <= S * STAGE && SMEM <= 232448, "shared memory of a CTA");
};

// hi + lo in bf16 of four f16 pairs.
__device__ __forceinline__ void gt_split_f16(uint4 u, uint4& hi, uint4& lo) {
  const uint32_t in[4] = {u.x, u.y, u.z, u.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = LoraType<false>::unpack(in[i]);
    lora_split_bf16(v.x, v.y, h[i], l[i]);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Four int8 codes as bf16, exactly and two at a time: with the code's low seven bits in the
// mantissa of 128 (128 + low) and its sign bit in that of another 128 (128 or 256), the
// difference is the code.
__device__ __forceinline__ uint2 gt_codes(uint32_t w) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = __byte_perm(w, 0u, i == 0 ? 0x4140u : 0x4342u);
    const uint32_t h = (v & 0x007f007fu) | 0x43004300u, z = (v & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&h),
                                     *reinterpret_cast<const __nv_bfloat162*>(&z));
    o[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
  return make_uint2(o[0], o[1]);
}
__device__ __forceinline__ uint4 gt_codes(uint32_t a, uint32_t b) {
  const uint2 x = gt_codes(a), y = gt_codes(b);
  return make_uint4(x.x, x.y, y.x, y.y);
}

template <int RP, bool F16>
__global__ void __launch_bounds__(GtShape<RP, F16>::THREADS, 1)
lora_grad_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                 LoraGradArgs ga, LoraGradArgs gb, LoraGradCommon c, int blocks_a, int split) {
  using Sh = GtShape<RP, F16>;
  using T = typename LoraType<!F16>::T;
  constexpr int GT_THREADS = Sh::THREADS;
  extern __shared__ __align__(1024) uint8_t gt_smem[];
  uint8_t* raws = gt_smem + Sh::S * Sh::STAGE;
  uint64_t* bars = (uint64_t*)(raws + Sh::RAW);
  uint64_t* full = bars;            // [8] the tile landed (in a slot, or in the raw ring)
  uint64_t* rawfree = bars + 8;     // [8] the raw tile is converted
  uint64_t* ready = bars + 16;      // [6] both operands are written
  uint64_t* empty = ready + 6;      // [6] the MMAs that read them are done
  uint64_t* done = empty + 6;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;
  int* scan = (int*)(tmem_slot + 3);  // GT_THREADS / 32 + 1 ints
  LoraPiece* table = (LoraPiece*)(raws + Sh::RAW + GT_BARS);
  static_assert((16 + 2 * 6 + 1) * 8 + 12 + 4 * (GT_THREADS / 32 + 1) <= GT_BARS, "fits");

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int part = (int)blockIdx.x % split, blk = (int)blockIdx.x / split;
  const bool second = blk >= blocks_a;
  const LoraGradArgs& g = second ? gb : ga;
  const CUtensorMap* map = second ? &bmap : &amap;
  const int col0 = (second ? blk - blocks_a : blk) * GT_C, ad = blockIdx.y;
  const bool codes = g.s_scales != nullptr;
  const bool convert = F16 || codes;
  // slots of the operands, their groups of warps, slots that the copies go round
  const int S = convert ? Sh::S : Sh::S_DIRECT, NG = convert ? Sh::NG : Sh::NG_DIRECT;
  const int R = codes ? Sh::R_CODES : F16 ? Sh::R_F16 : S;
  constexpr int TM = 2 * RP;  // TMEM columns
  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&rawfree[s], 4);
    }
    for (int s = 0; s < 6; ++s) {
      tc::mbar_init(&ready[s], 4);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    *issued = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(map);
  }
  pdl_wait();
  pdl_trigger();
  int np = lora_find_pieces<GT_THREADS>(c, GT_T, part, split, 0, table, GT_TABLE, scan, ad);
  if (warp == 1) tc::tmem_alloc(tmem_slot, TM);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto stage = [&](int it) { return gt_smem + (size_t)(it % S) * Sh::STAGE; };
  int base = 0;  // tiles of the tables before

  for (int chunk = 1; np > 0; ++chunk) {
    if (warp == 0) {
      if (lane == 0) {
        uint64_t* free = convert ? rawfree : empty;
        for (int i = 0; i < np; ++i) {
          const int it = base + i, q = it % R;
          if (it >= R && !tc::mbar_wait(&free[q], (uint32_t)(it / R - 1) & 1u, abort_flag, c.spin))
            break;
          const int t0 = table[i].t0;
          if (codes) {
            tc::mbar_arrive_expect_tx(&full[q], GT_ATOM);
            tc::tma_load_2d(raws + q * GT_ATOM, map, &full[q], col0, t0);
          } else {
            uint8_t* dst = F16 ? raws + q * (2 * GT_ATOM) : stage(q) + Sh::HI;
            tc::mbar_arrive_expect_tx(&full[q], 2 * GT_ATOM);
            tc::tma_load_2d(dst, map, &full[q], col0, t0);
            tc::tma_load_2d(dst + GT_ATOM, map, &full[q], col0 + 64, t0);
          }
          *issued = it + 1;
        }
      }
    } else if (warp == 1) {
      if (tc::elect_one()) {
        // bf16, both MN-major; S hi times W hi | lo, S lo (f16) times W hi
        const uint32_t id = tc::instr_desc(1, GT_C, 2 * RP, 1, 1);
        const uint32_t id_lo = tc::instr_desc(1, GT_C, RP, 1, 1);
        const uint64_t d0 = tc::smem_desc_sw128(tc::smem_u32(gt_smem), GT_ATOM, 1024);
        const bool split_s = F16 && !codes;
        int s = base % S;
        uint32_t ph = (uint32_t)(base / S) & 1u;
        for (int i = 0; i < np; ++i) {
          // the operand warps waited for the copy before they arrived
          if (!tc::mbar_wait(&ready[s], ph, abort_flag, c.spin)) break;
          tc::tc_fence_after();
          const uint64_t d = tc::desc_add(d0, (uint32_t)s * Sh::STAGE);
#pragma unroll
          for (int kk = 0; kk < GT_T / 16; ++kk) {
            const uint64_t w = tc::desc_add(d, Sh::W + kk * 2048);
            tc::mma_f16_ss(tmem, tc::desc_add(d, Sh::HI + kk * 2048), w, id,
                           kk > 0 ? 1u : (uint32_t)(base + i > 0));
            if (split_s) tc::mma_f16_ss(tmem, tc::desc_add(d, Sh::LO + kk * 2048), w, id_lo, 1u);
          }
          tc::mma_commit(&empty[s]);
          if (++s == S) s = 0, ph ^= 1u;
        }
      }
    } else {
      // ---- operands: group `grp` of four warps takes every NG-th tile ----
      const int grp = (warp - 2) / 4, gt = (warp - 2) % 4 * 32 + lane;
      constexpr int NCH = RP / 8;                 // 8-value chunks of a row of W
      constexpr int TASKS = GT_T * NCH / 128;     // chunks per thread: tokens wt + k WT
      constexpr int WT = 128 / NCH;               // a multiple of 8 where TASKS > 1
      const int nb = (g.C + 127) / 128;
      const int wt = gt / NCH, wc = gt % NCH, wl = NCH + wc;
      const bool wcol = 8 * wc < c.r;
      // places in shared memory (rows are 128 bytes; WT and 16 rows further on the swizzle
      // is the same): W hi and lo of task k at + k WT 128, codes of task k at + k 2048
      const int o_hi = Sh::W + (wc / 8) * GT_ATOM + wt * 128 + (((wc % 8) ^ (wt & 7)) << 4);
      const int o_lo = Sh::W + (wl / 8) * GT_ATOM + wt * 128 + (((wl % 8) ^ (wt & 7)) << 4);
      const int ct = gt / 8, cj = gt % 8, odd = cj / 4;
      // eight lanes write a row of both atoms, whose banks are the same: those of the second
      // atom write their odd chunk first
      const int o_c0 = Sh::HI + odd * GT_ATOM + ct * 128 + (((2 * (cj % 4) + odd) ^ (ct & 7)) << 4);
      const int o_c1 = o_c0 ^ 16;
      float4 w[TASKS][2];
      float sc[TASKS];
      auto fetch = [&](int i) {
        const LoraPiece p = table[i];
        const float* src = g.W + (int64_t)(p.t0 + wt) * c.r + 8 * wc;
        const float* ssc = codes ? g.s_scales + (int64_t)(p.t0 + wt) * nb + col0 / 128 : nullptr;
        const int left = p.cnt - wt;
#pragma unroll
        for (int k = 0; k < TASKS; ++k) {
          const bool have = wcol && k * WT < left;
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          w[k][0] = have ? __ldg(reinterpret_cast<const float4*>(src)) : z;
          w[k][1] = have ? __ldg(reinterpret_cast<const float4*>(src) + 1) : z;
          sc[k] = 1.f;
          if (codes) {
            if (have) sc[k] = __ldg(ssc);
            ssc += WT * nb;
          }
          src += WT * c.r;
        }
      };
      int i = grp < NG ? (grp - base % NG + NG) % NG : np;
      if (i < np) fetch(i);
      for (; i < np; i += NG) {
        const int it = base + i, s = it % S, q = it % R;
        const int cnt = table[i].cnt;
        if (!tc::mbar_wait_warp(&full[q], (uint32_t)(it / R) & 1u, abort_flag, c.spin)) break;
        if (convert && it >= S &&
            !tc::mbar_wait_warp(&empty[s], (uint32_t)(it / S - 1) & 1u, abort_flag, c.spin))
          break;
        uint8_t* sb = stage(s);
#pragma unroll
        for (int k = 0; k < TASKS; ++k) {
          uint4 hi, lo;
          if (codes) {
            const float f = sc[k];
            w[k][0].x *= f, w[k][0].y *= f, w[k][0].z *= f, w[k][0].w *= f;
            w[k][1].x *= f, w[k][1].y *= f, w[k][1].z *= f, w[k][1].w *= f;
          }
          lora_split_bf16(w[k][0].x, w[k][0].y, hi.x, lo.x);
          lora_split_bf16(w[k][0].z, w[k][0].w, hi.y, lo.y);
          lora_split_bf16(w[k][1].x, w[k][1].y, hi.z, lo.z);
          lora_split_bf16(w[k][1].z, w[k][1].w, hi.w, lo.w);
          *reinterpret_cast<uint4*>(sb + o_hi + k * (WT * 128)) = hi;
          *reinterpret_cast<uint4*>(sb + o_lo + k * (WT * 128)) = lo;
        }
        if (i + NG < np) fetch(i + NG);
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        if (codes) {
          const uint8_t* raw = raws + q * GT_ATOM + 16 * gt;
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // 16 codes each
            const uint4 u = *reinterpret_cast<const uint4*>(raw + 2048 * k);
            uint4 x = gt_codes(odd ? u.z : u.x, odd ? u.w : u.y);
            uint4 y = gt_codes(odd ? u.x : u.z, odd ? u.y : u.w);
            if (ct + 16 * k >= cnt) x = y = z;
            *reinterpret_cast<uint4*>(sb + o_c0 + 2048 * k) = x;
            *reinterpret_cast<uint4*>(sb + o_c1 + 2048 * k) = y;
          }
        } else if (F16) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 8 values each; the swizzle stays as TMA laid it
            const int e = gt + 128 * k;
            const bool have = (e % 512) / 8 < cnt;
            uint4 hi = z, lo = z;
            if (have)
              gt_split_f16(*reinterpret_cast<const uint4*>(raws + q * (2 * GT_ATOM) + 16 * e), hi, lo);
            *reinterpret_cast<uint4*>(sb + Sh::HI + 16 * e) = hi;
            *reinterpret_cast<uint4*>(sb + Sh::LO + 16 * e) = lo;
          }
        } else if (cnt < GT_T) {
          for (int e = gt; e < 2 * GT_ATOM / 16; e += 128)
            if ((e % 512) / 8 >= cnt) *reinterpret_cast<uint4*>(sb + Sh::HI + 16 * e) = z;
        }
        tc::fence_proxy_async_smem();  // the MMA reads what this thread wrote
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&ready[s]);
          if (convert) tc::mbar_arrive(&rawfree[q]);
        }
      }
    }
    __syncthreads();
    base += np;
    if (np < GT_TABLE || *abort_flag) break;
    np = lora_find_pieces<GT_THREADS>(c, GT_T, part, split, chunk * GT_TABLE, table, GT_TABLE, scan,
                                      ad);
  }
  // all MMAs done (their stages are free for the sums), all copies landed
  if (warp == 1) {
    if (tc::elect_one()) tc::mma_commit(done);  // the lane that issued them
  }
  const bool finished = tc::mbar_wait_warp(done, 0, abort_flag, tc::kSpinLimit);
  if (*abort_flag && threadIdx.x == 0)
    for (int p = max(0, *issued - R); p < *issued; ++p)
      for (uint32_t i = 0; i < tc::kSpinLimit; ++i)
        if (tc::mbar_try_wait(&full[p % R], (uint32_t)(p / R) & 1u)) break;
  __syncthreads();
  tc::tc_fence_after();
  const bool ok = finished && !*abort_flag;
  float* sums = (float*)gt_smem;  // [RP][GT_LD]
  if (warp >= 2 && warp < 10) {
    const int quarter = warp & 3, hf = (warp - 2) / 4, col = quarter * 32 + lane;
    constexpr int HC = RP / 2, CW = HC < 16 ? HC : 16;
#pragma unroll
    for (int q = 0; q < HC; q += CW) {
      float v[CW], l[CW];
      const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(hf * HC + q);
      if (CW == 8) tc::tmem_ld_32x32b_x8(ta, v), tc::tmem_ld_32x32b_x8(ta + RP, l);
      else tc::tmem_ld_32x32b_x16(ta, v), tc::tmem_ld_32x32b_x16(ta + RP, l);
      tc::tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < CW; ++e)
        sums[(hf * HC + q + e) * GT_LD + col] =
            !ok ? __int_as_float(0x7fc00000) : base > 0 ? v[e] + l[e] : 0.f;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, TM);
  if (split > 1) {
    cluster_arrive();
    cluster_wait();
  }
  // this CTA's share of the columns, summed over the cluster
  const int per = GT_C / split, c0 = part * per;
  T* out = (T*)g.out + (int64_t)ad * c.r * g.C;
  for (int e = threadIdx.x; e < per * c.r; e += GT_THREADS) {
    // neighbouring threads along the axis that is contiguous in the output
    const int cc = g.col_stride == 1 ? c0 + e % per : c0 + e / c.r;
    const int p = g.col_stride == 1 ? e / per : e % c.r;
    float v = 0.f;
    if (split == 1) {
      v = sums[p * GT_LD + cc];
    } else {
      const uint32_t at = tc::smem_u32(sums + p * GT_LD + cc);
      for (int q = 0; q < split; ++q) v += cluster_ld_f32(cluster_map(at, (uint32_t)q));
    }
    if (col0 + cc < g.C)
      out[(int64_t)(col0 + cc) * g.col_stride + (int64_t)p * g.rank_stride] = LoraType<!F16>::cvt(v);
  }
  if (split > 1) {  // no CTA leaves while another reads its sums
    cluster_arrive();
    cluster_wait();
  }
}

bool gt_supported(const LoraGradArgs& g) {
  const int64_t ldb = g.lds * (g.s_scales != nullptr ? 1 : 2);
  return (uintptr_t)g.S % 16 == 0 && ldb % 16 == 0 && (uintptr_t)g.W % 16 == 0 &&
         tensormap_encoder() != nullptr;
}

bool gt_map(CUtensorMap* map, const LoraGradArgs& g, int m, bool bf16) {
  const bool codes = g.s_scales != nullptr;
  cuuint64_t gdim[2] = {(cuuint64_t)g.C, (cuuint64_t)m};
  cuuint64_t gstride[1] = {(cuuint64_t)g.lds * (codes ? 1 : 2)};
  cuuint32_t box[2] = {codes ? 128u : 64u, GT_T};
  cuuint32_t es[2] = {1, 1};
  return tensormap_encoder()(
             map,
             codes  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
             : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             2, const_cast<void*>(g.S), gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dA and dB in one launch (`with_a`, `with_b`: those that TMA can read).
template <int RP, bool F16>
gptq_status launch_grad(const LoraGradArgs& ga, const LoraGradArgs& gb, const LoraGradCommon& c,
                        bool with_a, bool with_b, cudaStream_t s) {
  using Sh = GtShape<RP, F16>;
  CUtensorMap am, bm;
  bool ok = true;
  if (with_a) ok = ok && gt_map(&am, ga, c.m, !F16);
  if (with_b) ok = ok && gt_map(&bm, gb, c.m, !F16);
  if (!with_a) am = bm;
  if (!with_b) bm = am;
  if (!ok || smem_optin((const void*)lora_grad_kernel<RP, F16>, Sh::SMEM) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  const int ba = with_a ? (int)cdiv(ga.C, GT_C) : 0, bb = with_b ? (int)cdiv(gb.C, GT_C) : 0;
  // tokens split over a cluster while the CTAs still fit the device at once and keep a few
  // tiles each
  const int64_t ctas = (int64_t)(ba + bb) * c.na, tiles = cdiv(c.m, GT_T) / c.na;
  int split = 1;
  while (split < 8 && ctas * split * 2 <= sm_count() && tiles / (split * 2) >= 4) split *= 2;
  launch_cluster_pdl(lora_grad_kernel<RP, F16>, dim3((unsigned)((ba + bb) * split), (unsigned)c.na),
                     dim3(Sh::THREADS), Sh::SMEM, split, s, am, bm, ga, gb, c, ba, split);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <bool F16>
gptq_status grad_ranks(const LoraGradArgs& ga, const LoraGradArgs& gb, const LoraGradCommon& c,
                       bool with_a, bool with_b, cudaStream_t s) {
  if (c.r <= 16) return launch_grad<16, F16>(ga, gb, c, with_a, with_b, s);
  if (c.r <= 32) return launch_grad<32, F16>(ga, gb, c, with_a, with_b, s);
  if (c.r <= 64) return launch_grad<64, F16>(ga, gb, c, with_a, with_b, s);
  return launch_grad<128, F16>(ga, gb, c, with_a, with_b, s);
}

}  // namespace

// dA (na, r, k) and dB (na, n, r) from U, V (m, r).
gptq_status lora_grads_impl(const LoraGradArgs& ga, const LoraGradArgs& gb,
                            const LoraGradCommon& c, bool bf16, cudaStream_t s) {
  const bool with_a = c.m > 0 && c.nreq > 0 && gt_supported(ga);
  const bool with_b = c.m > 0 && c.nreq > 0 && gt_supported(gb);
  gptq_status st = GPTQ_OK;
  if (!with_a) st = grad_general(ga, c, bf16, s);
  if (st == GPTQ_OK && !with_b) st = grad_general(gb, c, bf16, s);
  if (st != GPTQ_OK || (!with_a && !with_b)) return st;
  return bf16 ? grad_ranks<false>(ga, gb, c, with_a, with_b, s)
              : grad_ranks<true>(ga, gb, c, with_a, with_b, s);
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
  c.min_len = 1, c.max_len = low.m;
  c.m = low.m, c.r = r, c.na = low.na, c.nreq = low.nreq, c.spin = low.spin;
  LoraGradArgs ga, gb;
  ga.S = X, ga.lds = ldx, ga.s_scales = x_scales, ga.W = low.V, ga.out = dA;
  ga.col_stride = 1, ga.rank_stride = k, ga.C = k;
  gb.S = low.X, gb.lds = low.ldx, gb.s_scales = nullptr, gb.W = V, gb.out = dB;
  gb.col_stride = r, gb.rank_stride = 1, gb.C = n;
  return lora_grads_impl(ga, gb, c, bf16, s);
}

}  // namespace gptq
