// Attention of chunks of new rows over a paged cache, on the sm_100a tensor
// cores (paged_attn.cu takes calls of a few rows a sequence).
//
// o = softmax(scale Q K^T + mask) V with the softmax's running maximum and sum
// over key tiles of 128 positions.  A work unit is one or two tiles of 128 rows of
// a sequence and kv head, row = token * group + head.  The exponentials (128 x 128
// a key tile and row tile) would bound it, then the products (4 HD flops each); what
// it does not reach of that goes to the chain of a row tile: scores, softmax and
// products, one after the other.  Two chains an SM fill each other's gaps:
//
// 8 bits, up to a head dimension of 64: a block has one row tile and half of an
// SM's tensor and shared memory, so two blocks share an SM.  One's start and end
// fall under the other's exponentials, and the last round of units leaves less idle
// (5 sequences of 200 to 1500 new tokens, 32 heads: 112 us, two tiles a block
// 130; 8192 rows: 445 and 519).
//
// bf16, or a head dimension of 128, whose tiles do not fit twice: a block has two
// row tiles that share its keys (bf16, head dimension 64, 4736 rows of 32 heads:
// 135 us, 147 with a tile a block, which copies the keys twice as often).  With
// 128 P takes the place of S, and S of the next key tile waits for P V.
//
// Four warps a row tile are its softmax, a thread a row: they bring their rows of
// Q to shared memory, read S from tensor memory, write P back and rescale O when
// the maximum grows by more than 2^8.  One warp copies pages (a lane a page), one a
// row tile issues the products.  One more (bf16 cache), two or four (8 bits) make a
// copied tile of V fit to be multiplied: positions that no row sees, whose content
// may be anything, become zeros, and e4m3 codes become f16 (exact).
//
// 8 bits: K's codes are multiplied as they are.  A row of Q, brought to a
// maximum of 2^7 to 2^8 by a power of two, is the sum of two e4m3 numbers, the
// nearest one and what that leaves: four significant bits each give bf16's
// eight, down to 2^-10 of the row's maximum (below, the error is 2^-18 of it).
// With value = code * scale a position's key scale multiplies its scores and the
// value scale's exponent joins the exponent of its probability, p' = 2^(s + e -
// m), m the running maximum of s + e; the sum takes p' 2^-e.  Both are constant
// over a page, so they cost one multiply a group of 16 positions, or of 64 where
// pages are as long (a compiled size, SPAN).  An 8-bit product takes 32 elements:
// with a head dimension of 16 the other half of Q and K is zeros, K's filled in by
// the copies, whose box is wider than the pool's rows.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "host.hpp"
#include "paged_plan.hpp"
#include "pdl.cuh"

namespace samba {

template <int HD, bool KV8>
struct ChunkCfg {
  static constexpr int NX = KV8 && HD <= 64 ? 1 : 2;        // row tiles a block (paged_unit has the same rule)
  static constexpr int RB = HD * 2 < 128 ? HD * 2 : 128;    // bytes of a panel's row = swizzle span
  static constexpr int NP = HD * 2 / RB;                    // panels a matrix
  static constexpr int PANEL = 128 * RB;
  static constexpr int TILE = NP * PANEL;                   // 128 rows of 16-bit elements
  static constexpr int RAW = 128 * HD;                      // 128 rows of codes
  static constexpr int KD = KV8 && HD < 32 ? 32 : HD;       // elements of a row of Q and K
  static constexpr int QRB = KV8 ? KD : RB;                 // the span of Q and K (Q: two matrices of codes)
  static constexpr int KTILE = KV8 ? 128 * KD : TILE, QTILE = KV8 ? 2 * KTILE : TILE;
  static constexpr int VS = HD == 128 || KV8 ? 2 : 4;       // tiles of V ready for the products
  static constexpr int RSTG = KV8 ? 2 : 0;                  // copied tiles of V's codes
  // Tiles of K: as many as the copies' waits for V free as well.  (Two row tiles:
  // these wait until V of tile it - VS was multiplied, though codes of it were
  // copied away before: 128, 8 bits, 1184 rows of 32 heads 60 us, 66 without,
  // as the row tiles then reach their exponentials together.)
  static constexpr int KS = NX == 2 ? VS : VS + RSTG;
  static constexpr int NFULL = KV8 ? RSTG : VS;
  static constexpr bool AHEAD = HD <= 64;                   // S of the next tile beside P
  static constexpr int Q_OFF = 0, K_OFF = NX * QTILE, V_OFF = K_OFF + KS * KTILE, RAW_OFF = V_OFF + VS * TILE;
  static constexpr int BAR_OFF = RAW_OFF + RSTG * RAW;
  static constexpr int SC_OFF = BAR_OFF + 512;              // [8 tiles][8] scale pairs
  static constexpr int SMEM = SC_OFF + (KV8 ? 512 : 0) + 1024;
  static constexpr int swz(int rb) { return rb == 128 ? 2 : rb == 64 ? 4 : 6; }  // descriptors' swizzle codes
  // Of each eight pairs of probabilities, so many go to the FMA pipe (bf16, 64,
  // 4736 rows: 1 of them 139 us, 2 135; 8 bits: none 156, 1 155)
  static constexpr int POLY = KV8 || HD == 128 ? 1 : 2;
  // warps: softmax, copies, products (one a row tile), V
  static constexpr int W_COPY = 4 * NX, W_MMA = W_COPY + 1, CONV_WARPS = !KV8 ? 1 : NX == 1 ? 2 : 4;
  static constexpr int WARPS = W_COPY + (KV8 && NX == 2 ? 8 : 4), W_CONV = WARPS - CONV_WARPS;
  static constexpr int THREADS = 32 * WARPS, BLOCKS = NX == 1 ? 2 : 1;
  // Registers a thread at launch, of the softmax warps and of the others: the
  // shares add up to the launch's.
  static constexpr int R0 = KV8 ? 128 : 168;
  static constexpr int R_SOFT = !KV8 ? 208 : NX == 2 ? 192 : 200, R_REST = !KV8 ? 88 : NX == 2 ? 64 : 56;
  static_assert(128 * NX * R_SOFT + (THREADS - 128 * NX) * R_REST == THREADS * R0, "registers");
  static constexpr uint32_t TMEM = NX == 2 ? 512 : 256;
  static constexpr uint32_t COL_S = 0, COL_P = !AHEAD ? 0 : 128 * NX, COL_O = !AHEAD ? 256 : 192 * NX,
                            STEP = AHEAD ? 64 : 128;  // (P's and O's columns of a tile after another's)
  static_assert(SMEM <= (NX == 1 ? 113 : 227) * 1024, "shared memory");
};

// Barriers, each per row tile x: Q written, S ready, S read, P ready, O done,
// all done; tile A's first P ready; then the stages'.
enum : int { CB_Q = 0, CB_S = 2, CB_SF = 4, CB_P = 6, CB_O = 8, CB_DONE = 10, CB_GO = 12, CB_STAGE = 13 };

struct ChunkParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* ws;
  const float* k_scale;
  const float* v_scale;
  samba_paged_batch batch;
  int64_t num_pages, window;
  int Hq, Hkv, group, page_shift, units, nsplit;  // units a sequence may have
  float scale_log2;
};

__device__ __forceinline__ float chunk_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maxima that keep a NaN: a row that sees one shows it.
__device__ __forceinline__ float chunk_max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float chunk_max2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Whether the phase is over, asked ahead of a wait so that the answer is there by
// then (a wait that need not wait still took 200 clocks of a key tile's 3000).
__device__ __forceinline__ bool chunk_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool F16>
__device__ __forceinline__ uint32_t chunk_pack(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Byte offset of 16-byte chunk c of row r in a tile of 128 rows, as panels of
// rows of RB bytes (the swizzle that the products' descriptors name).
template <int RB>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  constexpr int CPR = RB / 16;
  const int ci = c % CPR;
  const int x = RB == 128 ? ci ^ (r & 7) : RB == 64 ? ci ^ ((r >> 1) & 3) : ci ^ ((r >> 2) & 1);
  return static_cast<uint32_t>(c / CPR * (128 * RB) + r * RB + x * 16);
}

// umma_ss_w of common.cuh for e4m3 operands: 32 elements a step.
__device__ __forceinline__ void umma_ss8_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u), "r"(0u), "r"(0u), "r"(0u)
      : "memory");
}

// 2^x for a pair of arguments on the FMA pipe, to about 1e-4 (ample for
// probabilities that are rounded next): x = j + f, j = rint(x) by adding 1.5 *
// 2^23, 2^f a cubic fitted on [-1/2, 1/2] with value 1 at 0, j added to the
// exponent.  Arguments of -127 and less (hidden positions) give zero exactly: the
// cubic's 1 less 127 in the exponent is a float's zero; above -127 the result may
// be subnormal.  A NaN gives zero too, so the row's maximum has to carry it.
__device__ __forceinline__ float2 chunk_ex2_poly(float2 v) {
  const f2 x = pk2(fmaxf(v.x, -127.f), fmaxf(v.y, -127.f));
  const f2 magic = pk2(12582912.f, 12582912.f);
  const f2 t = add2(x, magic);
  const f2 f = sub2(x, sub2(t, magic));
  f2 q = pk2(0x1.c2a212p-5f, 0x1.c2a212p-5f);
  q = fma2(q, f, pk2(0x1.f00c4ep-3f, 0x1.f00c4ep-3f));
  q = fma2(q, f, pk2(0x1.62f5fap-1f, 0x1.62f5fap-1f));
  q = fma2(q, f, pk2(1.f, 1.f));
  const float2 tv = up2(t), qv = up2(q);
  return make_float2(__int_as_float(__float_as_int(qv.x) + (__float_as_int(tv.x) << 23)),
                     __int_as_float(__float_as_int(qv.y) + (__float_as_int(tv.y) << 23)));
}

template <int HD, bool KV8, int SPAN>
__global__ void __launch_bounds__(ChunkCfg<HD, KV8>::THREADS, ChunkCfg<HD, KV8>::BLOCKS)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const ChunkParams p) {
  using Cfg = ChunkCfg<HD, KV8>;
  constexpr int NX = Cfg::NX, KS = Cfg::KS, VS = Cfg::VS, RSTG = Cfg::RSTG, NFULL = Cfg::NFULL;
  static_assert(NX == 2 || KV8, "the copies' waits");
  static_assert(CB_STAGE + KS + NFULL + 2 * VS + RSTG <= 62, "barrier block");
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);  // (an offset: still known as shared memory)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cfg::BAR_OFF);
  uint64_t* kfull = bars + CB_STAGE;    // [KS] a tile of K landed (8 bits: and its scales were written)
  uint64_t* full = kfull + KS;          // [NFULL] a tile of V landed
  uint64_t* ready = full + NFULL;       // [VS] it may be multiplied
  uint64_t* vempty = ready + VS;        // [VS] its products are done
  uint64_t* rawempty = vempty + VS;     // [RSTG] its codes were converted
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 62);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* sc_tile = reinterpret_cast<float2*>(sm + Cfg::SC_OFF);  // [8][8] key scale, value scale exponent
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = 1 << p.page_shift;

  pdl_wait();
  // the unit: long ones (late rows) first
  const int split = blockIdx.x % p.nsplit;
  const int rest = blockIdx.x / p.nsplit;
  const int b = rest % static_cast<int>(p.batch.batch), g = blockIdx.y;
  const int unit = p.units - 1 - rest / static_cast<int>(p.batch.batch);
  const SeqSpan sq = seq_span(p.batch, P, b, unit == 0 && split == 0 && g == 0 && threadIdx.x == 0);
  const int row0 = unit * (128 * NX), nrow = min(128 * NX, sq.n * p.group - row0);
  if (nrow <= 0) return;
  const int first = sq.kv - sq.n;  // position of the sequence's first row
  const int hi = first + (row0 + nrow - 1) / p.group + 1;
  const int p_lo = first + row0 / p.group;
  const int lo = p.window > 0 && p_lo + 1 > p.window ? static_cast<int>(p_lo + 1 - p.window) : 0;
  // this split's key tiles
  const int m_all = lo / 128, n_all = (hi + 127) / 128 - m_all;
  const int m0 = m_all + static_cast<int>(static_cast<int64_t>(n_all) * split / p.nsplit);
  const int nt = m_all + static_cast<int>(static_cast<int64_t>(n_all) * (split + 1) / p.nsplit) - m0;
  auto row_of = [&](int r, int& tok, int& h) {
    tok = (row0 + r) / p.group;
    h = g * p.group + (row0 + r) - tok * p.group;
  };
  if (nt == 0) {  // more splits than tiles: an empty partial
    for (int r = threadIdx.x; r < nrow; r += Cfg::THREADS) {
      int tok, h;
      row_of(r, tok, h);
      p.ws[((((int64_t)b * p.batch.max_q + tok) * p.Hq + h) * p.nsplit + split) * (HD + 2)] = -INFINITY;
    }
    return;
  }

  const bool two = nrow > 128;  // the second row tile has rows
  if (threadIdx.x == 0) {
    for (int x = 0; x < NX; ++x) {
      mbar_init(&bars[CB_Q + x], 4);
      mbar_init(&bars[CB_S + x], KV8 ? 2 : 1);
      mbar_init(&bars[CB_SF + x], 4);
      mbar_init(&bars[CB_P + x], 4);
      mbar_init(&bars[CB_O + x], 1);
      mbar_init(&bars[CB_DONE + x], 1);
    }
    mbar_init(&bars[CB_GO], 4);
    for (int s = 0; s < KS; ++s) mbar_init(&kfull[s], 1);
    for (int s = 0; s < NFULL; ++s) mbar_init(&full[s], 1);
    for (int s = 0; s < VS; ++s) {
      mbar_init(&ready[s], Cfg::CONV_WARPS);
      mbar_init(&vempty[s], two ? 2 : 1);
    }
    for (int s = 0; s < RSTG; ++s) mbar_init(&rawempty[s], Cfg::CONV_WARPS);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == Cfg::W_MMA) {
    tmem_alloc(tmem_slot, Cfg::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Only now: a dependent kernel's block on this SM might else take the tensor
  // memory first and keep it while it waits for this one to end.
  pdl_launch_dependents();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
  };
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp >= Cfg::W_COPY) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::R_REST));
    if (warp == Cfg::W_COPY) {
      // ============================================================== copies
      if (lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
      const int brows = P < 128 ? P : 128, nbox = 128 / brows;  // a lane a box
      bool ok = true;
      int it = 0;
      auto lookup = [&](int t) {  // this lane's page of tile t
        const int at = (m0 + t) * 128 + lane * brows;
        if (t >= nt || lane >= nbox || at >= hi || at + brows <= lo) return static_cast<int>(p.num_pages);
        const int v = p.batch.block_table[(int64_t)b * p.batch.max_pages + (at >> p.page_shift)];
        if (v >= 0 && v < p.num_pages) return v;
        report_batch();
        return static_cast<int>(p.num_pages);  // past the pool: read as zeros
      };
      auto scales_of = [&](int pg) {
        if (!KV8 || pg >= p.num_pages) return make_float2(1.f, 0.f);
        const int64_t i = (int64_t)pg * p.Hkv + g;
        return make_float2(p.k_scale[i], p.v_scale[i]);
      };
      int pg = lookup(0);
      float2 sc = scales_of(pg);
      for (; it < nt; ++it) {
        const int blk = pg * p.Hkv + g, r = lane * brows, row = ((m0 + it) * 128 + r) & (P - 1);
        pg = lookup(it + 1);
        const int ks = it % KS, s = it % NFULL;
        // One row tile: V of tile it - RSTG was converted, for which V of tile it -
        // KS had been multiplied.  K of a tile is done with when its V is.
        if (NX == 2 && it >= VS && !wait(&vempty[it % VS], (it / VS - 1) & 1)) { ok = false; break; }
        if (KV8 && it >= RSTG && !wait(&rawempty[s], (it / NFULL - 1) & 1)) { ok = false; break; }
        if constexpr (KV8) {
          // The scales of each 16 positions.  (Slot it mod 8 was last read for tile
          // it - 8, and the softmax is past tile it - KS.)
          const float2 f = make_float2(exp2i(stored_exponent(sc.x)), static_cast<float>(stored_exponent(sc.y)));
          if (lane < nbox)
            for (int i = 0; i < brows / 16; ++i) sc_tile[it % 8 * 8 + lane * (brows / 16) + i] = f;
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&kfull[ks], Cfg::KTILE);
          mbar_arrive_expect_tx(&full[s], KV8 ? Cfg::RAW : Cfg::TILE);
        }
        __syncwarp();
        if (lane < nbox) {
#pragma unroll
          for (int pn = 0; pn < (KV8 ? 1 : Cfg::NP); ++pn)
            tma_load_3d(sm + Cfg::K_OFF + ks * Cfg::KTILE + pn * Cfg::PANEL + r * Cfg::QRB, &map_k, &kfull[ks], pn * (Cfg::RB / 2),
                        row, blk);
        }
        if (lane < nbox) {
          if constexpr (KV8) {
            tma_load_3d(sm + Cfg::RAW_OFF + s * Cfg::RAW + r * HD, &map_v, &full[s], 0, row, blk);
          } else {
#pragma unroll
            for (int pn = 0; pn < Cfg::NP; ++pn)
              tma_load_3d(sm + Cfg::V_OFF + s * Cfg::TILE + pn * Cfg::PANEL + r * Cfg::RB, &map_v, &full[s], pn * (Cfg::RB / 2), row,
                          blk);
          }
        }
        sc = scales_of(pg);
      }
      if (!ok && lane == 0) {  // copies still in flight after a wait that gave up
        volatile int never = 0;
        for (int i = it > NFULL ? it - NFULL : 0; i < it; ++i) mbar_wait(&full[i % NFULL], (i / NFULL) & 1, &never);
        for (int i = it > KS ? it - KS : 0; i < it; ++i) mbar_wait(&kfull[i % KS], (i / KS) & 1, &never);
      }
    } else if (warp == Cfg::W_MMA || (NX == 2 && warp == Cfg::W_MMA + 1 && two)) {
      // ============================================================ products
      const int x = warp - Cfg::W_MMA;
      const uint32_t fmt = KV8 ? 0u : (1u << 7) | (1u << 10);  // operands e4m3 or f16, or bf16
      const uint32_t idesc_s = (idesc_bf16_f32(128, 128, 0, 0) & ~((7u << 7) | (7u << 10))) | fmt;
      constexpr int NV = Cfg::RB / 2;                          // columns of O a product: one panel of V
      const uint32_t idesc_o = (idesc_bf16_f32(128, NV, 0, 1) & ~((7u << 7) | (7u << 10))) | fmt;
      const uint64_t dq = smem_desc(smem_u32(sm + Cfg::Q_OFF + x * Cfg::QTILE), 16, 8 * Cfg::QRB, Cfg::swz(Cfg::QRB));
      const uint64_t dk = smem_desc(smem_u32(sm + Cfg::K_OFF), 16, 8 * Cfg::QRB, Cfg::swz(Cfg::QRB));
      const uint64_t dv = smem_desc(smem_u32(sm + Cfg::V_OFF), 4096, 8 * Cfg::RB, Cfg::swz(Cfg::RB));
      constexpr uint32_t kTile = Cfg::TILE >> 4, kKTile = Cfg::KTILE >> 4, kPanel = Cfg::PANEL >> 4;
      constexpr int KPP = Cfg::RB / 32;  // steps of 32 bytes a panel
      bool ok = wait(&bars[CB_Q + x], 0);
      auto issue_s = [&](int t) {
        const int s = t % KS;
        if (!wait(&kfull[s], (t / KS) & 1)) return false;
        // S(t - 1) was read, or with P in its place, the products of that P are done
        // (one product is not ordered behind another that reads what it writes)
        if (t > 0 && !wait(&bars[(Cfg::AHEAD ? CB_SF : CB_O) + x], (t - 1) & 1)) return false;
        tc_fence_after();
        if constexpr (KV8) {
#pragma unroll
          for (int k = 0; k < Cfg::KD / 16; ++k) {  // the first parts of Q, then the second
            constexpr int STEPS = Cfg::KD / 32;
            umma_ss8_w(tmem + Cfg::COL_S + 128 * x, dq + k / STEPS * kKTile + 2 * (k % STEPS),
                       dk + s * kKTile + 2 * (k % STEPS), idesc_s, k > 0 ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t at = k / KPP * kPanel + 2 * (k % KPP);
            umma_ss_w(tmem + Cfg::COL_S + 128 * x, dq + at, dk + s * kKTile + at, idesc_s, k > 0 ? 1u : 0u);
          }
        }
        tc_commit_w(&bars[CB_S + x]);
        if (KV8 && lane == 0) mbar_arrive(&bars[CB_S + x]);  // passes the scales on to the softmax
        return true;
      };
      auto issue_pv = [&](int t) {
        const int s = t % VS;
        if constexpr (!KV8)
          if (!wait(&full[s], (t / VS) & 1)) return false;
        if (!wait(&ready[s], (t / VS) & 1)) return false;
        if (!wait(&bars[CB_P + x], t & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int pn = 0; pn < Cfg::NP; ++pn)
            umma_ts_w(tmem + Cfg::COL_O + Cfg::STEP * x + pn * NV, tmem + Cfg::COL_P + Cfg::STEP * x + 8 * k,
                      dv + s * kTile + pn * kPanel + k * Cfg::RB, idesc_o, t > 0 || k > 0 ? 1u : 0u);
        tc_commit_w(&bars[CB_O + x]);
        tc_commit_w(&vempty[s]);
        return true;
      };
      ok = ok && issue_s(0);
      for (int t = 0; t < nt && ok; ++t) {
        if (Cfg::AHEAD) ok = (t + 1 >= nt || issue_s(t + 1)) && issue_pv(t);
        else ok = issue_pv(t) && (t + 1 >= nt || issue_s(t + 1));
      }
      // every product of this warp has finished before tensor memory is released
      tc_commit_w(&bars[CB_DONE + x]);
      volatile int never = 0;
      mbar_wait(&bars[CB_DONE + x], 0, &never);
    } else if (warp >= Cfg::W_CONV) {
      // =================================== tiles of V fit to be multiplied
      const int cw = warp - Cfg::W_CONV;
      for (int t = 0; t < nt; ++t) {
        const int s = t % VS, k0 = (m0 + t) * 128;
        const bool edge = k0 < lo || k0 + 128 > hi;
        if constexpr (KV8) {
          constexpr int R = RSTG > 0 ? RSTG : 1;
          const int rs = t % R;
          if (!wait(&full[rs], (t / R) & 1)) break;
          if (t >= VS && !wait(&vempty[s], (t / VS - 1) & 1)) break;
          const unsigned char* raw = sm + Cfg::RAW_OFF + rs * Cfg::RAW;
          constexpr int CPR = HD / 16;  // 16-code chunks a row
#pragma unroll 1
          for (int i = cw * 32 + lane; i < 128 * CPR; i += 32 * Cfg::CONV_WARPS) {
            const int r = i / CPR, c = i % CPR;
            uint4 v = *reinterpret_cast<const uint4*>(raw + i * 16);
            if (edge && (k0 + r < lo || k0 + r >= hi)) v = make_uint4(0u, 0u, 0u, 0u);
            const uint4 a = make_uint4(e4m3x2_to_f16x2(v.x, false), e4m3x2_to_f16x2(v.x, true),
                                       e4m3x2_to_f16x2(v.y, false), e4m3x2_to_f16x2(v.y, true));
            const uint4 d = make_uint4(e4m3x2_to_f16x2(v.z, false), e4m3x2_to_f16x2(v.z, true),
                                       e4m3x2_to_f16x2(v.w, false), e4m3x2_to_f16x2(v.w, true));
            unsigned char* dst = sm + Cfg::V_OFF + s * Cfg::TILE;
            *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::RB>(r, 2 * c)) = a;
            *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::RB>(r, 2 * c + 1)) = d;
          }
          fence_proxy_async_shared();
          warp_arrive(&ready[s]);
          if (lane == 0) mbar_arrive(&rawempty[rs]);
        } else {
          if (!wait(&full[s], (t / VS) & 1)) break;
          if (edge) {
            constexpr int CPT = HD / 8;  // 16-byte chunks a row
            for (int i = lane; i < 128 * CPT; i += 32) {
              const int r = i / CPT;
              if (k0 + r < lo || k0 + r >= hi)
                *reinterpret_cast<uint4*>(sm + Cfg::V_OFF + s * Cfg::TILE + chunk_off<Cfg::RB>(r, i % CPT)) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_shared();
          }
          warp_arrive(&ready[s]);
        }
      }
    }
  } else {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::R_SOFT));
    const int x = warp >> 2, wq = warp & 3, r = wq * 32 + lane;  // row of the tile
    if (x == 0 || two) {
    const bool live = 128 * x + r < nrow;
    int tok = 0, h = 0;
    row_of(128 * x + (live ? r : 0), tok, h);
    tok = live ? tok : 0;
    const int pos = first + tok;
    const int64_t at = (int64_t)(sq.row0 + tok) * p.Hq + (live ? h : 0);
    float rowscale = p.scale_log2;
    {  // this row of Q
      unsigned char* dst = sm + Cfg::Q_OFF + x * Cfg::QTILE;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + at * HD);
      if constexpr (KV8) {
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < HD / 8; ++c) {
          const uint4 v = live ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            amax = chunk_max3(amax, fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u)));
        }
        const int ex = min(max(log2i(amax), -60), 126) - 7;  // 2^7 <= amax 2^-ex < 2^8
        // (e4m3 has no infinity: a row that holds one is NaN, which its softmax would be)
        const float by = amax <= 3.402823466e38f ? exp2i(-ex) : __int_as_float(0x7fffffff);
        rowscale *= exp2i(ex);
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {  // 16 elements
          float f[16];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 v = live ? src[2 * c + j] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              f[8 * j + 2 * i] = __uint_as_float(w[i] << 16) * by, f[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * by;
          }
          uint32_t u[4], e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = to_e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            const uint32_t l2 = e4m3x2_to_f16x2(u[i], false), h2 = e4m3x2_to_f16x2(u[i], true);
            const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&l2));
            const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            e[i] = to_e4m3x4(f[4 * i] - fl.x, f[4 * i + 1] - fl.y, f[4 * i + 2] - fh.x, f[4 * i + 3] - fh.y);
          }
          *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::QRB>(r, c)) = make_uint4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<uint4*>(dst + Cfg::KTILE + chunk_off<Cfg::QRB>(r, c)) = make_uint4(e[0], e[1], e[2], e[3]);
        }
#pragma unroll
        for (int c = HD / 16; c < Cfg::KD / 16; ++c) {
          *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::QRB>(r, c)) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(dst + Cfg::KTILE + chunk_off<Cfg::QRB>(r, c)) = make_uint4(0u, 0u, 0u, 0u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < HD / 8; ++c)
          *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::RB>(r, c)) = live ? src[c] : make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_shared();
      warp_arrive(&bars[CB_Q + x]);
    }
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + Cfg::COL_S + 128 * x;
    const uint32_t tP = tmem + lane_off + Cfg::COL_P + Cfg::STEP * x;
    const uint32_t tO = tmem + lane_off + Cfg::COL_O + Cfg::STEP * x;
    // positions of the tile's first and last row
    const int t_lo = first + (row0 + 128 * x) / p.group, t_hi = first + (row0 + min(nrow, 128 * x + 128) - 1) / p.group;
    const int r_lo = p.window > 0 && pos + 1 > p.window ? static_cast<int>(pos + 1 - p.window) : 0;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    // the second tile begins once the first has written its first P, so that
    // the two do not reach their exponentials together
    if (x == 1) ok = wait(&bars[CB_GO], 0);
    bool s_ready = false;  // S of the coming tile was seen to be there
    auto wait_after = [&](bool seen, uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, seen) || wait(bar, parity); };
    for (int t = 0; t < nt && ok; ++t) {
      if (!wait_after(s_ready, &bars[CB_S + x], t & 1)) { ok = false; break; }
      tc_fence_after();
      const int k0 = (m0 + t) * 128;
      const bool need_mask = k0 + 127 > t_lo || (p.window > 0 && k0 <= t_hi - p.window) || nrow < 128 * x + 128;
      // visible columns [lo_c, lo_c + span]; an empty interval for a row that sees nothing here
      const int lo_c = max(r_lo - k0, 0), span_i = (live ? pos - k0 : -1) - lo_c;
      const unsigned span = span_i < 0 ? 0u : static_cast<unsigned>(span_i);
      const int lo_e = span_i < 0 ? (1 << 20) : lo_c;
      const float2* tile_sc = sc_tile + t % 8 * 8;
      // the factor of a group's scores: above zero, so that a masked score stays -inf
      auto factor_of = [&](float2 f) { return fmaxf(rowscale * f.x, 1.17549435e-38f); };
      uint32_t sr[128];
      float* sc = reinterpret_cast<float*>(sr);
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(tS + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * i]));
      tc_wait_ld();
      auto read_done = [&] {
        tc_fence_before();
        if (Cfg::AHEAD) warp_arrive(&bars[CB_SF + x]);
      };
      // S of the next tile is early enough either way: with 8 bits told after the
      // maximum (112 us, 114 before it), with bf16 before (401 us, 406 after)
      if constexpr (!KV8) read_done();
      if (need_mask) {
#pragma unroll
        for (int c = 0; c < 128; ++c) sc[c] = (unsigned)(c - lo_e) <= span ? sc[c] : -INFINITY;
      }
      // the row's maximum; 8 bits: of each SPAN positions, scaled, then of those
      float m_tile = -INFINITY;
      constexpr int G = KV8 ? SPAN : 64;  // positions of one factor
#pragma unroll
      for (int q = 0; q < 128 / G; ++q) {
        float m4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = G * q + i;
          m4[i] = chunk_max3(sc[c], sc[c + 4], sc[c + 8]);
#pragma unroll
          for (int j = 12; j < G - 4; j += 8) m4[i] = chunk_max3(m4[i], sc[c + j], sc[c + j + 4]);
          m4[i] = chunk_max2(m4[i], sc[c + G - 4]);
        }
        const float mq = chunk_max2(chunk_max3(m4[0], m4[1], m4[2]), m4[3]);
        if constexpr (KV8) {
          const float2 f = tile_sc[q * SPAN / 16];
          m_tile = chunk_max2(m_tile, fmaf(mq, factor_of(f), f.y));
        } else {
          m_tile = chunk_max2(m_tile, mq * rowscale);
        }
      }
      if constexpr (KV8) read_done();
      // the row's reference m_run lies kRef below its maximum
      constexpr float kRef = KV8 ? kScaledRef : 0.f;
      float factor = 1.f;
      bool rescale = false;
      if (!(m_tile <= m_run + kRef + 8.f)) {  // (or NaN)
        // A score of NaN or infinity makes its row NaN from here on, as a softmax does.
        const float m_new = chunk_max2(m_run, fmaf(m_tile, 0.f, m_tile) - kRef);
        factor = chunk_ex2(m_run - m_new);
        m_run = m_new;
        rescale = true;
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      const bool o_done = t > 0 && chunk_test(&bars[CB_O + x], (t - 1) & 1);
      float sum = 0.f;
      f2 acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)}, a2 = pk2(rowscale, rowscale), c2 = pk2(-m_use, -m_use);
      float inv = 1.f;  // 1 / value scale of the group
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int c = 32 * k + 2 * j;
          if (KV8 && c % SPAN == 0) {
            const float2 f = tile_sc[c / 16];
            const float ga = factor_of(f);
            a2 = pk2(ga, ga);
            c2 = pk2(f.y - m_use, f.y - m_use);
            inv = exp2i(-static_cast<int>(f.y));
          }
          const float2 xv = up2(fma2(pk2(sc[c], sc[c + 1]), a2, c2));
          const float2 ev = j % 8 < Cfg::POLY ? chunk_ex2_poly(xv) : make_float2(chunk_ex2(xv.x), chunk_ex2(xv.y));
          acc[j & 1] = add2(acc[j & 1], pk2(ev.x, ev.y));
          pk[j] = chunk_pack<KV8>(ev.x, ev.y);
          if (KV8 && (c + 2) % SPAN == 0) {
            const float2 tot = up2(add2(acc[0], acc[1]));
            sum = fmaf(tot.x + tot.y, inv, sum);
            acc[0] = acc[1] = pk2(0.f, 0.f);
          }
        }
        if (k == 0) {  // until here the last product may read P and O
          if (t > 0) {
            ok = wait_after(o_done, &bars[CB_O + x], (t - 1) & 1);
            tc_fence_after();
          } else {
            __syncwarp();  // (as the vote in a wait: the store below is the whole warp's)
          }
        }
        tmem_st16(tP + 16 * k, pk);
      }
      if constexpr (!KV8) {
        const float2 tot = up2(add2(acc[0], acc[1]));
        sum = tot.x + tot.y;
      }
      l_run = l_run * factor + sum;
      if (__any_sync(0xffffffffu, t > 0 && rescale)) {  // factor is 1 in the rows that keep theirs
        uint32_t o[16];
#pragma unroll
        for (int q = 0; q < HD / 16; ++q) {
          tmem_ld16(tO + 16 * q, o);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * factor);
          tmem_st16(tO + 16 * q, o);
        }
      }
      s_ready = Cfg::AHEAD && chunk_test(&bars[CB_S + x], (t + 1) & 1);
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&bars[CB_P + x]);
      if (NX == 2 && t == 0 && x == 0 && lane == 0) mbar_arrive(&bars[CB_GO]);
    }
    if (ok && wait(&bars[CB_O + x], (nt - 1) & 1)) {
      tc_fence_after();
      const bool store = live && SAMBA_CHECK(sq.row0 + tok < p.batch.rows && h < p.Hq && split < p.nsplit);
      float* part = p.ws + ((((int64_t)b * p.batch.max_q + tok) * p.Hq + h) * p.nsplit + split) * (HD + 2);
      const float inv = 1.f / l_run;  // (infinite where every score was -infinity: NaN)
#pragma unroll
      for (int q = 0; q < HD / 16; ++q) {
        uint32_t o[16];
        __syncwarp();  // lanes without a row have stored nothing; the load is the whole warp's
        tmem_ld16(tO + 16 * q, o);
        tc_wait_ld();
        if (store) {
          if (p.nsplit == 1) {
            uint32_t v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
              v[c] = chunk_pack<false>(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv);
            uint4* dst = reinterpret_cast<uint4*>(p.o + at * HD + 16 * q);
            dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
            dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
          } else {
#pragma unroll
            for (int c = 0; c < 16; c += 2)
              *reinterpret_cast<float2*>(part + 2 + 16 * q + c) = make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1]));
          }
        }
      }
      if (store && p.nsplit > 1) *reinterpret_cast<float2*>(part) = make_float2(m_run, l_run);
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM);
  }
}

// ------------------------------------------------------------------- launcher
template <int HD, bool KV8, int SPAN>
static int chunk_go(const samba_paged_attn_args& a, const PagedPlan& pl, cudaStream_t s) {
  using Cfg = ChunkCfg<HD, KV8>;
  auto kern = paged_chunk_kernel<HD, KV8, SPAN>;
  static PerDeviceOnce attr;
  const int arc = once_per_device(attr, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM) == cudaSuccess
               ? SAMBA_OK
               : fail(SAMBA_ERR_CUDA, "samba_paged_attn: cannot set shared memory size");
  });
  if (arc != SAMBA_OK) return arc;
  const int P = a.kv.page_size, el = KV8 ? 1 : 2;
  CUtensorMap mk, mv;
  const uint64_t dims[3] = {(uint64_t)HD, (uint64_t)P, (uint64_t)a.kv.num_pages * a.kv.heads_kv};
  const uint64_t strides[2] = {(uint64_t)HD * el, (uint64_t)HD * el * P};
  const uint32_t box_k[3] = {(uint32_t)(KV8 ? Cfg::KD : Cfg::RB / 2), (uint32_t)std::min(P, 128), 1u};
  const uint32_t box_v[3] = {(uint32_t)(KV8 ? HD : Cfg::RB / 2), (uint32_t)std::min(P, 128), 1u};
  auto swizzle = [](int rb) {
    return rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  };
  const CUtensorMapSwizzle swk = swizzle(Cfg::QRB);
  const CUtensorMapSwizzle swv = KV8 ? CU_TENSOR_MAP_SWIZZLE_NONE : swizzle(Cfg::RB);
  const CUtensorMapDataType dt = KV8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int rc = encode_tiled(&mk, dt, 3, a.kv.k, dims, strides, box_k, swk, "samba_paged_attn K pool");
  if (rc) return rc;
  rc = encode_tiled(&mv, dt, 3, a.kv.v, dims, strides, box_v, swv, "samba_paged_attn V pool");
  if (rc) return rc;
  ChunkParams p;
  p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  p.o = reinterpret_cast<__nv_bfloat16*>(a.o);
  p.ws = reinterpret_cast<float*>(a.workspace);
  p.k_scale = a.kv.k_scale;
  p.v_scale = a.kv.v_scale;
  p.batch = a.batch;
  p.num_pages = a.kv.num_pages;
  p.window = a.window;
  p.Hq = a.heads_q;
  p.Hkv = a.kv.heads_kv;
  p.group = a.heads_q / a.kv.heads_kv;
  p.page_shift = 31 - __builtin_clz((unsigned)P);
  p.units = pl.ntile;
  p.nsplit = pl.nsplit;
  p.scale_log2 = paged_scale_log2(a);
  const int64_t gx = a.batch.batch * pl.ntile * pl.nsplit;
  if (gx > INT32_MAX) return fail(SAMBA_ERR_UNSUPPORTED, "samba_paged_attn: too many rows");
  const cudaError_t e =
      launch_pdl(kern, dim3((unsigned)gx, a.kv.heads_kv), dim3(Cfg::THREADS), Cfg::SMEM, s, mk, mv, p);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "samba_paged_attn: launch failed: %s", cudaGetErrorString(e));
  return check_launch("samba_paged_attn");
}

template <int HD>
static int chunk_hd(const samba_paged_attn_args& a, const PagedPlan& pl, cudaStream_t s) {
  if (a.kv.dtype == SAMBA_BF16) return chunk_go<HD, false, 64>(a, pl, s);
  return a.kv.page_size >= 64 ? chunk_go<HD, true, 64>(a, pl, s) : chunk_go<HD, true, 16>(a, pl, s);
}

int launch_paged_chunk(const samba_paged_attn_args& a, const PagedPlan& pl, cudaStream_t s) {
  switch (a.kv.head_dim) {
    case 16: return chunk_hd<16>(a, pl, s);
    case 32: return chunk_hd<32>(a, pl, s);
    case 64: return chunk_hd<64>(a, pl, s);
    default: return chunk_hd<128>(a, pl, s);
  }
}

int take_status_paged_chunk(cudaStream_t s) { return take_status_word(s); }

}  // namespace samba
