// Attention of chunks of new rows over a paged cache, on the sm_100a tensor
// cores (paged_attn.cu takes calls of a few rows a sequence).
//
// o = softmax(scale Q K^T + mask) V with the softmax's running maximum and sum
// over key tiles of 128 positions.  A work unit is 256 rows of one sequence
// and kv head, row = token * group + head, as two tiles of 128 rows that are
// processed in turn, so that every K/V tile serves 256 rows.  The exponentials
// (128 x 256 a key tile) bound it, then the products: 4 HD flops each.
//
// Warps 0-3 and 4-7 are the softmax of the two row tiles, a thread a row: they
// bring their rows of Q to shared memory, read S from tensor memory, write P
// back and rescale O when the maximum grows by more than 2^8.  Warp 8 copies
// pages (a lane a page), warps 9 and 10 issue the two tiles' products.  Warp 11
// (bf16 cache) or warps 12-15 (8 bits) make a copied tile fit to be
// multiplied: positions that no row sees become zeros in V, whose content may
// be anything, and e4m3 codes become f16 (exact).
//
// 8 bits: with value = code * scale a position's key scale multiplies its
// scores and the value scale's exponent joins the exponent of its probability,
// p' = 2^(s + e - m), m the running maximum of s + e; the sum takes p' 2^-e.
// Both are constant over a page, so they cost one multiply a group of 16
// positions, or of 64 where pages are as long (a compiled size, SPAN: 48.2 and
// 47.0 us for 1184 tokens of 32 heads over a window of 2048).  (A head dimension of 16 is below the 32
// elements of an 8-bit product: K and Q become f16 there.)
//
// A head dimension of 128 leaves no room in tensor memory for P beside S and
// O: P then takes the place of S, and S of the next tile waits for P V.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "host.hpp"
#include "paged_plan.hpp"
#include "pdl.cuh"

namespace samba {

template <int HD, bool KV8>
struct ChunkCfg {
  static constexpr bool QK8 = KV8 && HD >= 32;              // 8-bit products for S
  static constexpr int RB = HD * 2 < 128 ? HD * 2 : 128;    // bytes of a panel's row = swizzle span
  static constexpr int NP = HD * 2 / RB;                    // panels a matrix
  static constexpr int PANEL = 128 * RB;
  static constexpr int TILE = NP * PANEL;                   // 128 rows of 16-bit elements
  static constexpr int RAW = 128 * HD;                      // 128 rows of codes
  static constexpr int QRB = QK8 ? HD : RB;                 // the same for Q and K (Q: two matrices of codes)
  static constexpr int KTILE = QK8 ? RAW : TILE;
  static constexpr int STG = HD == 128 ? 2 : 4;             // K/V tiles ready for the products
  static constexpr int RSTG = KV8 ? 2 : 0;                  // copied tiles of codes (QK8: of V)
  static constexpr int RAWS = QK8 ? RAW : 2 * RAW;          // bytes of one
  static constexpr int NFULL = KV8 ? RSTG : STG;
  static constexpr bool AHEAD = HD <= 64;                   // S of the next tile beside P
  static constexpr int Q_OFF = 0, K_OFF = 2 * TILE, V_OFF = K_OFF + STG * KTILE, RAW_OFF = V_OFF + STG * TILE;
  static constexpr int BAR_OFF = RAW_OFF + RSTG * RAWS;
  static constexpr int SC_OFF = BAR_OFF + 256;              // [RSTG + STG][8] scale pairs
  static constexpr int SMEM = SC_OFF + (RSTG + STG) * 64 + 1024;
  static constexpr int swz(int rb) { return rb == 128 ? 2 : rb == 64 ? 4 : 6; }  // descriptors' swizzle codes
  // Of each eight pairs of probabilities, so many go to the FMA pipe (bf16, 64:
  // none, 1, 2 of them 459, 439, 414 us for 8192 rows of 32 heads)
  static constexpr int POLY = KV8 || HD == 128 ? 1 : 2;
  static constexpr int THREADS = KV8 ? 512 : 384;
  static constexpr int CONV_WARP0 = KV8 ? 12 : 11, CONV_WARPS = KV8 ? 4 : 1;
  static constexpr uint32_t COL_S = 0, COL_P = AHEAD ? 256 : 0, COL_O = AHEAD ? 384 : 256;
  static constexpr uint32_t P_STEP = AHEAD ? 64 : 128, O_STEP = AHEAD ? 64 : 128;  // tile B's columns after A's
  static_assert(SMEM <= 227 * 1024, "shared memory");
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
  int Hq, Hkv, group, page_shift, units, nsplit;  // units: pairs of row tiles a sequence may have
  float scale_log2;
};

__device__ __forceinline__ float chunk_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float chunk_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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
// exponent.  Arguments below -125 give 2^-125, which no sum can notice.
__device__ __forceinline__ float2 chunk_ex2_poly(float2 v) {
  const f2 x = pk2(fmaxf(v.x, -125.f), fmaxf(v.y, -125.f));
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
__global__ void __launch_bounds__(ChunkCfg<HD, KV8>::THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const ChunkParams p) {
  using Cfg = ChunkCfg<HD, KV8>;
  constexpr int STG = Cfg::STG, RSTG = Cfg::RSTG, NFULL = Cfg::NFULL;
  constexpr bool QK8 = Cfg::QK8;
  static_assert(CB_STAGE + 3 * STG + NFULL + RSTG <= 30, "barrier block");
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);  // (an offset: still known as shared memory)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cfg::BAR_OFF);
  uint64_t* full = bars + CB_STAGE;     // [NFULL] the copies of a stage landed
  uint64_t* ready = full + NFULL;       // [STG] a tile may be multiplied
  uint64_t* empty = ready + STG;        // [STG] both row tiles are done with it
  uint64_t* rawempty = empty + STG;     // [RSTG] the codes were converted
  uint64_t* kfull = rawempty + RSTG;    // [STG] QK8: the tile of K landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* sc_raw = reinterpret_cast<float2*>(sm + Cfg::SC_OFF);  // [RSTG][8] key scale, value scale exponent
  float2* sc_tile = sc_raw + RSTG * 8;                           // [STG][8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = 1 << p.page_shift;

  pdl_wait();
  // the unit: long ones (late rows) first
  const int split = blockIdx.x % p.nsplit;
  const int rest = blockIdx.x / p.nsplit;
  const int b = rest % static_cast<int>(p.batch.batch), g = blockIdx.y;
  const int unit = p.units - 1 - rest / static_cast<int>(p.batch.batch);
  const SeqSpan sq = seq_span(p.batch, P, b, unit == 0 && split == 0 && g == 0 && threadIdx.x == 0);
  const int row0 = unit * 256, nrow = min(256, sq.n * p.group - row0);
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
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[CB_Q + x], 4);
      mbar_init(&bars[CB_S + x], 1);
      mbar_init(&bars[CB_SF + x], 4);
      mbar_init(&bars[CB_P + x], 4);
      mbar_init(&bars[CB_O + x], 1);
      mbar_init(&bars[CB_DONE + x], 1);
    }
    mbar_init(&bars[CB_GO], 4);
    for (int s = 0; s < NFULL; ++s) mbar_init(&full[s], KV8 ? 2 : 1);  // (8 bits: copies, scales)
    for (int s = 0; s < STG && QK8; ++s) mbar_init(&kfull[s], 1);
    for (int s = 0; s < STG; ++s) {
      mbar_init(&ready[s], Cfg::CONV_WARPS);
      mbar_init(&empty[s], two ? 2 : 1);
    }
    for (int s = 0; s < RSTG; ++s) mbar_init(&rawempty[s], Cfg::CONV_WARPS);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
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

  if (warp >= 8) {
    // 512 threads start at 128 registers: 256 * 64 + 256 * 192 = 512 * 128;
    // 384 at 168: 128 * 88 + 256 * 208 = 384 * 168
    if constexpr (KV8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ============================================================== copies
      if (lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
      const int brows = P < 128 ? P : 128, nbox = 128 / brows;  // a lane a box
      bool ok = true;
      int it = 0;
      auto lookup = [&](int t) {                       // this lane's page of tile t
        const int at = (m0 + t) * 128 + lane * brows;
        if (t >= nt || lane >= nbox || at >= hi || at + brows <= lo) return static_cast<int>(p.num_pages);
        const int v = p.batch.block_table[(int64_t)b * p.batch.max_pages + (at >> p.page_shift)];
        if (v >= 0 && v < p.num_pages) return v;
        report_batch();
        return static_cast<int>(p.num_pages);          // past the pool: read as zeros
      };
      int pg_next = lookup(0);
      for (; it < nt; ++it) {
        const int pg = pg_next;
        float2 sc = make_float2(1.f, 0.f);
        if (KV8 && pg < p.num_pages) {
          const int64_t i = (int64_t)pg * p.Hkv + g;
          sc = make_float2(p.k_scale[i], p.v_scale[i]);
        }
        pg_next = lookup(it + 1);
        const int s = it % NFULL, st = it % STG;
        if (it >= NFULL && !wait(KV8 ? &rawempty[s] : &empty[s], (it / NFULL - 1) & 1)) { ok = false; break; }
        if (QK8 && it >= STG && !wait(&empty[st], (it / STG - 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[s], KV8 ? Cfg::RAWS : 2 * Cfg::TILE);
          if (QK8) mbar_arrive_expect_tx(&kfull[st], Cfg::KTILE);
        }
        __syncwarp();
        if (lane < nbox) {
          const int r = lane * brows, row = ((m0 + it) * 128 + r) & (P - 1), blk = pg * p.Hkv + g;
          if constexpr (KV8) {
            unsigned char* raw = sm + Cfg::RAW_OFF + s * Cfg::RAWS + r * HD;
            if constexpr (QK8) tma_load_3d(sm + Cfg::K_OFF + st * Cfg::KTILE + r * HD, &map_k, &kfull[st], 0, row, blk);
            else tma_load_3d(raw + Cfg::RAW, &map_k, &full[s], 0, row, blk);
            tma_load_3d(raw, &map_v, &full[s], 0, row, blk);
          } else {
#pragma unroll
            for (int pn = 0; pn < Cfg::NP; ++pn) {
              const int at = s * Cfg::TILE + pn * Cfg::PANEL + r * Cfg::RB;
              tma_load_3d(sm + Cfg::K_OFF + at, &map_k, &full[s], pn * (Cfg::RB / 2), row, blk);
              tma_load_3d(sm + Cfg::V_OFF + at, &map_v, &full[s], pn * (Cfg::RB / 2), row, blk);
            }
          }
          if constexpr (KV8) {  // the scales of each 16 positions, under the copies
            const float2 f = make_float2(exp2i(stored_exponent(sc.x)), static_cast<float>(stored_exponent(sc.y)));
            for (int i = 0; i < brows / 16; ++i) sc_raw[s * 8 + lane * (brows / 16) + i] = f;
          }
        }
        if (KV8) warp_arrive(&full[s]);
      }
      if (!ok && lane == 0) {  // copies still in flight after a wait that gave up
        volatile int never = 0;
        for (int i = it > NFULL ? it - NFULL : 0; i < it; ++i) mbar_wait(&full[i % NFULL], (i / NFULL) & 1, &never);
        for (int i = it > STG ? it - STG : 0; i < it && QK8; ++i) mbar_wait(&kfull[i % STG], (i / STG) & 1, &never);
      }
    } else if (warp == 9 || (warp == 10 && two)) {
      // ============================================================ products
      const int x = warp - 9;
      const uint32_t fmt = KV8 ? 0u : (1u << 7) | (1u << 10);  // operands f16 or bf16
      const uint32_t idesc_s = (idesc_bf16_f32(128, 128, 0, 0) & ~((7u << 7) | (7u << 10))) | fmt;
      constexpr int NV = Cfg::RB / 2;                          // columns of O a product: one panel of V
      const uint32_t idesc_o = (idesc_bf16_f32(128, NV, 0, 1) & ~((7u << 7) | (7u << 10))) | fmt;
      const uint64_t dq = smem_desc(smem_u32(sm + Cfg::Q_OFF + x * Cfg::TILE), 16, 8 * Cfg::QRB, Cfg::swz(Cfg::QRB));
      const uint64_t dk = smem_desc(smem_u32(sm + Cfg::K_OFF), 16, 8 * Cfg::QRB, Cfg::swz(Cfg::QRB));
      const uint64_t dv = smem_desc(smem_u32(sm + Cfg::V_OFF), 4096, 8 * Cfg::RB, Cfg::swz(Cfg::RB));
      constexpr uint32_t kTile = Cfg::TILE >> 4, kKTile = Cfg::KTILE >> 4, kPanel = Cfg::PANEL >> 4;
      constexpr int KPP = Cfg::RB / 32;  // steps of 32 bytes a panel
      bool ok = wait(&bars[CB_Q + x], 0);
      auto issue_s = [&](int t) {
        const int s = t % STG;
        if constexpr (!KV8)
          if (!wait(&full[s], (t / STG) & 1)) return false;
        if (!wait(QK8 ? &kfull[s] : &ready[s], (t / STG) & 1)) return false;
        if (Cfg::AHEAD && t > 0 && !wait(&bars[CB_SF + x], (t - 1) & 1)) return false;  // S(t - 1) was read
        tc_fence_after();
        if constexpr (QK8) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {  // the first parts of Q, then the second
            constexpr int KS = HD / 32;
            umma_ss8_w(tmem + Cfg::COL_S + 128 * x, dq + k / KS * (Cfg::RAW >> 4) + 2 * (k % KS), dk + s * kKTile + 2 * (k % KS),
                       idesc_s, k > 0 ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t at = k / KPP * kPanel + 2 * (k % KPP);
            umma_ss_w(tmem + Cfg::COL_S + 128 * x, dq + at, dk + s * kTile + at, idesc_s, k > 0 ? 1u : 0u);
          }
        }
        tc_commit_w(&bars[CB_S + x]);
        return true;
      };
      auto issue_pv = [&](int t) {
        const int s = t % STG;
        if (!wait(&bars[CB_P + x], t & 1)) return false;
        if (QK8 && !wait(&ready[s], (t / STG) & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int pn = 0; pn < Cfg::NP; ++pn)
            umma_ts_w(tmem + Cfg::COL_O + Cfg::O_STEP * x + pn * NV, tmem + Cfg::COL_P + Cfg::P_STEP * x + 8 * k,
                      dv + s * kTile + pn * kPanel + k * Cfg::RB, idesc_o, t > 0 || k > 0 ? 1u : 0u);
        tc_commit_w(&bars[CB_O + x]);
        tc_commit_w(&empty[s]);
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
    } else if (warp >= Cfg::CONV_WARP0) {
      // ======================================== tiles fit to be multiplied
      const int cw = warp - Cfg::CONV_WARP0;
      for (int t = 0; t < nt; ++t) {
        const int s = t % STG, k0 = (m0 + t) * 128;
        const bool edge = k0 < lo || k0 + 128 > hi;
        if constexpr (KV8) {
          const int rs = t % (RSTG > 0 ? RSTG : 1);
          if (!wait(&full[rs], (t / (RSTG > 0 ? RSTG : 1)) & 1)) break;
          if (t >= STG && !wait(&empty[s], (t / STG - 1) & 1)) break;
          const unsigned char* raw = sm + Cfg::RAW_OFF + rs * Cfg::RAWS;
          constexpr int CPR = HD / 16;  // 16-code chunks a row
#pragma unroll 4
          for (int i = cw * 32 + lane; i < Cfg::RAWS / 16; i += 128) {
            const bool is_k = i >= 128 * CPR;
            const int r = (is_k ? i - 128 * CPR : i) / CPR, c = i % CPR;
            uint4 v = *reinterpret_cast<const uint4*>(raw + i * 16);
            if (edge && !is_k && (k0 + r < lo || k0 + r >= hi)) v = make_uint4(0u, 0u, 0u, 0u);
            const uint4 a = make_uint4(e4m3x2_to_f16x2(v.x, false), e4m3x2_to_f16x2(v.x, true),
                                       e4m3x2_to_f16x2(v.y, false), e4m3x2_to_f16x2(v.y, true));
            const uint4 d = make_uint4(e4m3x2_to_f16x2(v.z, false), e4m3x2_to_f16x2(v.z, true),
                                       e4m3x2_to_f16x2(v.w, false), e4m3x2_to_f16x2(v.w, true));
            unsigned char* dst = sm + (is_k ? Cfg::K_OFF : Cfg::V_OFF) + s * Cfg::TILE;
            *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::RB>(r, 2 * c)) = a;
            *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::RB>(r, 2 * c + 1)) = d;
          }
          if (cw == 0 && lane < 8) sc_tile[s * 8 + lane] = sc_raw[rs * 8 + lane];
          fence_proxy_async_shared();
          warp_arrive(&ready[s]);
          if (lane == 0) mbar_arrive(&rawempty[rs]);
        } else {
          if (!wait(&full[s], (t / STG) & 1)) break;
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
    if constexpr (KV8) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
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
      unsigned char* dst = sm + Cfg::Q_OFF + x * Cfg::TILE;
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
        const int ex = min(max(log2i(amax), -60), 126) - (QK8 ? 7 : 0);  // 2^ex <= amax < 2^(ex + 1), or 2^7 of that
        const float by = exp2i(-ex);
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
          if constexpr (QK8) {
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
            *reinterpret_cast<uint4*>(dst + Cfg::RAW + chunk_off<Cfg::QRB>(r, c)) = make_uint4(e[0], e[1], e[2], e[3]);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float* q = f + 8 * j;
              *reinterpret_cast<uint4*>(dst + chunk_off<Cfg::RB>(r, 2 * c + j)) = make_uint4(
                  chunk_pack<true>(q[0], q[1]), chunk_pack<true>(q[2], q[3]), chunk_pack<true>(q[4], q[5]), chunk_pack<true>(q[6], q[7]));
            }
          }
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
    const uint32_t tP = tmem + lane_off + Cfg::COL_P + Cfg::P_STEP * x;
    const uint32_t tO = tmem + lane_off + Cfg::COL_O + Cfg::O_STEP * x;
    // positions of the tile's first and last row
    const int t_lo = first + (row0 + 128 * x) / p.group, t_hi = first + (row0 + min(nrow, 128 * x + 128) - 1) / p.group;
    const int r_lo = p.window > 0 && pos + 1 > p.window ? static_cast<int>(pos + 1 - p.window) : 0;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    // the second tile begins once the first has written its first P, so that
    // the two do not reach their exponentials together
    if (x == 1) ok = wait(&bars[CB_GO], 0);
    for (int t = 0; t < nt && ok; ++t) {
      const int k0 = (m0 + t) * 128, s = t % STG;
      const bool need_mask = k0 + 127 > t_lo || (p.window > 0 && k0 <= t_hi - p.window) || nrow < 128 * x + 128;
      if (!wait(&bars[CB_S + x], t & 1)) { ok = false; break; }
      tc_fence_after();
      uint32_t sr[128];
      tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
      tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
      tc_wait_ld();
      tc_fence_before();
      if (Cfg::AHEAD) warp_arrive(&bars[CB_SF + x]);
      float* sc = reinterpret_cast<float*>(sr);
      if (need_mask) {
        // visible columns [lo_c, lo_c + span]; an empty interval for a row that sees nothing here
        const int lo_c = max(r_lo - k0, 0), hi_c = live ? pos - k0 : -1;
        const int span_i = hi_c - lo_c;
        const unsigned span = span_i < 0 ? 0u : static_cast<unsigned>(span_i);
        const int lo_e = span_i < 0 ? (1 << 20) : lo_c;
#pragma unroll
        for (int c = 0; c < 128; ++c) sc[c] = (unsigned)(c - lo_e) <= span ? sc[c] : -INFINITY;
      }
      // the row's maximum; 8 bits: of each 16 positions, scaled, then of those
      float m_tile;
      if constexpr (KV8) {
        if (!wait(&ready[s], (t / STG) & 1)) { ok = false; break; }  // (passed long ago: orders the scales' reads)
        m_tile = -INFINITY;
#pragma unroll
        for (int q = 0; q < 128 / SPAN; ++q) {
          const float2 f = sc_tile[s * 8 + q * (SPAN / 16)];
          const float ga = fmaxf(rowscale * f.x, 1.17549435e-38f);  // above zero, so that a masked score stays -inf
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = SPAN * q + i;
            m4[i] = chunk_max3(sc[c], sc[c + 4], sc[c + 8]);
#pragma unroll
            for (int j = 12; j < SPAN - 4; j += 8) m4[i] = chunk_max3(m4[i], sc[c + j], sc[c + j + 4]);
            m4[i] = fmaxf(m4[i], sc[c + SPAN - 4]);
          }
          m_tile = fmaxf(m_tile, fmaf(fmaxf(chunk_max3(m4[0], m4[1], m4[2]), m4[3]), ga, f.y));
        }
      } else {
        float m8[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float m = chunk_max3(sc[q], sc[q + 8], sc[q + 16]);
#pragma unroll
          for (int c = 24; c < 120; c += 16) m = chunk_max3(m, sc[c + q], sc[c + 8 + q]);
          m8[q] = fmaxf(m, sc[120 + q]);
        }
        m_tile = fmaxf(chunk_max3(chunk_max3(m8[0], m8[1], m8[2]), chunk_max3(m8[3], m8[4], m8[5]), m8[6]), m8[7]) * rowscale;
      }
      float factor = 1.f;
      bool rescale = false;
      if (m_tile > m_run + 8.f) {
        factor = chunk_ex2(m_run - m_tile);
        m_run = m_tile;
        rescale = true;
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      if (t > 0) {  // the last product still reads P and O
        if (!wait(&bars[CB_O + x], (t - 1) & 1)) { ok = false; break; }
        tc_fence_after();
      }
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
            const float2 f = sc_tile[s * 8 + c / 16];
            const float ga = fmaxf(rowscale * f.x, 1.17549435e-38f);
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
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&bars[CB_P + x]);
      if (t == 0 && x == 0 && lane == 0) mbar_arrive(&bars[CB_GO]);
    }
    if (ok && wait(&bars[CB_O + x], (nt - 1) & 1)) {
      tc_fence_after();
      const bool store = live && SAMBA_CHECK(sq.row0 + tok < p.batch.rows && h < p.Hq && split < p.nsplit);
      float* part = p.ws + ((((int64_t)b * p.batch.max_q + tok) * p.Hq + h) * p.nsplit + split) * (HD + 2);
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll
      for (int q = 0; q < HD / 16; ++q) {
        uint32_t o[16];
        tmem_ld16(tO + 16 * q, o);
        tc_wait_ld();
        if (!store) continue;
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
      if (store && p.nsplit > 1) *reinterpret_cast<float2*>(part) = make_float2(m_run, l_run);
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
  const uint32_t box[3] = {(uint32_t)(KV8 ? HD : Cfg::RB / 2), (uint32_t)std::min(P, 128), 1u};
  auto swizzle = [](int rb) {
    return rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  };
  const CUtensorMapSwizzle swk = KV8 && !Cfg::QK8 ? CU_TENSOR_MAP_SWIZZLE_NONE : swizzle(Cfg::QRB);
  const CUtensorMapSwizzle swv = KV8 ? CU_TENSOR_MAP_SWIZZLE_NONE : swizzle(Cfg::RB);
  const CUtensorMapDataType dt = KV8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int rc = encode_tiled(&mk, dt, 3, a.kv.k, dims, strides, box, swk, "samba_paged_attn K pool");
  if (rc) return rc;
  rc = encode_tiled(&mv, dt, 3, a.kv.v, dims, strides, box, swv, "samba_paged_attn V pool");
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
