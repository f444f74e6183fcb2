// Attention of the newest rows of every sequence over a paged cache.
//
// o = sum_j softmax_j(scale q.k_j) v_j.  An e4m3 cache has a power-of-two
// scale a (page, kv head): with value = code * scale the key scale multiplies
// the score, and the value scale 2^e(j) goes into the exponent of the
// probability, p'_j = 2^(s_j + e(j) - m) with m the running maximum of
// s_j + e(j), so that
//   o = sum_j p'_j code_j / sum_j p'_j 2^-e(j)
// and no tile is ever rescaled element by element.
//
// A few rows of queries (the heads of a kv head by the sequence's new rows)
// meet a long cache, so reading K and V once bounds the call: 2 d bytes or
// 4 d bytes a position and kv head.  The positions are split over thread
// blocks; in a block each of the four warps streams its own share through its own ring
// of TMA stages (one box a page), so no warp waits for another until the
// warps' states are merged at the end.  Scores are computed transposed, S^T = K Q^T:
// 16 positions fill the 16 rows of an m16n8k16 product and 8 query rows its
// 8 columns, so nothing is spent on padding rows, and each thread
// holds the scores of two query rows.  P^T then enters O^T = V^T P^T through one
// in-register 8 x 8 transpose.  The running maximum moves only when a score exceeds
// it by more than 2^8 (a warp vote), so the common case needs no reduction across
// lanes at all.
//
// e4m3 codes become f16 in registers (exact), so the products run in f16:
// queries are scaled by a power of two a row into [1, 2) first, and p' between 2^7
// and 2^15 at a row's maximum fits and leaves f16's range to what lies below
// (paged.cuh).  A bf16 cache multiplies in bf16.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "host.hpp"
#include "paged_plan.hpp"
#include "pdl.cuh"

namespace samba {

// ------------------------------------------------------------- matrix pieces
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with C = 0.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_b16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_ap(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------ configuration
template <int HD, bool KV8, int NT>
struct PagedCfg {
  static constexpr int ES = KV8 ? 1 : 2;              // bytes an element
  static constexpr int ROWB = HD * ES;                // bytes a cache row
  static constexpr int RB = ROWB < 128 ? ROWB : 128;  // bytes a panel row = swizzle span
  static constexpr int NPANEL = ROWB / RB;
  static constexpr int PE = RB / ES;                  // elements a panel row
  // Positions a warp's stage: a whole number of 16-row pages, 8 KB or less a
  // stage, so that a block of three or four stages a warp stays near 48 KB
  // to 96 KB and several blocks share an SM.
  static constexpr int SW = ROWB >= 256 ? 16 : 32;
  static constexpr int MAT = SW * ROWB;               // bytes of K (or V) a stage
  static constexpr int STAGE = 2 * MAT;
  static constexpr int STG = 3;
  static constexpr int WARPS = 4;
  static constexpr int ROWS = 8 * NT;                 // query rows a block
  static constexpr int RING = WARPS * STG * STAGE;
  // the warps' results, then the block's: [WARPS + 1][ROWS][HD] and their maxima and sums
  static constexpr int MERGE = (WARPS + 1) * ROWS * (HD + 2) * 4;
  static constexpr int BAR_OFF = RING > MERGE ? RING : (MERGE + 127) / 128 * 128;
  static constexpr int TAB_OFF = BAR_OFF + 128;       // then the block's pages: scales, numbers
};

// Byte offset of 16-byte chunk c of row r in a stage matrix, as the tensor
// copy lays it out (panels of SW rows; chunks permuted by the swizzle of the span).
template <class Cfg>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  constexpr int CPR = Cfg::RB / 16;
  const int panel = c / CPR, ci = c % CPR;
  int x = ci;
  if constexpr (Cfg::RB == 128) x = ci ^ (r & 7);
  else if constexpr (Cfg::RB == 64) x = ci ^ ((r >> 1) & 3);
  else if constexpr (Cfg::RB == 32) x = ci ^ ((r >> 2) & 1);
  return static_cast<uint32_t>(panel * Cfg::SW * Cfg::RB + r * Cfg::RB + x * 16);
}

// e4m3: which position (of 8) row c = 2t + e of a product holds.  A thread's K
// read takes rows 2t, 2t + 1 in one phase and its V reads take the positions
// of t = 0..3 for one e; this order makes both free of bank conflicts for
// each row size (found by going through the swizzled banks).
template <int HD>
__device__ __forceinline__ int slot_of(int c) {
  const int e = c & 1, t0 = (c >> 1) & 1, t1 = c >> 2;
  if constexpr (HD == 128) return t1 + 2 * t0 + 4 * (e ^ t1);
  else if constexpr (HD == 64) return (e ^ t0) + 2 * t0 + 4 * t1;
  else if constexpr (HD == 32) return t0 + 2 * (e ^ t1) + 4 * e;
  else return c;
}

struct PagedParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* ws;           // [batch][max_q][Hq][npart][HD + 2] partial results, or null
  const float* k_scale;
  const float* v_scale;
  samba_paged_batch batch;
  int64_t num_pages;
  int64_t window;
  int Hq, Hkv, group, page_shift;
  int ntile;           // row tiles a sequence
  int nsplit, chunk;   // splits a row tile, positions a split at most (a multiple of 32)
  int cluster, npart;  // splits a cluster joins, results that leaves
  int ctab;            // pages a split can touch
  float scale_log2;
};

// The rows of one tile and what they see: positions [lo, hi).
struct TileSpan {
  int row0, nrow;    // first query row (within the sequence), rows: row = token * group + head
  int seq_row0, first;  // the sequence's first row of the call, its position
  int lo, hi;
};

__device__ __forceinline__ TileSpan tile_span(const PagedParams& p, int b, int tile, int rows, int page_size, bool report) {
  const SeqSpan s = seq_span(p.batch, page_size, b, report);
  TileSpan t;
  t.row0 = tile * rows;
  t.nrow = min(rows, s.n * p.group - t.row0);
  t.seq_row0 = s.row0;
  t.first = s.kv - s.n;
  if (t.nrow <= 0) {
    t.nrow = t.lo = t.hi = 0;
    return t;
  }
  const int p0 = t.first + t.row0 / p.group, p1 = t.first + (t.row0 + t.nrow - 1) / p.group;
  t.hi = p1 + 1;
  t.lo = p.window > 0 && p0 + 1 > p.window ? static_cast<int>(p0 + 1 - p.window) : 0;
  return t;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A float of another block of the cluster: `p` is this block's address of it.
__device__ __forceinline__ float cluster_load(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <int HD, bool KV8, int NT>
__global__ void __launch_bounds__(128) paged_split_kernel(const __grid_constant__ CUtensorMap map_k,
                                                          const __grid_constant__ CUtensorMap map_v,
                                                          const PagedParams p) {
  using Cfg = PagedCfg<HD, KV8, NT>;
  constexpr int SW = Cfg::SW, STG = Cfg::STG, NG = SW / 16, NMT = HD / 16, NKS = HD / 16, ROWS = Cfg::ROWS;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);  // (an offset: still known as shared memory)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cfg::BAR_OFF);  // [WARPS][STG]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + Cfg::WARPS * STG);
  float4* sct = reinterpret_cast<float4*>(sm + Cfg::TAB_OFF);  // [ctab] key scale, value scale 2^e: e, 2^-e
  int* tab = reinterpret_cast<int*>(sct + (KV8 ? p.ctab : 0));  // [ctab] page numbers (num_pages: none)
  float* Ow = reinterpret_cast<float*>(sm);                    // after the ring's last use: [WARPS + 1][ROWS][HD]
  float* wm = Ow + (Cfg::WARPS + 1) * ROWS * HD;               // [WARPS + 1][ROWS] maxima
  float* wl = wm + (Cfg::WARPS + 1) * ROWS;                    // sums
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int split = blockIdx.x % p.nsplit, tile = blockIdx.x / p.nsplit % p.ntile, b = blockIdx.x / p.nsplit / p.ntile;
  const int g = blockIdx.y, P = 1 << p.page_shift;

  if (tid < Cfg::WARPS * STG) mbar_init(&bars[tid], 1);
  if (tid == 0) {
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  pdl_launch_dependents();
  pdl_wait();
  const TileSpan t = tile_span(p, b, tile, ROWS, P, split == 0 && tile == 0 && g == 0 && tid == 0);
  if (t.nrow == 0) return;  // all blocks of the cluster
  // this block's positions: its share of the range that starts at a stage boundary
  const int base = t.lo / 32 * 32;
  const int share = p.cluster == 1 ? p.chunk : min(p.chunk, ((t.hi - base + p.nsplit - 1) / p.nsplit + 31) / 32 * 32);
  const int64_t c0 = base + static_cast<int64_t>(split) * share;
  const int c_lo = static_cast<int>(c0 < t.hi ? c0 : t.hi);
  const int c_hi = static_cast<int>(c0 + share < t.hi ? c0 + share : t.hi);
  const int nsub = (c_hi - c_lo + SW - 1) / SW;
  bool done = false;  // this block has a result
  if (nsub > 0) {
  // the pages of [c_lo, c_hi): those with a visible position are looked up, the rest read as nothing
  const int pg0 = c_lo >> p.page_shift, npg = ((c_hi - 1) >> p.page_shift) - pg0 + 1;
  int pg_first = static_cast<int>(p.num_pages);  // the thread's first page, whose scales are read below
  for (int i = tid; i < p.ctab; i += 128) {
    int pg = static_cast<int>(p.num_pages);
    if (i < npg && ((pg0 + i + 1) << p.page_shift) > t.lo) {
      const int v = p.batch.block_table[(int64_t)b * p.batch.max_pages + pg0 + i];
      if (v >= 0 && v < p.num_pages) pg = v;
      else report_batch();
    }
    tab[i] = pg;
    if (i == tid) pg_first = pg;
  }
  __syncthreads();

  // A lane issues one box: K or V, a panel, min(P, SW) rows of a page.
  const int brows = P < SW ? P : SW;
  unsigned char* ring = sm + warp * (STG * Cfg::STAGE);
  uint64_t* mybar = bars + warp * STG;
  const int bx_row = lane / (2 * Cfg::NPANEL) * brows, bx_pn = (lane >> 1) % Cfg::NPANEL;
  const bool bx_in = bx_row < SW;
  const uint32_t bx_dst = (lane & 1) * Cfg::MAT + bx_pn * SW * Cfg::RB + bx_row * Cfg::RB;
  const CUtensorMap* bx_map = (lane & 1) ? &map_v : &map_k;
  auto issue = [&](int st, int j) {  // positions j .. of the warp's stage st
    if (lane == 0) mbar_arrive_expect_tx(&mybar[st], Cfg::STAGE);
    __syncwarp();
    if (bx_in) {
      const int pg = tab[((j + bx_row) >> p.page_shift) - pg0];  // num_pages: past the pool, read as zeros
      tma_load_3d(ring + st * Cfg::STAGE + bx_dst, bx_map, &mybar[st], bx_pn * Cfg::PE, (j + bx_row) & (P - 1),
                  pg * p.Hkv + g);
    }
  };
  const int mine = (nsub - warp + Cfg::WARPS - 1) / Cfg::WARPS;  // stages of this warp
  for (int i = 0; i < STG && i < mine; ++i) issue(i, c_lo + (warp + i * Cfg::WARPS) * SW);
  if constexpr (KV8) {  // under the first copies
    for (int i = tid; i < p.ctab; i += 128) {
      const int pg = i == tid ? pg_first : tab[i];
      float4 sc = make_float4(1.f, 0.f, 1.f, 0.f);
      if (pg < p.num_pages) {
        const int64_t at = (int64_t)pg * p.Hkv + g;
        const int ke = stored_exponent(p.k_scale[at]), ve = stored_exponent(p.v_scale[at]);
        sc = make_float4(exp2i(ke), static_cast<float>(ve), exp2i(-ve), 0.f);
      }
      sct[i] = sc;
    }
  }

  // Query fragments (the B operand): column gq of tile nt is query row 8 nt + gq.
  uint32_t qb[NT][NKS][2];
  float rf[NT][2];  // score factors of the thread's two rows 8 nt + 2 tq, + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + gq;
    const bool in = r < t.nrow;
    const int rr = t.row0 + (in ? r : 0), tok = rr / p.group, h = g * p.group + rr % p.group;
    const __nv_bfloat16* qr = p.q + ((int64_t)(t.seq_row0 + tok) * p.Hq + h) * HD;
    float f = p.scale_log2;
    if constexpr (KV8) {
      // K's elements of a product step are four neighbours, so the row is read the same way
      constexpr int PER = HD >= 64 ? 16 : HD / 4;  // neighbours a thread takes of each 64 elements (or all)
      float v[NKS][4], amax = 0.f;
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        const int d0 = 64 * (s / 4) + PER * tq + 4 * (s % 4);
        uint2 w = make_uint2(0u, 0u);
        if (in) w = *reinterpret_cast<const uint2*>(qr + d0);
        v[s][0] = __uint_as_float(w.x << 16);
        v[s][1] = __uint_as_float(w.x & 0xffff0000u);
        v[s][2] = __uint_as_float(w.y << 16);
        v[s][3] = __uint_as_float(w.y & 0xffff0000u);
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(v[s][e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^ex <= amax < 2^(ex + 1); zero, tiny and infinite rows are left near as they are
      const int ex = min(max(log2i(amax), -100), 126);
      const float by = exp2i(-ex);
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        qb[nt][s][0] = pack_f16x2(v[s][0] * by, v[s][1] * by);
        qb[nt][s][1] = pack_f16x2(v[s][2] * by, v[s][3] * by);
      }
      f *= exp2i(ex);
    } else {
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        qb[nt][s][0] = in ? *reinterpret_cast<const uint32_t*>(qr + 16 * s + 2 * tq) : 0u;
        qb[nt][s][1] = in ? *reinterpret_cast<const uint32_t*>(qr + 16 * s + 2 * tq + 8) : 0u;
      }
    }
    rf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * tq);       // the lane of column 2 tq
    rf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
  }
  // what the thread's rows see: positions [rlo, rhi) of each
  int rlo[NT][2], rhi[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * tq + e;
      const int pos = t.first + (t.row0 + r) / p.group;
      rhi[nt][e] = r < t.nrow ? min(pos + 1, c_hi) : 0;
      rlo[nt][e] = p.window > 0 && pos + 1 > p.window ? static_cast<int>(pos + 1 - p.window) : 0;
    }
  // stages inside [full_lo, full_hi) are visible to every row of the tile
  const int last = t.hi - 1, firstp = t.first + t.row0 / p.group;
  const int full_lo = p.window > 0 && last + 1 > p.window ? static_cast<int>(last + 1 - p.window) : 0;
  const int full_hi = min(firstp + 1, c_hi);

  float o[NT][NMT][4], l[NT][2], m[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    l[nt][0] = l[nt][1] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
#pragma unroll
    for (int i = 0; i < NMT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
  }
  if constexpr (KV8) __syncthreads();  // the scales are there
  // A thread's places in a stage: rows 8 apart share the swizzle, so only the
  // first is worked out.
  uint32_t koff, voff[2];
  if constexpr (KV8) {
    const int r = slot_of<HD>(gq);
    koff = HD >= 64   ? tile_off<Cfg>(r, tq)
           : HD == 32 ? tile_off<Cfg>(r, tq >> 1) + 8 * (tq & 1)
                      : tile_off<Cfg>(r, 0) + 4 * tq;
    constexpr int NB = HD / 8;
    for (int e = 0; e < 2; ++e) voff[e] = tile_off<Cfg>(slot_of<HD>(2 * tq + e), NB * gq / 16) + (NB * gq) % 16;
  } else {
    koff = tile_off<Cfg>(lane & 15, lane >> 4);
    voff[0] = tile_off<Cfg>((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1);
    voff[1] = 0;
  }
  bool ok = true;
  int it = 0, st = 0, j0 = c_lo + warp * SW;
  uint32_t ph = 0;
  for (; it < mine; ++it, j0 += Cfg::WARPS * SW) {
    ok = __all_sync(0xffffffffu, mbar_wait(&mybar[st], ph, abort_flag));
    if (!ok) break;
    const unsigned char* Ks = ring + st * Cfg::STAGE + koff;
    const unsigned char* Vs = ring + st * Cfg::STAGE + Cfg::MAT;
    const bool edge = j0 < full_lo || j0 + SW > full_hi;
    // scores: S^T[position, row]; accumulator rows gq and gq + 8 of group u
    float s[NT][NG][4];
    float kv_e[NG], inv_v[NG];
    const uint32_t kaddr = smem_u32(Ks), vaddr = smem_u32(Vs) + voff[0];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      if constexpr (KV8) {
        constexpr int NB = HD >= 64 ? 16 : HD / 4;       // bytes a thread reads of each 64 (or all)
        constexpr int NH = HD >= 64 ? HD / 64 : 1;
        uint32_t wa[NH][NB / 4], wb[NH][NB / 4];
#pragma unroll
        for (int hf = 0; hf < NH; ++hf) {
          // (the second 64 elements: the chunk's bit 2, flipped)
          const unsigned char* pa = hf == 0 ? Ks : ring + st * Cfg::STAGE + (koff ^ 64u);
          pa += 16 * u * Cfg::RB;
          if constexpr (NB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(pa);
            const uint4 y = *reinterpret_cast<const uint4*>(pa + 8 * Cfg::RB);
            wa[hf][0] = x.x, wa[hf][1] = x.y, wa[hf][2] = x.z, wa[hf][3] = x.w;
            wb[hf][0] = y.x, wb[hf][1] = y.y, wb[hf][2] = y.z, wb[hf][3] = y.w;
          } else if constexpr (NB == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(pa);
            const uint2 y = *reinterpret_cast<const uint2*>(pa + 8 * Cfg::RB);
            wa[hf][0] = x.x, wa[hf][1] = x.y;
            wb[hf][0] = y.x, wb[hf][1] = y.y;
          } else {
            wa[hf][0] = *reinterpret_cast<const uint32_t*>(pa);
            wb[hf][0] = *reinterpret_cast<const uint32_t*>(pa + 8 * Cfg::RB);
          }
        }
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) {
          const uint32_t x = wa[ks / 4][ks % 4], y = wb[ks / 4][ks % 4];
          const uint32_t a[4] = {e4m3x2_to_f16x2(x, false), e4m3x2_to_f16x2(y, false), e4m3x2_to_f16x2(x, true),
                                 e4m3x2_to_f16x2(y, true)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (ks == 0) mma_f16_first(s[nt][u], a, qb[nt][ks][0], qb[nt][ks][1]);
            else mma_f16_16816(s[nt][u], a, qb[nt][ks][0], qb[nt][ks][1]);
          }
        }
        const float4 sc = sct[((j0 + 16 * u) >> p.page_shift) - pg0];
        kv_e[u] = sc.y;
        inv_v[u] = sc.z;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][u][e] = fmaf(s[nt][u][e], rf[nt][e & 1] * sc.x, kv_e[u]);
      } else {
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) {
          uint32_t a[4];
          constexpr int CPR = Cfg::RB / 16;
          ldsm4(a, (kaddr ^ (2 * ks % CPR * 16)) + 2 * ks / CPR * SW * Cfg::RB + 16 * u * Cfg::RB);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (ks == 0) mma_b16_first(s[nt][u], a, qb[nt][ks][0], qb[nt][ks][1]);
            else mma_b16_16816(s[nt][u], a, qb[nt][ks][0], qb[nt][ks][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][u][e] *= rf[nt][e & 1];
      }
      if (edge) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + 16 * u + (e >> 1) * 8 + (KV8 ? slot_of<HD>(gq) : gq);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (j < rlo[nt][e & 1] || j >= rhi[nt][e & 1]) s[nt][u][e] = -INFINITY;
        }
      }
    }
    // A row's reference lies kRef below its maximum and moves only when a score is
    // past that maximum by 2^8.
    constexpr float kRef = KV8 ? kScaledRef : 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e & 1] = fmaxf(mx[e & 1], s[nt][u][e]);
      if (__any_sync(0xffffffffu, mx[0] > m[nt][0] + kRef + 8.f || mx[1] > m[nt][1] + kRef + 8.f)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], x));
          const float mn = fmaxf(m[nt][e], mx[e] - kRef);
          f[e] = m[nt][e] == mn ? 1.f : exp2_ap(m[nt][e] - mn);  // 0 while nothing was seen
          m[nt][e] = mn;
          l[nt][e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < NMT; ++i) {
          o[nt][i][0] *= f[0];
          o[nt][i][1] *= f[1];
          o[nt][i][2] *= f[0];
          o[nt][i][3] *= f[1];
        }
      }
    }
    float mref[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) mref[nt][e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = mref[nt][0], m1 = mref[nt][1];
        const float x0 = exp2_ap(s[nt][u][0] - m0), x1 = exp2_ap(s[nt][u][1] - m1);
        const float x2 = exp2_ap(s[nt][u][2] - m0), x3 = exp2_ap(s[nt][u][3] - m1);
        if constexpr (KV8) {
          l[nt][0] = fmaf(x0 + x2, inv_v[u], l[nt][0]);
          l[nt][1] = fmaf(x1 + x3, inv_v[u], l[nt][1]);
          pb[nt][0] = transpose8x8(pack_f16x2(x0, x1));
          pb[nt][1] = transpose8x8(pack_f16x2(x2, x3));
        } else {
          l[nt][0] += x0 + x2;
          l[nt][1] += x1 + x3;
          pb[nt][0] = transpose8x8(pack_b16x2(x0, x1));
          pb[nt][1] = transpose8x8(pack_b16x2(x2, x3));
        }
      }
      if constexpr (KV8) {
        const bool tail = j0 + 16 * u + 16 > c_hi || j0 + 16 * u < t.lo;  // holds positions past the block's: as zeros
        constexpr int NB = HD / 8;  // bytes a thread reads of a V row: elements NB gq ..
        uint32_t w[4][NB >= 4 ? NB / 4 : 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // positions 2 tq, 2 tq + 1 of rows 0-7, then of rows 8-15
          const unsigned char* src = Vs + voff[i & 1] + (16 * u + (i >> 1) * 8) * Cfg::RB;
          if constexpr (NB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(src);
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
          } else if constexpr (NB == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(src);
            w[i][0] = x.x, w[i][1] = x.y;
          } else if constexpr (NB == 4) {
            w[i][0] = *reinterpret_cast<const uint32_t*>(src);
          } else {
            w[i][0] = *reinterpret_cast<const uint16_t*>(src);
          }
          if (tail) {
            const int j = j0 + 16 * u + (i >> 1) * 8 + slot_of<HD>(2 * tq + (i & 1));
            if (j >= c_hi || j < t.lo) {
#pragma unroll
              for (int x = 0; x < (NB >= 4 ? NB / 4 : 1); ++x) w[i][x] = 0u;
            }
          }
        }
        // product rows (elements) gq and gq + 8 of step i are bytes 2 i and 2 i + 1 of the thread's run
#pragma unroll
        for (int i = 0; i < NMT; ++i) {
          const int x = i / 2;
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          const uint32_t e0 = __byte_perm(w[0][x], w[1][x], sel), e1 = __byte_perm(w[2][x], w[3][x], sel);
          const uint32_t a[4] = {e4m3x2_to_f16x2(e0, false), e4m3x2_to_f16x2(e0, true), e4m3x2_to_f16x2(e1, false),
                                 e4m3x2_to_f16x2(e1, true)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][i], a, pb[nt][0], pb[nt][1]);
        }
      } else {
        const bool tail = j0 + SW > c_hi || j0 < t.lo;
        const int jb = j0 + 16 * u + 2 * tq;
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (tail) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = jb + 8 * h;
            keep[h] = (j < c_hi && j >= t.lo ? 0xffffu : 0u) | (j + 1 < c_hi && j + 1 >= t.lo ? 0xffff0000u : 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < NMT; ++i) {
          uint32_t a[4];  // matrices: positions 0-7 | 8-15 by elements 0-7 | 8-15 of step i
          constexpr int CPR = Cfg::RB / 16;
          ldsm4_t(a, (vaddr ^ (2 * i % CPR * 16)) + 2 * i / CPR * SW * Cfg::RB + 16 * u * Cfg::RB);
          if (tail) a[0] &= keep[0], a[1] &= keep[0], a[2] &= keep[1], a[3] &= keep[1];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_b16_16816(o[nt][i], a, pb[nt][0], pb[nt][1]);
        }
      }
    }
    __syncwarp();  // the stage has been read
    if (it + STG < mine) issue(st, j0 + STG * Cfg::WARPS * SW);
    if (++st == STG) st = 0, ph ^= 1;
  }
  if (!ok && lane == 0) {  // copies still in flight after a wait that gave up
    volatile int never = 0;
    for (int i = it + 1; i < mine && i < it + STG; ++i) mbar_wait(&mybar[i % STG], (i / STG) & 1, &never);
  }
  // sums over the positions a row's eight threads hold
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);

  // merge the warps in shared memory: each scales its share to the common maximum
  done = __syncthreads_and(ok);
  if (gq == 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        wm[warp * ROWS + 8 * nt + 2 * tq + e] = m[nt][e];
        wl[warp * ROWS + 8 * nt + 2 * tq + e] = l[nt][e];
      }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * tq + e;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < Cfg::WARPS; ++w) M = fmaxf(M, wm[w * ROWS + r]);
      const float f = m[nt][e] == M ? (M == -INFINITY ? 0.f : 1.f) : exp2_ap(m[nt][e] - M);
      float* dst = Ow + (warp * ROWS + r) * HD;
#pragma unroll
      for (int i = 0; i < NMT; ++i) {
        const int d0 = KV8 ? HD / 8 * gq + 2 * i : 16 * i + gq, d1 = KV8 ? d0 + 1 : d0 + 8;
        dst[d0] = o[nt][i][e] * f;
        dst[d1] = o[nt][i][2 + e] * f;
      }
    }
  __syncthreads();
  }
  // the block's result goes behind the warps'
  float* Ob = Ow + Cfg::WARPS * ROWS * HD;
  float* bm = wm + Cfg::WARPS * ROWS;
  float* bl = wl + Cfg::WARPS * ROWS;
  auto merged = [&](int i, float& M, float& L, float& acc) {
    const int r = i / HD;
    M = -INFINITY, L = acc = 0.f;
    if (!done) return;
#pragma unroll
    for (int w = 0; w < Cfg::WARPS; ++w) M = fmaxf(M, wm[w * ROWS + r]);
#pragma unroll
    for (int w = 0; w < Cfg::WARPS; ++w) {
      const float mw = wm[w * ROWS + r];
      L = fmaf(wl[w * ROWS + r], mw == M ? (M == -INFINITY ? 0.f : 1.f) : exp2_ap(mw - M), L);
      acc += Ow[w * ROWS * HD + i];
    }
  };
  const int total = t.nrow * HD;
  if (p.cluster > 1) {
    for (int i = tid; i < total; i += 128) {
      float M, L, acc;
      merged(i, M, L, acc);
      Ob[i] = acc;
      if (i % HD == 0) bm[i / HD] = M, bl[i / HD] = L;
    }
    cluster_sync();
  }
  // each block of the cluster finishes a part of the rows' elements
  const uint32_t rank = split % p.cluster;
  for (int i = rank * 128 + tid; i < total; i += 128 * p.cluster) {
    const int r = i / HD, d = i % HD;
    float M, L, acc;
    if (p.cluster == 1) {
      merged(i, M, L, acc);
    } else {
      float cm[8], cl[8], ca[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < p.cluster) cm[c] = cluster_load(bm + r, c), cl[c] = cluster_load(bl + r, c), ca[c] = cluster_load(Ob + i, c);
      M = -INFINITY, L = acc = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < p.cluster) M = fmaxf(M, cm[c]);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < p.cluster) {
          const float f = cm[c] == M ? (M == -INFINITY ? 0.f : 1.f) : exp2_ap(cm[c] - M);
          L = fmaf(cl[c], f, L);
          acc = fmaf(ca[c], f, acc);
        }
    }
    const int rr = t.row0 + r, tok = rr / p.group, h = g * p.group + rr % p.group;
    const int64_t at = (int64_t)(t.seq_row0 + tok) * p.Hq + h;
    if (!SAMBA_CHECK(t.seq_row0 + tok < p.batch.rows && h < p.Hq && split < p.nsplit)) continue;
    if (p.npart == 1) {
      p.o[at * HD + d] = __float2bfloat16_rn(acc / L);  // (0 / 0 where every score was -infinity)
    } else {
      float* dst = p.ws + ((((int64_t)b * p.batch.max_q + tok) * p.Hq + h) * p.npart + split / p.cluster) * (HD + 2);
      dst[2 + d] = acc;
      if (d == 0) {
        dst[0] = L == L ? M : L;  // a split that saw NaN alone has no maximum
        dst[1] = L;
      }
    }
  }
  if (p.cluster > 1) cluster_sync();  // the others have read this block's result
}

// Joins the partial results of each (row, head): a block each, its warps take
// every fourth one, E = HD / 32 elements a lane.
template <int HD>
__global__ void __launch_bounds__(128) paged_combine_kernel(const PagedParams p, int page_size) {
  constexpr int E = HD >= 32 ? HD / 32 : 1;
  __shared__ float sm[4][32][E + 1], sl[4];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const SeqSpan s = seq_span(p.batch, page_size, b, false);
  const int i = blockIdx.x;  // row within the sequence times Hq, plus head
  if (i >= s.n * p.Hq) return;
  const float* src = p.ws + ((int64_t)b * p.batch.max_q * p.Hq + i) * p.npart * (HD + 2);
  float M = -INFINITY;
  for (int k = lane; k < p.npart; k += 32) M = fmaxf(M, src[k * (HD + 2)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int k = warp; k < p.npart; k += 4) {
    const float* q = src + k * (HD + 2);
    const float mk = q[0];
    if (mk == -INFINITY) continue;  // an empty split wrote nothing else
    const float f = mk == M ? 1.f : exp2_ap(mk - M);
    L = fmaf(q[1], f, L);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (HD >= 32 || lane < HD) acc[e] = fmaf(q[2 + 32 * e + lane], f, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm[warp][lane][e] = acc[e];
  if (lane == 0) sl[warp] = L;
  __syncthreads();
  L = sl[0] + sl[1] + sl[2] + sl[3];
  const float inv = 1.f / L;  // (infinite where every score was -infinity: NaN)
  const int64_t at = (int64_t)s.row0 * p.Hq + i;
  if (!SAMBA_CHECK(s.row0 + i / p.Hq < p.batch.rows)) return;
  for (int d = threadIdx.x; d < HD; d += 128) {
    const int ln = d & 31, e = d >> 5;
    p.o[at * HD + d] = __float2bfloat16_rn((sm[0][ln][e] + sm[1][ln][e] + sm[2][ln][e] + sm[3][ln][e]) * inv);
  }
}

// ------------------------------------------------------------------ launcher
// Query rows a kv head up to which a call goes through the split kernel here:
// its tiles of 16 rows each read the keys again, so its time grows with the rows, and
// paged_chunk.cu's does not up to 128.  us here and there, 32 heads over 4 of 64:
//   rows                  32           64           96
//   1 x 8192, 8 bits      15.0 17.1    16.8 18.6    18.4 19.9
//   16 x 2048, 8 bits     17.8 24.6    25.7 28.0    43.2 31.7
//   16 x 2048, bf16       18.0 23.3    36.1 26.4    51.4 28.6
//   16 x 16384, 8 bits    63.7 101     131 105      190 109
//   64 x 4096, bf16       115 113      205 115      298 115
// 64 is the last multiple of 32 where some of these gain, not where all do.
constexpr int64_t kFewRows = 64;

// Splits of a row tile's positions: as many as the SMs hold at once (64
// sequences of 2048 positions, 8 bits: two splits each 20.8 us, one 26.4), of at
// least 128 positions (32 a warp) and at most kMaxChunk.  A sequence's length
// is shared out evenly.  Up to eight splits make one cluster, whose blocks join
// their results through shared memory (16 sequences of 2048: 11.0 us, 13.3 with
// a second kernel); more leave one result a cluster for the second kernel.
// Batches that fill the SMs several times over take splits of 2048 positions
// without clusters, so that a block without positions leaves at once.
constexpr int64_t kMaxChunk = 8192;
static PagedPlan paged_plan(const samba_paged_attn_args& a) {
  PagedPlan pl;
  const int64_t group = a.heads_q / a.kv.heads_kv;
  const int64_t rows = std::max<int64_t>(1, a.batch.max_q) * group;
  pl.chunk_kernel = rows > kFewRows;
  if (pl.chunk_kernel) {
    // one block of 256 rows an SM or two of 128: key tiles are split while units leave SMs idle, at least four tiles each
    const int64_t unit = paged_unit(a);
    pl.nt = pl.chunk = 0;
    pl.cluster = 1;
    pl.ntile = (int)((rows + unit - 1) / unit);
    int64_t span = a.batch.max_kv;
    if (a.window > 0) span = std::min<int64_t>(span, a.window + unit / group + 128);
    const int64_t units = (int64_t)pl.ntile * a.kv.heads_kv * std::max<int64_t>(1, a.batch.batch);
    pl.nsplit = pl.npart = (int)std::max<int64_t>(1, std::min<int64_t>(256 / unit * sm_count() / units, span / 512));
    return pl;
  }
  pl.nt = rows <= 8 ? 1 : 2;
  pl.ntile = (int)((rows + 8 * pl.nt - 1) / (8 * pl.nt));
  int64_t span = std::max<int64_t>(1, a.batch.max_kv);
  const int64_t toks = (8 * pl.nt + group - 1) / group;
  if (a.window > 0) span = std::min<int64_t>(span, a.window + toks);
  span += 32;  // a tile's range starts at the multiple of 32 below
  const int64_t tiles = (int64_t)pl.ntile * a.kv.heads_kv * a.batch.batch;
  const int row_bytes = a.kv.head_dim * (a.kv.dtype == SAMBA_E4M3 ? 1 : 2);
  const int64_t resident = row_bytes <= 64 ? 4 : 2;  // blocks an SM holds (their rings take 48 or 96 KB)
  // (seven eighths of them: clusters do not fill the last ones)
  const int64_t want = resident * sm_count() * 7 / 8 / std::max<int64_t>(1, tiles);
  const int64_t least = (span + kMaxChunk - 1) / kMaxChunk, most = (span + 127) / 128;
  int64_t n = std::max<int64_t>(1, std::min<int64_t>(most, want)), c = 1;
  if (least > n || n == 1) {
    n = (span + 2047) / 2048;
  } else {
    while (2 * c <= n && c < 8) c *= 2;
    if (c < 8 && c < least) c *= 2;
    n = std::max<int64_t>(n / c, (least + c - 1) / c) * c;
  }
  pl.cluster = (int)c;
  pl.nsplit = (int)n;
  pl.npart = pl.nsplit / pl.cluster;
  pl.chunk = (int)(((span + n - 1) / n + 31) / 32 * 32);
  return pl;
}

size_t paged_attn_workspace(const samba_paged_attn_args& a) {
  const PagedPlan pl = paged_plan(a);
  if (pl.npart <= 1) return 0;
  uint64_t n = 0;
  if (__builtin_mul_overflow((uint64_t)a.batch.batch, (uint64_t)a.batch.max_q, &n) ||
      __builtin_mul_overflow(n, (uint64_t)a.heads_q, &n) || __builtin_mul_overflow(n, (uint64_t)pl.npart, &n) || __builtin_mul_overflow(n, (uint64_t)(a.kv.head_dim + 2) * 4, &n))
    return SIZE_MAX;
  return (size_t)n;
}

// launch_pdl of pdl.cuh with `cluster` blocks along x in a cluster.
template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem, cudaStream_t s,
                                      Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int HD, bool KV8, int NT>
static int paged_go(const samba_paged_attn_args& a, const PagedPlan& pl, PagedParams& p, cudaStream_t s) {
  using Cfg = PagedCfg<HD, KV8, NT>;
  auto kern = paged_split_kernel<HD, KV8, NT>;
  const int P = a.kv.page_size;
  p.ctab = pl.chunk / P + 2;
  const int smem = Cfg::TAB_OFF + p.ctab * (KV8 ? 20 : 4) + 1024;
  constexpr int kMax = Cfg::TAB_OFF + ((kMaxChunk + 32) / 16 + 2) * 20 + 1024;
  static_assert(kMax <= 227 * 1024, "shared memory");
  static_assert(Cfg::WARPS * Cfg::STG * 8 + 4 <= 128, "barrier block");
  static PerDeviceOnce attr;
  const int arc = once_per_device(attr, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMax) == cudaSuccess
               ? SAMBA_OK
               : fail(SAMBA_ERR_CUDA, "samba_paged_attn: cannot set shared memory size");
  });
  if (arc != SAMBA_OK) return arc;
  // the pool as [num_pages * Hkv][P][d]; a box is one panel by min(P, SW) rows of one (page, head)
  CUtensorMap mk, mv;
  const uint64_t dims[3] = {(uint64_t)HD, (uint64_t)P, (uint64_t)a.kv.num_pages * a.kv.heads_kv};
  const uint64_t strides[2] = {(uint64_t)Cfg::ROWB, (uint64_t)Cfg::ROWB * P};
  const uint32_t box[3] = {(uint32_t)Cfg::PE, (uint32_t)std::min(P, Cfg::SW), 1u};
  const CUtensorMapSwizzle sw = Cfg::RB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : Cfg::RB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : Cfg::RB == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                : CU_TENSOR_MAP_SWIZZLE_NONE;
  const CUtensorMapDataType dt = KV8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int rc = encode_tiled(&mk, dt, 3, a.kv.k, dims, strides, box, sw, "samba_paged_attn K pool");
  if (rc) return rc;
  rc = encode_tiled(&mv, dt, 3, a.kv.v, dims, strides, box, sw, "samba_paged_attn V pool");
  if (rc) return rc;
  const int64_t gx = a.batch.batch * pl.ntile * pl.nsplit;
  if (gx > INT32_MAX) return fail(SAMBA_ERR_UNSUPPORTED, "samba_paged_attn: too many rows");
  const cudaError_t e = launch_pdl_cluster(kern, dim3((unsigned)gx, a.kv.heads_kv), dim3(128), pl.cluster, smem, s, mk, mv, p);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "samba_paged_attn: launch failed: %s", cudaGetErrorString(e));
  return check_launch("samba_paged_attn");
}

template <int HD>
static int paged_hd(const samba_paged_attn_args& a, const PagedPlan& pl, PagedParams& p, cudaStream_t s) {
  const bool kv8 = a.kv.dtype == SAMBA_E4M3;
  int rc = SAMBA_OK;
  if (pl.chunk_kernel) {}  // its splits are there already
  else if (pl.nt == 1) rc = kv8 ? paged_go<HD, true, 1>(a, pl, p, s) : paged_go<HD, false, 1>(a, pl, p, s);
  else rc = kv8 ? paged_go<HD, true, 2>(a, pl, p, s) : paged_go<HD, false, 2>(a, pl, p, s);
  if (rc != SAMBA_OK || pl.npart == 1) return rc;
  const int64_t cx = a.batch.max_q * a.heads_q;
  const cudaError_t e = launch_pdl(paged_combine_kernel<HD>, dim3((unsigned)cx, (unsigned)a.batch.batch), dim3(128), 0, s, p,
                                   (int)a.kv.page_size);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "samba_paged_attn: launch failed: %s", cudaGetErrorString(e));
  return check_launch("samba_paged_attn");
}

int launch_paged_attn(const samba_paged_attn_args& a, cudaStream_t s) {
  if (a.batch.batch == 0 || a.batch.rows == 0 || a.batch.max_q == 0) return SAMBA_OK;
  const PagedPlan pl = paged_plan(a);
  if (pl.chunk_kernel) {
    const int rc = launch_paged_chunk(a, pl, s);
    if (rc != SAMBA_OK || pl.npart == 1) return rc;
  }
  PagedParams p;
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
  p.page_shift = 31 - __builtin_clz((unsigned)a.kv.page_size);
  p.ntile = pl.ntile;
  p.nsplit = pl.nsplit;
  p.chunk = pl.chunk;
  p.cluster = pl.cluster;
  p.npart = pl.npart;
  p.scale_log2 = paged_scale_log2(a);
  switch (a.kv.head_dim) {
    case 16: return paged_hd<16>(a, pl, p, s);
    case 32: return paged_hd<32>(a, pl, p, s);
    case 64: return paged_hd<64>(a, pl, p, s);
    default: return paged_hd<128>(a, pl, p, s);
  }
}

int take_status_paged_attn(cudaStream_t s) { return take_status_word(s); }

}  // namespace samba
