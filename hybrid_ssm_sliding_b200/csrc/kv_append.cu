// New keys and values into a paged cache, with the position rotation of keys
// and queries on the way.
//
// The rotation turns pairs of elements by position * frequency.  The turn is
// reduced modulo one in fp64 (a position of 10^6 leaves fp32 with no digits
// of the angle), its sine and cosine are fp32, with what the turn loses in fp32
// put back to first order (without, the angle's error of 1e-7 is a key's largest).  An 8-bit cache holds e4m3
// codes with one power-of-two scale s a (page, kv head): the smallest with
// max |x| <= 448 s, so a block's largest value keeps the full three bits and
// growing a scale only shifts the codes stored before.
//
// Bytes bound the call (q in and out, k and v in, the cache rows out).  Its
// items are the (sequence, page) pairs, which is what a scale belongs to.  An
// item has blocks for some of its (matrix, kv head) pairs each, and blocks for a
// slice of its rows' queries each; a block brings the sines and cosines of its
// rows to shared memory once for all its heads.  Items of a sequence are
// numbered from floor(q_start / page) + 2 b, which needs no prefix sum and leaves
// each sequence at least as many numbers as it touches pages.
// A block asks for all of its rows at once (bulk copies into shared memory)
// before it works out the sines: the latency of loads, not the arithmetic, is
// what kept a version with loads to registers at 93 us where this one takes 74
// (41k rows of 32 + 2 x 4 heads of 64, 8 bits).
#include <algorithm>

#include "paged.cuh"
#include "host.hpp"
#include "pdl.cuh"

namespace samba {

struct AppendParams {
  samba_kv_append_args a;
  // blocks an item for keys and values, for queries; (matrix, kv head) units of
  // one of the former; slices of the query heads, heads and rows of one; bytes of
  // the sines before a block's rows
  int nkv, nq, kvu, nhead, qheads, qrows, kv_table_bytes, table_bytes;
};

constexpr int kAppendThreads = 256, kAppendBlocks = 3;  // three blocks an SM: 80 registers
constexpr int kKvBytes = 32 * 1024;                     // rows of keys and values a block
constexpr int kSliceBytes = 64 * 1024;                  // a slice of queries (48 KB, four blocks of 64 registers: 97 us)

__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A pair chunk: the 16 elements that one thread takes of a head's row, two
// runs of 8 at `lo` and `hi`.  Pair chunk c < rot / 16 is rotated with table
// entries 8c .. 8c + 7; the rest (c from rot / 16 on) is copied.
struct PairChunk {
  int lo, hi;
  bool rot;
};
__device__ __forceinline__ PairChunk pair_chunk(int c, int rot, bool inter) {
  if (16 * c >= rot || inter) return {16 * c, 16 * c + 8, 16 * c < rot};
  return {8 * c, rot / 2 + 8 * c, true};
}

// The pair chunk's two runs as loaded, the sines and cosines of its elements,
// and the runs rotated (x: run at lo, y: run at hi).
struct RawPair {
  uint4 x, y;
};
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ RawPair load_pair(const __nv_bfloat16* row, const PairChunk& pc) {
  return {*reinterpret_cast<const uint4*>(row + pc.lo), *reinterpret_cast<const uint4*>(row + pc.hi)};
}
__device__ __forceinline__ void load_turn(Turn& t, const float* co, const float* si) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<float4*>(t.c + 4 * i) = *reinterpret_cast<const float4*>(co + 4 * i);
    *reinterpret_cast<float4*>(t.s + 4 * i) = *reinterpret_cast<const float4*>(si + 4 * i);
  }
}
__device__ __forceinline__ void rotate(const RawPair& raw, bool rot, bool inter, const Turn& t, float (&x)[8], float (&y)[8]) {
  bf16x8_to_f32(raw.x, x);
  bf16x8_to_f32(raw.y, y);
  if (!rot) return;
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], w = x[2 * i + 1], u2 = y[2 * i], w2 = y[2 * i + 1];
      x[2 * i] = u * t.c[i] - w * t.s[i];
      x[2 * i + 1] = w * t.c[i] + u * t.s[i];
      y[2 * i] = u2 * t.c[4 + i] - w2 * t.s[4 + i];
      y[2 * i + 1] = w2 * t.c[4 + i] + u2 * t.s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[i], w = y[i];
      x[i] = u * t.c[i] - w * t.s[i];
      y[i] = w * t.c[i] + u * t.s[i];
    }
  }
}

__device__ __forceinline__ float finite_abs(float x) {  // |x|, 0 for NaN and infinities
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

template <bool KV8>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks) kv_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(128) float table[];  // [rows][rot / 2] cosines, then sines; a slice's queries
  __shared__ __align__(16) int found[kAppendThreads / 32];  // the item's sequence, if the warp came upon it
  __shared__ SeqSpan spans[kAppendThreads / 32];
  __shared__ uint64_t landed;                      // the slice's copies
  __shared__ float warp_max[kAppendThreads / 32];
  __shared__ int abort_flag;
  const samba_kv_append_args& a = p.a;
  const int P = a.kv.page_size, d = a.kv.head_dim, Hkv = a.kv.heads_kv, Hq = a.heads_q, rot = a.rot_dim;
  const int pshift = 31 - __clz(P), pcshift = 27 - __clz(d);  // log2 of P and of d / 16
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool inter = a.interleaved != 0;
  const int per_item = p.nkv + p.nq, item = blockIdx.x / per_item, part = blockIdx.x % per_item;
  if (tid == 0) {
    mbar_init(&landed, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  // The sequence that has this item among its numbers: one at most where the
  // sequences are in order, and one that is out of range has none.
  int b = -1, w = 0;
  SeqSpan s{0, 0, 0};
  for (int i = tid; i < (int)a.batch.batch; i += kAppendThreads) {
    const SeqSpan t = seq_span(a.batch, P, i, blockIdx.x == 0);  // one block reports what is out of range
    const int64_t at = item - (t.row0 / P + 2 * static_cast<int64_t>(i));
    if (t.n > 0 && at >= 0 && at <= ((t.kv - 1) >> pshift) - ((t.kv - t.n) >> pshift)) b = i, s = t;
  }
  const int top = __reduce_max_sync(0xffffffffu, b);
  if (b == top && (b >= 0 || lane == 0)) found[warp] = top, spans[warp] = s;
  __syncthreads();
  b = -1;
#pragma unroll
  for (int k = 0; k < kAppendThreads / 32; ++k)
    if (found[k] > b) b = found[k], w = k;
  if (b < 0) return;
  s = spans[w];
  const int j = item - s.row0 / P - 2 * b;       // page of the sequence's new rows
  const int first = s.kv - s.n;                  // position of the sequence's first new row
  const int col = (first >> pshift) + j;         // block_table column
  const int lo = j == 0 ? first : col << pshift; // positions [lo, hi) of this item
  const int hi = min(s.kv, (col + 1) << pshift);
  const bool keys = part < p.nkv;                // this block's part: keys and values, or queries
  const int row_lo = keys ? 0 : (part - p.nkv) / p.nhead * p.qrows;
  const int n = keys ? hi - lo : min(hi - lo - row_lo, p.qrows);  // its rows of the item, from row_lo
  if (n <= 0) return;
  const int row0 = s.row0 + lo - first + row_lo;
  const int half = rot / 2, PC = d >> 4;
  float* co = table;
  float* si = table + n * half;
  auto fill = [&]() {  // a lane a frequency, a warp every eighth row
    for (int c = lane; c < half; c += 32) {
      const double f = a.freqs[c] * 0.15915494309189535;  // turns a position: 1 / (2 pi)
      for (int r = warp; r < n; r += kAppendThreads / 32) {
        double turn = static_cast<double>(lo + row_lo + r) * f;
        turn -= rint(turn);
        const float near = static_cast<float>(turn);
        float sn, cs;
        sincospif(2.f * near, &sn, &cs);
        const float rest = 6.28318531f * static_cast<float>(turn - near);  // the angle that rounding the turn lost
        si[r * half + c] = fmaf(rest, cs, sn);
        co[r * half + c] = fmaf(-rest, sn, cs);
      }
    }
    __syncthreads();
  };

  if (!keys) {
    // Queries: a warp takes every eighth row of the slice (with few heads,
    // several rows at a time), a lane the same chunk of every 32 / PC-th head.
    const int h_lo = (part - p.nkv) % p.nhead * p.qheads, nh = min(p.qheads, Hq - h_lo), row_elems = nh * d;
    __nv_bfloat16* in = reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<unsigned char*>(table) + p.table_bytes);
    if (warp == 0) {
      const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)row0 * a.ldq + (int64_t)h_lo * d;
      if (lane == 0) mbar_arrive_expect_tx(&landed, n * row_elems * 2);
      __syncwarp();
      for (int r = lane; r < n; r += 32) bulk_load(in + r * row_elems, q + r * a.ldq, row_elems * 2, &landed);
    }
    fill();
    if (!mbar_wait(&landed, 0, &abort_flag)) {
      volatile int never = 0;
      if (tid == 0) mbar_wait(&landed, 0, &never);  // (copies still in flight)
      return;
    }
    const int per_row = nh * PC, rp = per_row < 32 ? 32 / per_row : 1;
    const int rsub = per_row < 32 ? lane / per_row : 0, k = per_row < 32 ? lane - rsub * per_row : lane;
    const int c = k & (PC - 1), h0 = k >> pcshift, hstep = 32 >> pcshift;
    const PairChunk pc = pair_chunk(c, rot, inter);
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.q_out) + ((int64_t)row0 * Hq + h_lo) * d;
    if (rsub >= rp) return;
    for (int r = warp * rp + rsub; r < n; r += kAppendThreads / 32 * rp) {
      Turn t;
      if (pc.rot) load_turn(t, co + r * half + 8 * c, si + r * half + 8 * c);
#pragma unroll 2
      for (int h = h0; h < nh; h += hstep) {
        float x[8], y[8];
        rotate(load_pair(in + r * row_elems + h * d, pc), pc.rot, inter, t, x, y);
        __nv_bfloat16* to = out + ((int64_t)r * Hq + h) * d;
        if (!SAMBA_CHECK(row0 + r < a.batch.rows && h_lo + h < Hq)) continue;
        *reinterpret_cast<uint4*>(to + pc.lo) = f32_to_bf16x8(x);
        *reinterpret_cast<uint4*>(to + pc.hi) = f32_to_bf16x8(y);
      }
    }
    return;
  }
  // Keys and values: the block's units are (matrix, kv head) pairs, keys first,
  // 8 / kvu warps each; their rows are copied to shared memory like the queries.
  const int page = a.batch.block_table[(int64_t)b * a.batch.max_pages + col];
  if (page < 0 || page >= a.kv.num_pages) {
    if (tid == 0 && part == 0) report_batch();
    return;
  }
  const int off = lo - (col << pshift);
  const int u0 = part * p.kvu, u1 = min(u0 + p.kvu, 2 * Hkv);
  const int kc = max(0, min(u1, Hkv) - u0), v0 = max(u0 - Hkv, 0), vc = u1 - u0 - kc, row_elems = (kc + vc) * d;
  __nv_bfloat16* in = reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<unsigned char*>(table) + p.kv_table_bytes);
  if (warp == 0) {
    if (lane == 0) mbar_arrive_expect_tx(&landed, n * row_elems * 2);
    __syncwarp();
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.k) + (int64_t)row0 * a.ldk + (int64_t)u0 * d;
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v) + (int64_t)row0 * a.ldv + (int64_t)v0 * d;
    for (int r = lane; r < n; r += 32) {
      if (kc > 0) bulk_load(in + r * row_elems, k + r * a.ldk, kc * d * 2, &landed);
      if (vc > 0) bulk_load(in + r * row_elems + kc * d, v + r * a.ldv, vc * d * 2, &landed);
    }
  }
  const int wpu = kAppendThreads / 32 / p.kvu, sw = warp & (wpu - 1), ul = warp / wpu, u = u0 + ul;
  const bool unit = u < u1, is_v = u >= Hkv;
  const int h = is_v ? u - Hkv : u;
  const int64_t block = (int64_t)page * Hkv + (unit ? h : 0);  // the (page, head) block
  float* scale = nullptr;
  float was_scale = 0.f;
  if constexpr (KV8) {
    scale = (is_v ? a.kv.v_scale : a.kv.k_scale) + block;
    if (unit && off > 0) was_scale = *scale;
  }
  if (kc > 0) fill();
  if (!__syncthreads_and(mbar_wait(&landed, 0, &abort_flag))) {
    volatile int never = 0;
    if (tid == 0) mbar_wait(&landed, 0, &never);  // (copies still in flight)
    return;
  }
  // a lane takes the same chunk of every rstep-th row
  const int c = lane & (PC - 1), r0 = (lane >> pcshift) + sw * (32 >> pcshift), rstep = wpu * (32 >> pcshift);
  const PairChunk pc = pair_chunk(c, is_v ? 0 : rot, inter);
  const __nv_bfloat16* src = in + ul * d;
  auto turned = [&](int r, float (&x)[8], float (&y)[8]) {
    Turn t;
    if (pc.rot) load_turn(t, co + r * half + 8 * c, si + r * half + 8 * c);
    rotate(load_pair(src + r * row_elems, pc), pc.rot, inter, t, x, y);
  };
  if constexpr (KV8) {
    float amax = 0.f;  // of finite values; infinities are looked at again only where there are any
    for (int finite = 0; finite < 2; ++finite) {
      amax = 0.f;
      if (unit)
#pragma unroll 2
        for (int r = r0; r < n; r += rstep) {
          float x[8], y[8];
          turned(r, x, y);
          if (finite) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = finite_abs(x[e]), y[e] = finite_abs(y[e]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e]), fabsf(y[e])));  // (NaN is passed over)
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (lane == 0) warp_max[warp] = amax;
      const bool all_finite = !__syncthreads_or(amax > 3.402823466e38f);
      for (int w = 0; w < wpu; ++w) amax = fmaxf(amax, warp_max[ul * wpu + w]);
      if (all_finite) break;
      __syncthreads();
    }
    if (!unit) return;
    uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? a.kv.v : a.kv.k) + block * P * d;
    int k = scale_exponent(amax);
    if (off > 0) {  // the page holds earlier rows at its old scale
      const int was = stored_exponent(was_scale);
      k = max(k, was);
      if (k > was) {  // code * 2^(was - k), re-rounded
        const float by = exp2i(was - k);
        uint4* old = reinterpret_cast<uint4*>(dst);
        for (int i = sw * 32 + lane; i < off * d / 16; i += 32 * wpu) {
          uint4 v = old[i];
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t l2 = e4m3x2_to_f16x2(w[e], false), h2 = e4m3x2_to_f16x2(w[e], true);
            const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&l2));
            const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            w[e] = to_e4m3x4(fl.x * by, fl.y * by, fh.x * by, fh.y * by);
          }
          if (SAMBA_CHECK(i * 16 + 16 <= P * d)) old[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    // (every warp of the unit read the old scale before the barriers above)
    if (lane == 0 && sw == 0 && SAMBA_CHECK(page < a.kv.num_pages && h < Hkv)) *scale = exp2i(k);
    const float inv = exp2i(-k);
#pragma unroll 2
    for (int r = r0; r < n; r += rstep) {
      float x[8], y[8];
      turned(r, x, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv, y[e] *= inv;
      uint8_t* to = dst + (off + r) * d;
      if (!SAMBA_CHECK(off + r < P)) continue;
      *reinterpret_cast<uint2*>(to + pc.lo) = make_uint2(to_e4m3x4(x[0], x[1], x[2], x[3]), to_e4m3x4(x[4], x[5], x[6], x[7]));
      *reinterpret_cast<uint2*>(to + pc.hi) = make_uint2(to_e4m3x4(y[0], y[1], y[2], y[3]), to_e4m3x4(y[4], y[5], y[6], y[7]));
    }
  } else {
    if (!unit) return;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? a.kv.v : a.kv.k) + block * P * d;
#pragma unroll 2
    for (int r = r0; r < n; r += rstep) {
      float x[8], y[8];
      turned(r, x, y);
      __nv_bfloat16* to = dst + (off + r) * d;
      if (!SAMBA_CHECK(off + r < P)) continue;
      *reinterpret_cast<uint4*>(to + pc.lo) = f32_to_bf16x8(x);
      *reinterpret_cast<uint4*>(to + pc.hi) = f32_to_bf16x8(y);
    }
  }
}

template <bool KV8>
static int kv_append_go(const AppendParams& p, unsigned grid, size_t smem, cudaStream_t s) {
  static PerDeviceOnce attr;
  const int rc = once_per_device(attr, [&] {
    return cudaFuncSetAttribute(kv_append_kernel<KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) == cudaSuccess
               ? SAMBA_OK
               : fail(SAMBA_ERR_CUDA, "samba_kv_append: cannot set shared memory size");
  });
  if (rc != SAMBA_OK) return rc;
  const cudaError_t e = launch_pdl(kv_append_kernel<KV8>, dim3(grid), dim3(kAppendThreads), smem, s, p);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "samba_kv_append: launch failed: %s", cudaGetErrorString(e));
  return check_launch("samba_kv_append");
}

int launch_kv_append(const samba_kv_append_args& a, cudaStream_t s) {
  if (a.batch.batch == 0 || a.batch.rows == 0 || a.batch.max_q == 0) return SAMBA_OK;
  const int P = a.kv.page_size;
  AppendParams p;
  p.a = a;
  const int page_rows = (int)std::min<int64_t>(P, a.batch.max_q), head_bytes = a.kv.head_dim * 2;
  // units of keys and values: as many as kKvBytes hold, one of 256 rows of 128 always
  p.kvu = kAppendThreads / 32;
  while (p.kvu > 1 && (p.kvu * page_rows * head_bytes > kKvBytes || p.kvu >= 4 * a.kv.heads_kv)) p.kvu /= 2;
  p.nkv = (2 * a.kv.heads_kv + p.kvu - 1) / p.kvu;
  p.kv_table_bytes = (page_rows * a.rot_dim * (int)sizeof(float) + 127) / 128 * 128;
  // a slice: whole rows, or for very wide ones a row's share of the heads
  p.qheads = std::min(std::max(1, a.heads_q), kSliceBytes / head_bytes);
  p.nhead = a.q ? (a.heads_q + p.qheads - 1) / p.qheads : 1;
  p.qrows = std::min(page_rows, std::max(1, kSliceBytes / (p.qheads * head_bytes)));
  if (p.qrows > 8) p.qrows = p.qrows / 8 * 8;
  p.nq = a.q ? (page_rows + p.qrows - 1) / p.qrows * p.nhead : 0;
  const int64_t grid = (a.batch.rows / P + 2 * a.batch.batch) * ((int64_t)p.nkv + p.nq);
  if (grid > INT32_MAX) return fail(SAMBA_ERR_UNSUPPORTED, "samba_kv_append: too many rows");
  // a block's rows are those of one page, and of one sequence (at most 128 KB of
  // sines; 192 KB with a slice of queries of one head)
  p.table_bytes = (p.qrows * a.rot_dim * (int)sizeof(float) + 127) / 128 * 128;
  const size_t smem = std::max<size_t>(p.kv_table_bytes + (size_t)p.kvu * page_rows * head_bytes,
                                       a.q ? p.table_bytes + (size_t)p.qrows * p.qheads * head_bytes : 0);
  return a.kv.dtype == SAMBA_E4M3 ? kv_append_go<true>(p, (unsigned)grid, smem, s)
                                  : kv_append_go<false>(p, (unsigned)grid, smem, s);
}

int take_status_kv_append(cudaStream_t s) { return take_status_word(s); }

}  // namespace samba
