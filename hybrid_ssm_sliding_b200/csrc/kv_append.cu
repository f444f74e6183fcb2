// New keys and values into a paged cache, with the position rotation of keys
// and queries on the way.
//
// The rotation turns pairs of elements by position * frequency.  The turn is
// reduced modulo one in fp64 (a position of 10^6 leaves fp32 with no digits
// of the angle), its sine and cosine are fp32.  An 8-bit cache holds e4m3
// codes with one power-of-two scale s a (page, kv head): the smallest with
// max |x| <= 448 s, so a block's largest value keeps the full three bits and
// growing a scale only shifts the codes stored before.
//
// Bytes bound the call (q in and out, k and v in, the cache rows out).  A
// thread block takes one (sequence, page) pair, which is what a scale
// belongs to, and a share of the heads: the sines and cosines of its rows go
// to shared memory once and serve all its heads.  Items of a sequence are
// numbered from floor(q_start / page) + 2 b, which needs no prefix sum and
// leaves each sequence at least as many numbers as it touches pages.
#include <algorithm>

#include "paged.cuh"
#include "host.hpp"
#include "pdl.cuh"

namespace samba {

struct AppendParams {
  samba_kv_append_args a;
  int nsplit;  // head shares an item is split into
};

constexpr int kAppendThreads = 256;

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

// The pair chunk's two runs, rotated (x: run at lo, y: run at hi).
__device__ __forceinline__ void load_rotated(const __nv_bfloat16* row, const PairChunk& pc, int c, bool inter,
                                             const float* co, const float* si, float (&x)[8], float (&y)[8]) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(row + pc.lo), x);
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(row + pc.hi), y);
  if (!pc.rot) return;
  float cv[8], sv[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<float4*>(cv + 4 * i) = *reinterpret_cast<const float4*>(co + 8 * c + 4 * i);
    *reinterpret_cast<float4*>(sv + 4 * i) = *reinterpret_cast<const float4*>(si + 8 * c + 4 * i);
  }
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], w = x[2 * i + 1], u2 = y[2 * i], w2 = y[2 * i + 1];
      x[2 * i] = u * cv[i] - w * sv[i];
      x[2 * i + 1] = w * cv[i] + u * sv[i];
      y[2 * i] = u2 * cv[4 + i] - w2 * sv[4 + i];
      y[2 * i + 1] = w2 * cv[4 + i] + u2 * sv[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[i], w = y[i];
      x[i] = u * cv[i] - w * sv[i];
      y[i] = w * cv[i] + u * sv[i];
    }
  }
}

__device__ __forceinline__ float finite_abs(float x) {  // |x|, 0 for NaN and infinities
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

template <bool KV8>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
  extern __shared__ float table[];  // [n][rot / 2] cosines, then sines
  const samba_kv_append_args& a = p.a;
  const int P = a.kv.page_size, d = a.kv.head_dim, Hkv = a.kv.heads_kv, Hq = a.heads_q, rot = a.rot_dim;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool inter = a.interleaved != 0;
  const int item = blockIdx.x / p.nsplit, share = blockIdx.x % p.nsplit;
  pdl_launch_dependents();
  pdl_wait();
  // the sequence: the last one whose first item number is at most this one
  const int B = (int)a.batch.batch;
  int b = -1;
  for (int i0 = 0; i0 < B; i0 += kAppendThreads) {
    const int i = i0 + tid;
    const bool below = i < B && static_cast<int64_t>(a.batch.q_start[i] / P) + 2 * i <= item;
    b += __syncthreads_count(below);
    if (blockIdx.x == 0 && i < B) seq_span(a.batch, P, i, true);  // one block reports what is out of range
  }
  if (b < 0) return;
  const int q0 = a.batch.q_start[b];
  const int j = item - q0 / P - 2 * b;  // page of the sequence's new rows
  const SeqSpan s = seq_span(a.batch, P, b, false);
  if (s.n == 0) return;
  const int first = s.kv - s.n;                       // position of the sequence's first new row
  const int col = first / P + j;                      // block_table column
  const int lo = j == 0 ? first : col * P;            // positions [lo, hi) of this item
  const int hi = min(s.kv, (col + 1) * P);
  const int n = hi - lo, off = lo - col * P, row0 = s.row0 + lo - first;
  if (j < 0 || n <= 0) return;
  const int page = a.batch.block_table[(int64_t)b * a.batch.max_pages + col];
  const bool page_ok = page >= 0 && page < a.kv.num_pages;
  if (!page_ok && tid == 0 && share == 0) report_batch();

  const int half = rot / 2;
  float* co = table;
  float* si = table + n * half;
  for (int i = tid; i < n * half; i += kAppendThreads) {
    const int r = i / half;
    double turn = static_cast<double>(lo + r) * a.freqs[i - r * half] * 0.15915494309189535;  // 1 / (2 pi)
    turn -= rint(turn);
    sincospif(2.f * static_cast<float>(turn), si + i, co + i);
  }
  __syncthreads();

  const int PC = d / 16;
  // keys and values: one warp a (matrix, kv head)
  if (page_ok) {
    for (int u = share * (kAppendThreads / 32) + warp; u < 2 * Hkv; u += p.nsplit * (kAppendThreads / 32)) {
      const bool is_v = u >= Hkv;
      const int h = is_v ? u - Hkv : u;
      const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) + (int64_t)row0 * (is_v ? a.ldv : a.ldk) +
                                 (int64_t)h * d;
      const int64_t ld = is_v ? a.ldv : a.ldk;
      const int64_t blk = ((int64_t)page * Hkv + h) * P;  // row of the (page, head) block
      const int urot = is_v ? 0 : rot;
      if constexpr (KV8) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? a.kv.v : a.kv.k) + blk * d;
        float* scale = (is_v ? a.kv.v_scale : a.kv.k_scale) + (int64_t)page * Hkv + h;
        float amax = 0.f;
        for (int i = lane; i < n * PC; i += 32) {
          const int r = i / PC, c = i - r * PC;
          float x[8], y[8];
          load_rotated(src + r * ld, pair_chunk(c, urot, inter), c, inter, co + r * half, si + r * half, x, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(finite_abs(x[e]), finite_abs(y[e])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int need = scale_exponent(amax);
        int k = need;
        if (off > 0) {  // the page holds earlier rows at its old scale
          const int was = stored_exponent(*scale);
          k = max(need, was);
          if (k > was) {  // code * 2^(was - k), re-rounded
            const float by = exp2i(max(was - k, -126));
            uint4* old = reinterpret_cast<uint4*>(dst);
            for (int i = lane; i < off * d / 16; i += 32) {
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
        __syncwarp();  // every lane has read the old scale
        if (lane == 0 && SAMBA_CHECK(page < a.kv.num_pages && h < Hkv)) *scale = exp2i(k);
        const float inv = exp2i(-k);
        for (int i = lane; i < n * PC; i += 32) {
          const int r = i / PC, c = i - r * PC;
          const PairChunk pc = pair_chunk(c, urot, inter);
          float x[8], y[8];
          load_rotated(src + r * ld, pc, c, inter, co + r * half, si + r * half, x, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv, y[e] *= inv;
          uint8_t* to = dst + (off + r) * d;
          if (!SAMBA_CHECK(off + r < P)) continue;
          *reinterpret_cast<uint2*>(to + pc.lo) = make_uint2(to_e4m3x4(x[0], x[1], x[2], x[3]), to_e4m3x4(x[4], x[5], x[6], x[7]));
          *reinterpret_cast<uint2*>(to + pc.hi) = make_uint2(to_e4m3x4(y[0], y[1], y[2], y[3]), to_e4m3x4(y[4], y[5], y[6], y[7]));
        }
      } else {
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? a.kv.v : a.kv.k) + blk * d;
        for (int i = lane; i < n * PC; i += 32) {
          const int r = i / PC, c = i - r * PC;
          const PairChunk pc = pair_chunk(c, urot, inter);
          float x[8], y[8];
          load_rotated(src + r * ld, pc, c, inter, co + r * half, si + r * half, x, y);
          __nv_bfloat16* to = dst + (off + r) * d;
          if (!SAMBA_CHECK(off + r < P)) continue;
          *reinterpret_cast<uint4*>(to + pc.lo) = f32_to_bf16x8(x);
          *reinterpret_cast<uint4*>(to + pc.hi) = f32_to_bf16x8(y);
        }
      }
    }
  }
  // this share's queries
  if (!a.q) return;
  const int h0 = Hq * share / p.nsplit, nh = Hq * (share + 1) / p.nsplit - h0;
  const int per_row = nh * PC;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)row0 * a.ldq + (int64_t)h0 * d;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.q_out) + ((int64_t)row0 * Hq + h0) * d;
  for (int i = tid; i < n * per_row; i += kAppendThreads) {
    const int r = i / per_row, k = i - r * per_row, h = k / PC, c = k - h * PC;
    const PairChunk pc = pair_chunk(c, rot, inter);
    float x[8], y[8];
    load_rotated(q + r * a.ldq + h * d, pc, c, inter, co + r * half, si + r * half, x, y);
    __nv_bfloat16* to = out + ((int64_t)r * Hq + h) * d;
    if (!SAMBA_CHECK(row0 + r < a.batch.rows && h0 + h < Hq)) continue;
    *reinterpret_cast<uint4*>(to + pc.lo) = f32_to_bf16x8(x);
    *reinterpret_cast<uint4*>(to + pc.hi) = f32_to_bf16x8(y);
  }
}

template <bool KV8>
static int kv_append_go(const AppendParams& p, unsigned grid, size_t smem, cudaStream_t s) {
  static PerDeviceOnce attr;
  const int rc = once_per_device(attr, [&] {
    return cudaFuncSetAttribute(kv_append_kernel<KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024) == cudaSuccess
               ? SAMBA_OK
               : fail(SAMBA_ERR_CUDA, "samba_kv_append: cannot set shared memory size");
  });
  if (rc != SAMBA_OK) return rc;
  const cudaError_t e = launch_pdl(kv_append_kernel<KV8>, dim3(grid), dim3(kAppendThreads), smem, s, p);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "samba_kv_append: launch failed: %s", cudaGetErrorString(e));
  return check_launch("samba_kv_append");
}

int launch_kv_append(const samba_kv_append_args& a, cudaStream_t s) {
  if (a.batch.batch == 0 || a.batch.rows == 0) return SAMBA_OK;
  const int P = a.kv.page_size;
  AppendParams p;
  p.a = a;
  // enough thread blocks for about four on each SM, at least two heads each
  const int64_t items = a.batch.rows / P + a.batch.batch;
  const int heads = std::max(a.q ? a.heads_q : 0, 2 * a.kv.heads_kv);
  p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>((heads + 1) / 2, (4 * (int64_t)sm_count() + items - 1) / items));
  const int64_t grid = (a.batch.rows / P + 2 * a.batch.batch) * p.nsplit;
  if (grid > INT32_MAX) return fail(SAMBA_ERR_UNSUPPORTED, "samba_kv_append: too many rows");
  // a block's rows are those of one page, and of one sequence
  const size_t smem = (size_t)std::min<int64_t>(P, a.batch.max_q) * a.rot_dim * sizeof(float);
  return a.kv.dtype == SAMBA_E4M3 ? kv_append_go<true>(p, (unsigned)grid, smem, s)
                                  : kv_append_go<false>(p, (unsigned)grid, smem, s);
}

int take_status_kv_append(cudaStream_t s) { return take_status_word(s); }

}  // namespace samba
