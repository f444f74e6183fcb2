// The norms around a block with its gate, residual scale and residual sum, and
// their gradients.  Per row of C elements, rms(x) = x / sqrt(mean(x^2) + eps):
//   t = rms(y) w_post,  r' = r + alpha sigmoid(gate) t,  n = rms(r') w_pre
// Everything is elementwise but the row sums, so HBM bandwidth bounds both
// directions: every tensor is read or written once.
//
// A block stays resident and walks over groups of rows (one row of 2048
// elements and more, several shorter ones, about 256 threads).  A group's
// tensors are contiguous, so one bulk copy each brings them into a ring of
// shared memory stages: the next groups' bytes are in flight while this one
// waits for its sums, at no cost in registers.  A call with no more groups
// than blocks reads global memory directly, which saves the copy's latency.  A thread has two runs of four
// elements, 128 apart (a warp 256 in a row), so that 16- and 32-bit tensors both
// move without a gap and the second run's addresses are the first's plus a constant.
//
// The backward pass needs one joint sum a row: with c = alpha s w_post yh and
// s1 = sum dn w_pre x, the second norm's sum is
//   sum c g = sum c (dr' + rstd dn w_pre) - rstd s1 / C sum c x.
// dw_post = alpha S and dalpha = w_post S share the column sums S = sum g s yh.
// They and dw_pre's stay in registers over all rows of a block; each block
// writes them once and a second kernel adds the blocks in a fixed order (no
// atomics, so results repeat bit for bit).
#include <algorithm>

#include "common.cuh"
#include "host.hpp"
#include "pdl.cuh"

namespace samba {

// Four elements as two packed pairs: the arithmetic here is in pairs (one
// instruction for two), which is what it takes to keep up with the memory.
__device__ __forceinline__ void load4(f2* f, const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = pk2(v.x, v.y), f[1] = pk2(v.z, v.w);
}
__device__ __forceinline__ void load4(f2* f, const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = pk2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
  f[1] = pk2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, const f2* f) {
  const float2 a = up2(f[0]), b = up2(f[1]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const f2* f) {
  const float2 u = up2(f[0]), v = up2(f[1]);
  const __nv_bfloat162 a = __floats2bfloat162_rn(u.x, u.y), b = __floats2bfloat162_rn(v.x, v.y);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ f2 both(float x) { return pk2(x, x); }
__device__ __forceinline__ float sum2(f2 v) {
  const float2 t = up2(v);
  return t.x + t.y;
}

// sigmoid of a pair; the fast divide gives 0 where 1 + exp(-x) passes 2^126
__device__ __forceinline__ float sigmoidf(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ f2 sigmoid2(f2 v) {
  const float2 t = up2(v);
  return pk2(sigmoidf(t.x), sigmoidf(t.y));
}

// The backward pass needs s = sigmoid(x) and 1 - s, each to a part of itself (1 less
// s has no digits left where s is near 1): with E = exp(-x) they are 1 / (1 + E) and E
// times that.  E is what is kept between the two places that use s; it stops
// short of infinity, where s is 0, and keeps a NaN.
__device__ __forceinline__ f2 exp_neg2(f2 x) {
  const float2 a = up2(mul2(x, both(-1.44269504f)));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(a.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(a.y));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.x) : "f"(3.402823466e38f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.y) : "f"(3.402823466e38f));
  return pk2(e.x, e.y);
}
__device__ __forceinline__ f2 one_over_one_plus2(f2 e) {
  const float2 d = up2(add2(e, both(1.f)));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return pk2(r.x, r.y);
}

// How a call is cut up: rows a group, threads a row (a multiple of 32), and
// where a tensor lies in a stage.
struct NormShape {
  uint32_t rows, groups;  // below 2^31, so that an index one step past the end still fits
  int C, rpb, tpr, stages, stage_bytes, off[5];
  float inv_c;
};

constexpr int kNormMaxStages = 4;

// Shared memory: [barriers][sum slots][stages].
struct NormShared {
  uint64_t full[kNormMaxStages];
  int abort_flag, pad[3];
  float slots[2][3][32];
};
constexpr int kNormHead = (int)((sizeof(NormShared) + 127) / 128 * 128);

// Sums of N values over the warps of a row, the same bits in every thread.
// The slots' two halves alternate, so one barrier per call is enough: a slot
// is written again only after the barrier of the call in between.
struct RowWarps {
  int nw, width;   // warps a row, the power of two from that
  float* out;      // the warp's slot
  const float* in; // the slot that the lane reads, null beyond the row's warps
  __device__ RowWarps(NormShared& sh, int tpr) : nw(tpr >> 5), width(1) {
    while (width < nw) width *= 2;
    const int warp = threadIdx.x >> 5, k = threadIdx.x & 31 & (width - 1);
    out = &sh.slots[0][0][warp];
    in = k < nw ? &sh.slots[0][0][warp / nw * nw + k] : nullptr;
  }
};
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int& ph, const RowWarps& rw) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (rw.nw == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) rw.out[ph + 32 * i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = rw.in ? rw.in[ph + 32 * i] : 0.f;
  for (int o = rw.width >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  ph ^= 96;
}

// The ring over a call's input tensors.
struct NormTensor {
  const void* p;  // null: not part of the call
  int elem;       // bytes an element
};
template <int NTEN>
struct NormInputs {
  NormTensor t[NTEN];
};

template <int NTEN>
__device__ __forceinline__ void norm_issue(const NormInputs<NTEN>& in, const NormShape& s, uint64_t* full,
                                           unsigned char* stage, uint32_t group) {
  const uint32_t row0 = group * s.rpb;
  const uint32_t n = min(s.rows - row0, static_cast<uint32_t>(s.rpb)) * s.C;
  uint32_t bytes = 0;
#pragma unroll
  for (int i = 0; i < NTEN; ++i)
    if (in.t[i].p) bytes += n * in.t[i].elem;
  mbar_arrive_expect_tx(full, bytes);
#pragma unroll
  for (int i = 0; i < NTEN; ++i)
    if (in.t[i].p)
      bulk_load(stage + s.off[i],
                reinterpret_cast<const unsigned char*>(in.t[i].p) + (int64_t)row0 * s.C * in.t[i].elem, n * in.t[i].elem, full);
}

// Walks over this block's groups of rows: read(at) loads the thread's row into
// registers, at(i) being tensor i's row (in the ring or in global memory);
// body(row, live, release) computes with them and calls release(synced) once
// all threads have read, that is after its first barrier (synced; release makes
// one otherwise): the stage is then refilled.  Threads without a row (behind
// the last one) keep an earlier row's values and store nothing.
template <bool RING, int NTEN, class Read, class Body>
__device__ __forceinline__ void norm_walk(const NormInputs<NTEN>& in, const NormShape& s, NormShared& sh,
                                          unsigned char* ring, Read&& read, Body&& body) {
  const int sub = threadIdx.x / s.tpr;
  uint32_t g = blockIdx.x, row = g * s.rpb + sub;
  int64_t o = (int64_t)row * s.C;
  if constexpr (!RING) {  // as many blocks as groups
    if (row < s.rows)
      read([&](int i) { return reinterpret_cast<const unsigned char*>(in.t[i].p) + o * in.t[i].elem; });
    body(row, o, row < s.rows, [](bool) {});
    return;
  }
  const uint32_t step = gridDim.x, ahead = s.stages * step;
  if (threadIdx.x == 0)
    for (uint32_t i = 0; i < s.stages && g + i * step < s.groups; ++i)
      norm_issue(in, s, &sh.full[i], ring + i * s.stage_bytes, g + i * step);
  int off[NTEN];
#pragma unroll
  for (int i = 0; i < NTEN; ++i) off[i] = s.off[i] + sub * s.C * in.t[i].elem;
  int stage = 0, parity = 0;
  for (; g < s.groups; g += step, row += step * s.rpb, o += (int64_t)step * s.rpb * s.C) {
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[stage], parity, &sh.abort_flag))) {
      // gave up: leave once the copies in flight have landed (threads that have
      // left do not hold up a barrier)
      if (threadIdx.x == 0) {
        volatile int never = 0;
        for (uint32_t i = 0; i < s.stages && g + i * step < s.groups; ++i)
          mbar_wait(&sh.full[(stage + i) % s.stages], parity ^ (stage + i >= s.stages ? 1 : 0), &never);
      }
      return;
    }
    unsigned char* base = ring + stage * s.stage_bytes;
    if (row < s.rows) read([&](int i) { return base + off[i]; });
    body(row, o, row < s.rows, [&](bool synced) {
      if (!synced) __syncthreads();
      if (threadIdx.x == 0 && g + ahead < s.groups) norm_issue(in, s, &sh.full[stage], base, g + ahead);
    });
    if (++stage == s.stages) stage = 0, parity ^= 1;
  }
}

template <bool RING>
__device__ __forceinline__ void norm_setup(NormShared& sh, const NormShape& s) {
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < s.stages; ++i) mbar_init(&sh.full[i], 1);
      sh.abort_flag = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  pdl_launch_dependents();
  pdl_wait();
}

struct NormFwdParams {
  NormInputs<3> in;  // r, y, gate
  const float* w_pre;
  const float* w_post;
  const float* alpha;
  void* r_out;
  void* n;
  float* rstd_pre;
  float* rstd_post;
  NormShape s;
  float eps;
};

// A vector's values for the thread's eight elements, 1 without one.
__device__ __forceinline__ void load_vec(f2 (&f)[4], const float* w, int e, const bool (&has)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (w && has[k]) load4(f + 2 * k, w + e + 128 * k);
    else f[2 * k] = f[2 * k + 1] = both(1.f);
  }
}

template <typename RT, typename YT, int MAXT, bool RING>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1024 / MAXT) block_norm_fwd_kernel(const __grid_constant__ NormFwdParams p) {
  extern __shared__ __align__(128) unsigned char sm[];
  NormShared& sh = *reinterpret_cast<NormShared*>(sm);
  const NormShape& s = p.s;
  const int lt = threadIdx.x % s.tpr;
  const int e = lt / 32 * 256 + lt % 32 * 4;
  const bool has[2] = {e < s.C, e + 128 < s.C};
  const bool has_y = p.in.t[1].p != nullptr, has_g = p.in.t[2].p != nullptr;
  const RowWarps rw(sh, s.tpr);
  norm_setup<RING>(sh, s);
  f2 wa[4], wp[4];  // w_post alpha, w_pre
  load_vec(wa, p.w_post, e, has);
  load_vec(wp, p.alpha, e, has);
#pragma unroll
  for (int i = 0; i < 4; ++i) wa[i] = mul2(wa[i], wp[i]);
  load_vec(wp, p.w_pre, e, has);
  f2 r[4], y[4], z[4];  // elements that the row does not have stay zero
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = y[i] = z[i] = both(0.f);
  int ph = 0;
  norm_walk<RING>(
      p.in, s, sh, sm + kNormHead,
      [&](auto at) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!has[k]) continue;
          load4(r + 2 * k, reinterpret_cast<const RT*>(at(0)) + e + 128 * k);
          if (has_y) load4(y + 2 * k, reinterpret_cast<const YT*>(at(1)) + e + 128 * k);
          if (has_g) load4(z + 2 * k, reinterpret_cast<const YT*>(at(2)) + e + 128 * k);
        }
      },
      [&](uint32_t row, int64_t o, bool live, auto release) {
        float sum[1];
        if (has_y) {
          f2 q = both(0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            q = fma2(y[i], y[i], q);
            y[i] = mul2(y[i], wa[i]);
          }
          if (has_g) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], sigmoid2(z[i]));
          }
          float rs = 1.f;
          if (p.w_post) {
            sum[0] = sum2(q);
            row_sum(sum, ph, rw);
            release(rw.nw > 1);
            rs = rsqrtf(fmaf(sum[0], s.inv_c, p.eps));
            if (p.rstd_post && live && lt == 0) p.rstd_post[row] = rs;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = fma2(y[i], both(rs), r[i]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (live && has[k] && SAMBA_CHECK(row < s.rows && e + 128 * k + 4 <= s.C))
              store4(reinterpret_cast<RT*>(p.r_out) + o + e + 128 * k, r + 2 * k);
        }
        if (p.n) {
          f2 q = both(0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) q = fma2(r[i], r[i], q);
          sum[0] = sum2(q);
          row_sum(sum, ph, rw);
          if (!p.w_post) release(rw.nw > 1);
          const float rs = rsqrtf(fmaf(sum[0], s.inv_c, p.eps));
          if (p.rstd_pre && live && lt == 0) p.rstd_pre[row] = rs;
          f2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = mul2(mul2(r[i], both(rs)), wp[i]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (live && has[k] && SAMBA_CHECK(row < s.rows && e + 128 * k + 4 <= s.C))
              store4(reinterpret_cast<YT*>(p.n) + o + e + 128 * k, w + 2 * k);
        } else if (!p.w_post) {
          release(false);
        }
      });
}

struct NormBwdParams {
  NormInputs<5> in;  // dn, r (with dn), dr_out, y, gate
  const float* w_pre;
  const float* rstd_pre;
  const float* w_post;
  const float* rstd_post;
  const float* alpha;
  void* dr;
  void* dy;
  void* dgate;
  float* part;  // [2][grid][C]: column sums of dn x and g s yh
  NormShape s;
};

template <typename RT, typename YT, int MAXT, bool RING>
__global__ void __launch_bounds__(MAXT) block_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  extern __shared__ __align__(128) unsigned char sm[];
  NormShared& sh = *reinterpret_cast<NormShared*>(sm);
  const NormShape& s = p.s;
  const int lt = threadIdx.x % s.tpr, sub = threadIdx.x / s.tpr;
  const int e = lt / 32 * 256 + lt % 32 * 4;
  const bool has[2] = {e < s.C, e + 128 < s.C};
  const bool has_n = p.in.t[0].p != nullptr, has_d = p.in.t[2].p != nullptr, has_y = p.in.t[3].p != nullptr,
             has_g = p.in.t[4].p != nullptr;
  const RowWarps rw(sh, s.tpr);
  norm_setup<RING>(sh, s);
  f2 wp[4], c[4];  // w_pre, w_post alpha
  load_vec(c, p.w_post, e, has);
  load_vec(wp, p.alpha, e, has);
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = mul2(c[i], wp[i]);
  load_vec(wp, p.w_pre, e, has);
  f2 a_pre[4], a_post[4], dn[4], x[4], g[4], yh[4], z[4];  // elements that the row does not have stay zero
#pragma unroll
  for (int i = 0; i < 4; ++i) a_pre[i] = a_post[i] = dn[i] = x[i] = g[i] = yh[i] = z[i] = both(0.f);
  float rs_next = 0.f, rsy_next = 1.f;
  auto stats = [&](uint32_t row) {  // a row's factors, read one group ahead
    if (row >= s.rows) return;
    if (has_n) rs_next = p.rstd_pre[row];
    if (p.w_post) rsy_next = p.rstd_post[row];
  };
  stats(blockIdx.x * s.rpb + sub);
  int ph = 0;
  norm_walk<RING>(
      p.in, s, sh, sm + kNormHead,
      [&](auto at) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!has[k]) continue;
          if (has_n) {
            load4(dn + 2 * k, reinterpret_cast<const YT*>(at(0)) + e + 128 * k);
            load4(x + 2 * k, reinterpret_cast<const RT*>(at(1)) + e + 128 * k);
          }
          if (has_d) load4(g + 2 * k, reinterpret_cast<const RT*>(at(2)) + e + 128 * k);
          if (has_y) load4(yh + 2 * k, reinterpret_cast<const YT*>(at(3)) + e + 128 * k);
          if (has_g) load4(z + 2 * k, reinterpret_cast<const YT*>(at(4)) + e + 128 * k);
        }
      },
      [&](uint32_t row, int64_t o, bool live, auto release) {
        // a thread without a row must add nothing to the column sums
        const float rs = live ? rs_next : 0.f, rsy = live ? rsy_next : 0.f;
        stats(row + gridDim.x * s.rpb);
        if (!live) {
#pragma unroll
          for (int i = 0; i < 4; ++i) dn[i] = x[i] = g[i] = yh[i] = both(0.f);
        }
        if (!has_d) {
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = both(0.f);
        }
        const f2 rs2 = both(rs), rsy2 = both(rsy);
        f2 q0 = both(0.f), q1 = both(0.f), q2 = both(0.f);
        if (has_n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], rs2);
            a_pre[i] = fma2(dn[i], x[i], a_pre[i]);
            dn[i] = mul2(dn[i], wp[i]);
            q0 = fma2(dn[i], x[i], q0);
            g[i] = fma2(rs2, dn[i], g[i]);
          }
        }
        if (has_y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = has_g ? exp_neg2(z[i]) : both(0.f);
            yh[i] = mul2(yh[i], rsy2);
            const f2 ci = mul2(mul2(c[i], has_g ? one_over_one_plus2(z[i]) : both(1.f)), yh[i]);
            q1 = fma2(ci, g[i], q1);
            q2 = fma2(ci, x[i], q2);
          }
        }
        float sum[3] = {sum2(q0), sum2(q1), sum2(q2)};
        const bool sums = has_n || p.w_post;
        if (sums) row_sum(sum, ph, rw);
        release(sums && rw.nw > 1);
        const float m1 = rs * sum[0] * s.inv_c;
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = fma2(both(-m1), x[i], g[i]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (live && has[k] && SAMBA_CHECK(row < s.rows && e + 128 * k + 4 <= s.C))
            store4(reinterpret_cast<RT*>(p.dr) + o + e + 128 * k, g + 2 * k);
        if (has_y) {
          const float m2 = p.w_post ? rsy * fmaf(-m1, sum[2], sum[1]) * s.inv_c : 0.f;
          f2 dz[4], dy[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f2 sg = has_g ? one_over_one_plus2(z[i]) : both(1.f);
            const f2 gs = mul2(g[i], sg), dt = mul2(gs, c[i]);
            a_post[i] = fma2(gs, yh[i], a_post[i]);
            dz[i] = mul2(mul2(dt, yh[i]), mul2(z[i], sg));
            dy[i] = fma2(rsy2, dt, mul2(both(-m2), yh[i]));
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (live && has[k] && SAMBA_CHECK(row < s.rows && e + 128 * k + 4 <= s.C)) {
              store4(reinterpret_cast<YT*>(p.dy) + o + e + 128 * k, dy + 2 * k);
              if (has_g) store4(reinterpret_cast<YT*>(p.dgate) + o + e + 128 * k, dz + 2 * k);
            }
        }
      });
  // this block's column sums: the row slots of a group added in order, then written once
  float* mine = p.part + (int64_t)blockIdx.x * s.C;
  float* acc = reinterpret_cast<float*>(sm + kNormHead);  // [rpb][C]
  auto put = [&](const f2 (&a)[4], float* dst) {
    if (s.rpb == 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (has[k]) store4(dst + e + 128 * k, a + 2 * k);
      return;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (has[k]) store4(acc + sub * s.C + e + 128 * k, a + 2 * k);
    __syncthreads();
    for (int i = 4 * threadIdx.x; i < s.C; i += 4 * blockDim.x) {
      f2 f[2], h[2];
      load4(f, acc + i);
      for (int q = 1; q < s.rpb; ++q) {
        load4(h, acc + q * s.C + i);
#pragma unroll
        for (int j = 0; j < 2; ++j) f[j] = add2(f[j], h[j]);
      }
      store4(dst + i, f);
    }
  };
  if (has_n) put(a_pre, mine);
  if (p.w_post || p.alpha) put(a_post, mine + (int64_t)gridDim.x * s.C);
}

// Adds the blocks' column sums: 8 threads x 4 columns by 32 slices of blocks,
// the slices then added in order.  Plane 0 is dw_pre, plane 1 the sums S of
// dw_post = alpha S and dalpha = w_post S.
__global__ void __launch_bounds__(256) block_norm_cols_kernel(const float* __restrict__ part, float* dw_pre,
                                                              float* dw_post, float* dalpha, const float* w_post,
                                                              const float* alpha, int nblk, int C) {
  __shared__ float4 sums[32][8];
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + 4 * tx;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.y == 0 ? !dw_pre : !dw_post && !dalpha) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < C) {
    const float* src = part + (int64_t)blockIdx.y * nblk * C + col;
#pragma unroll 4
    for (int b = ty; b < nblk; b += 32) {
      const float4 v = *reinterpret_cast<const float4*>(src + (int64_t)b * C);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
  sums[ty][tx] = a;
  __syncthreads();
  if (ty == 0 && col < C && SAMBA_CHECK(col + 4 <= C)) {
#pragma unroll 8
    for (int s = 1; s < 32; ++s) {
      const float4 v = sums[s][tx];
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    auto put = [&](float* out, const float* by) {
      float4 f = by ? *reinterpret_cast<const float4*>(by + col) : make_float4(1.f, 1.f, 1.f, 1.f);
      *reinterpret_cast<float4*>(out + col) = make_float4(a.x * f.x, a.y * f.y, a.z * f.z, a.w * f.w);
    };
    if (blockIdx.y == 0) {
      put(dw_pre, nullptr);
    } else {
      if (dw_post) put(dw_post, alpha);
      if (dalpha) put(dalpha, w_post);
    }
  }
}

// ------------------------------------------------------------------ launchers
// Threads an SM holds: forward 768 at 80 registers, or 1024 at 64 where a row
// takes more than 256 (2048 columns, bf16: 55 us where 1024 threads took 54, fp32
// stream: 55 where they took 66); backward 512, whose column sums and gradients
// take 120.  The stages take kFwdSmem or kBwdSmem of an SM's shared memory: enough
// in flight, and the forward pass loses with more (32768 x 2048, fp32 stream: 130
// KB 148 us, 200 KB 178).
constexpr int kBwdThreadsPerSm = 512;
constexpr int kFwdSmem = 130 * 1024, kBwdSmem = 200 * 1024;

struct NormCut {
  NormShape s;
  int grid, threads;
  size_t smem;
  bool ring;
};

static void norm_rows(int64_t C, int& tpr, int& rpb) {
  tpr = static_cast<int>((C + 255) / 256 * 32);
  rpb = std::max(1, 256 / tpr);
}

// Resident blocks by threads alone; a block's stage may take a whole SM, so
// the shared memory then allows fewer.
static int norm_blocks_per_sm(int64_t C, int threads_per_sm, int64_t stage_bytes, int smem) {
  int tpr, rpb;
  norm_rows(C, tpr, rpb);
  const int by_threads = std::max(1, threads_per_sm / (tpr * rpb));
  return std::max<int>(1, std::min<int64_t>(by_threads, smem / (stage_bytes + kNormHead)));
}

template <int NTEN>
static NormCut norm_cut(const NormInputs<NTEN>& in, int64_t rows, int64_t C, int threads_per_sm, int smem, bool colsums) {
  NormCut c;
  NormShape& s = c.s;
  s.rows = (uint32_t)rows;
  s.C = (int)C;
  norm_rows(C, s.tpr, s.rpb);
  s.groups = (uint32_t)((rows + s.rpb - 1) / s.rpb);
  s.inv_c = 1.f / (float)C;
  int64_t at = 0;
  for (int i = 0; i < NTEN; ++i) {
    s.off[i] = (int)at;
    if (in.t[i].p) at += (int64_t)s.rpb * C * in.t[i].elem;
  }
  s.stage_bytes = (int)at;
  const int per_sm = norm_blocks_per_sm(C, threads_per_sm, at, smem);
  const int64_t most = (int64_t)sm_count() * per_sm;
  c.grid = (int)std::min<int64_t>(s.groups, most);
  c.threads = s.tpr * s.rpb;
  c.ring = s.groups > most;
  s.stages = (int)std::min<int64_t>(kNormMaxStages, std::max<int64_t>(1, (smem / per_sm - kNormHead) / at));
  c.smem = kNormHead + (c.ring ? (size_t)s.stages * s.stage_bytes : 0);
  if (colsums && s.rpb > 1) c.smem = std::max(c.smem, kNormHead + (size_t)s.rpb * C * sizeof(float));
  return c;
}

template <auto KERN, class P>
static int norm_go(const NormCut& c, const P& p, cudaStream_t s, const char* who) {
  static PerDeviceOnce attr;
  const int rc = once_per_device(attr, [&] {
    return cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) == cudaSuccess
               ? SAMBA_OK
               : fail(SAMBA_ERR_CUDA, "%s: cannot set shared memory size", who);
  });
  if (rc != SAMBA_OK) return rc;
  const cudaError_t e = launch_pdl(KERN, dim3(c.grid), dim3(c.threads), c.smem, s, p);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return check_launch(who);
}

template <typename RT, typename YT>
static int norm_fwd_t(const NormCut& c, const NormFwdParams& p, cudaStream_t s) {
  const char* who = "samba_block_norm_fwd";
  if (c.threads <= 256)
    return c.ring ? norm_go<block_norm_fwd_kernel<RT, YT, 256, true>>(c, p, s, who)
                  : norm_go<block_norm_fwd_kernel<RT, YT, 256, false>>(c, p, s, who);
  if (c.threads <= 512)
    return c.ring ? norm_go<block_norm_fwd_kernel<RT, YT, 512, true>>(c, p, s, who)
                  : norm_go<block_norm_fwd_kernel<RT, YT, 512, false>>(c, p, s, who);
  return c.ring ? norm_go<block_norm_fwd_kernel<RT, YT, 1024, true>>(c, p, s, who)
                : norm_go<block_norm_fwd_kernel<RT, YT, 1024, false>>(c, p, s, who);
}

template <typename RT, typename YT>
static int norm_bwd_t(const NormCut& c, const NormBwdParams& p, cudaStream_t s) {
  const char* who = "samba_block_norm_bwd";
  if (c.threads <= 512)
    return c.ring ? norm_go<block_norm_bwd_kernel<RT, YT, 512, true>>(c, p, s, who)
                  : norm_go<block_norm_bwd_kernel<RT, YT, 512, false>>(c, p, s, who);
  return c.ring ? norm_go<block_norm_bwd_kernel<RT, YT, 1024, true>>(c, p, s, who)
                : norm_go<block_norm_bwd_kernel<RT, YT, 1024, false>>(c, p, s, who);
}

int launch_block_norm_fwd(const samba_block_norm_args& a, cudaStream_t s) {
  if (a.rows == 0) return SAMBA_OK;
  const bool rb = a.r_dtype == SAMBA_BF16, yb = a.y_dtype == SAMBA_BF16;
  const int re = rb ? 2 : 4, ye = yb ? 2 : 4;
  NormFwdParams p = {{{{a.r, re}, {a.y, ye}, {a.gate, ye}}}, a.w_pre, a.w_post, a.alpha, a.r_out, a.n, a.rstd_pre,
                     a.rstd_post, {}, a.eps};
  const NormCut c = norm_cut(p.in, a.rows, a.width, a.width <= 2048 ? 768 : 1024, kFwdSmem, false);
  p.s = c.s;
  if (rb && yb) return norm_fwd_t<__nv_bfloat16, __nv_bfloat16>(c, p, s);
  if (rb) return norm_fwd_t<__nv_bfloat16, float>(c, p, s);
  if (yb) return norm_fwd_t<float, __nv_bfloat16>(c, p, s);
  return norm_fwd_t<float, float>(c, p, s);
}

size_t block_norm_bwd_workspace(int64_t rows, int64_t C) {
  int tpr, rpb;
  norm_rows(C, tpr, rpb);
  const int64_t most = (int64_t)sm_count() * norm_blocks_per_sm(C, kBwdThreadsPerSm, 0, kBwdSmem);
  return (size_t)std::min<int64_t>((rows + rpb - 1) / rpb, most) * 2 * (size_t)C * sizeof(float);
}

int launch_block_norm_bwd(const samba_block_norm_bwd_args& a, cudaStream_t s) {
  const char* who = "samba_block_norm_bwd";
  const int C = (int)a.width;
  if (a.rows == 0) {  // no rows: the sums are empty
    for (float* d : {a.dw_pre, a.dw_post, a.dalpha})
      if (d && cudaMemsetAsync(d, 0, (size_t)C * sizeof(float), s) != cudaSuccess)
        return fail(SAMBA_ERR_CUDA, "%s: memset failed", who);
    return SAMBA_OK;
  }
  const bool rb = a.r_dtype == SAMBA_BF16, yb = a.y_dtype == SAMBA_BF16;
  const int re = rb ? 2 : 4, ye = yb ? 2 : 4;
  NormBwdParams p = {{{{a.dn, ye}, {a.dn ? a.r : nullptr, re}, {a.dr_out, re}, {a.y, ye}, {a.gate, ye}}},
                     a.w_pre, a.rstd_pre, a.w_post, a.rstd_post, a.alpha, a.dr, a.dy, a.dgate,
                     reinterpret_cast<float*>(a.workspace), {}};
  const NormCut c = norm_cut(p.in, a.rows, a.width, kBwdThreadsPerSm, kBwdSmem, true);
  p.s = c.s;
  int rc;
  if (rb && yb) rc = norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(c, p, s);
  else if (rb) rc = norm_bwd_t<__nv_bfloat16, float>(c, p, s);
  else if (yb) rc = norm_bwd_t<float, __nv_bfloat16>(c, p, s);
  else rc = norm_bwd_t<float, float>(c, p, s);
  if (rc != SAMBA_OK || !(a.dn || a.w_post || a.alpha)) return rc;
  const cudaError_t e = launch_pdl(block_norm_cols_kernel, dim3((C + 31) / 32, 2), dim3(256), 0, s, (const float*)p.part,
                                   a.dn ? a.dw_pre : nullptr, a.dw_post, a.dalpha, a.w_post, a.alpha, c.grid, C);
  if (e != cudaSuccess) return fail(SAMBA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return check_launch(who);
}

int take_status_block_norm(cudaStream_t s) { return take_status_word(s); }

}  // namespace samba
