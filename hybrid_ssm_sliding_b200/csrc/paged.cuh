// Device-side helpers of the paged cache kernels: the batch description with
// its checks, e4m3 conversions and power-of-two scales.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace samba {

__device__ __forceinline__ void report_batch() { atomicCAS(&g_status, 0, SAMBA_ERR_BATCH); }

// One sequence of a call: its rows [row0, row0 + n) and its length with them.
struct SeqSpan {
  int row0, n, kv;
};

// A sequence's entries, checked against the call's sizes; n = 0 where they are
// out of range (and reported, if `report`).
__device__ __forceinline__ SeqSpan check_span(const samba_paged_batch& bt, int page_size, int s0, int s1, int kv, bool report) {
  SeqSpan s{s0, s1 - s0, kv};
  const int64_t n = static_cast<int64_t>(s1) - s0;
  if (s0 < 0 || n < 0 || s1 > bt.rows || n > bt.max_q || kv < n || kv > bt.max_kv || kv > bt.max_pages * page_size) {
    if (report) report_batch();
    s.n = 0;
  }
  return s;
}
__device__ __forceinline__ SeqSpan seq_span(const samba_paged_batch& bt, int page_size, int b, bool report) {
  return check_span(bt, page_size, bt.q_start[b], bt.q_start[b + 1], bt.kv_len[b], report);
}

// Power of two 2^k as a float, k in [-126, 127].
__device__ __forceinline__ float exp2i(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }
// k of a power of two 2^k, k in [-126, 127].
__device__ __forceinline__ int log2i(float s) { return static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127; }

// Scales are powers of two within these exponents.  The range is narrow enough
// for one running maximum to serve scores s and value scales 2^e together: with
// p' = 2^(s + e - m), m at least kScaledRef below the largest s + e, the sum of
// p' 2^-e loses what lies below 2^-126, a part of under 2^-43 of it.
constexpr int kScaleMin = -60, kScaleMax = 30;

// The product with V takes p' rounded to f16, between 2^7 and 2^15 at a row's
// largest s + e: full precision down to 2^-21 of that, nothing below 2^-32.  So a
// page whose value scale is 2^20 times another's leaves the other's values (in
// elements where its own codes are small) five bits at equal scores; with the
// largest p' at 1 it left them none.
constexpr float kScaledRef = 7.f;

// The smallest k >= kScaleMin with amax <= 448 * 2^k (448 = 1.75 * 2^8), at
// most kScaleMax, in whole-number arithmetic on the bits: no rounding decides it.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127;
  const int k = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return k < kScaleMin ? kScaleMin : k > kScaleMax ? kScaleMax : k;
}

// A stored scale's exponent; anything that is no such scale (an uninitialised
// pool) counts as the smallest.
__device__ __forceinline__ int stored_exponent(float s) {
  const int k = log2i(s);
  return (s > 0.f && k >= kScaleMin && k <= kScaleMax) ? k : kScaleMin;
}

// Four floats to four e4m3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The low or high two codes of a word as packed f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w, bool high) {
  uint32_t r;
  const uint16_t h = static_cast<uint16_t>(high ? w >> 16 : w);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}

}  // namespace samba
