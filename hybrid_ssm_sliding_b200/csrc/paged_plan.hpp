// How a paged attention call is cut up (host side, shared by its two kernels).
#pragma once

#include <cmath>

#include "../../include/samba.h"

namespace samba {

struct PagedPlan {
  bool chunk_kernel;  // paged_chunk.cu (many rows a kv head) or paged_attn.cu
  int nt;             // paged_attn.cu: 8-row tiles of queries a block
  int ntile;          // row tiles (paged_chunk.cu: units) a sequence may have
  int nsplit, chunk;  // splits a row tile; positions a split at most (paged_attn.cu)
  int cluster, npart; // splits that a cluster joins; results that leaves
};

inline float paged_scale_log2(const samba_paged_attn_args& a) {
  const float scale = a.scale > 0.f ? a.scale : 1.f / std::sqrt(static_cast<float>(a.kv.head_dim));
  return scale * 1.4426950408889634f;
}

// Rows of a unit of paged_chunk.cu.
inline int paged_unit(const samba_paged_attn_args& a) { return a.kv.dtype == SAMBA_E4M3 && a.kv.head_dim <= 64 ? 128 : 256; }

int launch_paged_chunk(const samba_paged_attn_args& a, const PagedPlan& pl, cudaStream_t s);

}  // namespace samba
