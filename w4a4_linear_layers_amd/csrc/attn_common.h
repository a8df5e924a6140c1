// Device helpers that the attention kernels share.
#pragma once

#include "serq_attn.h"

namespace serq {
namespace attn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kNone = -__builtin_inff();

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const bf16x2 p = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, p);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The reference of the exponentials: the running maximum, or 0 while no
// score but -inf has been seen (2^(-inf - 0) = 0).
__device__ __forceinline__ float ref(float m) { return m == kNone ? 0.0f : m; }

// 1 / l, or 0 for a row without keys; NaN stays.
__device__ __forceinline__ float inverse(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }

// Partial results of a row and part, in the caller's workspace: D sums, then
// (m, l) pairs after all sums.
struct Parts {
  float* o;        // rows x splits x D
  float2* ml;      // rows x splits
  int splits;
};

__device__ __forceinline__ int bounded_len(const AttnArgs& a, int b) {
  const int n = a.kv_len[b];
  return n < 0 ? 0 : n < a.max_len ? n : a.max_len;
}

__device__ __forceinline__ int bounded_cu(const AttnArgs& a, int i) {
  const int n = a.cu_q[i];
  return n < 0 ? 0 : n < a.T ? n : a.T;
}

// The sequence that holds tile `tile` of tile_pos positions, counted over all
// sequences: its number, first packed row and rows, and the tile's number
// within it. 64 sequences at a time, one per lane. False past the last.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile_pos, int& tile, int& b, int& q0, int& nq) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < a.B; base += 64) {
    const int i = base + lane;
    const int first = i < a.B ? bounded_cu(a, i) : 0;
    const int n = i < a.B ? bounded_cu(a, i + 1) - first : 0;
    const int tiles = n > 0 ? (n + tile_pos - 1) / tile_pos : 0;
    int upto = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(upto, off, 64);
      if (lane >= off) upto += v;
    }
    const unsigned long long past = __ballot(upto > tile);
    if (past) {
      const int at = __builtin_ctzll(past);
      b = base + at;
      q0 = uniform(__shfl(first, at, 64));
      nq = uniform(__shfl(n, at, 64));
      tile -= uniform(__shfl(upto - tiles, at, 64));
      return true;
    }
    tile -= uniform(__shfl(upto, 63, 64));
  }
  return false;
}

// The first sequence that holds packed row t (its number, first row and
// rows); false if none does.
__device__ __forceinline__ bool find_row(const AttnArgs& a, int t, int& b, int& q0, int& nq) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < a.B; base += 64) {
    const int i = base + lane;
    const int first = i < a.B ? bounded_cu(a, i) : 0;
    const int end = i < a.B ? bounded_cu(a, i + 1) : 0;
    const unsigned long long here = __ballot(t >= first && t < end);
    if (here) {
      const int at = __builtin_ctzll(here);
      b = base + at;
      q0 = uniform(__shfl(first, at, 64));
      nq = uniform(__shfl(end - first, at, 64));
      return true;
    }
  }
  return false;
}

// Entry `i` (wave-uniform) of a row of page ids. No kernel writes the tables it
// reads, so this is a scalar load: as a vector load it would wait for the tile
// loads in flight around it.
__device__ __forceinline__ int page_entry(const int32_t* table, int i) {
  return ((const __attribute__((address_space(4))) int32_t*)table)[i];
}

// A page inside the cache, whatever the entry says.
__device__ __forceinline__ int in_cache(int page, int n_pages) {
  return page < 0 ? 0 : page >= n_pages ? n_pages - 1 : page;
}

}  // namespace attn

// What the tile kernel needs of a plan.
struct TileShape {
  int pack;            // query heads of a group per workgroup (prefill)
  int splits, chunk;   // parts of the keys
};

hipError_t launch_attn_tile(const AttnArgs& a, const TileShape& p, const attn::Parts& parts, hipStream_t stream);
hipError_t launch_attn_prefix_tile(const AttnArgs& a, const TileShape& p, const attn::Parts& parts, hipStream_t stream);

}  // namespace serq
