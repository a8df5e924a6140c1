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

// 1 / l, or 0 for a row without weights (no keys, or scores of -inf alone);
// NaN stays.
__device__ __forceinline__ float inverse(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }
// A sum of weighted values by that: 0 for such a row, whose sum may hold NaN
// (0 * inf).
__device__ __forceinline__ float normed(float o, float inv) { return inv == 0.0f ? 0.0f : o * inv; }

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

// Sums over the lanes up to each one, and over all.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);      // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);      // row_bcast:15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }

// One tile of tile_pos positions: sequence b (its first packed row, rows and
// keys), the tile's number within it; and how many tiles there are in all.
struct TileAt {
  int b, q0, nq, len, tile, total;
};

// Tile `idx` of all sequences; false past the last. Up to 64 sequences lie in
// the lanes and come in an order in which the workgroups that run last are
// short. BY_KEYS: by the keys a tile sees, most first: with class = (keys
// before the tile) / tile_pos, the class of tile idx is the largest c with
// more than idx tiles of class >= c, found by bisection. Otherwise sequence by
// sequence, the one with the most keys first, each one's longest tile first:
// sorted by counting, which takes a fifth of the bisection's 2000 cycles. (The
// fp32 kernel, whose workgroups share a CU, gains from the former, 112 us
// against 122 for three sequences of 500 to 2000 tokens; on LDS tiles both
// orders run alike.) More sequences than lanes come one after another, each
// one's longest tile first.
template <bool BY_KEYS>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile_pos, int idx, TileAt& at) {
  const int lane = threadIdx.x & 63;
  const auto load = [&](int i, int& first, int& n, int& len, int& tiles) {
    const bool in = i < a.B;
    first = in ? bounded_cu(a, i) : 0;
    n = in ? bounded_cu(a, i + 1) - first : 0;
    len = in ? bounded_len(a, i) : 0;
    tiles = n > 0 ? (n + tile_pos - 1) / tile_pos : 0;
  };
  const auto take = [&](int b, int from, int first, int n, int len, int tile) {
    at.b = uniform(b);
    at.q0 = __builtin_amdgcn_readlane(first, from);
    at.nq = __builtin_amdgcn_readlane(n, from);
    at.len = __builtin_amdgcn_readlane(len, from);
    at.tile = uniform(tile);
  };
  int first, n, len, tiles;
  if (a.B <= 64) {
    load(lane, first, n, len, tiles);
    if (a.B == 1) {
      at.total = __builtin_amdgcn_readfirstlane(tiles);
      if (idx >= at.total) return false;
      take(0, 0, first, n, len, at.total - 1 - idx);
      return true;
    }
    if constexpr (BY_KEYS) {
      at.total = wave_sum(tiles);
      if (idx >= at.total) return false;
      const int base = len > n ? (len - n) / tile_pos : 0;
      const auto from_class = [&](int c) {         // tiles of class >= c
        const int k = base + tiles - c;
        return wave_sum(k < 0 ? 0 : k < tiles ? k : tiles);
      };
      int lo = 0, hi = (a.max_len + a.T) / tile_pos + 2;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (from_class(mid) > idx) lo = mid;
        else hi = mid;
      }
      lo = uniform(lo);
      const int rank = idx - from_class(lo + 1);
      const bool has = base <= lo && lo < base + tiles;
      const unsigned long long all = __ballot(has);
      const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), 0));
      const int from = __builtin_ctzll(__ballot(has && before == rank));
      take(from, from, first, n, len, lo - __builtin_amdgcn_readlane(base, from));
    } else {
      int rank = 0;                                // sequences before this one; those past B stay last
      for (int j = 0; j < a.B; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane) ? 1 : 0;
      }
      rank = lane < a.B ? rank : lane;
      const int order = __builtin_amdgcn_ds_permute(rank << 2, lane);
      const int sorted = __builtin_amdgcn_ds_permute(rank << 2, tiles);
      const int upto = wave_scan(sorted);
      at.total = __builtin_amdgcn_readlane(upto, 63);
      if (idx >= at.total) return false;
      const int place = __builtin_ctzll(__ballot(upto > idx));
      const int from = __builtin_amdgcn_readlane(order, place);
      take(from, from, first, n, len, __builtin_amdgcn_readlane(upto, place) - 1 - idx);
    }
    return true;
  }
  bool found = false;
  at.total = 0;
  for (int start = 0; start < a.B; start += 64) {
    load(start + lane, first, n, len, tiles);
    const int upto = wave_scan(tiles);
    const int sum = __builtin_amdgcn_readlane(upto, 63);
    if (!found && idx < at.total + sum) {
      const int want = idx - at.total;
      const int from = __builtin_ctzll(__ballot(upto > want));
      take(start + from, from, first, n, len, __builtin_amdgcn_readlane(upto, from) - 1 - want);
      found = true;
    }
    at.total += sum;
  }
  return found;
}

// All tiles of a call.
__device__ __forceinline__ int count_tiles(const AttnArgs& a, int tile_pos) {
  int sum = 0;
  for (int i = threadIdx.x & 63; i < a.B; i += 64) {
    const int n = bounded_cu(a, i + 1) - bounded_cu(a, i);
    sum += n > 0 ? (n + tile_pos - 1) / tile_pos : 0;
  }
  return wave_sum(sum);
}

// How a prefill's keys are cut, known once its tiles are counted: as many
// parts as fill the card with the workgroups there are, at most the plan's.
// (The host knows bounds alone; a part too many for one round of workgroups
// costs a whole round.)
__device__ __forceinline__ int parts_for(const AttnArgs& a, const PrefillPlan& p, int total, int& chunk) {
  const int groups = total * (a.Hq / p.pack);
  int parts = groups > 0 ? p.target / groups : 1;
  parts = uniform(parts < 1 ? 1 : parts < p.splits ? parts : p.splits);
  chunk = uniform(((a.max_len + parts - 1) / parts + 63) & ~63);
  return parts;
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

hipError_t launch_attn_tile(const AttnArgs& a, const PrefillPlan& p, const attn::Parts& parts, hipStream_t stream);
// The prefix of a decode in `splits` parts of `chunk` keys.
hipError_t launch_attn_prefix_tile(const AttnArgs& a, int splits, int chunk, const attn::Parts& parts,
                                   hipStream_t stream);

}  // namespace serq
