// The decode kernel, over the kinds of rows (attention.hip, attention_f8.hip):
// a kind R holds sixteen query rows of one wave, and R::step takes kStep keys.
#pragma once

#include "attn_common.h"

namespace serq {
namespace attn {

// Maximum (sum) over the four lane groups that share a query.
__device__ __forceinline__ float max_groups(float v) {
  const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
__device__ __forceinline__ float sum_groups(float v) {
  const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

// One workgroup: 16 query rows over one part of the keys, its waves taking
// steps in turn and joined through LDS; eight of them where the part is all a
// sequence has, which is then written as it is. Prefix parts come first: their rows
// are those of all sequences (row R: sequence R / G, head R % G of the
// group); a sequence's own parts have its G rows.
template <typename R, typename T, int D, int kDecodeWaves>
__global__ __launch_bounds__(64 * kDecodeWaves, kDecodeWaves == 4 && sizeof(T) == 2 ? 3 : 2) void attn_decode_kernel(
    AttnArgs a, DecodePlan p, Parts parts) {
  __shared__ float so[kDecodeWaves][16][D + 4];
  __shared__ float sml[kDecodeWaves][2][16];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  int x = blockIdx.x;
  const int nprefix = p.ptiled ? 0 : a.Hkv * p.ptiles * p.psplits;
  const bool prefix = x < nprefix;
  int kvh, R0, rows, part, len, from, to;
  const int32_t* table;
  if (prefix) {
    kvh = x % a.Hkv;
    x /= a.Hkv;
    part = x % p.psplits;
    R0 = x / p.psplits * 16;
    rows = a.B * G;
    len = a.prefix_len;
    table = a.prefix_table;
    from = part * p.pchunk;
    to = from + p.pchunk;
  } else {
    x -= nprefix;
    kvh = x % a.Hkv;
    x /= a.Hkv;
    part = x % p.splits;
    x /= p.splits;
    const int b = x / p.tiles;
    R0 = b * G + x % p.tiles * 16;
    rows = (b + 1) * G;
    len = bounded_len(a, b);
    table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
    from = part * p.chunk;
    to = from + p.chunk;
    if (from >= len && (from > 0 || p.splits + p.psplits > 1)) return;   // nothing here, and the join knows it
    part += p.psplits;
  }
  if (to > len) to = len;
  const int at = R0 + n < rows ? R0 + n : rows - 1;
  const int b = at / G, h = kvh * G + at % G;
  R r;
  r.init();
  r.load_q(static_cast<const T*>(a.Q) + b * a.ldq + static_cast<int64_t>(h) * D, g);
  if (from < to) {
    const auto pg = R::pages(a, table, (len - 1) >> a.page_shift, kvh);
    for (int key = from + wave * r.kStep; key < to; key += kDecodeWaves * r.kStep)
      r.step(pg, key, to, a.scale_log2, n, g);
  }
  const float lw = sum_groups(r.l);
  r.store_f32(&so[wave][n][0], g);
  if (g == 0) {
    sml[wave][0][n] = r.m;
    sml[wave][1][n] = lw;
  }
  __syncthreads();
  // the waves' parts joined, all threads over the 16 rows
  constexpr int N = 4 * kDecodeWaves, W = D / N;
  const int q = threadIdx.x / N, d = threadIdx.x % N * W;
  if (R0 + q >= rows) return;
  float m = kNone;
#pragma unroll
  for (int w = 0; w < kDecodeWaves; ++w) m = fmaxf(m, sml[w][0][q]);
  float l = 0.0f, o[W] = {};
#pragma unroll
  for (int w = 0; w < kDecodeWaves; ++w) {
    const float f = exp2_(sml[w][0][q] - ref(m));
    l = __builtin_fmaf(f, sml[w][1][q], l);
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = __builtin_fmaf(f, so[w][q][d + i], o[i]);
  }
  const int bq = (R0 + q) / G, hq = kvh * G + (R0 + q) % G;
  if constexpr (kDecodeWaves == 4) {
    if (p.splits + p.psplits > 1) {
      const int64_t slot = (static_cast<int64_t>(bq) * a.Hq + hq) * parts.splits + part;
#pragma unroll
      for (int i = 0; i < W; i += 4)
        *reinterpret_cast<f32x4*>(parts.o + slot * D + d + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
      if (d == 0) parts.ml[slot] = float2{m, l};
      return;
    }
  }
  const float inv = inverse(l);
  T* out = static_cast<T*>(a.O) + bq * a.ldo + static_cast<int64_t>(hq) * D + d;
#pragma unroll
  for (int i = 0; i < W; ++i) out[i] = static_cast<T>(normed(o[i], inv));
}

}  // namespace attn
}  // namespace serq
