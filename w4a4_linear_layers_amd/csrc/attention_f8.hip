// Attention over a paged cache of FP8 (E4M3) codes (gfx950): the kernels that
// read codes straight into registers.
//
// A key is code * 2^e, e from the byte of its 16 tokens and head. Four bits of
// significand times a power of two are a bf16 number as they are, so
// v_cvt_scalef32_pk_bf16_fp8 makes two keys' values of two codes, scale
// included, and the products are those of a bf16 cache with half the bytes: no
// rounding is added to the stored values. (As for a bf16 cache, each softmax
// weight is rounded to bf16 for the product with the values, and sums are
// fp32.)
//
// Decode is bound by the codes' way from HBM: 48 sequences of 513 to 40000 keys, 8
// key/value heads of 128, 177 us at 5.2 TB/s (a large copy reaches 5.1); a bf16
// cache reads twice the bytes. fp32 queries take fp32 products, which bound them:
// a prefill as with an fp32 cache (124 us against 127, 475 against 493).

#include "attn_decode.h"

namespace serq {
namespace {

using namespace attn;

// One sequence's pages of one key/value head, for one wave.
struct Pages8 {
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const int32_t* table;
  int last;            // last page index in use (keys exist)
  int shift, n_pages, Hkv, h;

  // Block (16 tokens of this head) of key `key`, a multiple of 16, wave-uniform;
  // keys past the last page give that page again.
  __device__ __forceinline__ int64_t block(int key) const {
    const int i = key >> shift;
    const int page = uniform(in_cache(page_entry(table, uniform(i < last ? i : last)), n_pages));
    return ((static_cast<int64_t>(page) * Hkv + h) << (shift - 4)) + ((key & ((1 << shift) - 1)) >> 4);
  }
};

// A block's scale, 2^(byte - 127). Kernels that read scales write none, so this
// is a scalar load, of the dword that holds the byte (the arrays are 4-byte aligned,
// and their memory ends with a whole dword).
__device__ __forceinline__ float scale_of(const uint8_t* scales, int64_t block) {
  const uint32_t w = ((const __attribute__((address_space(4))) uint32_t*)scales)[block >> 2];
  return __uint_as_float((w >> (8 * (static_cast<int>(block) & 3)) & 0xFFu) << 23);
}

// Two codes of a word, as two bf16.
template <bool HIGH>
__device__ __forceinline__ uint32_t two_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HIGH));
}

template <typename T, int D>
struct Rows8;

// bf16 queries: TILES tiles of 16 keys a step, v_mfma_f32_16x16x32_bf16. Lane
// (n = lane % 16, g = lane / 16). K: codes 64 b + 16 g .. + 15 of row n in one
// load; product 2 b + i takes codes 8 i .. + 7 of them, and Q to match. V: lane
// n holds W = D / 16 codes W n .. of each of its keys 4 g + j; a code of two
// keys side by side makes a register of V^T, row n of product c is value W n +
// c, so O^T register (c, j) is value W (4 g + j) + c of query n.
template <int D>
struct Rows8<__bf16, D> {
  static constexpr int TILES = 4, kStep = 16 * TILES, B = D / 64, C = D / 32, W = D / 16;
  u32x4 q[C];
  f32x4 o[W];
  float m, l;

  static __device__ __forceinline__ Pages8 pages(const AttnArgs& a, const int32_t* table, int last, int kvh) {
    return {static_cast<const uint8_t*>(a.Kc), static_cast<const uint8_t*>(a.Vc), a.k_scale, a.v_scale, table, last,
            a.page_shift, a.n_pages, a.Hkv, kvh};
  }
  __device__ __forceinline__ void init() {
    m = kNone;
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < W; ++c) o[c] = f32x4{0, 0, 0, 0};
  }
  // The exponentials' reference follows the maximum only where that has
  // outgrown it by 2^8, so that the sums are rarely scaled.
  __device__ __forceinline__ void grow(float top) {
    if (__any(top > m + 8.0f)) {
      const float mn = top > m + 8.0f ? top : m;     // a query's own scores alone decide
      const float f = exp2_(m - ref(mn));
      m = mn;
      l *= f;
#pragma unroll
      for (int c = 0; c < W; ++c) o[c] *= f;
    }
  }

  __device__ __forceinline__ void load_q(const __bf16* row, int g) {
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] = *reinterpret_cast<const u32x4*>(row + 64 * (c / 2) + 16 * g + 8 * (c % 2));
  }

  __device__ __forceinline__ void step(const Pages8& pg, int key0, int limit, float scale, int n, int g) {
    u32x4 k[TILES][B];
    uint32_t v[TILES][4][W / 4];
    float sk[TILES], sv[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int64_t block = pg.block(key0 + 16 * t);
      const uint8_t* kp = pg.k + block * (16 * D) + n * D + 16 * g;
      const uint8_t* vp = pg.v + block * (16 * D) + 4 * g * D + W * n;
      sk[t] = scale_of(pg.k_scale, block);
      sv[t] = scale_of(pg.v_scale, block);
#pragma unroll
      for (int b = 0; b < B; ++b) k[t][b] = *reinterpret_cast<const u32x4*>(kp + 64 * b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (W == 8) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(vp + j * D);
          v[t][j][0] = x[0], v[t][j][1] = x[1];
        } else {
          v[t][j][0] = *reinterpret_cast<const uint32_t*>(vp + j * D);
        }
      }
    }
    const bool ends = key0 + kStep > limit;
    if (ends) {                     // what lies past the end may be anything
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = key0 + 16 * t + 4 * g + j < limit;
#pragma unroll
          for (int i = 0; i < W / 4; ++i) v[t][j][i] = in ? v[t][j][i] : 0;
        }
        sv[t] = key0 + 16 * t < limit ? sv[t] : 1.0f;
      }
    }
    float z[TILES][4];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      f32x4 s = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t w0 = k[t][c / 2][2 * (c % 2)], w1 = k[t][c / 2][2 * (c % 2) + 1];
        const u32x4 x = {two_bf16<false>(w0, sk[t]), two_bf16<true>(w0, sk[t]), two_bf16<false>(w1, sk[t]),
                         two_bf16<true>(w1, sk[t])};
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, q[c]), s,
                                                    0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) z[t][j] = s[j] * scale;
    }
    if (ends) {
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[t][j] = key0 + 16 * t + 4 * g + j < limit ? z[t][j] : kNone;
    }
    float top = z[0][0];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, z[t][j]);
    grow(max_groups(top));
    const float r = ref(m);
    uint32_t p[TILES][2];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float a = exp2_(z[t][j] - r), b = exp2_(z[t][j + 1] - r);
        l += a + b;
        p[t][j / 2] = pack2(a, b);
      }
#pragma unroll
    for (int t = 0; t < TILES; t += 2) {
      const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{p[t][0], p[t][1], p[t + 1][0], p[t + 1][1]});
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        // four values of pairs of keys: (key 2 y, key 2 y + 1) of values 4 i + 2 x, 4 i + 2 x + 1
        uint32_t w[2][2][2];                                   // [tile][y][x]
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            w[u][y][0] = __builtin_amdgcn_perm(v[t + u][2 * y + 1][i], v[t + u][2 * y][i], 0x05010400u);
            w[u][y][1] = __builtin_amdgcn_perm(v[t + u][2 * y + 1][i], v[t + u][2 * y][i], 0x07030602u);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const u32x4 lo = {two_bf16<false>(w[0][0][x], sv[t]), two_bf16<false>(w[0][1][x], sv[t]),
                            two_bf16<false>(w[1][0][x], sv[t + 1]), two_bf16<false>(w[1][1][x], sv[t + 1])};
          const u32x4 hi = {two_bf16<true>(w[0][0][x], sv[t]), two_bf16<true>(w[0][1][x], sv[t]),
                            two_bf16<true>(w[1][0][x], sv[t + 1]), two_bf16<true>(w[1][1][x], sv[t + 1])};
          o[4 * i + 2 * x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lo), pb, o[4 * i + 2 * x], 0, 0, 0);
          o[4 * i + 2 * x + 1] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, hi), pb, o[4 * i + 2 * x + 1], 0, 0, 0);
        }
      }
    }
  }

  // O^T as it lies in memory: for each j, W consecutive values from W (4 g + j).
  __device__ __forceinline__ void store_f32(float* row, int g) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < W; c += 4)
        *reinterpret_cast<f32x4*>(row + W * (4 * g + j) + c) = f32x4{o[c][j], o[c + 1][j], o[c + 2][j], o[c + 3][j]};
  }
};

// fp32 queries: 16 keys a step, v_mfma_f32_16x16x4_f32 (one summation slot per
// lane group). K: lane (n, g) holds codes 64 b + 16 g .. + 15 of row n; product
// (b, c) takes code c of them, and Q to match. V: lane n holds codes 64 b + 4 n
// .. + 3 of its keys 4 g + j; product (b, e, j) takes code e, so O^T register
// (b, e, i) is value 64 b + 4 (4 g + i) + e of query n.
template <int D>
struct Rows8<float, D> {
  static constexpr int kStep = 16, B = D / 64;
  f32x4 q[B * 4];
  f32x4 o[B * 4];
  float m, l;

  static __device__ __forceinline__ Pages8 pages(const AttnArgs& a, const int32_t* table, int last, int kvh) {
    return {static_cast<const uint8_t*>(a.Kc), static_cast<const uint8_t*>(a.Vc), a.k_scale, a.v_scale, table, last,
            a.page_shift, a.n_pages, a.Hkv, kvh};
  }
  __device__ __forceinline__ void init() {
    m = kNone;
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < B * 4; ++c) o[c] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void grow(float top) {              // (as for bf16)
    if (__any(top > m + 8.0f)) {
      const float mn = top > m + 8.0f ? top : m;
      const float f = exp2_(m - ref(mn));
      m = mn;
      l *= f;
#pragma unroll
      for (int c = 0; c < B * 4; ++c) o[c] *= f;
    }
  }
  __device__ __forceinline__ void load_q(const float* row, int g) {
#pragma unroll
    for (int c = 0; c < B * 4; ++c) q[c] = *reinterpret_cast<const f32x4*>(row + 64 * (c / 4) + 16 * g + 4 * (c % 4));
  }

  __device__ __forceinline__ void step(const Pages8& pg, int key0, int limit, float scale, int n, int g) {
    step(pg, key0, limit, limit, scale, n, g);
  }
  // `mine`: the keys that this lane's query sees, at most `limit`.
  __device__ __forceinline__ void step(const Pages8& pg, int key0, int limit, int mine, float scale, int n, int g) {
    const int64_t block = pg.block(key0);
    const uint8_t* kp = pg.k + block * (16 * D) + n * D + 16 * g;
    const uint8_t* vp = pg.v + block * (16 * D) + 4 * g * D + 4 * n;
    const float sk = scale_of(pg.k_scale, block), sv = scale_of(pg.v_scale, block);
    u32x4 k[B];
    uint32_t v[4][B];
#pragma unroll
    for (int b = 0; b < B; ++b) k[b] = *reinterpret_cast<const u32x4*>(kp + 64 * b);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < B; ++b) v[j][b] = *reinterpret_cast<const uint32_t*>(vp + j * D + 64 * b);
    f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(k[b][i], sk, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(k[b][i], sk, true);
        const float x[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], q[4 * b + i][e], s[e & 1], 0, 0, 0);
      }
    float z[4], p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = (s[0][j] + s[1][j]) * scale;
    const bool ends = key0 + 16 > limit, cut = __any(key0 + 16 > mine);
    if (cut) {
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = key0 + 4 * g + j < mine ? z[j] : kNone;
    }
    grow(max_groups(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]))));
    const float r = ref(m);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = exp2_(z[j] - r);
    l += (p[0] + p[1]) + (p[2] + p[3]);
    bool odd = sv >= kInfinities;
    float x[4][B][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = !ends || key0 + 4 * g + j < limit;          // what lies past the end may be anything
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint32_t w = in ? v[j][b] : 0;
        odd |= (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, sv, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, sv, true);
        x[j][b][0] = lo[0], x[j][b][1] = lo[1], x[j][b][2] = hi[0], x[j][b][3] = hi[1];
      }
    }
    if (cut && __any(odd)) {          // NaN or infinities on a key that some of these queries do not see: 0 * NaN is not 0
#pragma unroll
      for (int c = 0; c < B * 4; ++c)
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const int lim = __shfl(mine, i, 64);
          f32x4 t = o[c];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            t = __builtin_amdgcn_mfma_f32_16x16x4f32(key0 + 4 * g + j < lim ? x[j][c / 4][c % 4] : 0.0f, p[j], t, 0, 0, 0);
          o[c] = n == i ? t : o[c];
        }
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[4 * b + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j][b][e], p[j], o[4 * b + e], 0, 0, 0);
  }

  __device__ __forceinline__ void store_f32(float* row, int g) const {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(row + 64 * b + 4 * (4 * g + i)) =
            f32x4{o[4 * b][i], o[4 * b + 1][i], o[4 * b + 2][i], o[4 * b + 3][i]};
  }
};

// ------------------------------------------------------------------ prefill

// fp32 prompts (bf16 goes to attn_tile.hip). One workgroup: a tile of positions
// of one sequence for `pack` heads of a group, 32 rows in all; two waves hold
// 16 of them each, two more take the other half of the keys' steps, and the
// halves are joined through LDS.
template <int D>
__global__ __launch_bounds__(256, 2) void attn_prefill_f8_kernel(AttnArgs a, PrefillPlan p, Parts parts) {
  using R = Rows8<float, D>;
  __shared__ float so[4][16][D + 4];
  __shared__ float sml[4][2][16];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6), set = wave & 1, turn = wave >> 1;
  const int units = a.Hq / p.pack;
  const int unit = blockIdx.x % units;
  TileAt at;
  if (!find_tile<true>(a, p.tile_pos, blockIdx.x / units, at)) return;
  int chunk = 0, count = 1;
  if (p.splits > 1) {
    count = parts_for(a, p, at.total, chunk);
    if (static_cast<int>(blockIdx.y) >= count) return;
  }
  const int nq = at.nq, len = at.len;
  const int64_t first = static_cast<int64_t>(len) - nq + 1;        // keys that position 0 sees
  const int from = static_cast<int>(blockIdx.y) * chunk;
  const int h = unit * p.pack + set % p.pack, pos0 = at.tile * p.tile_pos + 16 * (set / p.pack);
  const int pos = pos0 + n;
  int mine = static_cast<int>(first + pos < 0 ? 0 : first + pos);
  if (mine > len) mine = len;
  const int top = pos0 + 15 < nq ? pos0 + 15 : nq - 1;
  int end = pos0 < nq && first + top > 0 ? static_cast<int>(first + top) : 0;
  if (count > 1 && end > from + chunk) end = from + chunk;
  R r;
  r.init();
  r.load_q(static_cast<const float*>(a.Q) + (at.q0 + (pos < nq ? pos : nq - 1)) * a.ldq + static_cast<int64_t>(h) * D, g);
  if (from < end) {
    const auto pg = R::pages(a, a.page_table + static_cast<int64_t>(at.b) * a.max_pages, (len - 1) >> a.page_shift,
                             unit * p.pack / (a.Hq / a.Hkv));
    for (int key = from + 16 * turn; key < end; key += 32) r.step(pg, key, len, mine, a.scale_log2, n, g);
  }
  const float lw = sum_groups(r.l);
  r.store_f32(&so[wave][n][0], g);
  if (g == 0) {
    sml[wave][0][n] = r.m;
    sml[wave][1][n] = lw;
  }
  __syncthreads();
  // the two halves of each set joined: a quarter of its values a wave's half
  const int x = lane >> 2, d = (lane & 3) * (D / 8) + turn * (D / 2);
  const int px = pos0 + x;
  if (px >= nq) return;
  const int64_t sees = first + px;
  const float m0 = sml[set][0][x], m1 = sml[set + 2][0][x], m = fmaxf(m0, m1);
  const float f0 = exp2_(m0 - ref(m)), f1 = exp2_(m1 - ref(m));
  const float l = __builtin_fmaf(f1, sml[set + 2][1][x], f0 * sml[set][1][x]);
  const int row = at.q0 + px;
  float* out = static_cast<float*>(a.O) + row * a.ldo + static_cast<int64_t>(h) * D;
  float inv = inverse(l);
  if (count > 1) {
    if (from >= sees && from > 0) return;                 // the join takes only parts that begin before a row's keys end
    const int64_t slot = (static_cast<int64_t>(row) * a.Hq + h) * parts.splits + blockIdx.y;
    out = parts.o + slot * D;
    inv = 1.0f;
    if (d == 0) parts.ml[slot] = float2{m, l};
  }
#pragma unroll
  for (int i = 0; i < D / 8; i += 4) {
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[e] = normed(__builtin_fmaf(f1, so[set + 2][x][d + i + e], f0 * so[set][x][d + i + e]), inv);
    *reinterpret_cast<f32x4*>(out + d + i) = y;
  }
}

template <typename T, int D>
void launch_decode_typed(const AttnArgs& a, const DecodePlan& p, const Parts& parts, dim3 grid, hipStream_t st) {
  if (p.waves == 8) attn_decode_kernel<Rows8<T, D>, T, D, 8><<<grid, 512, 0, st>>>(a, p, parts);
  else attn_decode_kernel<Rows8<T, D>, T, D, 4><<<grid, 256, 0, st>>>(a, p, parts);
}

}  // namespace

void launch_decode_f8(const AttnArgs& a, const DecodePlan& p, const Parts& parts, dim3 grid, hipStream_t st) {
  if (a.bf16) {
    if (a.D == 64) launch_decode_typed<__bf16, 64>(a, p, parts, grid, st);
    else launch_decode_typed<__bf16, 128>(a, p, parts, grid, st);
  } else {
    if (a.D == 64) launch_decode_typed<float, 64>(a, p, parts, grid, st);
    else launch_decode_typed<float, 128>(a, p, parts, grid, st);
  }
}

void launch_prefill_f8(const AttnArgs& a, const PrefillPlan& p, const Parts& parts, dim3 grid, hipStream_t st) {
  if (a.D == 64) attn_prefill_f8_kernel<64><<<grid, 256, 0, st>>>(a, p, parts);
  else attn_prefill_f8_kernel<128><<<grid, 256, 0, st>>>(a, p, parts);
}

}  // namespace serq
