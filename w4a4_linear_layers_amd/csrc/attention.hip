// Attention over the paged cache (gfx950): serq_attn_prefill and
// serq_attn_decode.
//
// Softmax over keys in one pass: with z_j = scale log2(e) q.k_j, the running
// maximum m, sum l = sum 2^(z_j - m) and o = sum 2^(z_j - m) v_j are kept in
// fp32; a larger maximum scales l and o by 2^(m_old - m_new). Parts of the
// keys are joined the same way.
//
// The kernels here read keys and values straight from the cache into registers.
// A decode's waves keep 16 query rows, a group's few heads, and read each key
// once, at the rate of HBM with matrix cores to spare (32 sequences of 513 to
// 32000 tokens, 64 query and 8 key/value heads of 128, 1.04 GB: 195 us, 5.3
// TB/s). fp32 prompts have a loop of their own with 32 rows a wave (three of 500
// to 2000 tokens, 16 heads of 64: 112 us, 96 TFLOP/s of the 154 that a large
// fp32 product reaches). bf16 prompts and long prefixes of many sequences go to
// attn_tile.hip.
//
// Both products are taken transposed. S^T = K Q^T leaves each lane with
// scores of one query (column = lane % 16) and four keys per 16 x 16 tile,
// so the statistics of a query are one value per lane; and as the index that
// a matrix instruction sums over may be renamed on both operands alike,
// those registers, converted, are the second operand of O^T = V^T P^T as
// they are: the lane group g = lane / 16 takes the keys it already holds
// (4 g .. 4 g + 3 of each tile) as its summation slots, and the values are
// loaded to match. Scores never pass through LDS.

#include "attn_common.h"

namespace serq {
namespace {

using namespace attn;

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

// One sequence's pages of one key/value head, for one wave.
template <typename T, int D>
struct Pages {
  const T* k;
  const T* v;
  const int32_t* table;
  int last;            // last page index in use (keys exist)
  int shift, n_pages, Hkv, h;

  // The table's entry of key `key` (a multiple of 16, wave-uniform); keys past
  // the last page give that page again.
  __device__ __forceinline__ int entry(int key) const {
    const int i = key >> shift;
    return page_entry(table, uniform(i < last ? i : last));
  }
  // Element offset of that key.
  __device__ __forceinline__ int64_t at(int key) const { return at(key, entry(key)); }
  __device__ __forceinline__ int64_t at(int key, int entry) const {
    const int page = uniform(in_cache(entry, n_pages));
    return (((static_cast<int64_t>(page) * Hkv + h) << shift) + (key & ((1 << shift) - 1))) * D;
  }
};

// Sixteen query rows of one wave: operands, running statistics, O^T.
template <typename T, int D>
struct Rows;

// bf16: 32 keys a step, v_mfma_f32_16x16x32_bf16. That instruction wants both
// operands in bf16, so each weight is rounded to 8 bits for the product with
// the values, which have no more; their sum l is of the unrounded ones. Whole
// outputs are then 0.0018 to 0.0024 from the 64-bit ones (relative norm),
// 0.0016 to 0.0017 of it their own rounding to bf16. Lane (n = lane % 16, g =
// lane / 16). Q and K operand c of D / 32: values 32 c + 8 g .. + 7 of row n.
// V: lane n holds W = D / 16 values W n .. of each of its eight keys; product
// c takes value W n + c of them as row n of V^T, so O^T register (c, j) is
// value W (4 g + j) + c of query n.
template <int D>
struct Rows<__bf16, D> {
  static constexpr int kStep = 32, C = D / 32, W = D / 16;
  u32x4 q[C];
  f32x4 o[W];
  float m, l;

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
    for (int c = 0; c < C; ++c) q[c] = *reinterpret_cast<const u32x4*>(row + 32 * c + 8 * g);
  }

  __device__ __forceinline__ void step(const Pages<__bf16, D>& pg, int key0, int limit, float scale, int n, int g) {
    const int64_t at0 = pg.at(key0), at1 = pg.at(key0 + 16);
    u32x4 k[2][C];
    uint32_t v[8][W / 2];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      k[0][c] = *reinterpret_cast<const u32x4*>(pg.k + at0 + n * D + 32 * c + 8 * g);
      k[1][c] = *reinterpret_cast<const u32x4*>(pg.k + at1 + n * D + 32 * c + 8 * g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __bf16* p = pg.v + (j < 4 ? at0 : at1) + (4 * g + (j & 3)) * D + W * n;
      if constexpr (W == 8) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = x[i];
      } else {
        const u32x2 x = *reinterpret_cast<const u32x2*>(p);
        v[j][0] = x[0];
        v[j][1] = x[1];
      }
    }
    if (key0 + 32 > limit) {        // what lies past the end may be anything
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = key0 + 16 * (j / 4) + 4 * g + (j & 3) < limit;
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[j][i] = in ? v[j][i] : 0;
      }
    }
    f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[t][c]),
                                                       __builtin_bit_cast(bf16x8, q[c]), s[t], 0, 0, 0);
    }
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = s[j / 4][j & 3] * scale;
    if (key0 + 32 > limit) {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = key0 + 16 * (j / 4) + 4 * g + (j & 3) < limit ? z[j] : kNone;
    }
    float top = z[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, z[j]);
    grow(max_groups(top));
    const float r = ref(m);
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float a = exp2_(z[j] - r), b = exp2_(z[j + 1] - r);
      l += a + b;
      p[j / 2] = pack2(a, b);       // (see above)
    }
    product(v, __builtin_bit_cast(bf16x8, u32x4{p[0], p[1], p[2], p[3]}), o);
  }

  static __device__ __forceinline__ void product(const uint32_t (&v)[8][W / 2], bf16x8 pb, f32x4 (&o)[W]) {
#pragma unroll
    for (int c = 0; c < W; ++c) {
      const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = __builtin_amdgcn_perm(v[2 * i + 1][c / 2], v[2 * i][c / 2], sel);
      o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), pb, o[c], 0, 0, 0);
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

// fp32: 16 keys a step, v_mfma_f32_16x16x4_f32 (one summation slot per lane
// group). Q and K: lane (n, g) holds values 16 c + 4 g .. + 3 of row n; the
// product (c, e) takes value e of them. V: lane n holds values 64 b + 4 n ..
// + 3 of its four keys 4 g + j; product (b, e, j) takes value e, so O^T
// register (b, e, i) is value 64 b + 4 (4 g + i) + e of query n.
template <int D>
struct Rows<float, D> {
  static constexpr int kStep = 16, C = D / 16, NB = D / 64;
  f32x4 q[C];
  f32x4 o[NB * 4];
  float m, l;

  __device__ __forceinline__ void init() {
    m = kNone;
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < NB * 4; ++c) o[c] = f32x4{0, 0, 0, 0};
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
      for (int c = 0; c < NB * 4; ++c) o[c] *= f;
    }
  }

  __device__ __forceinline__ void load_q(const float* row, int g) {
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] = *reinterpret_cast<const f32x4*>(row + 16 * c + 4 * g);
  }

  static __device__ __forceinline__ void fetch_k(const Pages<float, D>& pg, int64_t at, int n, int g, f32x4 (&k)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) k[c] = *reinterpret_cast<const f32x4*>(pg.k + at + n * D + 16 * c + 4 * g);
  }
  static __device__ __forceinline__ void fetch_v(const Pages<float, D>& pg, int64_t at, int n, int g,
                                                 f32x4 (&v)[4][NB]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        v[j][b] = *reinterpret_cast<const f32x4*>(pg.v + at + (4 * g + j) * D + 64 * b + 4 * n);
  }
  // Values of keys that are not there: 0, as 0 * inf is not.
  static __device__ __forceinline__ void clear(f32x4 (&v)[4][NB], int key0, int limit, int g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = key0 + 4 * g + j < limit;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][b][e] = in ? v[j][b][e] : 0.0f;
    }
  }

  __device__ __forceinline__ void step(const Pages<float, D>& pg, int key0, int limit, float scale, int n, int g) {
    const int64_t at = pg.at(key0);
    f32x4 k[C], v[4][NB];
    fetch_k(pg, at, n, g, k);
    fetch_v(pg, at, n, g, v);
    __builtin_amdgcn_sched_barrier(0);       // all loads at once (64 sequences of up to 2048: 119 us against 123)
    float z[4], p[4];
    scores(k, scale, z);
    if (key0 + 16 > limit) {
      clear(v, key0, limit, g);
      mask(z, key0, limit, g);
    }
    weigh(z, p);
    product(v, p, o);
  }

  __device__ __forceinline__ void scores(const f32x4 (&k)[C], float scale, float (&z)[4]) const {
    f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(k[c][e], q[c][e], s[e & 1], 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = (s[0][j] + s[1][j]) * scale;
  }
  static __device__ __forceinline__ void mask(float (&z)[4], int key0, int mine, int g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = key0 + 4 * g + j < mine ? z[j] : kNone;
  }
  __device__ __forceinline__ void weigh(const float (&z)[4], float (&p)[4]) {
    grow(max_groups(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]))));
    const float r = ref(m);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = exp2_(z[j] - r);
    l += (p[0] + p[1]) + (p[2] + p[3]);
  }

  // The product where a value that is not finite lies on a key that some of
  // these queries do not see, and 0 * inf is not 0: each query takes it over
  // its own keys with the others' values cleared.
  __device__ __forceinline__ void product_of_own(const f32x4 (&v)[4][NB], const float (&p)[4], int key0, int mine,
                                                 int n, int g) {
#pragma unroll
    for (int c = 0; c < NB * 4; ++c)
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int lim = __shfl(mine, i, 64);
        f32x4 t = o[c];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          t = __builtin_amdgcn_mfma_f32_16x16x4f32(key0 + 4 * g + j < lim ? v[j][c / 4][c % 4] : 0.0f, p[j], t, 0, 0, 0);
        o[c] = n == i ? t : o[c];
      }
  }

  static __device__ __forceinline__ bool finite(const f32x4 (&v)[4][NB]) {
    bool ok = true;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) ok &= (__float_as_uint(v[j][b][e]) & 0x7F800000u) != 0x7F800000u;
    return ok;
  }

  static __device__ __forceinline__ void product(const f32x4 (&v)[4][NB], const float (&p)[4], f32x4 (&o)[NB * 4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[4 * b + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[j][b][e], p[j], o[4 * b + e], 0, 0, 0);
  }

  __device__ __forceinline__ void store_f32(float* row, int g) const {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(row + 64 * b + 4 * (4 * g + i)) =
            f32x4{o[4 * b][i], o[4 * b + 1][i], o[4 * b + 2][i], o[4 * b + 3][i]};
  }
};

// ------------------------------------------------------------------ prefill

constexpr int kPrefillWaves = 4, kPrefillRows = 32;

// fp32 (bf16 goes to attn_tile.hip). One workgroup: a tile of positions of one
// sequence for `pack` heads of a group, 32 rows in all, which each of its
// waves holds: a wave takes every fourth 16 keys and uses each loaded value
// in two products, and the waves are joined through LDS. What bounds it is the
// matrix cores and, beside them, the cache's path into the registers: with 16
// rows a wave, and so twice the loads, two prompts of 2000 and 2100 (24 heads
// of 128) took 586 us against 462 (112 TFLOP/s), three of 500 to 2000 (16
// heads of 64) 139 against 124; eight of 40 tokens, whose time is the start
// and the join, 11.7 against 12.9. The loop over keys that all rows see is
// apart from the one with masks: together the first takes 627 us. Heads of 128
// fill all 256 registers and put 38 more in scratch (156 bytes a lane) around
// the loop with masks, which reads 16 bytes of them a step; the other has none.
template <int D>
__global__ __launch_bounds__(64 * kPrefillWaves, D == 64 ? 3 : 2) void attn_prefill_kernel(AttnArgs a, PrefillPlan p,
                                                                                      Parts parts) {
  using R = Rows<float, D>;
  constexpr int NO = R::NB * 4, kTurn = 16 * kPrefillWaves;
  __shared__ float2 so[2][2][kPrefillWaves][NO][64];      // [set of rows][half][wave]
  __shared__ float sml[2][kPrefillWaves][2][64];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
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
  R r[2];
  int pos[2], mine[2], end = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int h = unit * p.pack + s % p.pack, pos0 = at.tile * p.tile_pos + 16 * (s / p.pack);
    pos[s] = pos0 + n;
    mine[s] = static_cast<int>(first + pos[s] < 0 ? 0 : first + pos[s]);
    if (mine[s] > len) mine[s] = len;
    const int top = pos0 + 15 < nq ? pos0 + 15 : nq - 1;
    if (pos0 < nq && first + top > end) end = static_cast<int>(first + top);
    const int row = at.q0 + (pos[s] < nq ? pos[s] : nq - 1);
    r[s].init();
    r[s].load_q(static_cast<const float*>(a.Q) + row * a.ldq + static_cast<int64_t>(h) * D, g);
  }
  if (count > 1 && end > from + chunk) end = from + chunk;
  // keys that every row sees
  const int64_t low = first + static_cast<int64_t>(at.tile) * p.tile_pos;
  const int all = static_cast<int>(low < 0 ? 0 : low < len ? low : len);
  int key = from + 16 * wave;
  if (key < end) {
    Pages<float, D> pg{static_cast<const float*>(a.Kc), static_cast<const float*>(a.Vc),
                       a.page_table + static_cast<int64_t>(at.b) * a.max_pages, (len - 1) >> a.page_shift,
                       a.page_shift, a.n_pages, a.Hkv, unit * p.pack / (a.Hq / a.Hkv)};
    f32x4 k[R::C], v[4][R::NB];
    const int64_t at0 = pg.at(key);
    R::fetch_k(pg, at0, n, g, k);
    R::fetch_v(pg, at0, n, g, v);
    int entry = pg.entry(key + kTurn);
    // The next keys come while these ones' values are worked on, those values
    // while the next scores are; the page after them is looked up.
    auto step = [&](auto masked) __attribute__((always_inline)) {
      constexpr bool M = decltype(masked)::value;
      float z[2][4], w[2][4];
      r[0].scores(k, a.scale_log2, z[0]);
      r[1].scores(k, a.scale_log2, z[1]);
      __builtin_amdgcn_sched_barrier(0);
      const int64_t next = pg.at(key + kTurn, entry);
      R::fetch_k(pg, next, n, g, k);
      entry = pg.entry(key + 2 * kTurn);
      if constexpr (M) {
        R::mask(z[0], key, mine[0], g);
        R::mask(z[1], key, mine[1], g);
      }
      r[0].weigh(z[0], w[0]);
      r[1].weigh(z[1], w[1]);
      if (M && key + 16 > len) R::clear(v, key, len, g);
      if (M && __any(!R::finite(v))) {
        r[0].product_of_own(v, w[0], key, mine[0], n, g);
        r[1].product_of_own(v, w[1], key, mine[1], n, g);
      } else {
        R::product(v, w[0], r[0].o);
        R::product(v, w[1], r[1].o);
      }
      __builtin_amdgcn_sched_barrier(0);
      key += kTurn;
      R::fetch_v(pg, next, n, g, v);
    };
    while (key + 16 <= all && key < end) step(std::false_type{});
    while (key < end) step(std::true_type{});
  }
  // Each wave joins one half of the values of one set of rows, of the waves
  // that had keys.
  const int waves = end - from >= kTurn ? kPrefillWaves : (end - from + 15) / 16;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (wave >= waves) break;
    const float l = sum_groups(r[s].l);
#pragma unroll
    for (int c = 0; c < NO; ++c) {
      so[s][0][wave][c][lane] = float2{r[s].o[c][0], r[s].o[c][1]};
      so[s][1][wave][c][lane] = float2{r[s].o[c][2], r[s].o[c][3]};
    }
    sml[s][wave][0][lane] = r[s].m;
    sml[s][wave][1][lane] = l;
  }
  __syncthreads();
  const int s = wave & 1, half = wave >> 1;
  const int p0 = s ? pos[1] : pos[0], m0 = s ? mine[1] : mine[0];
  if (p0 >= nq) return;
  float m = kNone, l = 0.0f;
#pragma unroll
  for (int w = 0; w < kPrefillWaves; ++w)
    if (w < waves) m = fmaxf(m, sml[s][w][0][lane]);
  float2 o[NO] = {};
#pragma unroll
  for (int w = 0; w < kPrefillWaves; ++w) {
    if (w >= waves) break;
    const float f = exp2_(sml[s][w][0][lane] - ref(m));
    l = __builtin_fmaf(f, sml[s][w][1][lane], l);
#pragma unroll
    for (int c = 0; c < NO; ++c) {
      const float2 x = so[s][half][w][c][lane];
      o[c].x = __builtin_fmaf(f, x.x, o[c].x);
      o[c].y = __builtin_fmaf(f, x.y, o[c].y);
    }
  }
  const int row = at.q0 + p0, h = unit * p.pack + s % p.pack;
  float* out = static_cast<float*>(a.O) + row * a.ldo + static_cast<int64_t>(h) * D;
  float inv = inverse(l);
  if (count > 1) {
    if (from >= m0 && from > 0) return;              // the join takes only parts that begin before `mine`
    const int64_t slot = (static_cast<int64_t>(row) * a.Hq + h) * parts.splits + blockIdx.y;
    out = parts.o + slot * D;
    inv = 1.0f;
    if (half == 0 && g == 0) parts.ml[slot] = float2{m, l};
  }
#pragma unroll
  for (int b = 0; b < R::NB; ++b) {
    float* to = out + 64 * b + 4 * (4 * g + 2 * half);
    f32x4 x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = normed(o[4 * b + i].x, inv);
      y[i] = normed(o[4 * b + i].y, inv);
    }
    *reinterpret_cast<f32x4*>(to) = x;
    *reinterpret_cast<f32x4*>(to + 4) = y;
  }
}

// ------------------------------------------------------------------- decode

// One workgroup: 16 query rows over one part of the keys, its waves taking
// steps in turn and joined through LDS; eight of them where the part is all a
// sequence has, which is then written as it is. Prefix parts come first: their rows
// are those of all sequences (row R: sequence R / G, head R % G of the
// group); a sequence's own parts have its G rows.
template <typename T, int D, int kDecodeWaves>
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
  const int R = R0 + n < rows ? R0 + n : rows - 1;
  const int b = R / G, h = kvh * G + R % G;
  Rows<T, D> r;
  r.init();
  r.load_q(static_cast<const T*>(a.Q) + b * a.ldq + static_cast<int64_t>(h) * D, g);
  if (from < to) {
    Pages<T, D> pg{static_cast<const T*>(a.Kc), static_cast<const T*>(a.Vc), table, (len - 1) >> a.page_shift,
                   a.page_shift, a.n_pages, a.Hkv, kvh};
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

// --------------------------------------------------------------------- join

// The parts of a row's keys joined in their order. Rows of a prefill see parts
// that begin before their own limit, rows of a decode the prefix parts and
// those that begin before the sequence's length.
template <bool PREFILL>
__device__ __forceinline__ int parts_of_row(const AttnArgs& a, const PrefillPlan& p, int t, int psplits, int chunk) {
  int keys;
  if constexpr (PREFILL) {
    int b, q0, nq;
    if (parts_for(a, p, count_tiles(a, p.tile_pos), chunk) == 1) return -1;      // (the output is there)
    if (!find_row(a, t, b, q0, nq)) return -1;
    const int64_t first = static_cast<int64_t>(bounded_len(a, b)) - nq + 1;
    keys = static_cast<int>(first + (t - q0) < 0 ? 0 : first + (t - q0));
  } else {
    keys = bounded_len(a, t);
  }
  return psplits + (keys > 0 ? (keys - 1) / chunk + 1 : 0);
}

// Many rows: one wave each.
template <typename T, int D, bool PREFILL>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, PrefillPlan p, int psplits, int chunk,
                                                       Parts parts) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + uniform(threadIdx.x >> 6);
  const int t = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq);
  if (t >= (PREFILL ? a.T : a.B)) return;
  const int count = parts_of_row<PREFILL>(a, p, t, psplits, chunk);
  if (count < 0) return;
  const float2* ml = parts.ml + row * parts.splits;
  const float* po = parts.o + row * parts.splits * D + lane * W;
  // The parts' maxima and sums by lanes, 64 at a time; then their sums of
  // values, eight loads in flight.
  float m = kNone;
  for (int s = lane; s < count; s += 64) m = fmaxf(m, ml[s].x);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  const float r = ref(m);
  float l = 0.0f, o[W] = {};
  for (int s0 = 0; s0 < count; s0 += 64) {
    const int n = count - s0 < 64 ? count - s0 : 64;
    const float2 x = lane < n ? ml[s0 + lane] : float2{kNone, 0.0f};
    const float f = exp2_(x.x - r);                // this lane's part's weight
    l = __builtin_fmaf(f, x.y, l);
    for (int s = 0; s < n; s += 8) {
      float v[8][W];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) v[k][i] = s + k < n ? po[static_cast<int64_t>(s0 + s + k) * D + i] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __shfl(f, (s + k) & 63, 64);
        if (s + k < n) {
#pragma unroll
          for (int i = 0; i < W; ++i) o[i] = __builtin_fmaf(w, v[k][i], o[i]);
        }
      }
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off, 64);
  const float inv = inverse(l);
  T* out = static_cast<T*>(a.O) + t * a.ldo + static_cast<int64_t>(h) * D + lane * W;
#pragma unroll
  for (int i = 0; i < W; ++i) out[i] = static_cast<T>(normed(o[i], inv));
}

// Few rows: a workgroup each, D / 8 lanes to a part, so that the whole row is
// in flight at once. At most 256 parts (2 kMostSplits).
constexpr int kMostSplits = 128;
template <typename T, int D, bool PREFILL>
__global__ __launch_bounds__(256) void attn_join_few_kernel(AttnArgs a, PrefillPlan p, int psplits, int chunk,
                                                       Parts parts) {
  constexpr int L = D / 8, GROUPS = 256 / L;
  static_assert(2 * kMostSplits <= 256, "a thread per part");
  __shared__ float weight[256], so[GROUPS][D], red[2][4];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const int t = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq);
  const int count = parts_of_row<PREFILL>(a, p, t, psplits, chunk);
  if (count < 0) return;
  const float2 x = tid < count ? parts.ml[row * parts.splits + tid] : float2{kNone, 0.0f};
  const int group = tid / L, d = tid % L * 8;
  const float* po = parts.o + row * parts.splits * D + d;
  f32x4 v[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = group + GROUPS * k;
    if (s < count) {
      v[k][0] = *reinterpret_cast<const f32x4*>(po + static_cast<int64_t>(s) * D);
      v[k][1] = *reinterpret_cast<const f32x4*>(po + static_cast<int64_t>(s) * D + 4);
    }
  }
  float m = x.x;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((tid & 63) == 0) red[0][wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  const float f = exp2_(x.x - ref(m));
  weight[tid] = f;
  float l = f * x.y;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off, 64);
  if ((tid & 63) == 0) red[1][wave] = l;
  __syncthreads();
  l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float o[8] = {};
  for (int s = group, k = 0; s < count; s += GROUPS, ++k) {
    f32x4 p, q;
    if (k < 2) {
      p = k ? v[1][0] : v[0][0];
      q = k ? v[1][1] : v[0][1];
    } else {
      p = *reinterpret_cast<const f32x4*>(po + static_cast<int64_t>(s) * D);
      q = *reinterpret_cast<const f32x4*>(po + static_cast<int64_t>(s) * D + 4);
    }
    const float w = weight[s];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = __builtin_fmaf(w, p[i], o[i]);
      o[4 + i] = __builtin_fmaf(w, q[i], o[4 + i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i += 4) *reinterpret_cast<f32x4*>(&so[group][d + i]) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
  __syncthreads();
  if (tid >= D) return;
  float y = 0.0f;
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) y += so[k][tid];
  static_cast<T*>(a.O)[t * a.ldo + static_cast<int64_t>(h) * D + tid] = static_cast<T>(normed(y, inverse(l)));
}

// Which join: 32 sequences of 4096 keys, 256 rows: 26.9 us a call with a
// workgroup a row against 29.5 with a wave; 2048 rows 192 against 194; 3072
// rows of 1024 keys 83.8 against 82.1.
constexpr int64_t kFewRows = 2048;

template <typename T, int D, bool PREFILL>
void launch_join_typed(const AttnArgs& a, const PrefillPlan& p, int64_t rows, int psplits, int chunk,
                       const Parts& parts, hipStream_t st) {
  if (rows <= kFewRows)
    attn_join_few_kernel<T, D, PREFILL><<<dim3(static_cast<unsigned>(rows)), 256, 0, st>>>(a, p, psplits, chunk, parts);
  else
    attn_join_kernel<T, D, PREFILL><<<dim3(static_cast<unsigned>((rows + 3) / 4)), 256, 0, st>>>(a, p, psplits, chunk,
                                                                                                 parts);
}

template <bool PREFILL>
void launch_join(const AttnArgs& a, const PrefillPlan& p, int64_t rows, int psplits, int chunk, const Parts& parts,
                 hipStream_t st) {
  if (a.bf16) {
    if (a.D == 64) launch_join_typed<__bf16, 64, PREFILL>(a, p, rows, psplits, chunk, parts, st);
    else launch_join_typed<__bf16, 128, PREFILL>(a, p, rows, psplits, chunk, parts, st);
  } else {
    if (a.D == 64) launch_join_typed<float, 64, PREFILL>(a, p, rows, psplits, chunk, parts, st);
    else launch_join_typed<float, 128, PREFILL>(a, p, rows, psplits, chunk, parts, st);
  }
}

template <typename T, int D>
void launch_decode(const AttnArgs& a, const DecodePlan& p, const Parts& parts, dim3 grid, hipStream_t st) {
  if (p.waves == 8) attn_decode_kernel<T, D, 8><<<grid, 512, 0, st>>>(a, p, parts);
  else attn_decode_kernel<T, D, 4><<<grid, 256, 0, st>>>(a, p, parts);
}

Parts parts_of(void* workspace, int64_t rows, int D, int splits) {
  float* o = static_cast<float*>(workspace);
  return Parts{o, reinterpret_cast<float2*>(o + rows * splits * D), splits};
}

inline int64_t parts_bytes(int64_t rows, int D, int splits) {
  return splits > 1 ? rows * splits * (D + 2) * static_cast<int64_t>(sizeof(float)) : 0;
}

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// At most `splits` parts of [0, len), each a multiple of `unit` keys; returns the
// part's size and leaves in splits how many there are.
inline int cut(int len, int64_t& splits, int unit = 128) {
  if (splits < 1) splits = 1;
  if (splits > kMostSplits) splits = kMostSplits;
  int chunk = ceil_div(ceil_div(len, splits), unit) * unit;
  if (chunk < unit) chunk = unit;
  splits = len > 0 ? ceil_div(len, chunk) : 1;
  return chunk;
}

}  // namespace

constexpr int kTileRows = 256;       // rows of a workgroup of the tile kernel

// Work of a prefix (sequences * query heads * keys) from which it goes to the
// LDS tiles. They take ~13 us before they gain; the 16-row kernel reads the
// keys from L2 once for every 16 rows. Over 8 key/value heads of 128, bf16,
// join included, tiles against rows: 8192 keys, 64 rows a head 22.2 against
// 21.8 us, 96 rows 24.0 against 29.0, 384 rows 34.0 against 75.7; 2048 keys,
// 256 rows 30.4 against 22.2, 384 rows 24.3 against 27.5; 512 keys, 384 rows
// 18.6 against 12.8.
constexpr int64_t kPrefixTileWork = 6000000;

PrefillPlan plan_prefill(int bf16, int B, int T, int Hq, int Hkv, int D, int max_len) {
  PrefillPlan p{};
  const int G = Hq / Hkv;
  p.tiled = bf16;
  p.pack = p.tiled && G % 8 == 0 ? 8 : p.tiled && G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1;
  p.tile_pos = (p.tiled ? kTileRows : kPrefillRows) / p.pack;
  // Workgroups that run at once: one of the tile kernel's a CU, two or three of
  // the other (two prompts of 33 and 64 tokens over 4000 keys, 16 heads of 64:
  // 41 us for 512 of them, 35 for 768). Few new tokens over many keys leave CUs
  // idle unless the keys are cut: 16 tokens of 32 heads over 4096 keys take 20
  // us with parts and 79 without, 512 over 8192 80 against 153.
  p.target = p.tiled ? 256 : 768;
  int64_t splits = p.target / (static_cast<int64_t>(ceil_div(T, p.tile_pos)) * (Hq / p.pack));
  if (splits > max_len / 256) splits = max_len / 256;
  if (splits > kMostSplits) splits = kMostSplits;
  p.splits = splits < 1 ? 1 : static_cast<int>(splits);
  p.bytes = parts_bytes(static_cast<int64_t>(T) * Hq, D, p.splits);
  // (a launch takes fewer than 2^32 work items along x)
  const int64_t blocks = (static_cast<int64_t>(T / p.tile_pos) + B) * (Hq / p.pack);
  if (blocks * (p.tiled ? 512 : 64 * kPrefillWaves) > UINT32_MAX) p.bytes = -1;
  return p;
}

hipError_t launch_attn_prefill(const AttnArgs& a, const PrefillPlan& p, hipStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hq;
  const Parts parts = parts_of(a.workspace, rows, a.D, p.splits);
  if (p.tiled) {
    const hipError_t e = launch_attn_tile(a, p, parts, st);
    if (e != hipSuccess) return e;
  } else {
    const int64_t tiles = static_cast<int64_t>(a.T / p.tile_pos) + a.B;  // at least the sum of the sequences' tiles
    const dim3 grid(static_cast<unsigned>(tiles * (a.Hq / p.pack)), p.splits), block(64 * kPrefillWaves);
    if (a.D == 64) attn_prefill_kernel<64><<<grid, block, 0, st>>>(a, p, parts);
    else attn_prefill_kernel<128><<<grid, block, 0, st>>>(a, p, parts);
  }
  if (p.splits > 1) launch_join<true>(a, p, rows, 0, 0, parts, st);
  return hipGetLastError();
}

DecodePlan plan_decode(int bf16, int B, int Hq, int Hkv, int D, int prefix_len, int max_len) {
  DecodePlan p{};
  const int G = Hq / Hkv;
  const int64_t rows = static_cast<int64_t>(B) * G;
  p.tiles = ceil_div(G, 16);
  // About 8192 parts in all, so that ragged lengths balance (against 2048, 64
  // sequences of up to 4096 keys: 113 us against 130), of at least 128 keys;
  // of 256 where there are many sequences and heads (96 sequences of 8 heads
  // after a prefix: 50.6 us against 51.6; one of 4095 keys: 9.4 us against 8.4).
  const int64_t groups = static_cast<int64_t>(B) * Hkv * p.tiles;
  int64_t s = ceil_div(8192, groups);
  p.chunk = cut(max_len, s, groups >= 512 ? 256 : 128);
  p.splits = static_cast<int>(s);
  p.waves = 4;
  // Short caches whole: one launch and no join, eight waves a workgroup beyond
  // 256 keys. Against parts, 32 query heads of 8, up to 512 keys: one sequence
  // 7.0 us against 7.6 (launched one by one 8.9 against 12.8), 64 19.3 against
  // 23.8; up to 1024: 96 sequences of 64 heads 53 against 62, 32 of 32 heads
  // 19 against 20.5, but 8 of them 13.8 against 10.5; up to 2048 keys, 64
  // sequences: 71 against 67. Four waves up to 256 keys: 256 sequences 38
  // against 44.
  if (prefix_len == 0 && max_len <= (groups >= 256 ? 1024 : 512)) {
    p.splits = 1;
    p.chunk = max_len > 0 ? max_len : 1;
    p.waves = max_len > 256 ? 8 : 4;
  }
  if (prefix_len > 0) {
    p.ptiled = bf16 && static_cast<int64_t>(B) * Hq * prefix_len >= kPrefixTileWork;
    p.ptiles = ceil_div(rows, p.ptiled ? kTileRows : 16);
    s = ceil_div(p.ptiled ? 256 : 1024, static_cast<int64_t>(Hkv) * p.ptiles);
    p.pchunk = cut(prefix_len, s, p.ptiled ? 64 : 128);
    p.psplits = static_cast<int>(s);
  }
  p.bytes = parts_bytes(static_cast<int64_t>(B) * Hq, D, p.splits + p.psplits);
  return p;
}

// Sequences a launch: fewer than 2^32 work items, 512 of them to a sequence and
// query head at most (beyond this many rows there is one part each).
constexpr int kRowsOfLaunch = 1 << 22;

hipError_t launch_attn_decode(const AttnArgs& all, const DecodePlan& plan, hipStream_t st) {
  const int splits = plan.splits + plan.psplits;
  const Parts all_parts = parts_of(all.workspace, static_cast<int64_t>(all.B) * all.Hq, all.D, splits);
  const int64_t most = kRowsOfLaunch / all.Hq, bytes = all.bf16 ? 2 : 4;
  for (int64_t b = 0; b < all.B; b += most) {
    AttnArgs a = all;
    a.B = static_cast<int>(all.B - b < most ? all.B - b : most);
    a.Q = static_cast<const char*>(all.Q) + b * all.ldq * bytes;
    a.O = static_cast<char*>(all.O) + b * all.ldo * bytes;
    a.kv_len = all.kv_len + b;
    if (all.page_table) a.page_table = all.page_table + b * all.max_pages;
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
    const Parts parts{all_parts.o + b * a.Hq * splits * a.D, all_parts.ml + b * a.Hq * splits, splits};
    DecodePlan p = plan;
    if (p.psplits > 0) p.ptiles = ceil_div(rows / a.Hkv, p.ptiled ? kTileRows : 16);
    if (p.ptiled) {
      const hipError_t e = launch_attn_prefix_tile(a, p.psplits, p.pchunk, parts, st);
      if (e != hipSuccess) return e;
    }
    const int64_t blocks = (p.ptiled ? 0 : static_cast<int64_t>(a.Hkv) * p.ptiles * p.psplits) +
                           static_cast<int64_t>(a.B) * p.tiles * a.Hkv * p.splits;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.bf16) {
      if (a.D == 64) launch_decode<__bf16, 64>(a, p, parts, grid, st);
      else launch_decode<__bf16, 128>(a, p, parts, grid, st);
    } else {
      if (a.D == 64) launch_decode<float, 64>(a, p, parts, grid, st);
      else launch_decode<float, 128>(a, p, parts, grid, st);
    }
    if (splits > 1) launch_join<false>(a, PrefillPlan{}, rows, p.psplits, p.chunk, parts, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace serq
