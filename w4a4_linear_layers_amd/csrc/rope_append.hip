// Rotary positions, head norms and the paged cache write in one pass (gfx950).
//
// From row t of the q/k/v linear's output, head by head:
//     y = x * w / sqrt(mean(x^2) + eps),  (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s),
// queries to Q, keys and the unchanged values to slot[t] of the cache. Every
// value is read once and written once, so the kernel is bound by HBM for
// prompts (8192 tokens of 48 heads of 128 with norms, bf16, 206 MB: 46 us from
// HBM, 4.5 TB/s; 35 us with the inputs in the last-level cache) and by latency
// for single tokens (one token 2.4 us, about a launch).

#include "serq_attn.h"

namespace serq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;     // elements of a 16-byte chunk
  static __device__ __forceinline__ void unpack(u32x4 w, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[4]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    return w;
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ float round(float v) { return v; }
};
template <>
struct Elem<__bf16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf2 p = {static_cast<__bf16>(v[2 * i]), static_cast<__bf16>(v[2 * i + 1])};
      w[i] = __builtin_bit_cast(uint32_t, p);
    }
    return w;
  }
  static __device__ __forceinline__ float load(const __bf16* p) { return static_cast<float>(*p); }
  static __device__ __forceinline__ __bf16 round(float v) { return static_cast<__bf16>(v); }
};

// N floats in 8- or 16-byte loads (the table's rows and the norms are 16-byte
// aligned where the vector path runs): one dword a load, the sixteen cosines
// and sines and sixteen weights of a lane cost more than its data.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
  typedef float f32xk __attribute__((ext_vector_type(N < 4 ? N : 4)));
  constexpr int K = N < 4 ? N : 4;
#pragma unroll
  for (int i = 0; i < N; i += K) {
    const f32xk x = *reinterpret_cast<const f32xk*>(p + i);
#pragma unroll
    for (int j = 0; j < K; ++j) v[i + j] = x[j];
  }
}

// 1 / sqrt(x). The instruction takes numbers below the normal ones for 0.
__device__ __forceinline__ float inverse_root(float x) {
  const bool tiny = x < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(tiny ? x * 0x1p100f : x);
  return tiny ? r * 0x1p50f : r;
}

// Where token t's keys and values go: element offset of its slot for head 0
// (heads are D << page_shift apart), or -1.
__device__ __forceinline__ int64_t slot_base(const RopeArgs& a, int slot, bool pos_ok) {
  if (!pos_ok || slot < 0 || (slot >> a.page_shift) >= a.n_pages) return -1;
  const int64_t page = slot >> a.page_shift, in = slot & ((1 << a.page_shift) - 1);
  return ((page * a.Hkv << a.page_shift) + in) * a.D;
}

// A token's position on each axis, and whether all lie in the table.
struct Place {
  int pos[4];
  bool ok;
};
template <bool AXES>
__device__ __forceinline__ Place place_of(const RopeArgs& a, int t) {
  Place p{{0, 0, 0, 0}, true};
  if (a.rot) {
#pragma unroll
    for (int x = 0; x < (AXES ? 4 : 1); ++x)
      if (!AXES || x < a.n_axes) {
        p.pos[x] = a.pos[x * a.pos_stride + t];
        p.ok &= p.pos[x] >= 0 && p.pos[x] < a.max_pos;
      }
  }
  return p;
}

// Two bits for each pair from pair i on (i a multiple of the pairs asked for, at most 16).
__device__ __forceinline__ uint32_t axes_from(const RopeArgs& a, int i) {
  const uint32_t w = i < 32 ? (i < 16 ? a.axis_bits[0] : a.axis_bits[1]) : (i < 48 ? a.axis_bits[2] : a.axis_bits[3]);
  return w >> (2 * (i & 15));
}

// Cosines and sines of N pairs from pair i on. With several axes a pair takes
// them from the row of its axis' position: for each axis that one of the pairs
// has, its row is loaded whole and the pairs take their own.
template <int N, bool AXES>
__device__ __forceinline__ void load_turns(const RopeArgs& a, const Place& at, int i, float (&c)[N], float (&s)[N]) {
  const int half = a.rot / 2;
  if constexpr (!AXES) {
    const float* row = a.table + static_cast<int64_t>(at.pos[0]) * a.rot;
    load_floats<N>(row + i, c);
    load_floats<N>(row + half + i, s);
  } else {
    const uint32_t axes = axes_from(a, i);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      bool any = false;
#pragma unroll
      for (int j = 0; j < N; ++j) any |= (axes >> (2 * j) & 3) == x;
      if (x < a.n_axes && any) {
        float c1[N], s1[N];
        const float* row = a.table + static_cast<int64_t>(at.pos[x]) * a.rot;
        load_floats<N>(row + i, c1);
        load_floats<N>(row + half + i, s1);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const bool mine = (axes >> (2 * j) & 3) == x;
          c[j] = mine ? c1[j] : c[j];
          s[j] = mine ? s1[j] : s[j];
        }
      }
    }
  }
}

// The table's row for pair i.
template <bool AXES>
__device__ __forceinline__ const float* row_of(const RopeArgs& a, const Place& at, int i) {
  int pos = at.pos[0];
  if constexpr (AXES) {
    const uint32_t x = axes_from(a, i) & 3;
    pos = x < 2 ? (x == 0 ? at.pos[0] : at.pos[1]) : (x == 2 ? at.pos[2] : at.pos[3]);
  }
  return a.table + static_cast<int64_t>(pos) * a.rot;
}

// y = x A + partner B for the N values from d0 on (d0 below rot): A = c, B = -s
// in the first half of a pair and s in the second.
template <int N, bool INTER, bool AXES>
__device__ __forceinline__ void load_factors(const RopeArgs& a, const Place& at, int d0, float (&A)[N], float (&B)[N]) {
  if constexpr (INTER) {
    float c[N / 2] = {}, s[N / 2] = {};
    load_turns<N / 2, AXES>(a, at, d0 / 2, c, s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      A[i] = c[i / 2];
      B[i] = i & 1 ? s[i / 2] : -s[i / 2];
    }
  } else {
    const int half = a.rot / 2;
    const bool second = d0 >= half;
    load_turns<N, AXES>(a, at, second ? d0 - half : d0, A, B);
#pragma unroll
    for (int i = 0; i < N; ++i) B[i] = second ? B[i] : -B[i];
  }
}

// Vector path: 16-byte aligned rows, rot_dim made of whole chunks in each
// half (SERQ_ROPE_HALF) or in all (SERQ_ROPE_INTERLEAVED). A head is D / kVec
// lanes of one chunk each; a workgroup holds 256 / lanes heads of one token
// at a time and NB such sets, all of whose loads it starts before the first
// use, since the cosines and sines come only after the position they belong
// to. What depends on the lane's place in the head alone (cosines, sines, norm
// weights) is loaded once for all its heads; the other half's values come from
// the lane that holds them.
template <typename T, int D, bool INTER, bool NORM, bool AXES, int NB>
__device__ __forceinline__ void rope_heads(const RopeArgs& a, int t, int set, int heads) {
  using E = Elem<T>;
  constexpr int V = E::kVec, L = D / V, GROUPS = kThreads / L;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int d0 = lane * V;
  const int first = set * (GROUPS * NB) + group;
  const T* in = static_cast<const T*>(a.QKV) + t * a.ld + d0;
  u32x4 raw[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int h = first + GROUPS * k;
    if (h < heads) raw[k] = *reinterpret_cast<const u32x4*>(in + static_cast<int64_t>(h) * D);
  }
  const int slot = a.slot[t];
  const Place at = place_of<AXES>(a, t);
  const bool pos_ok = at.ok, turned = d0 < a.rot;
  const int half = a.rot / 2;
  float A[V], B[V], wq[V], wk[V];
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = 1.0f, B[i] = 0.0f;
  if (turned && pos_ok) load_factors<V, INTER, AXES>(a, at, d0, A, B);
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < V; ++i) wq[i] = wk[i] = 1.0f;
    if (a.q_norm) load_floats<V>(a.q_norm + d0, wq);
    if (a.k_norm) load_floats<V>(a.k_norm + d0, wk);
  }
  const int64_t base = slot_base(a, slot, pos_ok);
  const int step = half / V;                     // lanes to the other half
  const int mate = INTER || !turned ? lane : (d0 < half ? lane + step : lane - step);
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int h = first + GROUPS * k;
    if (h >= heads) break;
    const bool key = h >= a.Hq, value = h >= a.Hq + a.Hkv;
    u32x4 out = raw[k];
    if (!value) {
      float x[V], y[V];
      E::unpack(raw[k], x);
      if constexpr (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = __builtin_fmaf(x[i], x[i], ss);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor(ss, off, L);
        if (key ? a.k_norm != nullptr : a.q_norm != nullptr) {
          const float r = inverse_root(ss * (1.0f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] *= r * (key ? wk[i] : wq[i]);
        }
      }
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = x[i ^ 1];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = __shfl(x[i], mate, L);
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __builtin_fmaf(x[i], A[i], y[i] * B[i]);
      }
      if (!pos_ok) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __builtin_nanf("");
      }
      out = E::pack(x);
    }
    if (!key) {
      *reinterpret_cast<u32x4*>(static_cast<T*>(a.Q) + t * a.ldq + static_cast<int64_t>(h) * D + d0) = out;
    } else if (base >= 0) {
      const int kvh = h - a.Hq - (value ? a.Hkv : 0);
      T* c = static_cast<T*>(value ? a.Vc : a.Kc);
      *reinterpret_cast<u32x4*>(c + base + (static_cast<int64_t>(kvh) << a.page_shift) * D + d0) = out;
    }
  }
}

template <typename T, int D, bool INTER, bool NORM, bool AXES, int NB>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeArgs a) {
  rope_heads<T, D, INTER, NORM, AXES, NB>(a, blockIdx.x, blockIdx.y, a.Hq + 2 * a.Hkv);
}

// Scalar path, any row alignment and rot_dim: one wave per head, values
// d = lane + 64 e; partners are exchanged between lanes, so every value is
// read before any is written (Q may be QKV).
template <typename T, int D, bool AXES>
__global__ __launch_bounds__(64) void rope_append_scalar_kernel(RopeArgs a) {
  using E = Elem<T>;
  constexpr int N = D / 64;
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  const Place at = place_of<AXES>(a, t);
  const bool pos_ok = at.ok;
  const int64_t base = slot_base(a, a.slot[t], pos_ok);
  const bool key = h >= a.Hq, value = h >= a.Hq + a.Hkv;
  const T* in = static_cast<const T*>(a.QKV) + t * a.ld + static_cast<int64_t>(h) * D;
  float x[N];
  T raw[N];
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    raw[e] = in[lane + 64 * e];
    x[e] = E::load(&raw[e]);
    ss = __builtin_fmaf(x[e], x[e], ss);
  }
  if (!value) {
    const float* w = key ? a.k_norm : a.q_norm;
    if (w) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) ss += __shfl_xor(ss, off, 64);
      const float r = inverse_root(ss * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= r * w[lane + 64 * e];
    }
    const int half = a.rot / 2;
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int d = lane + 64 * e;
      const int m = d >= a.rot ? d : a.interleaved ? d ^ 1 : d < half ? d + half : d - half;
      float p = 0.0f;
#pragma unroll
      for (int f = 0; f < N; ++f) {
        const float v = __shfl(x[f], m & 63, 64);
        if (m / 64 == f) p = v;
      }
      y[e] = x[e];
      if (d < a.rot && pos_ok) {
        const bool second = a.interleaved ? (d & 1) : d >= half;
        const int i = a.interleaved ? d / 2 : second ? d - half : d;
        const float* row = row_of<AXES>(a, at, i);
        const float s = row[half + i];
        y[e] = __builtin_fmaf(x[e], row[i], p * (second ? s : -s));
      }
      if (!pos_ok) y[e] = __builtin_nanf("");
    }
#pragma unroll
    for (int e = 0; e < N; ++e) raw[e] = E::round(y[e]);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int d = lane + 64 * e;
    if (!key) {
      static_cast<T*>(a.Q)[t * a.ldq + static_cast<int64_t>(h) * D + d] = raw[e];
    } else if (base >= 0) {
      const int kvh = h - a.Hq - (value ? a.Hkv : 0);
      static_cast<T*>(value ? a.Vc : a.Kc)[base + (static_cast<int64_t>(kvh) << a.page_shift) * D + d] = raw[e];
    }
  }
}

// ---- A cache of FP8 codes (serq_rope_append_f8) ----
//
// Sixteen tokens (a block) of a head share a power of two 2^e, e the least with
// max |y| <= 448 * 2^e, so a block's codes need all of its new tokens: a run of
// consecutive rows that go to one block. Keys are taken
// in 64 bits and rounded to fp32 once, so that a cache does not depend on the
// order of a sum: next to the border of two codes, or of two scales, the last
// bit of a key would decide (8192 tokens of 8 normed heads of 128: 8 us of the
// 30 are this arithmetic).

// Least exponent >= kLeast with |y| <= 448 * 2^e for the finite fp32 number of bits `top`.
constexpr int kLeast = -117, kMost = 120;
__device__ __forceinline__ int exponent_for(uint32_t top) {
  const int e = static_cast<int>(top >> 23) - 135 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);    // 448 = 1.75 * 2^8
  return e < kLeast ? kLeast : e;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ uint32_t codes4(const float* y) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true));
}
__device__ __forceinline__ uint32_t recode4(uint32_t w, float f) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  const float y[4] = {a[0] * f, a[1] * f, b[0] * f, b[1] * f};
  return codes4(y);
}

// One window of 16 rows, one key/value head, keys or values: the runs that
// begin in it, whose rows are among 31. A row is the L lanes of a vector
// load; a wave's lanes also hold a row each (lane i + 1: row i) for what is
// known of rows: their slots, runs and maxima.
// VEC: as for the vector path above; otherwise every value and its partner are
// loaded one by one.
template <typename T, int D, bool INTER, bool NORM, bool VEC>
__device__ __forceinline__ void store_codes(const RopeArgs& a, int window, int kvh, bool value) {
  using E = Elem<T>;
  constexpr int V = E::kVec, L = D / V, GROUPS = kThreads / L, PASSES = GROUPS >= 32 ? 1 : 32 / GROUPS;
  __shared__ uint32_t tops[PASSES * GROUPS];
  const int wl = threadIdx.x & 63, mine_row = wl - 1;
  const int lane = threadIdx.x % L, group = threadIdx.x / L, d0 = lane * V;
  const int row0 = 16 * window;
  // the rows' slots and runs
  int slot = -1;
  if (wl <= 32 && row0 + mine_row >= 0 && row0 + mine_row < a.M) {
    slot = a.slot[row0 + mine_row];
    if (slot < 0 || (slot >> a.page_shift) >= a.n_pages || !place_of<true>(a, row0 + mine_row).ok) slot = -1;
  }
  const int before = __shfl_up(slot, 1, 64);
  const bool next = wl > 0 && slot >= 0 && before >= 0 && slot >> 4 == before >> 4;
  const uint64_t joined = __ballot(next) >> 1;                        // bit i: row i continues row i - 1
  const uint64_t starts = __ballot(slot >= 0 && !next) >> 1;
  const uint32_t upto = mine_row < 0 ? 0 : static_cast<uint32_t>(starts) & ((2u << (mine_row & 31)) - 1u);
  const int start = upto ? 31 - __builtin_clz(upto) : 16;
  const bool own = wl >= 1 && wl <= 32 && slot >= 0 && start < 16;
  const uint64_t rows = __ballot(own) >> 1;
  if (rows == 0) return;
  const int end = own ? mine_row + __builtin_ctzll(~(joined >> wl)) : 0;          // (bit 63 of a shifted mask is 0)
  uint8_t* scales = value ? a.v_scale : a.k_scale;
  const int per = a.page_shift - 4;                                               // blocks of a page: 1 << per
  const int64_t at_scale =
      own ? (((static_cast<int64_t>(slot >> a.page_shift) * a.Hkv + kvh) << per) + ((slot >> 4) & ((1 << per) - 1))) : 0;
  int old = kLeast;
  if (own && mine_row == start) {
    old = static_cast<int>(scales[at_scale]) - 127;
    old = old < kLeast ? kLeast : old > kMost ? kMost : old;
  }
  const bool norm = NORM && !value && a.k_norm;
  const bool turned = !value && d0 < a.rot;
  const int half = a.rot / 2;
  float y[PASSES][V];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = group + GROUPS * p, t = row0 + i;
    const bool in = i < 32 && (rows >> i & 1) != 0;
#pragma unroll
    for (int j = 0; j < V; ++j) y[p][j] = 0.0f;
    const T* src = static_cast<const T*>(a.QKV) + (in ? t : row0) * a.ld +
                   static_cast<int64_t>(a.Hq + (value ? a.Hkv : 0) + kvh) * D;
    if (in) {
      if constexpr (VEC) {
        E::unpack(*reinterpret_cast<const u32x4*>(src + d0), y[p]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) y[p][j] = E::load(src + d0 + j);
      }
    }
    if (!value) {
      double x[V], z[V];
      if constexpr (NORM) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) ss += static_cast<double>(y[p][j]) * y[p][j];
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor(ss, off, L);
        const double r = norm ? 1.0 / sqrt(ss * (1.0 / D) + static_cast<double>(a.eps)) : 1.0;
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = y[p][j] * r * (norm ? static_cast<double>(a.k_norm[d0 + j]) : 1.0);
        if constexpr (!VEC) {                 // the partner, normed alike
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int d = d0 + j, m = d >= a.rot ? d : INTER ? d ^ 1 : d < half ? d + half : d - half;
            z[j] = in ? static_cast<double>(E::load(src + m)) * r * (norm ? static_cast<double>(a.k_norm[m]) : 1.0) : 0.0;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = y[p][j];
        if constexpr (!VEC) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int d = d0 + j, m = d >= a.rot ? d : INTER ? d ^ 1 : d < half ? d + half : d - half;
            z[j] = in ? E::load(src + m) : 0.0f;
          }
        }
      }
      if constexpr (VEC) {
        if constexpr (INTER) {
#pragma unroll
          for (int j = 0; j < V; ++j) z[j] = x[j ^ 1];
        } else {
          const int step = half / V, mate = !turned ? lane : d0 < half ? lane + step : lane - step;
#pragma unroll
          for (int j = 0; j < V; ++j) z[j] = __shfl(x[j], mate, L);
        }
      }
      if (in && turned) {
        const Place at = place_of<true>(a, t);
        float A[V], B[V];
        if constexpr (VEC) {
          load_factors<V, INTER, true>(a, at, d0, A, B);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int d = d0 + j;
            A[j] = 1.0f, B[j] = 0.0f;
            if (d < a.rot) {
              const bool second = INTER ? (d & 1) : d >= half;
              const int pair = INTER ? d / 2 : second ? d - half : d;
              const float* row = row_of<true>(a, at, pair);
              A[j] = row[pair];
              B[j] = second ? row[half + pair] : -row[half + pair];
            }
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = x[j] * A[j] + z[j] * B[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) y[p][j] = static_cast<float>(x[j]);
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t b = __float_as_uint(y[p][j]) & 0x7FFFFFFFu;
      top = b < 0x7F800000u && b > top ? b : top;                     // (NaN and infinities become NaN codes)
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) {
      const uint32_t o = __shfl_xor(top, off, L);
      top = o > top ? o : top;
    }
    if (lane == 0) tops[i] = in ? top : 0;
  }
  __syncthreads();
  // the runs' maxima, exponents and blocks
  uint32_t top = own ? tops[mine_row] : 0, tokens = own ? 1u << (slot & 15) : 0;
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) {
    const uint32_t o = __shfl_up(top, off, 64), s = __shfl_up(tokens, off, 64);
    if (own && mine_row - off >= start) {
      top = o > top ? o : top;
      tokens |= s;
    }
  }
  top = __shfl(top, end + 1, 64);
  tokens = __shfl(tokens, end + 1, 64);                               // of the block: those of this run
  const int was = __shfl(old, (own ? start : 0) + 1, 64);
  const int now = exponent_for(top);
  const int e = (tokens & 1) == 0 && was > now ? was : now;             // (token 0 begins the block anew)
  if (threadIdx.x < 64 && own && mine_row == start) scales[at_scale] = static_cast<uint8_t>(e + 127);
  uint8_t* cache = static_cast<uint8_t*>(value ? a.Vc : a.Kc);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = group + GROUPS * p;
    const int li = (i < 32 ? i : 31) + 1;                             // (all lanes take part in the shuffles)
    const int se = __shfl(e, li, 64), sw = __shfl(was, li, 64), ss = __shfl(slot, li, 64), st = __shfl(start, li, 64);
    const uint32_t tk = __shfl(tokens, li, 64);
    if (!(i < 32 && (rows >> i & 1) != 0)) continue;
    const float f = two_to(-se);
    const int64_t at = slot_base(a, ss, true) + (static_cast<int64_t>(kvh) << a.page_shift) * D + d0;
    float z[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool finite = (__float_as_uint(y[p][j]) & 0x7F800000u) != 0x7F800000u;
      z[j] = finite ? y[p][j] * f : __builtin_nanf("");
    }
    uint32_t w[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) w[j] = codes4(z + 4 * j);
    if constexpr (V == 8) *reinterpret_cast<u32x2*>(cache + at) = u32x2{w[0], w[1]};
    else *reinterpret_cast<uint32_t*>(cache + at) = w[0];
    if (i == st && (tk & 1) == 0 && se > sw) {                              // the block's other tokens, by 2^(old - new)
      const float g = two_to(sw - se < -30 ? -30 : sw - se);
      uint8_t* block = cache + at - static_cast<int64_t>(ss & 15) * D;
      uint32_t c[16][V / 4];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if ((tk >> k & 1) == 0) {
          if constexpr (V == 8) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(block + k * D);
            c[k][0] = x[0], c[k][1] = x[1];
          } else {
            c[k][0] = *reinterpret_cast<const uint32_t*>(block + k * D);
          }
        }
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if ((tk >> k & 1) == 0) {
          if constexpr (V == 8) *reinterpret_cast<u32x2*>(block + k * D) = u32x2{recode4(c[k][0], g), recode4(c[k][1], g)};
          else *reinterpret_cast<uint32_t*>(block + k * D) = recode4(c[k][0], g);
        }
    }
  }
}

// Workgroups for the windows' keys and values (of one window side by side),
// then, with QUERIES, sets of query heads as above. `first`: the first token
// of this launch, a multiple of 16.
template <typename T, int D, bool INTER, bool NORM, bool VEC>
__global__ __launch_bounds__(kThreads) void rope_append_f8_kernel(RopeArgs a, int first, int tokens, int sets) {
  const int windows = (tokens + 15) / 16;
  const int stores = windows * 2 * a.Hkv;
  const int b = blockIdx.x;
  if (b < stores) {
    const int h = b % (2 * a.Hkv);
    store_codes<T, D, INTER, NORM, VEC>(a, first / 16 + b / (2 * a.Hkv), h % a.Hkv, h >= a.Hkv);
  } else if constexpr (VEC) {
    const int x = b - stores;
    rope_heads<T, D, INTER, NORM, true, 1>(a, first + x / sets, x % sets, a.Hq);
  }
}

// A workgroup per set of heads, or per three sets where many tokens are normed:
// their weights are then loaded once for three heads a lane instead of one.
// (8192 tokens of 48 heads with norms, bf16: 42 us against 52; 2048 tokens
// 13.9 against 13.0, 8192 without norms 38.9 against 37.9, one token 3.3
// against 2.9.)
constexpr int kManyTokens = 4096;

template <typename T, int D, bool INTER, bool NORM, bool AXES>
void launch_vector(const RopeArgs& a, hipStream_t st) {
  constexpr int GROUPS = kThreads / (D / Elem<T>::kVec);
  const int sets = (a.Hq + 2 * a.Hkv + GROUPS - 1) / GROUPS;
  if constexpr (NORM) {
    if (a.M >= kManyTokens && sets > 1) {
      rope_append_kernel<T, D, INTER, NORM, AXES, 3><<<dim3(a.M, (sets + 2) / 3), kThreads, 0, st>>>(a);
      return;
    }
  }
  rope_append_kernel<T, D, INTER, NORM, AXES, 1><<<dim3(a.M, sets), kThreads, 0, st>>>(a);
}

// Whether rows and rot_dim suit the vector path.
template <typename T>
bool vector_path(const RopeArgs& a) {
  constexpr int V = Elem<T>::kVec;
  auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool whole = a.interleaved ? a.rot % V == 0 : a.rot % (2 * V) == 0;
  return whole && al16(a.QKV) && a.ld % V == 0 && (a.Hq == 0 || (al16(a.Q) && a.ldq % V == 0));
}

template <typename T, int D, bool AXES>
hipError_t launch_typed(const RopeArgs& a, hipStream_t st) {
  if (!vector_path<T>(a)) {
    const dim3 grid(a.M, a.Hq + 2 * a.Hkv);
    rope_append_scalar_kernel<T, D, AXES><<<grid, 64, 0, st>>>(a);
  } else {
    const bool norm = a.q_norm || a.k_norm;
    if (a.interleaved) norm ? launch_vector<T, D, true, true, AXES>(a, st) : launch_vector<T, D, true, false, AXES>(a, st);
    else norm ? launch_vector<T, D, false, true, AXES>(a, st) : launch_vector<T, D, false, false, AXES>(a, st);
  }
  return hipGetLastError();
}

template <typename T, bool AXES>
hipError_t launch_by_dim(const RopeArgs& a, hipStream_t st) {
  return a.D == 64 ? launch_typed<T, 64, AXES>(a, st) : launch_typed<T, 128, AXES>(a, st);
}

// Tokens [first, first + tokens) of a call onto a cache of codes.
template <typename T, int D, bool INTER, bool NORM>
hipError_t launch_f8(const RopeArgs& a, int first, int tokens, hipStream_t st) {
  constexpr int GROUPS = kThreads / (D / Elem<T>::kVec);
  const int sets = (a.Hq + GROUPS - 1) / GROUPS;
  const int64_t stores = static_cast<int64_t>((tokens + 15) / 16) * 2 * a.Hkv;
  if (vector_path<T>(a)) {
    rope_append_f8_kernel<T, D, INTER, NORM, true>
        <<<dim3(static_cast<unsigned>(stores + static_cast<int64_t>(tokens) * sets)), kThreads, 0, st>>>(a, first, tokens, sets);
  } else {
    rope_append_f8_kernel<T, D, INTER, NORM, false><<<dim3(static_cast<unsigned>(stores)), kThreads, 0, st>>>(a, first, tokens, 0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.Hq > 0) {                                        // (the keys first: Q may lie in QKV's query part alone)
      RopeArgs x = a;
      x.QKV = static_cast<const T*>(a.QKV) + first * a.ld;
      x.Q = static_cast<T*>(a.Q) + first * a.ldq;
      if (a.rot > 0) x.pos = a.pos + first;
      x.slot = a.slot + first;
      rope_append_scalar_kernel<T, D, true><<<dim3(tokens, a.Hq), 64, 0, st>>>(x);
    }
  }
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_f8_typed(const RopeArgs& a, int first, int tokens, hipStream_t st) {
  const bool norm = a.q_norm || a.k_norm;
  if (a.interleaved) return norm ? launch_f8<T, D, true, true>(a, first, tokens, st) : launch_f8<T, D, true, false>(a, first, tokens, st);
  return norm ? launch_f8<T, D, false, true>(a, first, tokens, st) : launch_f8<T, D, false, false>(a, first, tokens, st);
}

}  // namespace

// A launch takes fewer than 2^32 work items along x, 2^24 tokens of 256.
constexpr int kTokensOfLaunch = 1 << 23;

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
  if (a.k_scale) {
    // workgroups of 16 tokens: at most a set of heads each for 8 of them
    const int64_t sixteen = 2 * static_cast<int64_t>(a.Hkv) + 16 * ((static_cast<int64_t>(a.Hq) + 7) / 8);
    const int64_t most = ((int64_t{1} << 24) - 1) / sixteen * 16;
    for (int64_t t = 0; t < a.M; t += most) {
      const int first = static_cast<int>(t), tokens = static_cast<int>(a.M - t < most ? a.M - t : most);
      hipError_t e;
      if (a.bf16) e = a.D == 64 ? launch_f8_typed<__bf16, 64>(a, first, tokens, st) : launch_f8_typed<__bf16, 128>(a, first, tokens, st);
      else e = a.D == 64 ? launch_f8_typed<float, 64>(a, first, tokens, st) : launch_f8_typed<float, 128>(a, first, tokens, st);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int64_t bytes = a.bf16 ? 2 : 4;
  for (int64_t t = 0; t < a.M; t += kTokensOfLaunch) {
    RopeArgs x = a;
    x.M = static_cast<int>(a.M - t < kTokensOfLaunch ? a.M - t : kTokensOfLaunch);
    x.QKV = static_cast<const char*>(a.QKV) + t * a.ld * bytes;
    if (a.Hq > 0) x.Q = static_cast<char*>(a.Q) + t * a.ldq * bytes;
    if (a.rot > 0) x.pos = a.pos + t;
    x.slot = a.slot + t;
    hipError_t e;
    if (a.n_axes > 1) e = a.bf16 ? launch_by_dim<__bf16, true>(x, st) : launch_by_dim<float, true>(x, st);
    else e = a.bf16 ? launch_by_dim<__bf16, false>(x, st) : launch_by_dim<float, false>(x, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace serq
