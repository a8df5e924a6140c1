// Rotary positions, head norms and the paged cache write in one pass (gfx950).
//
// From row t of the q/k/v linear's output, head by head:
//     y = x * w / sqrt(mean(x^2) + eps),  (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s),
// queries to Q, keys and the unchanged values to slot[t] of the cache. Every
// value is read once and written once, so the kernel is bound by HBM for
// prompts (8192 tokens of 48 heads of 128 with norms, bf16, 206 MB: 46 us from
// HBM, 4.5 TB/s; 35 us with the inputs in the last-level cache) and by latency
// for single tokens (one token 2.4 us, about a launch).

#include <type_traits>
#include <utility>

#include "serq_attn.h"

namespace serq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

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
// bit of a key would decide. What that costs shows beside the values, which are
// coded as they are: 8192 tokens of 8 normed heads of 128 take 19 us for the keys,
// 10 for the values, each alone (24 in one launch; 28 for 32 heads of queries, at 4.8
// TB/s).

// Least exponent >= kLeast with |y| <= 448 * 2^e for the finite fp32 number of bits `top`.
constexpr int kLeast = -117, kMost = 120;
__device__ __forceinline__ int exponent_for(uint32_t top) {
  const int e = static_cast<int>(top >> 23) - 135 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);    // 448 = 1.75 * 2^8
  return e < kLeast ? kLeast : e;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// 1 / sqrt(x) for positive x, by two Newton steps from the instruction's 2^-26 or
// so (2048 tokens of 32 and 8 normed heads 21.4 us, with a square root and a
// division 23.9).
__device__ __forceinline__ double inverse_root64(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double e = __builtin_fma(-x * y, y, 1.0);
    y = __builtin_fma(0.5 * e, y, y);
  }
  return x > 0.0 && x < static_cast<double>(__builtin_inff()) ? y : __builtin_amdgcn_rsq(x);
}

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

// Sum, and maximum, over the aligned groups of L lanes.
template <int L, typename X, typename F>
__device__ __forceinline__ X over_lanes(X v, F&& f) {
  static_assert(L == 8 || L == 16 || L == 32, "lanes of a head");
  const auto moved = [](X x, auto ctrl) {
    constexpr int C = decltype(ctrl)::value;
    constexpr int N = sizeof(X) / 4;
    struct Words { int w[N]; } a = __builtin_bit_cast(Words, x);
#pragma unroll
    for (int i = 0; i < N; ++i) a.w[i] = __builtin_amdgcn_update_dpp(0, a.w[i], C, 0xf, 0xf, true);
    return __builtin_bit_cast(X, a);
  };
  v = f(v, moved(v, std::integral_constant<int, 0xB1>{}));          // lane ^ 1, lane ^ 2
  v = f(v, moved(v, std::integral_constant<int, 0x4E>{}));
  v = f(v, moved(v, std::integral_constant<int, 0x141>{}));         // the other four of eight, the other eight of sixteen
  if constexpr (L >= 16) v = f(v, moved(v, std::integral_constant<int, 0x140>{}));
  if constexpr (L == 32) v = f(v, __shfl_xor(v, 16, 32));
  return v;
}

// One window of 16 rows, HB * SUB key/value heads from h0 on, keys or values: the
// runs that begin in the window, whose rows are among 31. A pass is RP rows of
// L lanes each, for SUB heads side by side; what depends on the row alone
// serves its HB heads. Which rows go together is found by each wave from the
// slots (lane i + 1: row i); the rows' maxima and slots meet in LDS, where the
// lanes of a row read those of its run. Few runs reach past their window:
// their later rows are computed twice, for the maximum and to be stored,
// instead of kept.
// VEC: as for the vector path above; otherwise every value and its partner are
// loaded one by one.
template <typename T, int D, bool INTER, bool NORM, bool VEC, int HB, bool value>
__device__ __forceinline__ void store_codes(const RopeArgs& a, int window, int h0) {
  using E = Elem<T>;
  constexpr int V = E::kVec, L = D / V, RP = kThreads / L < 16 ? kThreads / L : 16, SUB = kThreads / (L * RP), EARLY = 16 / RP;
  // bf16 values stay as they are: their codes come from pairs of bf16
  constexpr bool kPairs = value && VEC && V == 8;
  __shared__ uint32_t tops[HB * SUB][32];
  __shared__ int slots[32];
  const int wl = threadIdx.x & 63;
  const int lane = threadIdx.x % L, group = threadIdx.x / L % RP, sub = threadIdx.x / (L * RP), d0 = lane * V;
  const int row0 = 16 * window;
  const bool norm = NORM && !value && a.k_norm;
  const bool turned = !value && d0 < a.rot;
  const int half = a.rot / 2;
  const auto partner = [&](int d) { return d >= a.rot ? d : INTER ? d ^ 1 : d < half ? d + half : d - half; };

  // y = r (x (w A) + z (w' B)), z and w' the partner's: w A and w' B are exact.
  struct Factors { double wa[V], wb[V]; };
  const auto load_row = [&](int t, bool in, Factors& f) __attribute__((always_inline)) {
    float A[V], B[V], wx[V], wz[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = wx[j] = wz[j] = 1.0f, B[j] = 0.0f;
    if (in && turned) {
      const Place at = place_of<true>(a, t);
      if (at.ok) {
        if constexpr (VEC) {
          load_factors<V, INTER, true>(a, at, d0, A, B);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int d = d0 + j;
            if (d < a.rot) {
              const bool second = INTER ? (d & 1) : d >= half;
              const int pair = INTER ? d / 2 : second ? d - half : d;
              const float* row = row_of<true>(a, at, pair);
              A[j] = row[pair];
              B[j] = second ? row[half + pair] : -row[half + pair];
            }
          }
        }
      }
    }
    if (norm) {
      load_floats<V>(a.k_norm + d0, wx);
      if constexpr (VEC) {
        if constexpr (INTER) {
#pragma unroll
          for (int j = 0; j < V; ++j) wz[j] = wx[j ^ 1];
        } else {
          load_floats<V>(a.k_norm + partner(d0), wz);
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) wz[j] = a.k_norm[partner(d0 + j)];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f.wa[j] = static_cast<double>(wx[j]) * A[j];
      f.wb[j] = static_cast<double>(wz[j]) * B[j];
    }
  };
  struct Raw {
    u32x4 w;                    // kPairs
    float y[V], z[V];
  };
  const auto load_raw = [&](int t, int h, bool in, Raw& r) __attribute__((always_inline)) {
    r.w = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < V; ++j) r.y[j] = r.z[j] = 0.0f;
    if (!in) return;
    const T* src = static_cast<const T*>(a.QKV) + t * a.ld + static_cast<int64_t>(a.Hq + (value ? a.Hkv : 0) + h) * D;
    if constexpr (kPairs) {
      r.w = *reinterpret_cast<const u32x4*>(src + d0);
    } else if constexpr (VEC) {
      E::unpack(*reinterpret_cast<const u32x4*>(src + d0), r.y);
      if (!INTER && turned) E::unpack(*reinterpret_cast<const u32x4*>(src + partner(d0)), r.z);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        r.y[j] = E::load(src + d0 + j);
        if (turned) r.z[j] = E::load(src + partner(d0 + j));
      }
    }
  };
  // The keys themselves in r.y (all lanes take part).
  const auto finish = [&](Raw& r, const Factors& f) __attribute__((always_inline)) {
    if constexpr (!value) {
      double x[V], s = 1.0;
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = r.y[j];
      if constexpr (NORM) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) ss = __builtin_fma(x[j], x[j], ss);
        ss = over_lanes<L>(ss, [](double u, double v) { return u + v; });
        if (norm) s = inverse_root64(ss * (1.0 / D) + static_cast<double>(a.eps));
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        double u = x[j] * f.wa[j];
        if (VEC ? turned : d0 + j < a.rot) u = __builtin_fma(INTER && VEC ? x[j ^ 1] : static_cast<double>(r.z[j]), f.wb[j], u);
        r.y[j] = static_cast<float>(NORM ? u * s : u);
      }
    }
  };
  // Largest finite magnitude of a row, as the bits of an fp32 number. (NaN and
  // infinities, which become NaN codes, make the lane look at each value.)
  const auto top_of = [&](const Raw& r) __attribute__((always_inline)) {
    uint32_t top = 0;
    if constexpr (kPairs) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      const auto mag = [&](int j) { return __builtin_bit_cast(u16x2, r.w[j] & 0x7FFF7FFFu); };
      const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(0), mag(1)), __builtin_elementwise_max(mag(2), mag(3)));
      top = static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
      if (top >= 0x7F800000u) {
        top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b = (r.w[j / 2] >> (16 * (j & 1)) & 0x7FFFu) << 16;
          top = b < 0x7F800000u && b > top ? b : top;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t b = __float_as_uint(r.y[j]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
      }
      if (top >= 0x7F800000u) {
        top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const uint32_t b = __float_as_uint(r.y[j]) & 0x7FFFFFFFu;
          top = b < 0x7F800000u && b > top ? b : top;
        }
      }
    }
    return over_lanes<L>(top, [](uint32_t u, uint32_t v) { return u > v ? u : v; });
  };
  const auto head = [&](int k) { return h0 + k * SUB + sub; };

  // The window's own rows are loaded before it is known which of them are stored.
  Raw raw[EARLY][HB];
  Factors fac[EARLY];
#pragma unroll
  for (int p = 0; p < EARLY; ++p) {
    const int t = row0 + group + RP * p;
#pragma unroll
    for (int k = 0; k < HB; ++k) load_raw(t, head(k), t < a.M && head(k) < a.Hkv, raw[p][k]);
    if constexpr (!value) load_row(t, t < a.M, fac[p]);
  }
  // the rows' slots and runs
  int slot = -1;
  if (wl <= 32 && row0 + wl - 1 >= 0 && row0 + wl - 1 < a.M) {
    const int s = a.slot[row0 + wl - 1];
    const bool ok = place_of<true>(a, row0 + wl - 1).ok;
    slot = ok && s >= 0 && (s >> a.page_shift) < a.n_pages ? s : -1;
  }
  const int before = __shfl_up(slot, 1, 64);
  const bool next = wl > 0 && wl <= 32 && slot >= 0 && before >= 0 && slot >> 4 == before >> 4;
  const uint64_t joined = __ballot(next) >> 1;                        // bit i: row i continues row i - 1
  const uint32_t starts = static_cast<uint32_t>(__ballot(slot >= 0 && !next) >> 1);
  // the run that row i is of: its first and last row
  const auto start_of = [&](int i) {
    const uint32_t upto = starts & ((2u << i) - 1u);
    return upto ? 31 - __builtin_clz(upto) : 16;
  };
  const auto end_of = [&](int i) { return i + __builtin_ctzll(~(joined >> (i + 1))); };
  const uint32_t rows = static_cast<uint32_t>(__ballot(wl > 0 && slot >= 0 && start_of((wl - 1) & 31) < 16) >> 1);
  if (rows == 0) return;
  if (threadIdx.x - 1u < 32u) slots[threadIdx.x - 1] = slot;
  const int past = rows >> 16 ? 32 - __builtin_clz(rows) : 16;         // rows past the window to look at: 16 .. past - 1
#pragma unroll
  for (int p = 0; p < EARLY; ++p)
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int i = group + RP * p;
      finish(raw[p][k], fac[p]);
      const uint32_t top = top_of(raw[p][k]);
      if (lane == 0) tops[k * SUB + sub][i] = (rows >> i & 1) ? top : 0;
    }
  const auto later = [&](auto&& use) __attribute__((always_inline)) {  // use(row, head's number, values)
#pragma unroll 1
    for (int i0 = 16; i0 < past; i0 += RP) {
      const int i = i0 + group;
      const bool in = (rows >> i & 1) != 0;
      Factors f;
      if constexpr (!value) load_row(row0 + i, in, f);
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        Raw r;
        load_raw(row0 + i, head(k), in && head(k) < a.Hkv, r);
        finish(r, f);
        use(i, k, r);
      }
    }
  };
  later([&](int i, int k, const Raw& r) __attribute__((always_inline)) {
    const uint32_t top = top_of(r);
    if (lane == 0) tops[k * SUB + sub][i] = (rows >> i & 1) ? top : 0;
  });
  __syncthreads();

  uint8_t* const scales = value ? a.v_scale : a.k_scale;
  uint8_t* const cache = static_cast<uint8_t*>(value ? a.Vc : a.Kc);
  const int per = a.page_shift - 4;                                    // blocks of a page: 1 << per
  constexpr auto most = [](uint32_t u, uint32_t v) { return u > v ? u : v; };
  // Row i's codes of head k; the run's first row writes the scale and takes care
  // of the block's other codes. (All lanes take part.)
  const auto store = [&](int i, int k, const Raw& r) __attribute__((always_inline)) {
    const bool mine = (rows >> i & 1) != 0;
    const int start = mine ? start_of(i) : i, end = mine ? end_of(i) : i;
    // the run's tokens (a bit each) and maximum: a row of it a lane
    uint32_t tokens = 0, top = 0;
#pragma unroll
    for (int n = 0; n < 16; n += (L < 16 ? L : 16)) {
      const int j = start + (lane & 15) + n;
      if (j <= end) {
        tokens |= 1u << (slots[j] & 15);
        top = most(top, tops[k * SUB + sub][j]);
      }
    }
    tokens = over_lanes<L>(tokens, [](uint32_t u, uint32_t v) { return u | v; });
    top = over_lanes<L>(top, most);
    if (!mine || head(k) >= a.Hkv) return;
    const int s = slots[i];
    const int64_t block = ((static_cast<int64_t>(s >> a.page_shift) * a.Hkv + head(k)) << per) + ((s >> 4) & ((1 << per) - 1));
    int e = exponent_for(top), was = kLeast;
    if ((tokens & 1) == 0) {                                          // (token 0 begins the block anew)
      was = static_cast<int>(scales[block]) - 127;
      was = was < kLeast ? kLeast : was > kMost ? kMost : was;
      e = e > was ? e : was;
    }
    uint8_t* const to = cache + block * (16 * D) + d0;                // the lane's codes of the block's tokens, D apart
    uint32_t w[V / 4];
    if constexpr (kPairs) {
      typedef short s16x2 __attribute__((ext_vector_type(2)));
      u32x4 x = r.w;
      if (__any((x[0] & 0x7F80u) == 0x7F80u || (x[0] & 0x7F800000u) == 0x7F800000u || (x[1] & 0x7F80u) == 0x7F80u ||
                (x[1] & 0x7F800000u) == 0x7F800000u || (x[2] & 0x7F80u) == 0x7F80u || (x[2] & 0x7F800000u) == 0x7F800000u ||
                (x[3] & 0x7F80u) == 0x7F80u || (x[3] & 0x7F800000u) == 0x7F800000u)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {                                 // infinities to NaN
          if ((x[j] & 0x7F80u) == 0x7F80u) x[j] |= 0x7FFFu;
          if ((x[j] & 0x7F800000u) == 0x7F800000u) x[j] |= 0x7FFF0000u;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t x0 = x[2 * j], x1 = x[2 * j + 1];
        const s16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(s16x2{0, 0}, __builtin_bit_cast(bf16x2, x0), two_to(e), false);
        w[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2, x1), two_to(e), true));
      }
    } else {
      const float f = two_to(-e);
      float z[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool finite = (__float_as_uint(r.y[j]) & 0x7F800000u) != 0x7F800000u;
        z[j] = finite ? r.y[j] * f : __builtin_nanf("");
      }
#pragma unroll
      for (int j = 0; j < V / 4; ++j) w[j] = codes4(z + 4 * j);
    }
    if constexpr (V == 8) *reinterpret_cast<u32x2*>(to + (s & 15) * D) = u32x2{w[0], w[1]};
    else *reinterpret_cast<uint32_t*>(to + (s & 15) * D) = w[0];
    if (i != start) return;
    if (lane == 0) scales[block] = static_cast<uint8_t>(e + 127);
    if ((tokens & 1) == 0 && e > was) {                               // by 2^(old - new)
      const float g = two_to(was - e < -30 ? -30 : was - e);
      uint32_t c[16][V / 4];
#pragma unroll
      for (int n = 0; n < 16; ++n)
        if ((tokens >> n & 1) == 0) {
          if constexpr (V == 8) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(to + n * D);
            c[n][0] = v[0], c[n][1] = v[1];
          } else {
            c[n][0] = *reinterpret_cast<const uint32_t*>(to + n * D);
          }
        }
#pragma unroll
      for (int n = 0; n < 16; ++n)
        if ((tokens >> n & 1) == 0) {
          if constexpr (V == 8) *reinterpret_cast<u32x2*>(to + n * D) = u32x2{recode4(c[n][0], g), recode4(c[n][1], g)};
          else *reinterpret_cast<uint32_t*>(to + n * D) = recode4(c[n][0], g);
        }
    }
  };
#pragma unroll
  for (int p = 0; p < EARLY; ++p)
#pragma unroll
    for (int k = 0; k < HB; ++k) store(group + RP * p, k, raw[p][k]);
  later(store);
}

// Workgroups for the windows' keys and values (of one window side by side),
// then, with sets, sets of query heads as above. `first`: the first token of
// this launch, a multiple of 16.
template <typename T, int D>
constexpr int heads_side_by_side() {
  return kThreads / (D / Elem<T>::kVec) <= 16 ? 1 : kThreads / (D / Elem<T>::kVec) / 16;
}
template <typename T, int D, bool INTER, bool NORM, bool VEC>
__global__ __launch_bounds__(kThreads) void rope_append_f8_kernel(RopeArgs a, int first, int tokens, int sets) {
  constexpr int HB = 1, EACH = heads_side_by_side<T, D>();
  const int windows = (tokens + 15) / 16, parts = (a.Hkv + EACH - 1) / EACH;
  const int stores = windows * 2 * parts;
  const int b = blockIdx.x;
  if (b < stores) {
    const int h = b % (2 * parts);
    const int window = first / 16 + b / (2 * parts), h0 = h % parts * EACH;
    if (h >= parts) store_codes<T, D, false, false, VEC, HB, true>(a, window, h0);
    else store_codes<T, D, INTER, NORM, VEC, HB, false>(a, window, h0);
  } else if constexpr (VEC) {
    const int x = b - stores;
    rope_heads<T, D, INTER, NORM, true, 1>(a, first + x / sets, x % sets, a.Hq);
  }
}

// Keys and values without the queries: `keys` workgroups of KB heads' keys, then
// those of VB heads' values.
template <typename T, int D, bool INTER, bool NORM, int KB, int VB>
__global__ __launch_bounds__(kThreads) void store_f8_kernel(RopeArgs a, int first, int keys) {
  constexpr int EACH = heads_side_by_side<T, D>();
  const int b = blockIdx.x;
  if (b < keys) {
    const int parts = (a.Hkv + KB * EACH - 1) / (KB * EACH);
    store_codes<T, D, INTER, NORM, true, KB, false>(a, first / 16 + b / parts, b % parts * (KB * EACH));
  } else {
    const int parts = (a.Hkv + VB * EACH - 1) / (VB * EACH), x = b - keys;
    store_codes<T, D, false, false, true, VB, true>(a, first / 16 + x / parts, x % parts * (VB * EACH));
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

// From so many tokens times heads (of all three kinds) on, keys and values of a
// call onto a cache of codes take a launch and the queries another, each with its
// own registers and heads of a workgroup. One launch against two, bf16, 2048 normed
// tokens unless said otherwise: 32 and 8 heads of 128, 1024 tokens 11.5 us and 11.3,
// 1536 16.5 and 14.7, 2048 21.3 and 17.4, 8192 75 and 48 (fp32, 1536 24.2 and 22.1);
// 64 and 8 heads 30.4 and 23.3, 512 tokens 9.2 and 11.1; 32 and 32 39.0 and 30.8; 8
// and 1 7.4 and 9.7, 8192 tokens 24.6 and 19.8 (fp32 7.2 and 11.5, 25.1 and 24.2);
// heads of 64, 32 and 8, 1024 tokens 7.3 and 9.1, 1536 10.0 and 10.1; 16 and 16 15.8
// and 11.2; 8 and 8 without norms 8.9 and 8.4, 3000 tokens 12.1 and 9.9. The two
// change places between 43 and 82 thousand. (Keys and values in a launch each: 8192
// tokens of 32 and 8 heads 52; all in one with these heads of a workgroup 51.)
constexpr int64_t kManyStored = 1 << 16;

// Tokens [first, first + tokens) of a call onto a cache of codes. Where they are
// many, a workgroup takes two heads of keys (alone 8192 tokens 18.4 us, one head
// 22.3, four 21.1) or four of values (9.7, two alike, one 11.2), which load what
// depends on the token once.
template <typename T, int D, bool INTER, bool NORM>
hipError_t launch_f8(const RopeArgs& a, int first, int tokens, hipStream_t st) {
  constexpr int GROUPS = kThreads / (D / Elem<T>::kVec), KB = 2, VB = 4;
  const int sets = (a.Hq + GROUPS - 1) / GROUPS;
  const auto stores = [&](int heads) {                     // workgroups of so many heads each
    const int64_t each = heads * heads_side_by_side<T, D>();
    return static_cast<int64_t>((tokens + 15) / 16) * ((a.Hkv + each - 1) / each);
  };
  const auto queries = [&] {                               // of these tokens alone
    RopeArgs x = a;
    x.QKV = static_cast<const T*>(a.QKV) + first * a.ld;
    x.Q = static_cast<T*>(a.Q) + first * a.ldq;
    if (a.rot > 0) x.pos = a.pos + first;
    x.slot = a.slot + first;
    x.M = tokens;
    x.Hkv = 0;
    return x;
  };
  const bool vector = vector_path<T>(a), many = static_cast<int64_t>(tokens) * (a.Hq + 2 * a.Hkv) >= kManyStored;
  if (vector && !many) {
    rope_append_f8_kernel<T, D, INTER, NORM, true>
        <<<dim3(static_cast<unsigned>(2 * stores(1) + static_cast<int64_t>(tokens) * sets)), kThreads, 0, st>>>(a, first, tokens, sets);
    return hipGetLastError();
  }
  if (vector) {
    const int keys = static_cast<int>(stores(KB));
    store_f8_kernel<T, D, INTER, NORM, KB, VB>
        <<<dim3(static_cast<unsigned>(keys + stores(VB))), kThreads, 0, st>>>(a, first, keys);
  } else {
    rope_append_f8_kernel<T, D, INTER, NORM, false><<<dim3(static_cast<unsigned>(2 * stores(1))), kThreads, 0, st>>>(a, first, tokens, 0);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.Hq == 0) return e;
  const RopeArgs x = queries();                            // (the keys first: Q may lie in QKV's query part alone)
  if (!vector) rope_append_scalar_kernel<T, D, true><<<dim3(tokens, a.Hq), 64, 0, st>>>(x);
  else if (a.n_axes > 1) launch_vector<T, D, INTER, NORM, true>(x, st);
  else launch_vector<T, D, INTER, NORM, false>(x, st);
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
