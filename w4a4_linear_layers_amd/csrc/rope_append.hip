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

// Vector path: 16-byte aligned rows, rot_dim made of whole chunks in each
// half (SERQ_ROPE_HALF) or in all (SERQ_ROPE_INTERLEAVED). A head is D / kVec
// lanes of one chunk each; a workgroup holds 256 / lanes heads of one token
// at a time and NB such sets, all of whose loads it starts before the first
// use, since the cosines and sines come only after the position they belong
// to. What depends on the lane's place in the head alone (cosines, sines, norm
// weights) is loaded once for all its heads; the other half's values come from
// the lane that holds them.
template <typename T, int D, bool INTER, bool NORM, int NB>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeArgs a) {
  using E = Elem<T>;
  constexpr int V = E::kVec, L = D / V, GROUPS = kThreads / L;
  const int t = blockIdx.x;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int d0 = lane * V;
  const int heads = a.Hq + 2 * a.Hkv;
  const int first = blockIdx.y * (GROUPS * NB) + group;
  const T* in = static_cast<const T*>(a.QKV) + t * a.ld + d0;
  u32x4 raw[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int h = first + GROUPS * k;
    if (h < heads) raw[k] = *reinterpret_cast<const u32x4*>(in + static_cast<int64_t>(h) * D);
  }
  const int slot = a.slot[t];
  const int pos = a.rot ? a.pos[t] : 0;
  const bool pos_ok = !a.rot || (pos >= 0 && pos < a.max_pos);
  const bool turned = d0 < a.rot;
  const int half = a.rot / 2;
  // y = x A + partner B with A = c, B = -s in the first half of a pair and s in the second
  float A[V], B[V], wq[V], wk[V];
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = 1.0f, B[i] = 0.0f;
  if (turned && pos_ok) {
    const float* row = a.table + static_cast<int64_t>(pos) * a.rot;
    if constexpr (INTER) {
      float c[V / 2], s[V / 2];
      load_floats<V / 2>(row + d0 / 2, c);
      load_floats<V / 2>(row + half + d0 / 2, s);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        A[i] = c[i / 2];
        B[i] = i & 1 ? s[i / 2] : -s[i / 2];
      }
    } else {
      const bool second = d0 >= half;
      const int i0 = second ? d0 - half : d0;
      load_floats<V>(row + i0, A);
      load_floats<V>(row + half + i0, B);
#pragma unroll
      for (int i = 0; i < V; ++i) B[i] = second ? B[i] : -B[i];
    }
  }
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

// Scalar path, any row alignment and rot_dim: one wave per head, values
// d = lane + 64 e; partners are exchanged between lanes, so every value is
// read before any is written (Q may be QKV).
template <typename T, int D>
__global__ __launch_bounds__(64) void rope_append_scalar_kernel(RopeArgs a) {
  using E = Elem<T>;
  constexpr int N = D / 64;
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  const int pos = a.rot ? a.pos[t] : 0;
  const bool pos_ok = !a.rot || (pos >= 0 && pos < a.max_pos);
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
        const float* row = a.table + static_cast<int64_t>(pos) * a.rot;
        const bool second = a.interleaved ? (d & 1) : d >= half;
        const int i = a.interleaved ? d / 2 : second ? d - half : d;
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

// A workgroup per set of heads, or per three sets where many tokens are normed:
// their weights are then loaded once for three heads a lane instead of one.
// (8192 tokens of 48 heads with norms, bf16: 42 us against 52; 2048 tokens
// 13.9 against 13.0, 8192 without norms 38.9 against 37.9, one token 3.3
// against 2.9.)
constexpr int kManyTokens = 4096;

template <typename T, int D, bool INTER, bool NORM>
void launch_vector(const RopeArgs& a, hipStream_t st) {
  constexpr int GROUPS = kThreads / (D / Elem<T>::kVec);
  const int sets = (a.Hq + 2 * a.Hkv + GROUPS - 1) / GROUPS;
  if constexpr (NORM) {
    if (a.M >= kManyTokens && sets > 1) {
      rope_append_kernel<T, D, INTER, NORM, 3><<<dim3(a.M, (sets + 2) / 3), kThreads, 0, st>>>(a);
      return;
    }
  }
  rope_append_kernel<T, D, INTER, NORM, 1><<<dim3(a.M, sets), kThreads, 0, st>>>(a);
}

template <typename T, int D>
hipError_t launch_typed(const RopeArgs& a, hipStream_t st) {
  constexpr int V = Elem<T>::kVec;
  auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool whole = a.interleaved ? a.rot % V == 0 : a.rot % (2 * V) == 0;
  const bool vec = whole && al16(a.QKV) && a.ld % V == 0 && (a.Hq == 0 || (al16(a.Q) && a.ldq % V == 0));
  if (!vec) {
    const dim3 grid(a.M, a.Hq + 2 * a.Hkv);
    rope_append_scalar_kernel<T, D><<<grid, 64, 0, st>>>(a);
  } else {
    const bool norm = a.q_norm || a.k_norm;
    if (a.interleaved) norm ? launch_vector<T, D, true, true>(a, st) : launch_vector<T, D, true, false>(a, st);
    else norm ? launch_vector<T, D, false, true>(a, st) : launch_vector<T, D, false, false>(a, st);
  }
  return hipGetLastError();
}

}  // namespace

// A launch takes fewer than 2^32 work items along x, 2^24 tokens of 256.
constexpr int kTokensOfLaunch = 1 << 23;

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
  const int64_t bytes = a.bf16 ? 2 : 4;
  for (int64_t t = 0; t < a.M; t += kTokensOfLaunch) {
    RopeArgs x = a;
    x.M = static_cast<int>(a.M - t < kTokensOfLaunch ? a.M - t : kTokensOfLaunch);
    x.QKV = static_cast<const char*>(a.QKV) + t * a.ld * bytes;
    if (a.Hq > 0) x.Q = static_cast<char*>(a.Q) + t * a.ldq * bytes;
    if (a.rot > 0) x.pos = a.pos + t;
    x.slot = a.slot + t;
    hipError_t e;
    if (a.bf16) e = a.D == 64 ? launch_typed<__bf16, 64>(x, st) : launch_typed<__bf16, 128>(x, st);
    else e = a.D == 64 ? launch_typed<float, 64>(x, st) : launch_typed<float, 128>(x, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace serq
