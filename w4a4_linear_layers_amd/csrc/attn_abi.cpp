// C ABI entry points of the attention half: host-side argument validation and
// dispatch of serq_rope_append, serq_attn_prefill and serq_attn_decode onto
// the caller's HIP stream. serq_rope_table (host) lives in rope_table.cpp.

#include <hip/hip_runtime.h>

#include <cmath>

#include "serq.h"
#include "serq_attn.h"

namespace {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// log2 of a page size the calls take, or -1.
inline int page_shift(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

constexpr int kMaxHeads = 16384;

inline bool valid_heads(int Hq, int Hkv) {
  return Hkv > 0 && Hq > 0 && Hq <= kMaxHeads && Hkv <= kMaxHeads && Hq % Hkv == 0;
}

inline bool valid_dtype(serq_dtype t) { return t == SERQ_F32 || t == SERQ_BF16; }

// Bounds of one call: rows * heads and keys of a sequence.
inline bool valid_rows(int64_t rows, int Hq) { return rows * Hq <= (int64_t{1} << 30); }
constexpr int kMaxKeys = 1 << 30;

}  // namespace

extern "C" int serq_rope_append(const void* QKV, serq_dtype dtype, int64_t ld, int M, int Hq, int Hkv, int D,
                                const float* q_norm, const float* k_norm, float eps, const float* table, int rot_dim,
                                int max_pos, serq_rope_layout layout, const int32_t* pos, const int32_t* slot, void* Q,
                                int64_t ldq, void* Kc, void* Vc, int n_pages, int page_size, void* stream) {
  if (!valid_dtype(dtype) || (layout != SERQ_ROPE_HALF && layout != SERQ_ROPE_INTERLEAVED)) return SERQ_EINVAL;
  if (M < 0 || Hq < 0 || Hkv <= 0 || Hq > kMaxHeads || Hkv > kMaxHeads || D <= 0 || page_size <= 0 || n_pages <= 0)
    return SERQ_EINVAL;
  if ((Hq % Hkv) != 0) return SERQ_EINVAL;
  if (D != 64 && D != 128) return SERQ_EUNSUPPORTED;
  const int shift = page_shift(page_size);
  if (shift < 0) return SERQ_EUNSUPPORTED;
  if (static_cast<int64_t>(n_pages) << shift > INT32_MAX) return SERQ_EINVAL;      // slots are int32
  if (ld < static_cast<int64_t>(Hq + 2 * Hkv) * D || (Hq > 0 && ldq < static_cast<int64_t>(Hq) * D))
    return SERQ_EINVAL;
  if (rot_dim < 0 || rot_dim > D || (rot_dim % 2) != 0) return SERQ_EINVAL;
  if (rot_dim > 0 && (!table || max_pos <= 0)) return SERQ_EINVAL;
  if ((q_norm || k_norm) && !(std::isfinite(eps) && eps >= 0.0f)) return SERQ_EINVAL;
  if (!Kc || !Vc) return SERQ_EINVAL;
  if (!aligned(Kc, 16) || !aligned(Vc, 16) || !aligned(table, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16))
    return SERQ_EALIGN;
  if (M == 0) return SERQ_OK;
  if (!QKV || !slot || (rot_dim > 0 && !pos) || (Hq > 0 && !Q)) return SERQ_EINVAL;
  const uintptr_t eb = dtype == SERQ_BF16 ? 2 : 4;
  if (!aligned(QKV, eb) || (Hq > 0 && !aligned(Q, eb)) || !aligned(pos, 4) || !aligned(slot, 4)) return SERQ_EALIGN;
  serq::RopeArgs a{};
  a.QKV = QKV;
  a.ld = ld;
  a.M = M;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.eps = eps;
  a.table = table;
  a.rot = rot_dim;
  a.max_pos = max_pos;
  a.interleaved = layout == SERQ_ROPE_INTERLEAVED;
  a.pos = pos;
  a.slot = slot;
  a.Q = Q;
  a.ldq = ldq;
  a.Kc = Kc;
  a.Vc = Vc;
  a.n_pages = n_pages;
  a.page_shift = shift;
  a.bf16 = dtype == SERQ_BF16;
  return serq::launch_rope_append(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SERQ_OK : SERQ_EHIP;
}

namespace {

// What the two attention calls check alike. `rows`: T or B.
int check_attention(const void* Q, serq_dtype dtype, int64_t ldq, int rows, int Hq, int Hkv, int D, const void* Kc,
                    const void* Vc, int n_pages, int page_size, int max_pages, int max_len, float scale, const void* O,
                    int64_t ldo) {
  if (!valid_dtype(dtype) || !valid_heads(Hq, Hkv) || D <= 0 || page_size <= 0 || n_pages <= 0) return SERQ_EINVAL;
  if (max_pages < 0 || max_len < 0 || max_len > kMaxKeys || !std::isfinite(scale)) return SERQ_EINVAL;
  if (D != 64 && D != 128) return SERQ_EUNSUPPORTED;
  if (page_shift(page_size) < 0) return SERQ_EUNSUPPORTED;
  if (ldq < static_cast<int64_t>(Hq) * D || ldo < static_cast<int64_t>(Hq) * D || !valid_rows(rows, Hq))
    return SERQ_EINVAL;
  if (!Kc || !Vc) return SERQ_EINVAL;
  const int eb = dtype == SERQ_BF16 ? 2 : 4;
  if (!aligned(Kc, 16) || !aligned(Vc, 16) || (ldq * eb) % 16 != 0 || (ldo * eb) % 16 != 0 || !aligned(Q, 16) ||
      !aligned(O, 16))
    return SERQ_EALIGN;
  return SERQ_OK;
}

serq::AttnArgs attention_args(const void* Q, serq_dtype dtype, int64_t ldq, int B, int Hq, int Hkv, int D,
                              const void* Kc, const void* Vc, int n_pages, int page_size, const int32_t* page_table,
                              int max_pages, const int32_t* kv_len, int max_len, float scale, void* O, int64_t ldo,
                              void* workspace) {
  serq::AttnArgs a{};
  a.Q = Q;
  a.ldq = ldq;
  a.Kc = Kc;
  a.Vc = Vc;
  a.n_pages = n_pages;
  a.page_shift = page_shift(page_size);
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.kv_len = kv_len;
  const int64_t room = static_cast<int64_t>(max_pages) << a.page_shift;
  a.max_len = max_len < room ? max_len : static_cast<int>(room);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.O = O;
  a.ldo = ldo;
  a.workspace = workspace;
  a.bf16 = dtype == SERQ_BF16;
  return a;
}

}  // namespace

extern "C" int64_t serq_attn_prefill_workspace(serq_dtype dtype, int B, int T, int Hq, int Hkv, int D, int max_len) {
  if (!valid_dtype(dtype) || B < 0 || T < 0 || !valid_heads(Hq, Hkv) || (D != 64 && D != 128) || max_len < 0 ||
      max_len > kMaxKeys || !valid_rows(T, Hq) || !valid_rows(B, Hq))
    return -1;
  return B == 0 || T == 0 ? 0 : serq::plan_prefill(dtype == SERQ_BF16, B, T, Hq, Hkv, D, max_len).bytes;
}

extern "C" int serq_attn_prefill(const void* Q, serq_dtype dtype, int64_t ldq, const int32_t* cu_q, int B, int T,
                                 int Hq, int Hkv, int D, const void* Kc, const void* Vc, int n_pages, int page_size,
                                 const int32_t* page_table, int max_pages, const int32_t* kv_len, int max_len,
                                 float scale, void* O, int64_t ldo, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
  if (B < 0 || T < 0 || !valid_rows(B, Hq)) return SERQ_EINVAL;
  const int bad = check_attention(Q, dtype, ldq, T, Hq, Hkv, D, Kc, Vc, n_pages, page_size, max_pages, max_len, scale,
                                  O, ldo);
  if (bad != SERQ_OK) return bad;
  if (B == 0 || T == 0) return SERQ_OK;
  if (!Q || !O || !cu_q || !kv_len) return SERQ_EINVAL;
  if (!page_table && max_pages > 0 && max_len > 0) return SERQ_EINVAL;
  if (!aligned(cu_q, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4)) return SERQ_EALIGN;
  const serq::PrefillPlan plan = serq::plan_prefill(dtype == SERQ_BF16, B, T, Hq, Hkv, D, max_len);
  if (plan.bytes < 0) return SERQ_EINVAL;
  if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes)) return SERQ_EINVAL;
  if (!aligned(workspace, 16)) return SERQ_EALIGN;
  serq::AttnArgs a = attention_args(Q, dtype, ldq, B, Hq, Hkv, D, Kc, Vc, n_pages, page_size, page_table, max_pages,
                                    kv_len, max_len, scale, O, ldo, workspace);
  a.cu_q = cu_q;
  a.T = T;
  return serq::launch_attn_prefill(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SERQ_OK : SERQ_EHIP;
}

extern "C" int64_t serq_attn_decode_workspace(serq_dtype dtype, int B, int Hq, int Hkv, int D, int prefix_len,
                                              int max_len) {
  if (!valid_dtype(dtype) || B < 0 || !valid_heads(Hq, Hkv) || (D != 64 && D != 128) || prefix_len < 0 ||
      prefix_len > kMaxKeys || max_len < 0 || max_len > kMaxKeys || !valid_rows(B, Hq))
    return -1;
  return B == 0 ? 0 : serq::plan_decode(dtype == SERQ_BF16, B, Hq, Hkv, D, prefix_len, max_len).bytes;
}

extern "C" int serq_attn_decode(const void* Q, serq_dtype dtype, int64_t ldq, int B, int Hq, int Hkv, int D,
                                const void* Kc, const void* Vc, int n_pages, int page_size,
                                const int32_t* prefix_table, int prefix_len, const int32_t* page_table, int max_pages,
                                const int32_t* kv_len, int max_len, float scale, void* O, int64_t ldo, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  if (B < 0 || prefix_len < 0 || prefix_len > kMaxKeys) return SERQ_EINVAL;
  const int bad = check_attention(Q, dtype, ldq, B, Hq, Hkv, D, Kc, Vc, n_pages, page_size, max_pages, max_len, scale,
                                  O, ldo);
  if (bad != SERQ_OK) return bad;
  if (B == 0) return SERQ_OK;
  if (!Q || !O || !kv_len || (prefix_len > 0 && !prefix_table)) return SERQ_EINVAL;
  if (!page_table && max_pages > 0 && max_len > 0) return SERQ_EINVAL;
  if (!aligned(prefix_table, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4)) return SERQ_EALIGN;
  const serq::DecodePlan plan = serq::plan_decode(dtype == SERQ_BF16, B, Hq, Hkv, D, prefix_len, max_len);
  if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes)) return SERQ_EINVAL;
  if (!aligned(workspace, 16)) return SERQ_EALIGN;
  serq::AttnArgs a = attention_args(Q, dtype, ldq, B, Hq, Hkv, D, Kc, Vc, n_pages, page_size, page_table, max_pages,
                                    kv_len, max_len, scale, O, ldo, workspace);
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  return serq::launch_attn_decode(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SERQ_OK : SERQ_EHIP;
}
