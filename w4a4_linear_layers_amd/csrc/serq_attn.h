// Internal declarations of the attention half (serq_rope_append,
// serq_attn_prefill, serq_attn_decode): argument structs, the plans made on
// the host from the call's sizes alone, and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace serq {

struct RopeArgs {
  const void* QKV;
  int64_t ld;
  int M, Hq, Hkv, D;
  const float* q_norm;    // may be null
  const float* k_norm;    // may be null
  float eps;
  const float* table;     // max_pos x rot: cosines, then sines (null when rot == 0)
  int rot, max_pos;
  int interleaved;
  const int32_t* pos;     // axis a of token t at a * pos_stride + t
  int64_t pos_stride;
  int n_axes;
  uint32_t axis_bits[4];  // two bits a pair: its axis
  const int32_t* slot;
  void* Q;
  int64_t ldq;
  void* Kc;
  void* Vc;
  uint8_t* k_scale;       // of a cache of codes, else null
  uint8_t* v_scale;
  int n_pages, page_shift;
  int bf16;               // of QKV and Q
};

// One attention call (device pointers, validated sizes).
struct AttnArgs {
  const void* Q;
  int64_t ldq;
  const void* Kc;
  const void* Vc;
  const uint8_t* k_scale;       // of a cache of FP8 codes, else null
  const uint8_t* v_scale;
  int n_pages, page_shift;
  const int32_t* page_table;
  int max_pages;
  const int32_t* kv_len;
  int max_len;                  // at most max_pages << page_shift
  const int32_t* cu_q;          // prefill
  int T;                        // prefill: packed rows
  const int32_t* prefix_table;  // decode
  int prefix_len;
  int B, Hq, Hkv, D;
  float scale_log2;             // scale * log2(e): softmax weights are taken in base 2
  void* O;
  int64_t ldo;
  void* workspace;
  int bf16;
};

// How serq_attn_prefill is cut: `pack` query heads of a group and tile_pos
// positions per workgroup; keys in up to `splits` parts, so many that there
// are about `target` workgroups.
struct PrefillPlan {
  int tiled;              // on LDS tiles (attn_tile.hip)
  int pack, tile_pos;
  int splits, target;
  int64_t bytes;          // workspace; -1: more than one launch takes
};

// How serq_attn_decode is cut: the sequences' own keys in `splits` parts of
// `chunk` (one, with no join, where they are few), the prefix in `psplits`
// parts of `pchunk`; row tiles of 16.
struct DecodePlan {
  int splits, chunk, tiles, waves;      // waves of a workgroup
  int psplits, pchunk, ptiles;
  int ptiled;             // the prefix on LDS tiles (attn_tile.hip)
  int64_t bytes;          // workspace
};

// `kind`: kBf16 for bf16 queries (else fp32), kCodes over a cache of FP8 codes.
constexpr int kBf16 = 1, kCodes = 2;
PrefillPlan plan_prefill(int kind, int B, int T, int Hq, int Hkv, int D, int max_len);
DecodePlan plan_decode(int kind, int B, int Hq, int Hkv, int D, int prefix_len, int max_len);

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t stream);
hipError_t launch_attn_prefill(const AttnArgs& a, const PrefillPlan& p, hipStream_t stream);
hipError_t launch_attn_decode(const AttnArgs& a, const DecodePlan& p, hipStream_t stream);

}  // namespace serq
