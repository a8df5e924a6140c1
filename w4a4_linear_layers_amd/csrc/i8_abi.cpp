// C ABI entry points of the linear in 8-bit integers: host-side argument
// validation and dispatch of serq_linear_i8 onto the caller's HIP stream.
// serq_calibrate_i8 (host) lives in calibrate.cpp.

#include <hip/hip_runtime.h>

#include "serq.h"
#include "serq_i8.h"

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// int32 sums of products up to 2^14 in magnitude; outputs that a launch's grid takes.
constexpr int kMostK = (1 << 17) - 1, kMostN = 1 << 26;
inline bool valid_sizes(int M, int K, int N) {
  return M >= 0 && K > 0 && K <= kMostK && N > 0 && N <= kMostN && static_cast<int64_t>(M) * N <= int64_t{1} << 37;
}

}  // namespace

extern "C" int64_t serq_linear_i8_workspace(int M, int K, int N) {
  if (!valid_sizes(M, K, N)) return -1;
  return M == 0 ? 0 : serq::plan_linear_i8(M, K, N).bytes;
}

extern "C" const char* serq_linear_i8_kernel_name(int M, int K, int N) {
  return valid_sizes(M, K, N) ? serq::plan_linear_i8(M, K, N).name : nullptr;
}

extern "C" int serq_linear_i8(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, int M, int K, int N,
                              void* Y, serq_dtype y_dtype, int32_t* acc_dbg, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  if (y_dtype != SERQ_F32 && y_dtype != SERQ_BF16) return SERQ_EINVAL;
  if (!valid_sizes(M, K, N)) return SERQ_EINVAL;
  if (!Wq || !sw) return SERQ_EINVAL;
  if (!aligned16(Wq) || !aligned16(sw)) return SERQ_EALIGN;
  if (M == 0) return SERQ_OK;  // the M-sized buffers may then be empty (NULL)
  if (!Xq || !sx || !Y) return SERQ_EINVAL;
  if (!aligned16(Xq) || !aligned16(sx) || !aligned16(Y) || !aligned16(acc_dbg) || !aligned16(workspace)) return SERQ_EALIGN;
  const serq::I8Plan plan = serq::plan_linear_i8(M, K, N);
  if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes)) return SERQ_EINVAL;
  serq::I8Args a{};
  a.Xq = Xq;
  a.sx = sx;
  a.Wq = Wq;
  a.sw = sw;
  a.Y = Y;
  a.dbg = acc_dbg;
  a.partial = plan.bytes > 0 ? static_cast<int32_t*>(workspace) : nullptr;
  a.M = M;
  a.K = K;
  a.N = N;
  a.y_bf16 = y_dtype == SERQ_BF16;
  return serq::launch_linear_i8(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SERQ_OK : SERQ_EHIP;
}
