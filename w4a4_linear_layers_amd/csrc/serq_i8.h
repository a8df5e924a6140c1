// Internal declarations of the linear in 8-bit integers (serq_linear_i8).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace serq {

struct I8Args {
  const int8_t* Xq;      // M x K
  const float* sx;       // M
  const int8_t* Wq;      // N x K
  const float* sw;       // N
  void* Y;               // M x N, fp32 or bf16
  int32_t* dbg;          // optional M x N
  int32_t* partial;      // splits x M x N, where the plan has splits
  int M, K, N;
  int y_bf16;
};

enum class I8Kernel { kStream, kTile64, kTile64x128, kTile128, kTile256, kTile256x128, kGeneric };

struct I8Plan {
  I8Kernel kind;
  int rt, nt;            // kStream: tiles of 16 weight rows and of 16 tokens of a workgroup
  int splits, per;       // tiles: parts of K, of `per` k-tiles each
  int64_t bytes;         // workspace
  const char* name;
};

I8Plan plan_linear_i8(int M, int K, int N);
hipError_t launch_linear_i8(const I8Args& a, const I8Plan& p, hipStream_t stream);

}  // namespace serq
