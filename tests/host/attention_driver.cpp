// Host-side driver for the sanitizer build of the attention calls' host
// code (attn_abi.cpp, rope_table.cpp): stubs stand in for the device
// launchers and plans; tables of exactly their documented size.

#include <cstdio>
#include <cstdlib>
#include <memory>

#include "serq.h"
#include "serq_attn.h"

namespace serq {
static int g_launches = 0;
static AttnArgs g_last{};
PrefillPlan plan_prefill(int, int, int, int, int, int, int) { return PrefillPlan{}; }
DecodePlan plan_decode(int, int, int, int, int, int, int) {
  DecodePlan p{};
  p.bytes = 4096;
  return p;
}
hipError_t launch_rope_append(const RopeArgs&, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_attn_prefill(const AttnArgs& a, const PrefillPlan&, hipStream_t) {
  ++g_launches;
  g_last = a;
  return hipSuccess;
}
hipError_t launch_attn_decode(const AttnArgs& a, const DecodePlan&, hipStream_t) {
  ++g_launches;
  g_last = a;
  return hipErrorUnknown;
}
}  // namespace serq

static int g_fail = 0;
#define EXPECT(cond)                                                  \
  do {                                                                \
    if (!(cond)) {                                                    \
      std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                       \
    }                                                                 \
  } while (0)

int main() {
  for (int rot : {2, 6, 64, 128})
    for (int n : {1, 3, 100})
      for (int kind = SERQ_ROPE_PLAIN; kind <= SERQ_ROPE_BANDS; ++kind) {
        std::unique_ptr<float[]> t(new float[static_cast<size_t>(rot) * n]);
        const int want = kind == SERQ_ROPE_BASE && rot == 2 ? SERQ_EINVAL : SERQ_OK;
        EXPECT(serq_rope_table(rot, n, 1e4, static_cast<serq_rope_scaling>(kind), 2.0, 64, 1.0, 4.0, 1.0, t.get()) ==
               want);
      }
  char* const P = reinterpret_cast<char*>(uintptr_t{1} << 20);
  float* const F = reinterpret_cast<float*>(P);
  int32_t* const I = reinterpret_cast<int32_t*>(P);
  EXPECT(serq_rope_append(P, SERQ_BF16, 768, 4, 4, 1, 128, F, nullptr, 1e-5f, F, 128, 9, SERQ_ROPE_HALF, I, I, P, 512,
                          P, P, 4, 16, nullptr) == SERQ_OK);
  EXPECT(serq_rope_append(P, SERQ_F32, 1 << 30, 1, 16384, 16384, 128, F, F, 1e-5f, F, 128, 9, SERQ_ROPE_HALF, I, I, P,
                          1 << 30, P, P, 1, 1024, nullptr) == SERQ_OK);
  EXPECT(serq_attn_prefill(P, SERQ_BF16, 512, I, 2, 9, 4, 1, 128, P, P, 4, 16, I, 4, I, 1 << 30, 0.1f, P, 512, nullptr,
                           0, nullptr) == SERQ_OK);
  EXPECT(serq::g_last.max_len == 64 && serq::g_last.page_shift == 4);     // the table's room
  EXPECT(serq_attn_prefill(P, SERQ_BF16, 512, I, 2, 9, 4, 1, 128, P, P, 4, 1024, I, INT32_MAX, I, 1 << 30, 0.1f, P, 512,
                           nullptr, 0, nullptr) == SERQ_OK);
  EXPECT(serq::g_last.max_len == 1 << 30);
  EXPECT(serq_attn_decode(P, SERQ_F32, 512, 2, 4, 1, 128, P, P, 4, 16, nullptr, 0, nullptr, 0, I, 64, 0.1f, P, 512, P,
                          4096, nullptr) == SERQ_EHIP);
  EXPECT(serq::g_last.max_len == 0);
  EXPECT(serq_attn_decode(P, SERQ_F32, 512, 2, 4, 1, 128, P, P, 4, 16, I, 5, I, 4, I, 64, 0.1f, P, 512, P, 4095,
                          nullptr) == SERQ_EINVAL);
  EXPECT(serq::g_launches == 5);
  if (g_fail) {
    std::fprintf(stderr, "%d checks failed\n", g_fail);
    return 1;
  }
  std::printf("attention host driver: all checks passed\n");
  return 0;
}
