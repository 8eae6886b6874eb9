// The attention's launches, one unit per head width (attend64.cu and so on).
#pragma once
#include "attend.cuh"
#include "host.cuh"

namespace sv {

template <int D>
bool attend_prepare();  // shared-memory limits on the current device
template <int D>
bool attend_launch(const AttendParams& p, int num_sms, cudaStream_t stream);

#ifdef SV_ATTEND_WIDTH
namespace {  // every unit has its own
// Rows of a row tile by eights up to 32, then by sixteens: the softmax's registers
// and instructions go by them.
template <int D, class F>
bool attend_each(F f) {
  bool ok = f.template operator()<8>() && f.template operator()<16>() && f.template operator()<24>() &&
            f.template operator()<32>();
  if constexpr (D < 256) ok = ok && f.template operator()<48>() && f.template operator()<64>();
  return ok;
}

struct AttendPrepare {
  template <int NP>
  bool operator()() const {
    return cudaFuncSetAttribute(k_attend<SV_ATTEND_WIDTH, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(AttendGeo<SV_ATTEND_WIDTH, NP>::kSmemBytes)) == cudaSuccess;
  }
};
// The first size that holds the rows is launched.
struct AttendRun {
  const AttendParams& p;
  int num_sms;
  cudaStream_t stream;
  bool* started;
  template <int NP>
  bool operator()() const {
    if (*started || p.rp > NP) return true;
    *started = true;
    using G = AttendGeo<SV_ATTEND_WIDTH, NP>;
    return launch_waiting(k_attend<SV_ATTEND_WIDTH, NP>, dim3(num_sms), G::kThreads, G::kSmemBytes, stream, p) &&
           launch_waiting(k_attend_join<SV_ATTEND_WIDTH, NP>, dim3(num_sms, (p.rp + kJoinRows - 1) / kJoinRows),
                          join_threads(SV_ATTEND_WIDTH), 0, stream, p);
  }
};
}  // namespace

template <>
bool attend_prepare<SV_ATTEND_WIDTH>() {
  return attend_each<SV_ATTEND_WIDTH>(AttendPrepare{});
}
template <>
bool attend_launch<SV_ATTEND_WIDTH>(const AttendParams& p, int num_sms, cudaStream_t stream) {
  bool started = false;
  return attend_each<SV_ATTEND_WIDTH>(AttendRun{p, num_sms, stream, &started}) && started;
}
#endif

}  // namespace sv
