// gdn_selftest.cu -- the bounded-wait path of the fused kernels, exercised on its own.
//
// Every mbarrier wait in the tensor-core kernels goes through sm100::mbar_wait with a time
// limit; when a wait gives up, the kernel sets GDN_DEV_TIMEOUT in the caller's status word,
// drains what it has in flight and returns instead of hanging.  This entry point runs that wait
// in a one-thread kernel with nothing in flight: on an mbarrier that nobody arrives on (the
// wait must give up after limit_ns and report the timeout), or on one the thread has already
// arrived on (the wait must succeed and report nothing).
//
// The gated linear recurrence counts tries instead of reading the clock; its two kinds of waits are run
// likewise.
#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_recurrence.cuh"
#include "gdn_sm100.cuh"

namespace {

__global__ void wait_selftest_kernel(int* dev_status, unsigned long long limit_ns, int arrive_first,
                                     unsigned long long* waited_ns) {
  using namespace gdn::sm100;
  __shared__ uint64_t bar;
  if (threadIdx.x != 0) return;
  mbar_init(&bar, 1);
  fence_mbar_init();
  if (arrive_first) mbar_arrive(&bar);
  const uint64_t t0 = globaltimer_ns();
  const bool ok = mbar_wait(&bar, 0u, limit_ns);
  if (waited_ns) *waited_ns = globaltimer_ns() - t0;
  if (!ok) gdn::report(dev_status, GDN_DEV_TIMEOUT);
}

// One lane waits for a message and for a copy that do not come, each twice: what has run out once is not waited
// for again.  (Of the second kind two are under way, and each of them is given the same time.)
__global__ void recurrence_wait_selftest_kernel(int* dev_status, int tries, int arrive_first,
                                                unsigned long long* waited_ns) {
  using namespace gdn;
  __shared__ uint64_t message, copies[2][1];
  if (threadIdx.x != 0) return;
  mbar_init(&message, 1);
  for (int k = 0; k < 2; ++k) mbar_init(&copies[k][0], 1);
  fence_mbar_init();
  if (arrive_first) {
    mbar_arrive(&message);
    for (int k = 0; k < 2; ++k) mbar_arrive(&copies[k][0]);
  }
  unsigned lost = 0;
  uint64_t at = globaltimer_ns();
  auto lap = [&](int n) {
    const uint64_t now = globaltimer_ns();
    waited_ns[n] = now - at;
    at = now;
  };
  for (int n = 0; n < 2; ++n) {
    wait_or_report(&message, 0u, &lost, dev_status, tries);
    lap(n);
  }
  for (int n = 0; n < 2; ++n) {
    wait_for_copies<2>(copies, 0, 0, 2, &lost, dev_status, tries);
    lap(2 + n);
  }
  waited_ns[4] = kTries;
}

}  // namespace

extern "C" gdn_status_t gdn_selftest_recurrence_wait(int* dev_status, int tries, int arrive_first,
                                                     unsigned long long* waited_ns, void* stream) {
  if (!dev_status || !waited_ns) return GDN_ERR_NULL;
  if (tries <= 0 || tries > 10000) return GDN_ERR_SHAPE;
  recurrence_wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(dev_status, tries, arrive_first, waited_ns);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" gdn_status_t gdn_selftest_wait_timeout(int* dev_status, unsigned long long limit_ns,
                                                  int arrive_first, unsigned long long* waited_ns,
                                                  void* stream) {
  if (!dev_status) return GDN_ERR_NULL;
  if (limit_ns == 0 || limit_ns > 100000000ull) return GDN_ERR_SHAPE;   // (0, 100 ms]
  wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(dev_status, limit_ns,
                                                                        arrive_first, waited_ns);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
