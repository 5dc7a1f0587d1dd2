// selftest.cu -- kernels whose bounded mbarrier waits are made to run out, or their block to
// give up while they wait.
//
// It initialises an mbarrier that nothing will ever arrive on and waits for it
// with the same bounded-wait helper the tensor-core kernels use.  The wait gives
// up after limit_ns, sets DEVERR_TIMEOUT in the error word and returns, so the
// host sees a timeout status and the context stays usable.  In the second kernel 128 threads
// wait together, as those that join parts of a tile do (few_rows.cu), and four warps each for
// themselves, as those that drain accumulators do: threads begin some tens of microseconds
// apart, while another one says that the block gives up, arrives, or both.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

__global__ void wait_selftest_kernel(unsigned* flag, unsigned* err, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  const uint32_t b = smem_u32(&bar);
  if (threadIdx.x == 0) {
    mbar_init(b, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool ok = mbar_wait(b, 0, err, limit_ns);
    flag[0] = ok ? 1u : 2u;
  }
}

constexpr int kTogether = 128, kApart = 128;

__device__ void spin_ns(uint64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) {}
}

// answers[t]: 1 the thread went on, 2 it stopped; of the kTogether threads, then of kApart / 32 warps
__global__ void together_selftest_kernel(int posted, int aborted, unsigned* answers, unsigned* err, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ volatile int abort_flag;
  const uint32_t b = smem_u32(&bar);
  const int t = threadIdx.x;
  if (t == 0) {
    mbar_init(b, 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (t < kTogether) {
    spin_ns(t / 32 * 20000u);
    answers[t] = all_meet<1, kTogether>(!abort_flag && mbar_wait(b, 0, err, limit_ns)) ? 1u : 2u;
  } else if (t < kTogether + kApart) {
    spin_ns(t % 32 * 2000u);
    answers[t] = warp_wait(&abort_flag, b, 0, err, limit_ns) ? 1u : 2u;
  } else if (t == kTogether + kApart) {
    spin_ns(30000u);
    if (aborted) abort_flag = 1;
    if (posted) mbar_arrive(b);
  }
}

}  // namespace

bool selftest_together_agrees(const unsigned* answers, bool* stopped) {
  *stopped = false;
  for (int t = 0; t < kTogether + kApart; ++t) {
    const int first = t < kTogether ? 0 : t / 32 * 32;
    if ((answers[t] != 1u && answers[t] != 2u) || answers[t] != answers[first]) return false;
    *stopped = *stopped || answers[t] == 2u;
  }
  return true;
}

static_assert(kTogether + kApart <= kSelftestAnswers, "answers");
cudaError_t launch_together_selftest(bool posted, bool aborted, unsigned* answers, unsigned* err, uint64_t limit_ns,
                                     cudaStream_t st) {
  together_selftest_kernel<<<1, kTogether + kApart + 32, 0, st>>>(posted, aborted, answers, err, limit_ns);
  return cudaGetLastError();
}

cudaError_t launch_wait_selftest(unsigned* flag, unsigned* err, uint64_t limit_ns, cudaStream_t st) {
  wait_selftest_kernel<<<1, 32, 0, st>>>(flag, err, limit_ns);
  return cudaGetLastError();
}

}  // namespace moe
