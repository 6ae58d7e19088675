// Test-only kernel: a warp whose lanes wait with the chunk kernels' own wait, for a barrier that
// has completed (even lanes) and for one that nothing arrives on (odd lanes, if `odd`). What the
// wait returned on each lane and how long it took come back; the kernel returns normally.
#include "tcgen05.cuh"

__global__ void warp_waits(int odd, int32_t* status, int32_t* done,
                           unsigned long long* elapsed_ns) {
  __shared__ uint64_t bars[2];
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    pda::mbar_init(&bars[0], 1);
    pda::mbar_init(&bars[1], 1);
    pda::fence_mbar_init();
    pda::mbar_arrive(&bars[0]);
  }
  __syncwarp();
  const unsigned long long t0 = pda::global_timer_ns();
  const bool ok = pda::warp_wait(&bars[odd != 0 ? lane & 1 : 0], 0);
  done[lane] = ok;
  if (lane == 0) {
    *elapsed_ns = pda::global_timer_ns() - t0;
    if (!ok) pda::atomic_or_error(status, PDA_DEVERR_TIMEOUT);
  }
}

extern "C" int pda_test_warp_wait(int odd, int32_t* status, int32_t* done,
                                  unsigned long long* elapsed_ns, cudaStream_t stream) {
  warp_waits<<<1, 32, 0, stream>>>(odd, status, done, elapsed_ns);
  return static_cast<int>(cudaGetLastError());
}
