// attend_tiles_int8.cu -- attend_tiles.cuh for int8 codes.
#include "attend_tiles.cuh"

namespace sv {
cudaError_t launch_attend_tiles_int8(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  return a.D <= 64    ? launch_tiles<false, 64>(a, sms, bytes, s)
         : a.D <= 128 ? launch_tiles<false, 128>(a, sms, bytes, s)
                      : launch_tiles<false, 256>(a, sms, bytes, s);
}

// Test probe of the kernel's waits (one warp): one on an mbarrier that has been arrived at, and one on an mbarrier
// that nothing arrives at.  flags[0]: the first was taken as run out; [1]: the second was;
// [2]: how often a wait after it may look again.
__global__ void attend_wait_probe_kernel(uint32_t* flags) {
  __shared__ unsigned long long bar[2];
  __shared__ Waits waits;
  if (threadIdx.x == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    waits.tries = mbar_tries(spin_limit());
    waits.out = 0;
    mbar_arrive(&bar[0]);
  }
  __syncwarp();
  bounded_wait(waits, &bar[0], 0);
  __syncwarp();
  if (threadIdx.x == 0) flags[0] = waits.out;
  bounded_wait(waits, &bar[1], 0);
  __syncwarp();
  if (threadIdx.x == 0) flags[1] = waits.out, flags[2] = waits.tries;
}
cudaError_t attend_wait_probe(uint32_t* flags_host) {
  uint32_t* flags = nullptr;
  cudaError_t e = cudaMalloc(&flags, 3 * sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  attend_wait_probe_kernel<<<1, 32>>>(flags);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpy(flags_host, flags, 3 * sizeof(uint32_t), cudaMemcpyDeviceToHost);
  const cudaError_t e2 = cudaFree(flags);
  return e != cudaSuccess ? e : e2;
}
cudaError_t attend_tiles_int8_set_spin_limit(unsigned n) { return set_spin_limit_here(n); }
}  // namespace sv
