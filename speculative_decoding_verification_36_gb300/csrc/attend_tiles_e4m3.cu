// attend_tiles_e4m3.cu -- attend_tiles.cuh for e4m3 codes.
#include "attend_tiles.cuh"

namespace sv {
cudaError_t launch_attend_tiles_e4m3(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  return a.D <= 64    ? launch_tiles<true, 64>(a, sms, bytes, s)
         : a.D <= 128 ? launch_tiles<true, 128>(a, sms, bytes, s)
                      : launch_tiles<true, 256>(a, sms, bytes, s);
}
cudaError_t attend_tiles_e4m3_set_spin_limit(unsigned n) { return set_spin_limit_here(n); }
}  // namespace sv
