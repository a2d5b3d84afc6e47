// attend_tiles_int8.cu -- attend_tiles.cuh for int8 codes.
#include "attend_tiles.cuh"

namespace sv {
cudaError_t launch_attend_tiles_int8(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  return a.D <= 64    ? launch_tiles<false, 64>(a, sms, bytes, s)
         : a.D <= 128 ? launch_tiles<false, 128>(a, sms, bytes, s)
                      : launch_tiles<false, 256>(a, sms, bytes, s);
}
cudaError_t attend_tiles_int8_set_spin_limit(unsigned n) { return set_spin_limit_here(n); }
}  // namespace sv
