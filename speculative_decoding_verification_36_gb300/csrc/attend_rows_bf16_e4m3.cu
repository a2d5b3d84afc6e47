// attend_rows_bf16_e4m3.cu -- attend_rows.cuh for bf16 queries and e4m3 codes.
#include "attend_rows.cuh"

namespace sv {
cudaError_t launch_attend_rows_bf16_e4m3(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  return launch_rows_of<uint16_t, true>(a, sms, bytes, s);
}
}  // namespace sv
