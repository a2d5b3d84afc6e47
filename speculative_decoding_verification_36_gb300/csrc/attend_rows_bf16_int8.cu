// attend_rows_bf16_int8.cu -- attend_rows.cuh for bf16 queries and int8 codes.
#include "attend_rows.cuh"

namespace sv {
cudaError_t launch_attend_rows_bf16_int8(const KvAttendArgs& a, int sms, size_t* bytes, cudaStream_t s) {
  return launch_rows_of<uint16_t, false>(a, sms, bytes, s);
}
}  // namespace sv
