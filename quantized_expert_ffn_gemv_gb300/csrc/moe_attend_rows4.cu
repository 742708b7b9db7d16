// attend_rows_kernel over caches of 4 bits.
#include "moe_attend_rows.cuh"

namespace moe {

moe_status_t launch_rows4(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st) {
  return launch_rows<4>(kv, t, dim, bf16, st);
}

}  // namespace moe
