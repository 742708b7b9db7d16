// attend_tiles_kernel over caches of 8 bits.
#include "moe_attend_tiles.cuh"

namespace moe {

moe_status_t launch_tiles8(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st) {
  return launch_tiles<8>(kv, t, dim, bf16, st);
}

}  // namespace moe
