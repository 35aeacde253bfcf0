// Attention of several new tokens over a bfloat16 cache (see paged_tree_impl.h).
#include "paged_tree_impl.h"

namespace orbit {
namespace block {
hipError_t launch_tree_bf16(const TreeArgs& a, bool few, dim3 grid, hipStream_t stream) {
  return launch_tree<ORBIT_KV_BF16, ORBIT_KV_BF16>(a, few, grid, stream);
}
}  // namespace block
}  // namespace orbit
