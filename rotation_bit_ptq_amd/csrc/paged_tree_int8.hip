// Attention of several new tokens over an int8 cache (see paged_tree_impl.h).
#include "paged_tree_impl.h"

namespace orbit {
namespace block {
hipError_t launch_tree_int8(const TreeArgs& a, int q_dtype, bool few, dim3 grid, hipStream_t stream) {
  return q_dtype == ORBIT_BF16 ? launch_tree<ORBIT_KV_BF16, ORBIT_KV_INT8>(a, few, grid, stream)
                               : launch_tree<ORBIT_KV_F16, ORBIT_KV_INT8>(a, few, grid, stream);
}
}  // namespace block
}  // namespace orbit
