// Single-token attention over an int8 paged cache (see paged_attention_impl.h).
#include "paged_attention_impl.h"

namespace orbit {
namespace block {

hipError_t launch_attend_coded(const AttentionArgs& a, int q_dtype, dim3 grid, hipStream_t stream) {
  return q_dtype == ORBIT_BF16 ? launch_attend<ORBIT_KV_BF16, ORBIT_KV_INT8>(a, grid, stream)
                               : launch_attend<ORBIT_KV_F16, ORBIT_KV_INT8>(a, grid, stream);
}

}  // namespace block
}  // namespace orbit
