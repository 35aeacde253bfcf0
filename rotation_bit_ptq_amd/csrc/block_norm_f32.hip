// Norms around a residual sum, float32 residual stream (see block_norm_impl.h).
#include "block_norm_impl.h"

namespace orbit {
namespace block {

template <class BT>
static hipError_t by_output(NormArgs& a, int y_dtype, hipStream_t stream) {
  switch (y_dtype) {
    case ORBIT_BF16: return launch_norm<float, BT, __bf16>(a, stream);
    case ORBIT_F16: return launch_norm<float, BT, _Float16>(a, stream);
    default: return launch_norm<float, BT, float>(a, stream);
  }
}

hipError_t launch_norm_f32(NormArgs& a, int b_dtype, int y_dtype, hipStream_t stream) {
  switch (b_dtype) {
    case ORBIT_BF16: return by_output<__bf16>(a, y_dtype, stream);
    case ORBIT_F16: return by_output<_Float16>(a, y_dtype, stream);
    default: return by_output<float>(a, y_dtype, stream);
  }
}

}  // namespace block
}  // namespace orbit
