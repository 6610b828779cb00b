// k_linear_f32_128.hip -- instantiations of the linear-attention scan for f32 I/O, x and y rows of up to 128 channels.
#include "k_linear.hpp"

namespace m3 {

hipError_t launch_linear_f32_128(const LinParams &p, int dz, bool out, hipStream_t s) {
    return launch_linear_dx<float, 128>(p, dz, out, s);
}

} // namespace m3
