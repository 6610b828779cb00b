// k_linear_f32_32.hip -- instantiations of the linear-attention scan for f32 I/O, x and y rows of up to 32 channels.
#include "k_linear.hpp"

namespace m3 {

hipError_t launch_linear_f32_32(const LinParams &p, int dz, bool out, hipStream_t s) {
    return launch_linear_dx<float, 32>(p, dz, out, s);
}

} // namespace m3
