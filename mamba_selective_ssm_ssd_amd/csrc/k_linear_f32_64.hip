// k_linear_f32_64.hip -- instantiations of the linear-attention scan for f32 I/O, x and y rows of up to 64 channels.
#include "k_linear.hpp"

namespace m3 {

hipError_t launch_linear_f32_64(const LinParams &p, int dz, bool out, hipStream_t s) {
    return launch_linear_dx<float, 64>(p, dz, out, s);
}

} // namespace m3
