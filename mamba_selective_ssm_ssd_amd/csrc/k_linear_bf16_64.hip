// k_linear_bf16_64.hip -- instantiations of the linear-attention scan for bf16 I/O, x and y rows of up to 64 channels.
#include "k_linear.hpp"

namespace m3 {

hipError_t launch_linear_bf16_64(const LinParams &p, int dz, bool out, hipStream_t s) {
    return launch_linear_dx<bf16, 64>(p, dz, out, s);
}

} // namespace m3
