// Kernels of a layer's products on fp32 operands.
#include "layer_tables.hpp"

namespace dg {

const void *layer_kernel_f32(int config, int variant) { return layer_kernel_of<float>(config, variant); }

}  // namespace dg
