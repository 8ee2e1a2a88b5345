// Kernels of a layer's products on bf16 operands.
#include "layer_tables.hpp"

namespace dg {

const void *layer_kernel_bf16(int config, int variant) { return layer_kernel_of<__bf16>(config, variant); }

}  // namespace dg
