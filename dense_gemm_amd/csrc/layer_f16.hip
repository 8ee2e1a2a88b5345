// Kernels of a layer's products on fp16 operands.
#include "layer_tables.hpp"

namespace dg {

const void *layer_kernel_f16(int config, int variant) { return layer_kernel_of<_Float16>(config, variant); }

}  // namespace dg
