// k_layer_f16.cu -- the layer norm's kernels (layer.cuh) for binary16 rows.
#include "layer.cuh"

namespace tcr {

const void *layer_kernel_f16(size_t nvec, bool elem, int &team)
{
    return layer_kernel_of<kF16>(nvec, elem, team);
}

}  // namespace tcr
