// k_layer_bf16.cu -- the layer norm's kernels (layer.cuh) for bfloat16 rows.
#include "layer.cuh"

namespace tcr {

const void *layer_kernel_bf16(size_t nvec, bool elem, int &team)
{
    return layer_kernel_of<kBF16>(nvec, elem, team);
}

}  // namespace tcr
