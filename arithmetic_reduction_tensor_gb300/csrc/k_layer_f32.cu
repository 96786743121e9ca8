// k_layer_f32.cu -- the layer norm's kernels (layer.cuh) for binary32 rows.
#include "layer.cuh"

namespace tcr {

const void *layer_kernel_f32(size_t nvec, bool elem, int &team)
{
    return layer_kernel_of<kF32>(nvec, elem, team);
}

}  // namespace tcr
