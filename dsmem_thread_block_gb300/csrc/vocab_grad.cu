// vocab_grad.cu -- the gradient of the logits' tiles (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_grad_kernel(int dtype, VocabTile t) {
    return dtype ? vocab_kernel_of<GradOut<bf16>, false>(t) : vocab_kernel_of<GradOut<float>, true>(t);
}
}  // namespace credit
