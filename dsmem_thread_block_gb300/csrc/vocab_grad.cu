// vocab_grad.cu -- the gradient of the logits' tiles (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_grad_kernel(int dtype, VocabTile t) {
    return dtype
               ? vocab_kernel_of<GradOut<bf16>, vocab_promotes(kVocabGrad, 1), 1>(t)
               : vocab_kernel_of<GradOut<float>, vocab_promotes(kVocabGrad, 0), 3>(t);
}
}  // namespace credit
