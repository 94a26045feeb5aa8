// vocab_grad.cu -- the gradient of the logits' tiles (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_grad_kernel(VocabTerms terms, VocabTile t) {
    return terms == kTerms1   ? vocab_kernel_of<GradOut<kTerms1>, kVocabGrad, kTerms1>(t)
           : terms == kTerms2 ? vocab_kernel_of<GradOut<kTerms2>, kVocabGrad, kTerms1>(t)
                              : vocab_kernel_of<GradOut<kTerms3>, kVocabGrad, kTerms3>(t);
}
}  // namespace credit
