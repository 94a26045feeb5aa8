// vocab_product.cu -- the products of the logits' gradient (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_product_kernel(VocabTerms terms, VocabTile t) {
    return terms == kTerms1   ? vocab_kernel_of<ProductRow<bf16>, kVocabProduct, kTerms1>(t)
           : terms == kTerms2 ? vocab_kernel_of<ProductRow<bf16>, kVocabProduct, kTerms2>(t)
                              : vocab_kernel_of<ProductRow<float>, kVocabProduct, kTerms3>(t);
}
}  // namespace credit
