// vocab_product.cu -- the products of the logits' gradient (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_product_kernel(VocabTerms terms, VocabTile t) {
    return terms == kTerms1   ? vocab_kernel_of<ProductRow<bf16>, kVocabProduct, kTerms1>(t)
           : terms == kTerms2 ? vocab_kernel_of<ProductRow<bf16>, kVocabProduct, kTerms2>(t)
                              : vocab_kernel_of<ProductRow<float>, kVocabProduct, kTerms3>(t);
}
const void* vocab_sums_kernel(VocabTerms terms) {
    return terms == kTerms3 ? (const void*)vocab_tiles<ProductRow<float>, kVocabSums, kTerms3, 128, 1>
                            : (const void*)vocab_tiles<ProductRow<float>, kVocabSums, kTerms1, 128, 1>;
}
}  // namespace credit
