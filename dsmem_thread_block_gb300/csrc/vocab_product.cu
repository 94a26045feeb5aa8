// vocab_product.cu -- the products of the logits' gradient (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_product_kernel(int dtype, VocabTile t) {
    return dtype
               ? vocab_kernel_of<ProductRow<bf16>, vocab_promotes(kVocabProduct, 1), 1>(t) : vocab_kernel_of<ProductRow<float>, vocab_promotes(kVocabProduct, 0), 3>(t);
}
}  // namespace credit
