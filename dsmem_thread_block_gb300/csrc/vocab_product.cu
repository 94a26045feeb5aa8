// vocab_product.cu -- the products of the logits' gradient (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_product_kernel(int dtype, VocabTile t) {
    return dtype ? vocab_kernel_of<ProductRow<bf16>, false>(t) : vocab_kernel_of<ProductRow<float>, true>(t);
}
}  // namespace credit
