// vocab_stats.cu -- statistics of the logits' tiles (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_stats_kernel(VocabTerms terms, VocabTile t) {
    return terms == kTerms3 ? vocab_kernel_of<StatsOut, kVocabStats, kTerms3>(t)
                            : vocab_kernel_of<StatsOut, kVocabStats, kTerms1>(t);
}
}  // namespace credit
