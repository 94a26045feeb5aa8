// vocab_stats.cu -- statistics of the logits' tiles (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_stats_kernel(int dtype, VocabTile t) {
    return dtype ? vocab_kernel_of<StatsOut, vocab_promotes(kVocabStats, 1), 1>(t)
                 : vocab_kernel_of<StatsOut, vocab_promotes(kVocabStats, 0), 3>(t);
}
}  // namespace credit
