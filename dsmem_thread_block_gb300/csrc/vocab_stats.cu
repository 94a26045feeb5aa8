// vocab_stats.cu -- statistics of the logits' tiles (vocab_tiles.cuh).
#include "vocab_tiles.cuh"

namespace credit {
const void* vocab_stats_kernel(VocabTile t) { return vocab_kernel_of<StatsOut, vocab_promotes(kVocabStats, 0)>(t); }
}  // namespace credit
