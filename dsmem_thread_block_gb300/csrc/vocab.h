// vocab.h -- the linear head's cross entropy: launch arguments and launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace credit {

constexpr int kTileM = 128;   // rows of a CTA's output tile
constexpr int kTileK = 64;    // k of a stage

// The output tile of a CTA or pair of CTAs: rows x columns.
enum VocabTile : int {
    kPair256,   // 256 x 256, a pair
    kOne256,    // 128 x 256
    kOne128,    // 128 x 128
};
constexpr int vocab_tile_rows(VocabTile t) { return t == kPair256 ? 2 * kTileM : kTileM; }
constexpr int vocab_tile_cols(VocabTile t) { return t == kOne128 ? 128 : 256; }
constexpr int vocab_tile_ctas(VocabTile t) { return t == kPair256 ? 2 : 1; }
// parts of the statistics: one for an epilogue warp's columns
constexpr int kPartCols = 64;
constexpr int vocab_tile_parts(VocabTile t) { return vocab_tile_cols(t) / kPartCols; }

// A matrix of bf16 terms: `terms` planes of rows x cols, rows `pitch` bytes and
// planes `plane` bytes apart, all 16-byte aligned.
struct TermMatrix {
    const void* p;
    int64_t rows, cols, pitch, plane;
    int terms;
};

// The tiles of one matrix product, C = A B summed over k.
struct TileWork {
    int32_t mt, nt;        // tiles of C
    int32_t splits;        // parts of k, each summed apart
    int32_t kb, per;       // stages of k in all, and in a part
    int32_t group;         // tile rows that are walked together
    int32_t a_mn, b_mn;    // operand lies with M (N) innermost
    int32_t b_y0;          // first row of B's matrix
    int32_t a_bytes;       // of A that a CTA's stage receives
    int32_t both;          // A in two terms, both in a stage
};

// Where a product goes: rows x cols at `out` (of the call's type), or the
// fp32 sums of its splits, rows x pitch each.
struct ProductOut {
    void* out;
    float* sums;
    int64_t pitch;         // elements
    int32_t rows, cols;
    int32_t add;           // to what the sums hold
    int32_t vec;           // rows of `out` are whole 16-byte lines
    const float* unit;     // what the logits' gradient was divided by (null: 1; not for sums)
    int64_t room;          // bytes at `sums`, or else at `out` (looked at by the checked build)
};

struct VocabArgs {
    TileWork work[2];
    int32_t jobs;          // products
    int32_t lead;          // rounds of the second product that some units start early
    int32_t a_room;        // of A in a stage: a_bytes at least, a multiple of 1024
    int32_t rows, cols;    // tokens, vocabulary rows of this piece
    int32_t v0;            // the piece's first vocabulary row
    int64_t vocab;
    const int64_t* target;
    int64_t ignore;
    // statistics: per (kPartCols columns, token) maximum and sum of exponentials, and
    // the target's logit per token
    float2* parts;
    float* picked;
    int64_t parts_room;    // bytes of it, as grad_room (looked at by the checked build)
    // gradient of the logits
    const float* lse;
    const float* dloss;
    const float* dlse;     // or null
    void* grad;            // terms planes, tokens x grad_pitch
    int64_t grad_pitch, grad_plane;  // elements
    const float* unit;     // of one term: what it is divided by (vocab_unit)
    int64_t grad_room;
    ProductOut out[2];
    unsigned* err;
    int32_t alone;         // a self-test: nothing brings B, every wait runs out
};

// kVocabSums: the logits themselves, as fp32 sums of their splits.
enum VocabOut : int { kVocabStats, kVocabGrad, kVocabProduct, kVocabSums };
// What a call's operands are: bf16, bf16 with the logits' gradient in two terms, or
// fp32 in three.
enum VocabTerms : int { kTerms1 = 1, kTerms2 = 2, kTerms3 = 3 };
// Results that the tensor cores' sums alone are not good enough for: all but bf16
// products.
constexpr bool vocab_promotes(VocabOut out, VocabTerms t) { return out != kVocabProduct || t == kTerms3; }

// A call of a few tokens (vocab_few.cu).
struct FewArgs {
    const void* h;
    const void* w;
    int32_t tokens, cols, pitch;   // pitch: floats of a token in shared memory
    int32_t shaped;                // the kernel is that of so many tokens
    int64_t vocab;
    const int64_t* target;
    int64_t ignore;
    float2* parts;                 // per (block, token), blocks parts_pitch apart
    int64_t parts_pitch;
    float* picked;
    // the logits' gradient, vocab x few_tokens(tokens), written and then read; null:
    // the statistics are wanted
    float* grad;
    const float* lse;
    const float* dloss;
    const float* dlse;             // or null
    float* sums;                   // of dhidden, per slice; null: not wanted
    int64_t sums_pitch;
    void* dw;                      // null: not wanted
    // bytes of parts, grad and sums, and the error word (looked at by the checked build)
    int64_t parts_room, grad_room, sums_room;
    unsigned* err;
};
constexpr int kFewTokens = 8;      // most of them
// the tokens that a kernel counts with
constexpr int few_tokens(int tokens) { return tokens == 1 ? 1 : tokens <= 4 ? 4 : 8; }
int few_blocks(int tokens, int pitch, int64_t vocab, int sms);
int few_slices(int64_t cols, int dtype, bool vec, int64_t vocab, int sms);
cudaError_t launch_few_logits(int dtype, bool vec, const FewArgs& a, int blocks, cudaStream_t s);
cudaError_t launch_few_products(int dtype, bool vec, const FewArgs& a, int slices, cudaStream_t s);

// box_rows: of a box (K innermost: the tile's rows; else the stage's k).
bool term_map(const TermMatrix& m, int box_rows, CUtensorMap* map);

const void* vocab_stats_kernel(VocabTerms terms, VocabTile t);
const void* vocab_grad_kernel(VocabTerms terms, VocabTile t);
const void* vocab_product_kernel(VocabTerms terms, VocabTile t);

const void* vocab_sums_kernel(VocabTerms terms);   // kOne128 alone

cudaError_t launch_vocab(VocabOut out, VocabTerms terms, VocabTile tile, const CUtensorMap (&maps)[4],
                         const VocabArgs& a, int sms, cudaStream_t s);
// The tiles' kernel with nothing that brings B; allocates its scratch and waits for it.
cudaError_t run_tiles_alone(int dev, int sms, VocabTile tile);
// loss and lse from the tiles' parts
cudaError_t launch_vocab_merge(const VocabArgs& a, int nparts, float* loss, float* lse,
                               cudaStream_t s);
// From the splits' sums of the logits, splits x tokens x pitch (a.out[0].room bytes): loss and lse, or with
// a.grad the logits' gradient in `terms` terms.
cudaError_t launch_vocab_rows(const VocabArgs& a, const float* sums, int splits, int64_t pitch,
                              VocabTerms terms, float* loss, float* lse, cudaStream_t s);
// n matrices of the call's type and of one width as bf16 terms
cudaError_t launch_vocab_pack(int dtype, const void* const (&src)[2], const TermMatrix (&dst)[2], int n,
                              unsigned* err, int sms, cudaStream_t s);
// out = the splits' sums (`room` bytes) added in order, times *unit (null: 1)
cudaError_t launch_vocab_sum(int dtype, const float* sums, int splits, int64_t rows, int64_t cols,
                             int64_t pitch, const float* unit, void* out, int64_t room, unsigned* err, int sms,
                             cudaStream_t s);
// What a logits' gradient of one term is divided by.
cudaError_t launch_vocab_unit(const float* dloss, const int64_t* target, int64_t ignore, int64_t tokens,
                              float* unit, cudaStream_t s);

}  // namespace credit
