// vocab_api.cu -- the C ABI of the linear head's cross entropy (see
// include/credit.h): argument checks, the pieces of the vocabulary and their
// workspace, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "credit.h"
#include "internal.h"
#include "planner.h"
#include "vocab.h"

using namespace credit;

namespace {

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// Bytes of the logits' gradient that a piece of the vocabulary may take, and of the
// statistics' parts that a piece of the tokens may.
constexpr int64_t kPieceBytes = (int64_t)256 << 20;
// Most parts of a sum over the vocabulary.
constexpr int kMaxSplits = 64;
// Most tokens whose logits' gradient takes two bf16 terms unasked: those whose two terms
// are rows of one tile, so that dhidden's products cost no more for the second.  Rounded
// to one, a token's target is off by up to 2^-8, uniformly: the root mean square over T
// tokens varies by 0.45 / sqrt(T) of itself, 6 % for 64.
constexpr int kTwoTerms = kTileM / 2;
// Fewest stages of a part.
constexpr int kMinPart = 8;
// Most stages of a part of a product that is summed in the tensor cores' accumulators
// alone.  Every addition of sixteen k drops up to 2^-25 of the sum, always towards zero:
// four a stage, 2^-12 in all, where the rounding to bf16 behind it is up to 2^-8 (in one
// part 4194304 tokens of one sign lost 0.8 %).
constexpr int kLongPart = 2048;

// Widest tile: a piece of the vocabulary, or of the tokens, is whole tiles of any shape.
constexpr int kTileN = vocab_tile_cols(kPair256);

struct Shape {
    int64_t tokens, hidden, vocab;
    int dtype, es, terms;  // terms of the operands
    VocabTerms kind;       // and of the logits' gradient
    bool pack_h, pack_w;   // the operand is copied as bf16 terms first
    bool few;              // takes the form for a few tokens
    // rows of A in dhidden's product: two terms lie one behind the other
    int64_t grad_rows() const { return kind == kTerms2 ? 2 * tokens : tokens; }
};

// Floats of a token in the shared memory of the form for a few tokens: whole steps
// of a warp.
int64_t few_pitch(int64_t hidden) { return round_up(hidden, 256); }
// Columns that it takes at most: two CTAs to an SM, of eight tokens one of twice the
// threads.
constexpr int64_t few_columns(int tokens) { return (tokens == 8 ? 200 << 10 : 100 << 10) / (4 * tokens); }
// fp32 tokens and elements of the weight of a forward pass that takes it eight tokens at
// a time: up to 16 read the weight twice, where the tiles read it, write its three bf16
// terms and read those (16 tokens of 32768 x 4096: 235 and 387 us, of 16384 x 1024 46 and
// 52, 12 of 131072 x 256 77 and 110; of 4096 x 1024 24 and 22, of 10000 x 256 23 and 16;
// 24 of 32768 x 4096 361 and 384, of 10000 x 6000 254 and 205, of 8192 x 4096 110 and 102).
constexpr int64_t kFewForward = 16, kFewForwardWeight = 1 << 24;

// backward: 0 the loss, 1 its gradient, 2 its precise gradient.
credit_status_t shape_of(int backward, const void* h, const void* w, int64_t tokens, int64_t hidden,
                         int64_t vocab, credit_dtype_t dtype, Shape* s) {
    if (tokens < 0 || hidden < 1 || vocab < 1 || backward < 0 || backward > 2) return CREDIT_ERR_INVALID_ARG;
    if (dtype != CREDIT_F32 && dtype != CREDIT_BF16) return CREDIT_ERR_UNSUPPORTED;
    // rows and columns are counted in 32 bits, tiles of 128 past them too
    const int64_t limit = ((int64_t)1 << 31) - 1024;
    if (tokens > limit || vocab > limit || hidden > ((int64_t)1 << 24)) return CREDIT_ERR_INVALID_ARG;
    // (tiles of a launch, too)
    const int64_t tiles = ceil_div(tokens, kTileM) * ceil_div(vocab, kTileM);
    const int64_t wide = ceil_div(std::max(tokens, vocab), kTileM) * ceil_div(hidden, kTileM);
    if (tiles > ((int64_t)1 << 28) || wide > ((int64_t)1 << 28)) return CREDIT_ERR_INVALID_ARG;
    s->tokens = tokens;
    s->hidden = hidden;
    s->vocab = vocab;
    s->dtype = (int)dtype;
    s->es = dtype == CREDIT_F32 ? 4 : 2;
    s->terms = dtype == CREDIT_F32 ? 3 : 1;
    s->kind = dtype == CREDIT_F32 ? kTerms3 : tokens <= kTwoTerms || backward == 2 ? kTerms2 : kTerms1;
    // (two terms of a token are two rows)
    if (s->kind == kTerms2 && tokens > limit / 2) return CREDIT_ERR_INVALID_ARG;
    if (!aligned(h, s->es) || !aligned(w, s->es)) return CREDIT_ERR_INVALID_ARG;
    const bool lines = hidden * s->es % 16 == 0;
    s->pack_h = s->terms > 1 || !lines || !aligned(h, 16);
    s->pack_w = s->terms > 1 || !lines || !aligned(w, 16);
    // One token is bound by reading the weight (131072 x 4096 bf16: 162 us in the form
    // for a few, 175 in tiles).  More take it where the tiles would copy the weight
    // first (4 tokens of 50000 x 1001 bf16: 47 and 73 us; 8 of 131072 x 2048 fp32: 212
    // and 900; 8 of bf16 223 and 99).
    const int64_t most =
        !backward && dtype == CREDIT_F32 && vocab * hidden >= kFewForwardWeight ? kFewForward : kFewTokens;
    s->few = tokens <= most && (tokens <= 1 || s->pack_w) &&
             few_pitch(hidden) <= few_columns(few_tokens((int)std::min<int64_t>(tokens, kFewTokens)));
    return CREDIT_OK;
}

// An operand of the call as the tensor maps see it, packed to `at` or not.
TermMatrix operand(const Shape& s, const void* p, int64_t rows, bool pack, char* at) {
    const int64_t pitch = pack ? round_up(s.hidden, 8) * 2 : s.hidden * 2;
    return {pack ? at : p, rows, s.hidden, pitch, pitch * rows, s.terms};
}
int64_t operand_bytes(const Shape& s, int64_t rows, bool pack) {
    return pack ? round_up(s.hidden, 8) * 2 * rows * s.terms : 0;
}

// The workspace of a call, in the order of its parts.
struct Layout {
    int64_t h, w, parts, picked, unit, logits, grad, sums, dw, bytes;  // offsets
    int64_t piece;      // vocabulary rows (backward) or tokens (forward) at a time
    int32_t pieces;
    int64_t sums_pitch;
    bool add;           // dhidden is the sums' sum
    int64_t parts_room, logits_room, grad_room, dw_room, sums_room;  // bytes
    int64_t place(int64_t* at, int64_t n) {
        *at = bytes;
        bytes += round_up(n, 256);
        return n;
    }
};

// A tile's time in a launch, in stages of a pair: four products of sixteen k take
// 512 cycles whatever the tile's shape (a CTA alone with 256 columns, which stages
// half as much again, takes a tenth longer: backward 4096 x 4096 x 65536 3.83 ms
// instead of 3.49); the epilogue, which runs beside the next tile's products, some
// eight of that for 256 columns a CTA.
double tile_cost(VocabTile t, double stages) {
    return std::max(t == kOne256 ? 1.1 * stages : stages, vocab_tile_cols(t) / 32.0) + 1.0;
}
// What the first tile waits for besides: a pair's CTAs meet, and a wide tile's
// epilogue stands alone at the end.
double launch_cost(VocabTile t) { return t == kPair256 ? 10.0 : t == kOne256 ? 4.0 : 0.0; }
constexpr VocabTile kTiles[] = {kPair256, kOne256, kOne128};
// The shape whose tiles end first.
VocabTile tile_for(int64_t rows, int64_t cols, int64_t stages, int sms) {
    VocabTile best = kPair256;
    double least = 0;
    for (const VocabTile t : kTiles) {
        const int64_t tiles = ceil_div(rows, vocab_tile_rows(t)) * ceil_div(cols, vocab_tile_cols(t));
        const double time = (double)ceil_div(tiles, sms / vocab_tile_ctas(t)) *
                                tile_cost(t, (double)stages) + launch_cost(t);
        if (t == kPair256 || time < least) {
            best = t;
            least = time;
        }
    }
    return best;
}

VocabTile logits_tile(const Shape& s, int64_t rows, int64_t cols, int sms) {
    return tile_for(rows, cols, ceil_div(s.hidden, kTileK) * (s.terms == 1 ? 1 : 6), sms);
}

// Parts of k of a product whose tiles of 128 x 128 would leave half of the SMs idle
// (1: it is not split); `pairs` products a stage, a part of four stages' at least.
// The parts' sums go through memory and another kernel, some 6 us: what a tile saves
// has to be worth them, 32 stages of 0.27 us (bf16 loss of 32, 1024 x 4096, 12 stages
// less: 11.5 us split, 9.8 whole; of 200, 2048 x 2048, 24 less: 13.1 and 12.6; of 64,
// 4096 x 4096, 48 less: 14.4 and 18.7; fp32 of 38, 4864 x 246: 19 and 90; dweight of
// 8192, 64 x 128 with its call: 14 and 31).
struct Split {
    int32_t splits, per;
    int64_t pitch;      // of a row's sums
};
Split split_for(int64_t rows, int64_t cols, int64_t k, int pairs, int sms) {
    const int64_t kb = ceil_div(k, kTileK), least = pairs > 1 ? 2 : 4;
    const int64_t tiles = ceil_div(rows, vocab_tile_rows(kOne128)) * ceil_div(cols, vocab_tile_cols(kOne128));
    const int64_t want = std::min<int64_t>({sms / tiles, kb / least, kMaxSplits});
    const int64_t per = want > 1 ? ceil_div(kb, want) : kb;
    const bool worth = (kb - per) * pairs >= 32;
    return {worth ? (int32_t)ceil_div(kb, per) : 1, (int32_t)(worth ? per : kb), round_up(cols, 4)};
}
Split logits_split(const Shape& s, int64_t cols, int sms) {
    return split_for(s.tokens, cols, s.hidden, s.terms == 1 ? 1 : 6, sms);
}

// The tokens are walked in equal pieces whose parts fit kPieceBytes, however wide the
// tiles (16384 tokens of 131072 words: one piece).
Layout forward_layout(const Shape& s, int sms, VocabTile* t, Split* split) {
    Layout l{};
    const Split k = *split = logits_split(s, s.vocab, sms);
    const int64_t token = ceil_div(s.vocab, kTileN) * vocab_tile_parts(kPair256) * 8;
    const int64_t most = std::max<int64_t>(kTileN, kPieceBytes / token / kTileN * kTileN);
    l.pieces = k.splits > 1 ? 1 : (int32_t)ceil_div(s.tokens, most);
    l.piece = l.pieces > 1 ? round_up(ceil_div(s.tokens, l.pieces), kTileN) : s.tokens;
    l.pieces = (int32_t)ceil_div(s.tokens, l.piece);
    *t = k.splits > 1 ? kOne128 : logits_tile(s, l.piece, s.vocab, sms);
    l.place(&l.h, operand_bytes(s, s.tokens, s.pack_h));
    l.place(&l.w, operand_bytes(s, s.vocab, s.pack_w));
    if (k.splits > 1) {
        l.logits_room = l.place(&l.logits, k.splits * s.tokens * k.pitch * 4);
        return l;
    }
    l.parts_room = l.place(&l.parts, ceil_div(s.vocab, vocab_tile_cols(*t)) * vocab_tile_parts(*t) * l.piece * 8);
    l.place(&l.picked, l.piece * 4);
    return l;
}

// The two products of a piece of the vocabulary in one launch: the tiles' shape and
// the parts of the sum over the piece that dhidden takes.  Where its tiles alone
// would keep SMs waiting, a part is at most half of what each SM has to do.
struct Products {
    VocabTile tile;
    int32_t splits, per;
    Split dw;            // of dweight's sum over the tokens
};
Products products_for(const Shape& s, int64_t piece, bool dh, bool dw, int sms) {
    Products best{};
    double least = 0;
    const int64_t kb = ceil_div(piece, kTileK), kt = ceil_div(s.tokens, kTileK) * (s.kind == kTerms2 ? 2 : 1);
    const int64_t rows_h = s.grad_rows();
    const int pairs = s.kind == kTerms3 ? 6 : 1;  // products a stage of k
    for (const VocabTile t : kTiles) {
        const int rows = vocab_tile_rows(t), cols = vocab_tile_cols(t), units = sms / vocab_tile_ctas(t);
        const int64_t nt = ceil_div(s.hidden, cols);
        const int64_t th = dh ? ceil_div(rows_h, rows) * nt : 0, tw = dw ? ceil_div(piece, rows) * nt : 0;
        const double all = (double)th * tile_cost(t, (double)(kb * pairs)) +
                           (double)tw * tile_cost(t, (double)(kt * pairs));
        Products p{t, 1, (int32_t)kb, {}};
        double time = all / units;
        if (dh) {
            const int64_t share = std::max<int64_t>(kMinPart, (int64_t)(all / units / 2 / pairs));
            int64_t want = std::min<int64_t>(ceil_div(kb, share), kMaxSplits);
            if (s.kind != kTerms3) want = std::max<int64_t>(want, ceil_div(kb, kLongPart));
            p.per = (int32_t)ceil_div(kb, want);
            p.splits = (int32_t)ceil_div(kb, p.per);
            const double part = tile_cost(t, (double)p.per * pairs);
            time = dw ? std::max(time, part) : (double)ceil_div(th * p.splits, units) * part;
        } else {
            time = (double)ceil_div(tw, units) * tile_cost(t, (double)(kt * pairs));
        }
        time += launch_cost(t);
        if (t == kPair256 || time < least) {
            best = p;
            least = time;
        }
    }
    return best;
}

// The vocabulary is walked in equal pieces whose logits' gradient fits kPieceBytes.
Layout backward_layout(const Shape& s, bool dh, bool dw, int sms, Products* products) {
    Layout l{};
    l.place(&l.h, operand_bytes(s, s.tokens, s.pack_h));
    l.place(&l.w, operand_bytes(s, s.vocab, s.pack_w));
    const int64_t most = std::max<int64_t>(kTileN, kPieceBytes / (s.tokens * 2 * s.kind) / kTileN * kTileN);
    l.pieces = (int32_t)ceil_div(s.vocab, most);
    l.piece = round_up(ceil_div(s.vocab, l.pieces), kTileN);
    l.pieces = (int32_t)ceil_div(s.vocab, l.piece);
    l.grad_room = l.place(&l.grad, s.tokens * l.piece * 2 * s.kind);
    if (s.kind == kTerms1) l.place(&l.unit, 4);
    *products = products_for(s, std::min(l.piece, s.vocab), dh, dw, sms);
    const Split k = logits_split(s, l.piece, sms);
    if (k.splits > 1) l.logits_room = l.place(&l.logits, k.splits * s.tokens * k.pitch * 4);
    Split& d = products->dw;
    d = split_for(l.piece, s.hidden, s.tokens, s.terms == 1 ? 1 : 6, sms);
    if (dw && d.splits > 1) products->tile = kOne128;
    // (a stage adds both terms' products)
    const int64_t kt = ceil_div(s.tokens, kTileK), longest = s.kind == kTerms2 ? kLongPart / 2 : kLongPart;
    if (s.kind != kTerms3 && d.per > longest) {
        d.splits = (int32_t)ceil_div(kt, longest);
        d.per = (int32_t)ceil_div(kt, d.splits);
    }
    if (dw && d.splits > 1) l.dw_room = l.place(&l.dw, d.splits * std::min(l.piece, s.vocab) * d.pitch * 4);
    l.sums_pitch = round_up(s.hidden, 4);
    l.add = dh && (products->splits > 1 || l.pieces > 1 || s.kind == kTerms2);
    if (l.add) l.sums_room = l.place(&l.sums, products->splits * s.grad_rows() * l.sums_pitch * 4);
    return l;
}

// The same of a call of a few tokens.
struct FewLayout {
    int64_t parts, picked, grad, sums, bytes = 0;
    int64_t parts_room = 0, grad_room = 0, sums_room = 0;
    int blocks, slices;
    int64_t sums_pitch;
};
FewLayout few_layout(const Shape& s, bool backward, bool dh, bool vec, int sms) {
    FewLayout l;
    Layout place{};
    const int shaped = (int)std::min<int64_t>(s.tokens, kFewTokens);
    l.blocks = few_blocks(shaped, (int)few_pitch(s.hidden), s.vocab, sms);
    l.slices = few_slices(s.hidden, s.dtype, vec, s.vocab, sms);
    l.sums_pitch = round_up(s.hidden, 4);
    if (!backward) {
        l.parts_room = place.place(&l.parts, l.blocks * s.tokens * 8);
        place.place(&l.picked, s.tokens * 4);
    } else {
        l.grad_room = place.place(&l.grad, s.vocab * few_tokens(shaped) * 4);
        if (dh) l.sums_room = place.place(&l.sums, l.slices * s.tokens * l.sums_pitch * 4);
    }
    l.bytes = place.bytes;
    return l;
}
FewArgs few_args(const Shape& s, const void* h, const void* w, const int64_t* target, int64_t ignore) {
    FewArgs a{};
    a.h = h;
    a.w = w;
    a.tokens = a.shaped = (int32_t)s.tokens;
    a.cols = (int32_t)s.hidden;
    a.pitch = (int32_t)few_pitch(s.hidden);
    a.vocab = s.vocab;
    a.target = target;
    a.ignore = ignore;
    return a;
}

credit_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CREDIT_OK : CREDIT_ERR_CUDA; }

credit_status_t device(const DevInfo** info) {
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return CREDIT_ERR_CUDA; }
    *info = device_info(dev);
    return *info ? CREDIT_OK : CREDIT_ERR_CUDA;
}

struct Span {
    const void* p;
    uint64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// Every output is disjoint from every input and every other output.
bool disjoint(const Span* in, int nin, const Span* out, int nout) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(out[i], in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

// Tiles of a product of rows x cols.  Tile rows are walked together in groups of
// 2048 rows, which stay in L2 while the other operand's pass by.
TileWork work_of(VocabTile t, int64_t rows, int64_t cols, int64_t k, bool a_mn, bool b_mn) {
    TileWork w{};
    w.mt = (int32_t)ceil_div(rows, vocab_tile_rows(t));
    w.nt = (int32_t)ceil_div(cols, vocab_tile_cols(t));
    w.splits = 1;
    w.kb = w.per = (int32_t)ceil_div(k, kTileK);
    w.group = std::min(w.mt, 2048 / vocab_tile_rows(t));
    w.a_mn = a_mn;
    w.b_mn = b_mn;
    w.a_bytes = kTileM * kTileK * 2;
    return w;
}

// The rows of a box of A with K innermost: of a single tile only those there are
// (the others of a stage keep what they held, and their products go nowhere).
int box_rows(VocabTile t, int64_t rows, TileWork* w) {
    int box = kTileM;
    if (vocab_tile_ctas(t) == 1 && rows < kTileM) box = (int)round_up(rows, 8);
    w->a_bytes = box * kTileK * 2;
    return box;
}

// The logits of a.rows tokens and a.cols columns as the sums of their splits.
void logits_out(const Split& k, float* sums, int64_t room, VocabArgs* a) {
    a->work[0].per = k.per;
    a->work[0].splits = k.splits;
    a->out[0] = ProductOut{nullptr, sums, k.pitch, a->rows, a->cols, 0, 1, nullptr, room};
}

// Copies the operands that the tensor maps cannot take as they are.
cudaError_t pack(const Shape& s, const void* hidden, const TermMatrix& h, const void* weight,
                 const TermMatrix& w, unsigned* err, int sms, cudaStream_t stream) {
    const void* src[2];
    TermMatrix dst[2];
    int n = 0;
    if (s.pack_h) { src[n] = hidden; dst[n++] = h; }
    if (s.pack_w) { src[n] = weight; dst[n++] = w; }
    return n ? launch_vocab_pack(s.dtype, src, dst, n, err, sms, stream) : cudaSuccess;
}

}  // namespace

extern "C" {

credit_status_t credit_linear_ce_workspace(int backward, const void* hidden, const void* weight,
                                           int64_t tokens, int64_t hidden_size, int64_t vocab,
                                           credit_dtype_t dtype, int device, size_t* bytes) {
    if (!bytes) return CREDIT_ERR_INVALID_ARG;
    Shape s;
    const credit_status_t st = shape_of(backward, hidden, weight, tokens, hidden_size, vocab, dtype, &s);
    if (st != CREDIT_OK) return st;
    *bytes = 0;
    if (tokens == 0) return CREDIT_OK;
    const DevInfo* d = device_info(device);
    if (!d) return CREDIT_ERR_CUDA;
    if (s.few) {  // (either access)
        *bytes = (size_t)std::max(few_layout(s, backward, true, true, d->sms).bytes,
                                  few_layout(s, backward, true, false, d->sms).bytes);
        return CREDIT_OK;
    }
    if (!backward) {
        VocabTile t;
        Split k;
        *bytes = (size_t)forward_layout(s, d->sms, &t, &k).bytes;
        return CREDIT_OK;
    }
    Products p;  // (whichever gradients are asked for)
    *bytes = (size_t)std::max(backward_layout(s, true, true, d->sms, &p).bytes,
                              backward_layout(s, true, false, d->sms, &p).bytes);
    return CREDIT_OK;
}

credit_status_t credit_linear_ce_forward(const void* hidden, const void* weight,
                                         const int64_t* target, int64_t ignore_index, float* loss,
                                         float* lse, int64_t tokens, int64_t hidden_size,
                                         int64_t vocab, credit_dtype_t dtype, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    Shape s;
    credit_status_t st = shape_of(0, hidden, weight, tokens, hidden_size, vocab, dtype, &s);
    if (st != CREDIT_OK) return st;
    if (tokens == 0) return CREDIT_OK;
    if (!hidden || !weight || !target || !loss || !lse) return CREDIT_ERR_INVALID_ARG;
    if (!aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4)) return CREDIT_ERR_INVALID_ARG;
    const uint64_t hb = (uint64_t)(tokens * hidden_size) * s.es, wb = (uint64_t)(vocab * hidden_size) * s.es;
    const Span in[] = {{hidden, hb}, {weight, wb}, {target, (uint64_t)tokens * 8}};
    const Span out[] = {{loss, (uint64_t)tokens * 4}, {lse, (uint64_t)tokens * 4},
                        {workspace, workspace ? workspace_bytes : 0}};
    if (!disjoint(in, 3, out, 3)) return CREDIT_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16)) return CREDIT_ERR_INVALID_ARG;
    const DevInfo* d;
    st = device(&d);
    if (st != CREDIT_OK) return st;
    if (s.few) {
        const bool vec = aligned(weight, 16) && hidden_size * s.es % 16 == 0;
        const FewLayout l = few_layout(s, false, false, vec, d->sms);
        if (workspace_bytes < (uint64_t)l.bytes) return CREDIT_ERR_INVALID_ARG;
        cudaStream_t q = (cudaStream_t)stream;
        FewArgs f = few_args(s, hidden, weight, target, ignore_index);
        f.parts = reinterpret_cast<float2*>(static_cast<char*>(workspace) + l.parts);
        f.parts_pitch = tokens;
        f.parts_room = l.parts_room;
        f.err = checked_error_word();
        f.picked = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.picked);
        float2* const parts = f.parts;
        float* const picked = f.picked;
        // (as many at a time as the first, so that each leaves as many parts)
        for (int64_t t = 0; t < tokens; t += kFewTokens) {
            f.h = static_cast<const char*>(hidden) + t * hidden_size * s.es;
            f.tokens = (int32_t)std::min<int64_t>(kFewTokens, tokens - t);
            f.shaped = (int32_t)std::min<int64_t>(kFewTokens, tokens);
            f.target = target + t;
            f.parts = parts + t;
            f.parts_room = l.parts_room - t * (int64_t)sizeof(*parts);
            f.picked = picked + t;
            if ((st = from_cuda(launch_few_logits(s.dtype, vec, f, l.blocks, q))) != CREDIT_OK) return st;
        }
        f.parts = parts;
        f.picked = picked;
        VocabArgs a{};
        a.rows = (int32_t)tokens;
        a.vocab = vocab;
        a.target = target;
        a.ignore = ignore_index;
        a.parts = f.parts;
        a.picked = f.picked;
        a.parts_room = l.parts_room;
        a.err = f.err;
        return from_cuda(launch_vocab_merge(a, l.blocks, loss, lse, q));
    }
    Split split;
    VocabTile tile;
    const Layout l = forward_layout(s, d->sms, &tile, &split);
    if (workspace_bytes < (uint64_t)l.bytes) return CREDIT_ERR_INVALID_ARG;
    unsigned* err = device_error_word();
    if (!err) return CREDIT_ERR_CUDA;
    cudaStream_t q = (cudaStream_t)stream;
    char* const ws = static_cast<char*>(workspace);
    const TermMatrix h = operand(s, hidden, tokens, s.pack_h, ws + l.h);
    const TermMatrix w = operand(s, weight, vocab, s.pack_w, ws + l.w);
    CUtensorMap maps[4] = {};
    if (!term_map(w, vocab_tile_cols(tile) / vocab_tile_ctas(tile), &maps[1])) return CREDIT_ERR_CUDA;
    if ((st = from_cuda(pack(s, hidden, h, weight, w, err, d->sms, q))) != CREDIT_OK) return st;
    VocabArgs a{};
    a.jobs = 1;
    a.cols = (int32_t)vocab;
    a.vocab = vocab;
    a.ignore = ignore_index;
    a.err = err;
    if (split.splits > 1) {
        a.work[0] = work_of(tile, tokens, vocab, hidden_size, false, false);
        if (!term_map(h, box_rows(tile, tokens, &a.work[0]), &maps[0])) return CREDIT_ERR_CUDA;
        a.rows = (int32_t)tokens;
        a.target = target;

        float* const sums = reinterpret_cast<float*>(ws + l.logits);
        logits_out(split, sums, l.logits_room, &a);
        if ((st = from_cuda(launch_vocab(kVocabSums, s.kind, tile, maps, a, d->sms, q))) != CREDIT_OK)
            return st;
        return from_cuda(launch_vocab_rows(a, sums, split.splits, split.pitch, s.kind, loss, lse, q));
    }
    a.parts = reinterpret_cast<float2*>(ws + l.parts);
    a.picked = reinterpret_cast<float*>(ws + l.picked);
    a.parts_room = l.parts_room;
    for (int64_t t = 0; t < tokens; t += l.piece) {
        const int64_t n = std::min(l.piece, tokens - t);
        TermMatrix rows = h;
        rows.p = static_cast<const char*>(h.p) + t * h.pitch;
        rows.rows = n;
        a.work[0] = work_of(tile, n, vocab, hidden_size, false, false);
        if (!term_map(rows, box_rows(tile, n, &a.work[0]), &maps[0])) return CREDIT_ERR_CUDA;
        a.rows = (int32_t)n;
        a.target = target + t;
        if ((st = from_cuda(launch_vocab(kVocabStats, s.kind, tile, maps, a, d->sms, q))) != CREDIT_OK)
            return st;
        st = from_cuda(launch_vocab_merge(a, a.work[0].nt * vocab_tile_parts(tile), loss + t, lse + t, q));
        if (st != CREDIT_OK) return st;
    }
    return CREDIT_OK;
}

}  // extern "C"

namespace {

credit_status_t gradient(int backward, const float* dloss, const float* dlse, const void* hidden,
                         const void* weight, const int64_t* target, int64_t ignore_index,
                         const float* lse, void* dhidden, void* dweight, int64_t tokens,
                         int64_t hidden_size, int64_t vocab, credit_dtype_t dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
    Shape s;
    credit_status_t st = shape_of(backward, hidden, weight, tokens, hidden_size, vocab, dtype, &s);
    if (st != CREDIT_OK) return st;
    cudaStream_t q = (cudaStream_t)stream;
    const uint64_t hb = (uint64_t)(tokens * hidden_size) * s.es, wb = (uint64_t)(vocab * hidden_size) * s.es;
    if (!aligned(dhidden, s.es) || !aligned(dweight, s.es)) return CREDIT_ERR_INVALID_ARG;
    if (!dhidden && !dweight) return CREDIT_OK;
    if (tokens == 0) return dweight ? from_cuda(cudaMemsetAsync(dweight, 0, wb, q)) : CREDIT_OK;
    if (!dloss || !hidden || !weight || !target || !lse) return CREDIT_ERR_INVALID_ARG;
    if (!aligned(dloss, 4) || !aligned(dlse, 4) || !aligned(target, 8) || !aligned(lse, 4))
        return CREDIT_ERR_INVALID_ARG;
    const uint64_t tb = (uint64_t)tokens * 4;
    const Span in[] = {{hidden, hb}, {weight, wb}, {target, 2 * tb}, {dloss, tb}, {dlse, tb}, {lse, tb}};
    const Span out[] = {{dhidden, hb}, {dweight, wb}, {workspace, workspace ? workspace_bytes : 0}};
    if (!disjoint(in, 6, out, 3)) return CREDIT_ERR_INVALID_ARG;
    const DevInfo* d;
    st = device(&d);
    if (st != CREDIT_OK) return st;
    if (s.few) {
        const bool vec = aligned(weight, 16) && aligned(dweight, 16) && hidden_size * s.es % 16 == 0;
        const FewLayout l = few_layout(s, true, dhidden != nullptr, vec, d->sms);
        if (!workspace || workspace_bytes < (uint64_t)l.bytes || !aligned(workspace, 16))
            return CREDIT_ERR_INVALID_ARG;
        FewArgs f = few_args(s, hidden, weight, target, ignore_index);
        f.lse = lse;
        f.dloss = dloss;
        f.dlse = dlse;
        f.grad = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.grad);
        if (dhidden) f.sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.sums);
        f.sums_pitch = l.sums_pitch;
        f.grad_room = l.grad_room;
        f.sums_room = l.sums_room;
        f.err = checked_error_word();
        f.dw = dweight;
        const bool lines = aligned(weight, 16) && hidden_size * s.es % 16 == 0;
        if ((st = from_cuda(launch_few_logits(s.dtype, lines, f, l.blocks, q))) != CREDIT_OK) return st;
        if ((st = from_cuda(launch_few_products(s.dtype, vec, f, l.slices, q))) != CREDIT_OK) return st;
        return dhidden ? from_cuda(launch_vocab_sum(s.dtype, f.sums, l.slices, tokens, hidden_size,
                                                    l.sums_pitch, nullptr, dhidden, l.sums_room, f.err, d->sms,
                                                    q))
                       : CREDIT_OK;
    }
    Products products;
    const Layout l = backward_layout(s, dhidden != nullptr, dweight != nullptr, d->sms, &products);
    if (!workspace || workspace_bytes < (uint64_t)l.bytes || !aligned(workspace, 16))
        return CREDIT_ERR_INVALID_ARG;
    unsigned* err = device_error_word();
    if (!err) return CREDIT_ERR_CUDA;
    char* const ws = static_cast<char*>(workspace);
    const TermMatrix h = operand(s, hidden, tokens, s.pack_h, ws + l.h);
    const TermMatrix w = operand(s, weight, vocab, s.pack_w, ws + l.w);
    float* const unit = s.kind == kTerms1 ? reinterpret_cast<float*>(ws + l.unit) : nullptr;
    if (unit && (st = from_cuda(launch_vocab_unit(dloss, target, ignore_index, tokens, unit, q))) != CREDIT_OK)
        return st;
    if ((st = from_cuda(pack(s, hidden, h, weight, w, err, d->sms, q))) != CREDIT_OK) return st;

    const Split split = logits_split(s, l.piece, d->sms);
    const VocabTile pt = products.tile, gt = split.splits > 1 ? kOne128 : logits_tile(s, tokens, l.piece, d->sms);
    // what the logits' gradient is formed from, and what it is multiplied with
    CUtensorMap logits[4] = {}, operands[4] = {};
    for (int p = 0; p < l.pieces; ++p) {
        const int64_t v0 = p * l.piece, pv = std::min(l.piece, vocab - v0);
        VocabArgs a{};
        a.jobs = 1;
        a.work[0] = work_of(gt, tokens, pv, hidden_size, false, false);
        a.work[0].b_y0 = (int32_t)v0;
        const int box = box_rows(gt, tokens, &a.work[0]);
        if (p == 0 && (!term_map(h, box, &logits[0]) ||
                       !term_map(w, vocab_tile_cols(gt) / vocab_tile_ctas(gt), &logits[1])))
            return CREDIT_ERR_CUDA;
        a.rows = (int32_t)tokens;
        a.cols = (int32_t)pv;
        a.v0 = (int32_t)v0;
        a.vocab = vocab;
        a.target = target;
        a.ignore = ignore_index;
        a.lse = lse;
        a.dloss = dloss;
        a.dlse = dlse;
        a.grad = ws + l.grad;
        a.grad_pitch = l.piece;
        a.grad_plane = l.piece * tokens;
        a.grad_room = l.grad_room;
        a.unit = unit;
        a.err = err;
        if (split.splits > 1) {
            float* const sums = reinterpret_cast<float*>(ws + l.logits);
            logits_out(split, sums, l.logits_room, &a);
            if ((st = from_cuda(launch_vocab(kVocabSums, s.kind, gt, logits, a, d->sms, q))) != CREDIT_OK)
                return st;
            st = from_cuda(launch_vocab_rows(a, sums, split.splits, split.pitch, s.kind, nullptr, nullptr, q));
            if (st != CREDIT_OK) return st;
        } else if ((st = from_cuda(launch_vocab(kVocabGrad, s.kind, gt, logits, a, d->sms, q))) != CREDIT_OK) {
            return st;
        }
        const TermMatrix g{ws + l.grad, tokens, pv, l.piece * 2, l.piece * tokens * 2, s.kind};
        a.jobs = 0;
        if (dhidden) {
            // (a piece starts at a whole stage of k, and past its end g is zero)
            TermMatrix rows = g;  // (terms as rows)
            if (s.kind == kTerms2) {
                rows.rows = s.grad_rows();
                rows.terms = 1;
                rows.plane *= 2;
            }
            TileWork& k = a.work[0] = work_of(pt, rows.rows, hidden_size, pv, false, true);
            k.b_y0 = (int32_t)v0;
            // (a shorter last piece may leave parts without a stage: they add nothing)
            k.per = std::min(products.per, k.kb);
            k.splits = (int32_t)ceil_div(k.kb, k.per);
            ProductOut& o = a.out[0];
            o.out = dhidden;
            o.sums = l.add ? reinterpret_cast<float*>(ws + l.sums) : nullptr;
            o.pitch = l.add ? l.sums_pitch : hidden_size;
            o.room = l.add ? l.sums_room : (int64_t)hb;
            o.rows = (int32_t)rows.rows;
            o.cols = (int32_t)hidden_size;
            o.add = p > 0;
            o.vec = aligned(dhidden, 16) && hidden_size * s.es % 16 == 0;
            o.unit = unit;
            if (!term_map(rows, box_rows(pt, rows.rows, &k), &operands[0]) || !term_map(w, kTileK, &operands[1]))
                return CREDIT_ERR_CUDA;
            a.jobs = 1;
        }
        if (dweight) {
            const int j = a.jobs++;
            a.work[j] = work_of(pt, pv, hidden_size, tokens, true, true);
            if (s.kind == kTerms2) {
                a.work[j].both = 1;
                a.work[j].a_bytes *= 2;
            }
            ProductOut& o = a.out[j];
            o = ProductOut{};
            o.out = static_cast<char*>(dweight) + v0 * hidden_size * s.es;
            o.pitch = hidden_size;
            o.room = pv * hidden_size * s.es;
            o.rows = (int32_t)pv;
            o.cols = (int32_t)hidden_size;
            o.vec = aligned(dweight, 16) && hidden_size * s.es % 16 == 0;
            o.unit = unit;
            if (products.dw.splits > 1) {
                TileWork& k = a.work[j];
                k.per = std::min(products.dw.per, k.kb);
                k.splits = (int32_t)ceil_div(k.kb, k.per);
                o.sums = reinterpret_cast<float*>(ws + l.dw);
                o.pitch = products.dw.pitch;
                o.room = l.dw_room;
            }
            if (!term_map(g, kTileK, &operands[2 * j]) || !term_map(h, kTileK, &operands[2 * j + 1]))
                return CREDIT_ERR_CUDA;
        }
        if ((st = from_cuda(launch_vocab(kVocabProduct, s.kind, pt, operands, a, d->sms, q))) !=
            CREDIT_OK)
            return st;
        if (dweight && products.dw.splits > 1) {
            st = from_cuda(launch_vocab_sum(s.dtype, reinterpret_cast<float*>(ws + l.dw), products.dw.splits, pv,
                                            hidden_size, products.dw.pitch, unit,
                                            static_cast<char*>(dweight) + v0 * hidden_size * s.es, l.dw_room, err,
                                            d->sms, q));
            if (st != CREDIT_OK) return st;
        }
    }
    if (dhidden && l.add)  // (a split's terms lie one behind the other, as splits do)
        return from_cuda(launch_vocab_sum(s.dtype, reinterpret_cast<float*>(ws + l.sums),
                                          products.splits * (s.kind == kTerms2 ? 2 : 1), tokens,
                                          hidden_size, l.sums_pitch, unit, dhidden, l.sums_room, err, d->sms, q));
    return CREDIT_OK;
}

}  // namespace

extern "C" {

credit_status_t credit_linear_ce_backward(const float* dloss, const float* dlse, const void* hidden,
                                          const void* weight, const int64_t* target,
                                          int64_t ignore_index, const float* lse, void* dhidden,
                                          void* dweight, int64_t tokens, int64_t hidden_size,
                                          int64_t vocab, credit_dtype_t dtype, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    return gradient(1, dloss, dlse, hidden, weight, target, ignore_index, lse, dhidden, dweight, tokens,
                    hidden_size, vocab, dtype, workspace, workspace_bytes, stream);
}

credit_status_t credit_linear_ce_backward_precise(const float* dloss, const float* dlse,
                                                  const void* hidden, const void* weight,
                                                  const int64_t* target, int64_t ignore_index,
                                                  const float* lse, void* dhidden, void* dweight,
                                                  int64_t tokens, int64_t hidden_size, int64_t vocab,
                                                  credit_dtype_t dtype, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
    return gradient(2, dloss, dlse, hidden, weight, target, ignore_index, lse, dhidden, dweight, tokens,
                    hidden_size, vocab, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
