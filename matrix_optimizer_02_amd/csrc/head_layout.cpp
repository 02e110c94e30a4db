// How a call of the output-head losses is cut: pieces of the vocabulary, tiles,
// splits and the workspace (head_layout.h).
#include "head_layout.h"

#include <algorithm>
#include <cmath>

namespace dmuon {

namespace {

// Bytes of ds a piece of the vocabulary may take (one part): it is written
// once and read by two products, so it should stay in the 256 MB last-level
// cache next to what those stream.
constexpr int64_t kPieceBytes = int64_t(256) << 20;
constexpr int64_t kCachedBytes = int64_t(240) << 20;  // ... and does, with those streams' share left
constexpr int64_t kLowTokens = 128;
// Bytes that a forward call of the log probabilities holds for its alternatives.
constexpr int64_t kProbsBytes = int64_t(1) << 30;
constexpr int64_t kPieceMin = 8192;  // vocab rows: fewer would leave dW's launch short of tiles

// Tiles with the time a workgroup takes for 64 of K, in microseconds, when it has
// the chip to itself (loads' latency) and when every slot is taken, and per tile.
// Taken with loops that read, wait and multiply.  The loops pipelined in registers
// since are 1 to 10% faster, that of 256 x 256 bf16 tiles, by four waves, 17% (1.57 for
// 1.9); a three-part fp32 slab is counted as six bf16 ones, which it beats by some
// 20%.  Only the order of the shapes is used, and the first is put too low in it where it
// and the second lie close: with 1.57, forward and backward, 640 x 4096 x 128256 would take
// 2.55 ms for 2.77, 777 x 1536 x 50257 587 us for 600, 1100 x 1024 x 32000 348 for 367, and
// nothing measured longer.  (Another tile changes a call's last bits.)
struct TileCost {
    HeadTile tile;
    double alone, full, fixed;
};
constexpr TileCost kTiles[] = {
    {{256, 256}, 1.2, 1.9, 6.0}, {{256, 128}, 0.63, 1.09, 4.0}, {{256, 64}, 0.5, 1.05, 3.0}, {{64, 64}, 0.18, 0.54, 2.0}};

// Estimated microseconds of `tiles` tiles of `slabs` slabs each: rounds of the
// chip's slots.
double rounds_cost(const TileCost& c, int64_t tiles, double slabs) {
    const int64_t slots = head_slots(c.tile.tp);
    const double busy = std::min(1.0, (double)tiles / slots);
    return (double)ceil_div(tiles, slots) * (slabs * (c.alone + (c.full - c.alone) * busy) + c.fixed);
}

// The tile of a product with p rows of P, q of Q and K of `slabs` slabs.
HeadTile pick_tile(int64_t p, int64_t q, double slabs, int max_tq) {
    HeadTile best{256, max_tq};
    double least = 1e300;
    for (const TileCost& c : kTiles) {
        if (c.tile.tq > max_tq) continue;
        const double cost = rounds_cost(c, ceil_div(p, c.tile.tp) * ceil_div(q, c.tile.tq), slabs);
        if (cost < least) {
            least = cost;
            best = c.tile;
        }
    }
    return best;
}

// The same for the gradients: the K axis (dH: the vocabulary, dW: the tokens) is
// split until every slot of the chip has a tile; the splits' fp32 sums are written
// and read once more (dH's always are: they add up over the pieces).
HeadTile pick_split_tile(int64_t p, int64_t q, double slabs, int max_tq, bool sums_anyway, int64_t* splits) {
    HeadTile best{256, max_tq};
    double least = 1e300;
    for (const TileCost& c : kTiles) {
        if (c.tile.tq > max_tq) continue;
        const int64_t tiles = ceil_div(p, c.tile.tp) * ceil_div(q, c.tile.tq);
        const int64_t s = std::max<int64_t>(1, std::min<int64_t>(head_slots(c.tile.tp) / tiles, (int64_t)slabs));
        // at 4 TB/s, and a launch for dW
        const double sums = s > 1 || sums_anyway ? 8.0 * s * tiles * c.tile.tp * c.tile.tq / 4e6 + (sums_anyway ? 0 : 8) : 0;
        const double cost = rounds_cost(c, tiles * s, std::ceil(slabs / s)) + sums;
        if (cost < least) {
            least = cost;
            best = c.tile;
            *splits = s;
        }
    }
    return best;
}

}  // namespace

dmuon_status head_check_desc(const dmuon_head_desc* d) {
    if (d == nullptr) return DMUON_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->hidden < 1 || d->vocab < 1 || d->top_k < 0) return DMUON_ERR_INVALID_ARG;
    if (d->dtype != DMUON_BF16 && d->dtype != DMUON_F32) return DMUON_ERR_INVALID_ARG;
    if (d->tokens > kHeadMaxTokens || d->hidden > kHeadMaxHidden || d->vocab > kHeadMaxVocab ||
        d->top_k > kHeadMaxTopK || d->tokens > kHeadMaxLogits / d->vocab)
        return DMUON_ERR_UNSUPPORTED;
    return DMUON_OK;
}

HeadLayout head_layout_of(dmuon_head_desc d, bool backward, bool split_live) {
    HeadLayout L{};
    d.tokens = std::max<int64_t>(d.tokens, 1);
    L.tokens = d.tokens;
    L.hidden = d.hidden;
    L.vocab = d.vocab;
    L.top_k = d.top_k;
    L.planes = head_planes(d.dtype);
    L.esize = d.dtype == DMUON_BF16 ? 2 : 4;
    L.t_pad = std::max<int64_t>(round_up(d.tokens, kHeadTile), kHeadTile);
    L.d_pad = round_up(d.hidden, kHeadSlab);
    // bf16 rows of whole slabs are read in place; others go through a padded copy
    L.pack_weight = L.planes > 1 || d.hidden != L.d_pad;
    // ... unless tokens are few: then the copy costs more than what the stream kernels
    // lose per tile.  Measured (us, stream against copy): bf16 256 x 4090 x 50000
    // forward 314 / 443, 512 tokens 573 / 534; backward without dW 128 tokens 360 / 502,
    // 256 tokens 668 / 567; fp32 forward 256 tokens 883 / 1247, 512 x 1000 x 32000 219 /
    // 153; backward without dW 512 x 1000 x 32000 426 / 429, 256 x 4090 x 50000 1531 / 2171.
    const int64_t few = !backward ? 256 : L.planes > 1 ? 384 : 128;
    L.stream_weight = L.pack_weight && d.tokens <= few;
    if (L.stream_weight) L.pack_weight = 0;
    const int64_t v_pad = round_up(d.vocab, kHeadTile);
    const int64_t fit = kPieceBytes / (L.t_pad * 2 * L.planes) / kHeadTile * kHeadTile;
    int64_t piece = std::max(fit, kPieceMin);
    if (L.pack_weight) {  // ... and the copies of W's piece
        const int64_t w = (2 * kPieceBytes) / (L.d_pad * 2 * L.planes) / kHeadTile * kHeadTile;
        piece = std::min(piece, std::max(w, kPieceMin));
    }
    L.pieces = (int32_t)ceil_div(v_pad, piece);
    L.piece = round_up(ceil_div(v_pad, L.pieces), kHeadTile);
    L.pieces = (int32_t)ceil_div(v_pad, L.piece);
    const bool f32 = L.planes > 1;
    // one launch covers the vocabulary (forward, read in place) or a piece of it
    const int64_t s_rows = backward || L.pack_weight ? L.piece : v_pad;
    // bf16 batches of few tokens hold ds in two bf16 parts: a few entries' roundings
    // would not average out, and while W's bytes bound the call the further rows are
    // next to free.  By the tokens of the call, not by those with a loss: their number
    // is known on the device only, and the arrays and launches are laid out here.
    // Larger batches round ds to bf16 once: a second part would make dH and dW, half of
    // a training step's products, twice as many.  What it costs them, as the gradients'
    // relative error against 64 bits with the plain form's, which only rounds the
    // results: 8192 tokens 1.69e-3 (1.48e-3), distillation of 4096 tokens 2.34e-3
    // (1.66e-3), of 777 2.33e-3 (1.67e-3).
    L.low = backward && !f32 && d.tokens <= kLowTokens;
    const int64_t ds_rows = L.low ? 2 * head_low_row((int)d.tokens) : d.tokens;
    const int max_tq = L.stream_weight || L.low ? 128 : 256;
    const double s_slabs = (double)(L.d_pad / kHeadSlab) * (!f32 ? 1 : L.stream_weight ? 6 : 3);
    L.s_tile = pick_tile(std::min(s_rows, d.vocab), d.tokens, s_slabs, max_tq);
    const double parts = f32 ? 6 : 1;
    int64_t dw_splits = 1;
    L.dw_tile = pick_split_tile(d.hidden, std::min(L.piece, d.vocab), (double)ceil_div(ds_rows, kHeadSlab) * parts, 256,
                                false, &dw_splits);
    L.dw_splits = (int32_t)std::min(dw_splits, ceil_div(ds_rows, kHeadSlab));
    const int64_t k = round_up(std::min(L.piece, d.vocab), kHeadSlab);  // of the first, longest piece
    int64_t splits = 1;
    L.dh_tile = pick_split_tile(d.hidden, ds_rows, (double)(k / kHeadSlab) * parts, max_tq, true, &splits);
    L.split_k = round_up(ceil_div(k, std::min(splits, k / kHeadSlab)), kHeadSlab);
    L.splits = (int32_t)ceil_div(k, L.split_k);

    // ds is written past the caches, which the tiles of its operands are read from again.  Not
    // where dH, in 64 x 64 tiles for want of columns, is bound by reading ds, and ds stays in the
    // last-level cache.  Backward, us, written through the caches against past them: 2048 x 128 x
    // 50257 197 / 223, 1024 x 320 x 50257 201 / 224, 4096 x 64 x 30000 (236 MB of ds) 196 / 206; 4096 x
    // 64 x 32700 (256 MB) 229 / 221; with larger tiles 1024 x 320 x 120000 427 / 410, 8192 x 256 x
    // 128256 2482 / 2381.
    L.g_cached = backward && !f32 && L.dh_tile.tp == 64 && 2 * L.t_pad * L.piece <= kCachedBytes;
    // So is dW, but for rows that are not whole 128-byte lines: past the caches their ends are
    // written in parts.  What that takes shows where few tokens leave dW bound by its writes, and
    // the caches hold it.  Backward, us, through against past them: 16 x 1000 x 32000 69 / 75, 96 x 712 x
    // 50257 116 / 123, 48 x 1672 x 32000 118 / 126; 48 x 1416 x 50257 (142 MB) 147 / 145, 96 x 2760 x 32000
    // (177 MB) 248 / 227; whole lines 100 x 1024 x 32000 87 / 85.  Up to 256 tokens it shows while
    // less of the caches is dW's: 200 x 1000 x 32000 (64 MB) 97 / 103, 256 x 1112 x 32000 (71 MB) 119 / 121,
    // 200 x 1288 x 32000 (82 MB) 131 / 129, 200 x 1112 x 50257 (112 MB) 182 / 180.
    const int64_t dw_held = d.tokens <= kLowTokens ? int64_t(112) << 20 : d.tokens <= 256 ? int64_t(72) << 20 : 0;
    L.dw_cached = backward && !f32 && d.hidden % 64 != 0 && 2 * d.hidden * d.vocab <= dw_held;

    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = at;
        at += align_up((size_t)bytes);
        return o;
    };
    L.off_count = take(8);
    L.off_norm = take(4);
    L.off_src = take(4 * L.t_pad);
    L.off_tgt = take(4 * L.t_pad);
    L.off_lse = take(4 * L.t_pad);
    L.off_cp = take(4 * L.t_pad);
    L.off_ct = take(4 * L.t_pad);
    L.off_tl = take(4 * L.t_pad);
    L.off_q = take(8 * L.t_pad);
    L.off_flag = take(4 * L.t_pad);
    L.off_h = take(2 * L.planes * L.t_pad * L.d_pad);
    // a packed piece of W, or the copy of its last, partial tile
    if (!L.pack_weight && !L.stream_weight) L.off_w = take(2 * kHeadTile * L.d_pad);
    else if (L.pack_weight && (!f32 || backward)) L.off_w = take(2 * L.planes * L.piece * L.d_pad);
    if (f32 && L.pack_weight) {
        L.off_h2 = take(4 * L.t_pad * L.d_pad);
        L.off_hs = take(4 * L.t_pad);
        L.off_w2 = take(4 * L.piece * L.d_pad);
        L.off_ws = take(4 * L.piece);
        L.off_rh = take(8 * kHeadRangeBlocks);
        L.off_rw = take(8 * kHeadRangeBlocks);
    }
    if (backward) {
        L.off_g = take(2 * L.planes * L.t_pad * L.piece);
        // Tiles of rows that take no part leave slots empty, which only the device knows: with
        // room for twice the splits it fills them (8192 tokens, hidden 4096, 5734 of them
        // live: 368 tiles on 256 slots take two rounds, 736 of half the length three).  Backward
        // without dW, us, against the splits of all rows: 8192 x 4096 x 128256, 30% dead 10201 /
        // 11098, 40% 8969 / 10199, 90% 1862 / 3272, none 13460 / 13456.  Calls of
        // so many tiles that a round is a small part keep theirs; so do the losses, whose
        // results would round differently.
        int64_t splits_held = L.splits;
        const int64_t dh_tiles = ceil_div(L.hidden, kHeadTile) * (L.t_pad / kHeadTile);
        if (split_live && !f32 && L.dh_tile.tq == kHeadTile && dh_tiles * L.splits <= 4 * head_slots(kHeadTile)) {
            splits_held = 2 * L.splits;
            L.dh_room = (int32_t)(splits_held * dh_tiles);
        }
        L.off_dh = take(4 * splits_held * L.t_pad * round_up(L.hidden, kHeadTile));
        if (L.dw_splits > 1) L.off_dw = take(4 * L.dw_splits * L.piece * round_up(L.hidden, kHeadTile));
    } else {
        // Distillation needs K logits a token.  Dots of H's rows with the gathered rows of W
        // read K hidden elements of W a token; written out and gathered, the logits cost 4
        // bytes each and some: the cheaper one, as long as they stay a small buffer.
        const int64_t kept = 4 * L.t_pad * v_pad;
        L.keep_logits = L.top_k > 0 && kept <= kPieceBytes && (int64_t)L.top_k * L.hidden * L.esize > 5 * v_pad;
        if (L.keep_logits) L.off_logits = take(kept);
        L.off_part = take(8 * (v_pad / L.s_tile.tp) * head_wave_rows(L.s_tile.tp, L.s_tile.tq) * L.t_pad);
    }
    L.bytes = at;
    return L;
}

dmuon_status probs_check_desc(const dmuon_head_desc* d, bool backward) {
    const dmuon_status st = head_check_desc(d);
    if (st != DMUON_OK) return st;
    if (backward ? d->top_k != 0 : d->top_k > d->vocab) return DMUON_ERR_INVALID_ARG;
    return d->top_k > kHeadMaxAlternatives ? DMUON_ERR_UNSUPPORTED : DMUON_OK;
}

namespace {

// Alternatives come from the largest logit of every group of 16 words, which the
// products' epilogue leaves (8 bytes a group); where a row's alternatives share a group, the
// group's other logits are formed again.  With K alternatives spread over V / 16 groups that are
// 8 K^2 / V groups: from one in eight alternatives on, the logits themselves are kept.
bool probs_keep(const dmuon_head_desc& d) { return d.top_k > 0 && d.vocab < 64 * (int64_t)d.top_k; }

}  // namespace

int64_t probs_chunk(const dmuon_head_desc& d) {
    if (d.top_k == 0) return std::max<int64_t>(d.tokens, 1);
    const int64_t v_pad = round_up(d.vocab, kHeadTile), row = probs_keep(d) ? 4 * v_pad : v_pad / 2;
    return std::max<int64_t>(kProbsBytes / row / kHeadTile, 1) * kHeadTile;
}

ProbsLayout probs_layout_of(const dmuon_head_desc& d, bool backward) {
    ProbsLayout L{};
    dmuon_head_desc h = d;
    h.top_k = 0;
    L.head = head_layout_of(h, backward, true);
    // Few rows read W at the rate of the memory, which a last round of the chip's slots that is
    // not full costs less than the tiles' rule counts: 256 x 64 tiles wherever each slot has one.
    // Against 64 x 64, us: 40 x 3584 x 152064, 20 alternatives, 249 / 274; 16 x 5120 x 151936
    // 334 / 380; with half of the slots taken 64 x 2048 x 32000 63 / 57.
    // (Fewer parts a row than of 64 x 64: the arrays hold them.)
    if (!backward && L.head.planes == 1 && !L.head.stream_weight && d.tokens <= 64 && L.head.s_tile.tp == 64 &&
        ceil_div(d.vocab, 256) >= head_slots(256))
        L.head.s_tile = HeadTile{256, 64};
    size_t at = L.head.bytes;
    auto take = [&](int64_t bytes) {
        const size_t o = at;
        at += align_up((size_t)bytes);
        return o;
    };
    const int64_t v_pad = round_up(d.vocab, kHeadTile), t_pad = L.head.t_pad;
    const HeadTile s = L.head.s_tile;
    L.keep_logits = !backward && probs_keep(d);
    if (backward) {
        L.off_ce = take(4 * t_pad);
    } else {
        // a row's parts and groups lie together: one workgroup reads them
        L.row_parts = (v_pad / s.tp) * head_wave_rows(s.tp, s.tq);
        L.row_groups = v_pad / 16;
        L.off_part_e = take(4 * L.row_parts * t_pad);
        if (L.keep_logits) L.off_logits = take(4 * t_pad * v_pad);
        else if (d.top_k > 0) L.off_top = take(v_pad / 2 * t_pad);
    }
    L.bytes = at;
    return L;
}

}  // namespace dmuon
