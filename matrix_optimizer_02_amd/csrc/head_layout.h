// Sizes of the output-head losses, the shapes of their tiles and how a call is cut:
// host C++ without any HIP, shared by the entry points (head.hip), the kernels and
// the host tests.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/dmuon_head.h"
#include "dmuon_internal.h"

namespace dmuon {

constexpr int64_t kHeadMaxTokens = (int64_t(1) << 24) - 1;
constexpr int64_t kHeadMaxHidden = 65536;
constexpr int64_t kHeadMaxVocab = (int64_t(1) << 27) - 1;
constexpr int32_t kHeadMaxTopK = 1024;
constexpr int32_t kHeadMaxAlternatives = 128;
constexpr int64_t kHeadMaxLogits = int64_t(1) << 42;  // tokens x vocab: keeps every launch's tile count in 31 bits

constexpr int kHeadTile = 256;  // every tile edge divides it: arrays are padded to it
constexpr int kHeadSlab = 64;   // K slab
constexpr int kHeadMaxPlanes = 3;

// bf16 parts of the gradients' operands: 1 (bf16) or 3 (fp32).
inline int head_planes(int32_t dtype) { return dtype == DMUON_BF16 ? 1 : kHeadMaxPlanes; }

// First row of the low parts of ds behind n token rows.
#if defined(__HIPCC__)
__host__ __device__
#endif
inline int head_low_row(int n) { return n <= kHeadSlab ? kHeadSlab : (n + kHeadSlab - 1) / kHeadSlab * kHeadSlab; }

// An output tile: tp rows of P by tq rows of Q.
struct HeadTile {
    int32_t tp, tq;
};
constexpr int head_waves(int tp) { return tp == 64 ? 4 : 8; }
// Waves along a tile's P rows: rows of statistics written per vocab tile.
constexpr int head_wave_rows(int tp, int tq) { return tp == 64 || tq == 256 ? 2 : 4; }
// Workgroups the chip holds at once (two of the 64 x 64 tiles' to a CU).
constexpr int head_slots(int tp) { return tp == 64 ? 512 : 256; }

// Blocks that pack rows as two fp16 parts, at most: each leaves the largest element
// and the largest sum of magnitudes of its rows.
constexpr int kHeadRangeBlocks = 8192;
inline int head_range_blocks(int64_t rows) {
    const int64_t b = (rows + 3) / 4;  // a wave a row
    return (int)(b < kHeadRangeBlocks ? b : kHeadRangeBlocks);
}

// Where everything lies in the workspace, and how the work is cut.
struct HeadLayout {
    int64_t tokens, hidden, vocab;
    int32_t top_k, planes, esize;
    HeadTile s_tile, dh_tile, dw_tile;  // of the logits, dH and dW
    int64_t t_pad;          // token rows of the padded arrays (multiple of 256)
    int64_t d_pad;          // K extent of packed rows (multiple of 64)
    int32_t pack_weight;    // 1: pieces of W are copied (split) into the workspace
    int32_t stream_weight;  // 1: the stream kernels read W in place
    int32_t low;            // 1: ds in two bf16 parts, the low ones as further token rows
    int64_t piece;          // vocab rows of a piece (multiple of 256)
    int32_t pieces;
    int64_t split_k;        // dH: vocab rows of a split (multiple of 64)
    int32_t splits;         // ... splits of a full piece
    int32_t dh_room;        // tiles that the sums of dH hold, where the device chooses the splits (else 0)
    int32_t g_cached, dw_cached;  // 256 x 256 tiles of bf16 ds, of dW, are written through the caches
    int32_t dw_splits;      // dW: splits of the tokens
    int32_t keep_logits;    // distillation, small vocabularies: see head_layout.cpp
    // byte offsets
    size_t off_count, off_norm, off_src, off_tgt, off_lse, off_cp, off_ct, off_tl, off_q, off_flag;
    size_t off_h, off_w, off_part, off_g, off_dh, off_dw, off_logits;
    size_t off_h2, off_w2, off_hs, off_ws;  // fp32: the logits' operands and their row scales
    size_t off_rh, off_rw;                  // ... and ranges (kHeadRangeBlocks pairs each)
    size_t bytes;
};

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t x, int64_t a) { return (x + a - 1) / a; }

// Splits of dH's K, of `slabs` slabs, for so many tiles of 256 x 256 in an array that holds
// `room` of them: the fewest rounds of the chip's slots.  A round's sums are written, and
// read to be added to, at what kHeadSumSlabs slabs take.
constexpr int kHeadSumSlabs = 20, kHeadMostSplits = 16;
constexpr int head_dh_splits(int tiles, int slabs, int room) {
    int best = 1, least = INT32_MAX;
    for (int s = 1; s <= kHeadMostSplits && s <= slabs && s * tiles <= room; ++s) {
        const int cost = ((s * tiles + 255) / 256) * ((slabs + s - 1) / s + kHeadSumSlabs);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// INVALID_ARG or UNSUPPORTED for sizes out of range.
dmuon_status head_check_desc(const dmuon_head_desc* d);
// The cut of one call (a descriptor that head_check_desc accepts).  With split_live the
// device cuts dH's K by the rows that take part (dh_room).
HeadLayout head_layout_of(dmuon_head_desc d, bool backward, bool split_live = false);

// The log probabilities: arrays beside those of a head loss.  The forward call takes a
// chunk of the tokens at a time.
struct ProbsLayout {
    HeadLayout head;
    int32_t keep_logits;  // forward: the logits lie in memory
    int64_t row_parts, row_groups;  // of a row (row_parts even: pairs of groups are 16-byte aligned)
    size_t off_logits;
    size_t off_part_e;    // forward otherwise: sums for the entropy, the groups' largest
    size_t off_top;
    size_t off_ce;      // backward
    size_t bytes;
};
// INVALID_ARG or UNSUPPORTED for sizes out of range.
dmuon_status probs_check_desc(const dmuon_head_desc* d, bool backward);
// Tokens of a forward call's chunk, and the cut of one of d.tokens <= that (or of a
// whole backward call).
int64_t probs_chunk(const dmuon_head_desc& d);
ProbsLayout probs_layout_of(const dmuon_head_desc& d, bool backward);

}  // namespace dmuon
