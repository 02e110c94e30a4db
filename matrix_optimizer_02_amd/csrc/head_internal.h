// Internal types of the output-head losses: the workspace layout and the
// kernels' launchers (k_head_gemm.hip, k_head_rows.hip, head.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/dmuon_head.h"
#include "dmuon_internal.h"

namespace dmuon {

constexpr int64_t kHeadMaxTokens = (int64_t(1) << 24) - 1;
constexpr int64_t kHeadMaxHidden = 65536;
constexpr int64_t kHeadMaxVocab = (int64_t(1) << 27) - 1;
constexpr int32_t kHeadMaxTopK = 1024;
constexpr int64_t kHeadMaxLogits = int64_t(1) << 42;  // tokens x vocab: keeps every launch's tile count in 31 bits

constexpr int kHeadTile = 256;  // rows of the P operand a tile covers (vocab, or hidden columns)
constexpr int kHeadSlab = 64;   // K slab
constexpr int kHeadMinK = 128;  // K extents are padded to at least two slabs
constexpr int kHeadMaxPlanes = 3;

// bf16 parts of an operand element: 1 (bf16) or 3 (fp32).
inline int head_planes(int32_t dtype) { return dtype == DMUON_BF16 ? 1 : kHeadMaxPlanes; }

// Where everything lies in the workspace, and how the work is cut.
struct HeadLayout {
    int64_t tokens, hidden, vocab;
    int32_t top_k, planes, esize;
    int32_t tq;             // token rows a tile of the logits covers (64 or 256)
    int64_t t_pad;          // token rows of the padded arrays (multiple of 256)
    int64_t d_pad;          // K extent of packed rows (multiple of 64, >= 128)
    int32_t pack_weight;    // 1: pieces of W are copied (split) into the workspace
    int64_t piece;          // vocab rows of a piece (multiple of 256)
    int32_t pieces;
    int64_t split_k;        // dH: vocab rows of a split (multiple of 128)
    int32_t splits;         // ... splits of a full piece
    // byte offsets
    size_t off_count, off_src, off_tgt, off_lse, off_cp, off_ct, off_tl, off_q, off_flag;
    size_t off_h, off_w, off_part, off_g, off_dh;
    size_t bytes;
};

// One launch of tile products: C[r][c] = sum over k of P[r][k] Q[c][k].
enum HeadMode : int32_t {
    kHeadLse = 0,   // P = W rows, Q = H rows: softmax statistics of each tile (and the targets' logits)
    kHeadGrad = 1,  // P = W rows, Q = H rows: ds as bf16 parts
    kHeadDh = 2,    // P = W (k = vocab rows, columns of hidden), Q = ds rows: fp32 sums, added per piece
    kHeadDw = 3     // P = H (k = tokens, columns of hidden), Q = ds (k = tokens, columns of vocab): dW rows
};

struct HeadGemmArgs {
    const int32_t* count;        // token rows that carry a loss
    const char* p;               // P operand of this piece
    const char* p_tail;          // a zero-padded copy of the last, partial vocab tile ...
    int32_t tail_row;            // ... which stands for P rows >= tail_row of this piece (INT32_MAX: none)
    const char* q;
    int64_t p_plane, q_plane;    // bytes between the parts of an operand
    int32_t p_ld, q_ld;          // elements between rows
    int32_t parts;               // bf16 parts of the operands: 1, or 3 (six products)
    int32_t k;                   // K extent (dH: of the piece; dW: taken from count)
    int32_t split_k, splits;     // dH
    int32_t tiles_i;             // tiles along P's rows (or columns)
    int32_t tiles_j;             // tiles along Q's (dW: vocab); else from count
    // softmax
    int64_t v0;                  // first vocab row of the piece
    int64_t vocab;
    float inv_temp;
    const int32_t* target;       // per compact row (cross entropy; else null)
    float2* part;                // statistics: part[(tile * WR + wr) * t_pad + row]
    int64_t t_pad;
    int32_t first_tile;          // vocab tile index of the piece's first tile
    float* target_logit;
    const float* lse;            // per compact row
    const float* cp;             // coefficient of p
    const float* ct;             // coefficient at the target
    char* g;                     // ds out
    int64_t g_plane;             // bytes
    int32_t g_ld;
    float* dh;                   // fp32 sums, tile by tile in the accumulators' own order
    int32_t accumulate;          // dH: add to what earlier pieces left
    void* dw;                    // dW out (row v0 of it is at dw)
    int64_t dw_rows;             // rows of dW left from v0
    int32_t dw_ld;               // hidden
};

hipError_t launch_head_gemm(int mode, int tq, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream);
// Waves along a tile's P rows: statistics rows written per vocab tile.
inline int head_wave_rows(int tq) { return tq == 256 ? 2 : 4; }

// ---- row kernels (k_head_rows.hip) ---------------------------------------------

struct HeadTeacher {
    const int64_t* ids;
    const float* logits;
    int32_t k;
    int64_t vocab;
    float inv_temp;
};
// Per token: (max, log sum) of the teacher's z / T in q (NaN for a bad id), the
// flag that the row carries a loss; zeros student_logits (null: not).
hipError_t launch_head_teacher(const HeadTeacher& t, int64_t tokens, float2* q, int32_t* flag, float* student,
                               hipStream_t stream);
// The rows that carry a loss: count, src (a permutation of the tokens, those
// rows first, in order) and, for cross entropy, each one's target (-1 in the
// padding, -2 where out of range); zeros losses and lse (null: not) of the others.
struct HeadRowsArgs {
    const int64_t* targets;  // null: flag decides
    const int32_t* flag;
    int64_t ignore_index, vocab;
    int32_t tokens, t_pad;
    int32_t* count;
    int32_t* src;
    int32_t* target;
    float* losses;
    float* lse;
};
hipError_t launch_head_rows(const HeadRowsArgs& a, hipStream_t stream);
// Rows of a rows x cols matrix to bf16 parts with rows of ld elements: row r of
// the output is row src[r] (src null: r) for r < limit (limit from device memory
// when given), zero above up to out_rows.
struct HeadPackArgs {
    const void* in;
    int32_t esize;
    int64_t cols;
    const int32_t* src;
    const int32_t* count;  // device row count, or null:
    int64_t rows;          // rows of the input
    uint16_t* out;
    int64_t out_rows, ld, plane;  // plane in elements
    int32_t planes;
};
hipError_t launch_head_pack(const HeadPackArgs& a, hipStream_t stream);
// Joins the tiles' softmax statistics: lse (compact, natural units) and, for
// cross entropy, losses and lse of the caller.
struct HeadMergeArgs {
    const int32_t* count;
    const int32_t* src;
    const float2* part;
    int64_t t_pad;
    int32_t parts;
    int64_t tokens;
    float inv_temp;
    const int32_t* target;      // cross entropy, else null
    const float* target_logit;
    float* lse_c;
    float* losses;              // cross entropy
    float* lse;
};
hipError_t launch_head_merge(const HeadMergeArgs& a, hipStream_t stream);
// Distillation: the student's logits at the teacher's ids and the losses.
struct HeadStudentArgs {
    const int32_t* count;
    const int32_t* src;
    HeadTeacher t;
    const float2* q;
    const void* hidden;
    const void* weight;
    int32_t esize;
    int64_t cols;
    const float* lse_c;
    float temp;
    float* student;
    float* losses;
    int64_t tokens;
};
hipError_t launch_head_student(const HeadStudentArgs& a, hipStream_t stream);
// Backward coefficients per compact row (zero in the padding).
struct HeadCoefArgs {
    const int32_t* count;
    const int32_t* src;
    const int32_t* target;  // cross entropy, else null
    const float2* q;        // distillation, else null
    const float* lse;
    const float* grad_losses;
    const float* grad_lse;  // or null
    float temp;
    float *lse_c, *cp, *ct;
    int64_t t_pad;
};
hipError_t launch_head_coef(const HeadCoefArgs& a, hipStream_t stream);
// Distillation: ds at the teacher's ids inside one piece.
struct HeadFixArgs {
    const int32_t* count;
    const int32_t* src;
    HeadTeacher t;
    const float2* q;
    const float* student;
    const float* lse_c;
    const float* cp;
    uint16_t* g;
    int64_t g_plane;  // elements
    int64_t g_ld;
    int32_t planes;
    int64_t v0, v1;
    int64_t tokens;
};
hipError_t launch_head_fix(const HeadFixArgs& a, hipStream_t stream);
// dH from the fp32 tile sums: splits added in order, rows scattered to their
// tokens, zeros for rows without a loss.
struct HeadDhArgs {
    const int32_t* count;
    const int32_t* src;
    const float* dh;
    int32_t splits;
    int32_t tiles_i;
    int32_t tq;
    void* out;
    int32_t esize;
    int64_t tokens, cols;
};
hipError_t launch_head_dh(const HeadDhArgs& a, hipStream_t stream);
hipError_t launch_head_zero(void* p, int64_t bytes, hipStream_t stream);

}  // namespace dmuon
