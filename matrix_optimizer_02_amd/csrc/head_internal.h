// Internal types of the output-head losses: the kernels' arguments and launchers
// (k_head_gemm.hip, k_head_rows.hip, head.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "head_layout.h"

namespace dmuon {

// Parts of an operand element (fp32 operands of dH and dW: three bf16 parts).
enum HeadKind : int32_t {
    kHeadBf16 = 0,    // as it is
    kHeadHalf2 = 1    // fp32 as two fp16 parts, rows scaled (logits)
};

// One launch of tile products: C[r][c] = sum over k of P[r][k] Q[c][k].
enum HeadMode : int32_t {
    kHeadLse = 0,   // P = W rows, Q = H rows: softmax statistics of each tile (and the targets' logits)
    kHeadGrad = 1,  // P = W rows, Q = H rows: ds as bf16 parts
    kHeadDh = 2,    // P = W (k = vocab rows, columns of hidden), Q = ds rows: fp32 sums, added per piece
    kHeadDw = 3,    // P = H (k = tokens, columns of hidden), Q = ds (k = tokens, columns of vocab): dW rows
    kHeadDwSum = 4  // the same in splits of the tokens: fp32 sums
};

struct HeadGemmArgs {
    const int32_t* count;        // token rows that carry a loss (dH, dW: rows of ds)
    const char* p;               // P operand of this piece
    const char* p_tail;          // a zero-padded copy of the last, partial vocab tile ...
    int32_t tail_row;            // ... which stands for P rows >= tail_row of this piece (INT32_MAX: none)
    const char* q;
    int64_t p_plane, q_plane;    // bytes between the parts of an operand
    const float *p_scale, *q_scale;  // fp32 logits: what the rows' products are multiplied by
    const float2 *p_range, *q_range; // stream kernels: run only where two fp16 parts do not hold these ranges (null: run)
    int32_t p_ranges, q_ranges;
    int32_t p_ld, q_ld;          // elements between rows
    int64_t p_rows;              // rows of W left from the piece's first (stream kernels)
    int32_t parts;               // 1: bf16; 3: fp32
    int32_t k;                   // K extent (dH: of the piece; dW: taken from count)
    int32_t split_k, splits;     // dH: K of a split; DwSum: splits of the tokens
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
    float* logits;               // Lse: the logits too (row stride logits_ld), or null
    int32_t logits_ld;
    const float* lse;            // per compact row
    const float* cp;             // coefficient of p
    const float* ct;             // coefficient at the target
    const float* norm;           // the largest coefficient: ds is held as multiples of it
    int32_t low;                 // Grad: the rows' low parts go to head_low_row(n) rows further
    char* g;                     // ds out
    int64_t g_plane;             // bytes
    int32_t g_ld;
    float* sums;                 // fp32 sums (dH; dW in splits), tile by tile in the accumulators' own order
    int32_t accumulate;          // dH: add to what earlier pieces left
    void* dw;                    // dW out (row v0 of it is at dw)
    int64_t dw_rows;             // rows of dW left from v0
    int32_t dw_ld;               // hidden
};

hipError_t launch_head_gemm(int mode, HeadTile tile, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream);
// ... dH and dW of fp32 operands (k_head_x3.hip).
hipError_t launch_head_x3(int mode, HeadTile tile, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream);
// The same with W read in place whatever its width and type (Lse, Grad, dH;
// tiles 256 x 128, 256 x 64 and 64 x 64).
hipError_t launch_head_stream(int mode, HeadTile tile, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream);

// ---- row kernels (k_head_rows.hip) ---------------------------------------------

struct HeadTeacher {
    const int64_t* ids;
    const float* logits;
    int32_t k;
    int64_t vocab;
    float inv_temp;
};
// Per token: (largest z, log sum of exp((z - it) / T)) of the teacher in q (NaN for a bad id), the
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
    int32_t* count;          // the rows, then the rows of ds
    int32_t low;
    float* norm;             // zeroed
    int32_t* src;
    int32_t* target;
    float* losses;
    float* lse;
};
// Up to this many tokens the launch that packs the rows finds them too.
constexpr int kScanTokens = 1024;
// Rows of a matrix to its operand parts, rows of ld elements: row r of the output
// is row src[r] of the input (W: row r) below the row count, zero above up to
// out_rows or a whole tile.
struct HeadPackArgs {
    const void* in;
    int64_t cols;
    int64_t rows;          // W: rows of the input
    uint16_t* out;         // bf16: the rows; fp32: three bf16 parts (null: not)
    int64_t out_rows, ld, plane;  // plane in elements
    int32_t low;           // 1: every row again, head_low_row(count) rows further
    uint16_t* half2;       // fp32: 32 hi, 32 lo fp16 values of every 32 columns, rows of 2 ld
    float* scale;          // ... and the factor that restores a row's scale
    float2* range;         // ... and per block the largest element and the largest sum of magnitudes of a row
};
// Distillation: the student's logits at the teacher's ids.
struct HeadStudentArgs {
    const int32_t* count;
    const int32_t* src;
    HeadTeacher t;
    const void* hidden;
    const void* weight;
    int32_t esize;
    int64_t cols;
    float* student;
    int64_t tokens;
};
hipError_t launch_head_student(const HeadStudentArgs& a, hipStream_t stream);
// Joins the tiles' softmax statistics: the caller's lse and losses.
struct HeadMergeArgs {
    const int32_t* count;
    const int32_t* src;
    const float2* part;
    int64_t t_pad;
    int32_t parts;
    int64_t tokens;
    float inv_temp, temp;
    const int32_t* target;      // cross entropy, else null
    const float* target_logit;
    HeadTeacher t;              // distillation
    const float2* q;
    float* student;
    const float* logits;        // distillation: the logits themselves (written to student), or null
    int64_t logits_ld;
    float* losses;
    float* lse;
};
hipError_t launch_head_merge(const HeadMergeArgs& a, hipStream_t stream);
// Backward coefficients per compact row (zero in the padding).
struct HeadCoefArgs {
    const float2* q;        // distillation, else null
    const float* lse;
    const float* grad_losses;
    const float* grad_lse;  // or null
    float temp;
    float *lse_c, *cp, *ct;
    float* norm;            // the largest |cp|, |ct|, within 2^100 either way
    int64_t t_pad;
};
// The rows that carry a loss (rows.tokens 0: found before), then up to three
// independent jobs: those rows packed, W packed (out_rows 0: not) and the
// coefficients (t_pad 0: not).
struct HeadPrepareArgs {
    HeadRowsArgs rows;
    HeadPackArgs h, w;
    HeadCoefArgs coef;
    int32_t esize;
    int32_t h_blocks, w_blocks, coef_blocks;  // set by the launcher
};
hipError_t launch_head_prepare(const HeadPrepareArgs& a, hipStream_t stream);
// Distillation: ds at the teacher's ids inside one piece.
struct HeadFixArgs {
    const int32_t* count;
    const int32_t* src;
    HeadTeacher t;
    const float2* q;
    const float* student;
    const float* lse_c;
    const float* cp;
    const float* norm;
    int32_t low;
    uint16_t* g;
    int64_t g_plane;  // elements
    int64_t g_ld;
    int32_t planes;
    int64_t v0, v1;
    int64_t tokens;
};
hipError_t launch_head_fix(const HeadFixArgs& a, hipStream_t stream);
// dH (or dW) from the fp32 tile sums: splits added in order, rows scattered to
// their tokens, zeros for rows without a loss.
struct HeadSumArgs {
    const int32_t* count;  // null: rows
    int64_t rows;          // rows of the output
    const int32_t* src;    // null: in place
    const float* norm;
    int32_t low;
    const float* sums;
    int32_t splits;
    int32_t tiles_i;
    HeadTile tile;
    void* out;
    int32_t esize;
    int64_t cols;
};
hipError_t launch_head_sum(const HeadSumArgs& a, hipStream_t stream);
hipError_t launch_head_zero(void* p, int64_t bytes, hipStream_t stream);

}  // namespace dmuon
