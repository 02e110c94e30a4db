// Entry points of the output-head losses: argument checks and the launch sequences
// (head_layout.cpp: tiles, splits and the workspace)
//   forward   (teacher) rows -> pack H -> [pack W piece ->] tile statistics -> join
//             (-> student logits and loss)
//   backward  (teacher) rows -> pack H, coefficients -> per piece of the
//             vocabulary: [pack W piece,] ds, (teacher's ids,) dH sums, dW -> dH
// fp32 with W packed: behind statistics and ds the same from three bf16 parts, by a
// launch that returns at once unless a row's range needs it (launch_logits).
// No device memory is allocated and nothing is synchronised.  The number of
// rows that carry a loss stays on the device: the launches are sized for every
// token and their workgroups read it.
#include <algorithm>
#include <climits>
#include <cmath>
#include <new>
#include <vector>

#include "head_internal.h"

using namespace dmuon;

namespace {

struct Span {
    uintptr_t lo, hi;
    bool written;
};

// Non-null, aligned, and no written buffer overlapping another one.
struct Buffers {
    std::vector<Span> spans;
    bool ok = true;
    void add(const void* p, int64_t bytes, bool written) {
        if (bytes == 0) return;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (p == nullptr || (a & 15u) != 0) ok = false;
        spans.push_back({a, a + (uintptr_t)bytes, written});
    }
    bool good() const {
        if (!ok) return false;
        for (size_t i = 0; i < spans.size(); ++i)
            for (size_t j = 0; j < i; ++j)
                if ((spans[i].written || spans[j].written) && spans[i].lo < spans[j].hi && spans[j].lo < spans[i].hi)
                    return false;
        return true;
    }
};

struct Call {
    const dmuon_head_desc* desc;
    const void* hidden;
    const void* weight;
    const int64_t* targets;  // cross entropy
    int64_t ignore_index;
    const int64_t* ids;      // distillation
    const float* teacher;
    float temp;
    void* workspace;
    size_t workspace_bytes;
    hipStream_t stream;
};

dmuon_status check_call(const Call& c, bool distill, Buffers& b) {
    const dmuon_status st = head_check_desc(c.desc);
    if (st != DMUON_OK) return st;
    const dmuon_head_desc& d = *c.desc;
    if (distill ? d.top_k < 1 : d.top_k != 0) return DMUON_ERR_INVALID_ARG;
    // the losses are multiplied by T^2, the logits by 1 / T
    if (distill && !(c.temp > 0.f && std::isnormal(c.temp * c.temp))) return DMUON_ERR_INVALID_ARG;
    const int64_t e = d.dtype == DMUON_BF16 ? 2 : 4;
    b.add(c.hidden, d.tokens * d.hidden * e, false);
    b.add(c.weight, d.vocab * d.hidden * e, false);
    if (distill) {
        b.add(c.ids, 8 * d.tokens * d.top_k, false);
        b.add(c.teacher, 4 * d.tokens * d.top_k, false);
    } else {
        b.add(c.targets, 8 * d.tokens, false);
    }
    return DMUON_OK;
}

dmuon_status check_rest(const Call& c, const HeadLayout& L, Buffers& b) {
    if (!b.good()) return DMUON_ERR_INVALID_ARG;
    if (c.workspace == nullptr || (reinterpret_cast<uintptr_t>(c.workspace) & (kAlign - 1)) != 0 ||
        c.workspace_bytes < L.bytes)
        return DMUON_ERR_WORKSPACE;
    b.add(c.workspace, (int64_t)L.bytes, true);
    return b.good() ? DMUON_OK : DMUON_ERR_INVALID_ARG;
}

#define HEAD_TRY(X)                                  \
    do {                                             \
        if ((X) != hipSuccess) return DMUON_ERR_HIP; \
    } while (0)

// The arrays of the workspace.
struct Views {
    char* ws;
    const HeadLayout& L;
    template <typename T>
    T* at(size_t off) const {
        return reinterpret_cast<T*>(ws + off);
    }
    int32_t* count() const { return at<int32_t>(L.off_count); }
    float* norm() const { return at<float>(L.off_norm); }
    int32_t* src() const { return at<int32_t>(L.off_src); }
    int32_t* target() const { return at<int32_t>(L.off_tgt); }
    float* lse() const { return at<float>(L.off_lse); }
    float* cp() const { return at<float>(L.off_cp); }
    float* ct() const { return at<float>(L.off_ct); }
    float* target_logit() const { return at<float>(L.off_tl); }
    float2* q() const { return at<float2>(L.off_q); }
    int32_t* flag() const { return at<int32_t>(L.off_flag); }
};

HeadTeacher teacher_of(const Call& c) {
    return HeadTeacher{c.ids, c.teacher, c.desc->top_k, c.desc->vocab, 1.f / c.temp};
}

// W's rows v0 .. v0 + rows - 1 to be packed (all parts a backward call needs).
HeadPackArgs pack_weight(const Call& c, const Views& v, bool backward, int64_t v0, int64_t rows) {
    const HeadLayout& L = v.L;
    HeadPackArgs p{};
    p.in = static_cast<const char*>(c.weight) + v0 * L.hidden * L.esize;
    p.cols = L.hidden;
    p.rows = rows;
    p.out_rows = round_up(rows, kHeadTile);
    p.out = L.planes == 1 || backward ? v.at<uint16_t>(L.off_w) : nullptr;
    p.ld = L.d_pad;
    p.plane = L.piece * L.d_pad;
    p.half2 = v.at<uint16_t>(L.off_w2);
    p.scale = v.at<float>(L.off_ws);
    if (L.planes > 1) p.range = v.at<float2>(L.off_rw);
    return p;
}

// Which rows carry a loss; then their hidden states packed together, the first
// piece of W (or its last, partial tile, where it is read in place) and, where
// given, the coefficients of the gradient.
dmuon_status gather_rows(const Call& c, const Views& v, float* losses, float* lse, float* student,
                         const HeadCoefArgs* coef) {
    const HeadLayout& L = v.L;
    const bool backward = coef != nullptr;
    if (c.ids != nullptr) HEAD_TRY(launch_head_teacher(teacher_of(c), L.tokens, v.q(), v.flag(), student, c.stream));
    HeadPrepareArgs a{};
    a.esize = L.esize;
    a.rows.targets = c.ids != nullptr ? nullptr : c.targets;
    a.rows.flag = v.flag();
    a.rows.ignore_index = c.ignore_index;
    a.rows.vocab = L.vocab;
    a.rows.tokens = (int32_t)L.tokens;
    a.rows.t_pad = (int32_t)L.t_pad;
    a.rows.count = v.count();
    a.rows.low = L.low;
    a.rows.norm = v.norm();
    a.rows.src = v.src();
    a.rows.target = v.target();
    a.rows.losses = losses;
    a.rows.lse = lse;
    a.h.in = c.hidden;
    a.h.cols = L.hidden;
    a.h.out = v.at<uint16_t>(L.off_h);
    a.h.low = L.low;
    a.h.out_rows = L.t_pad;
    a.h.ld = L.d_pad;
    a.h.plane = L.t_pad * L.d_pad;
    a.h.half2 = L.pack_weight ? v.at<uint16_t>(L.off_h2) : nullptr;
    a.h.scale = v.at<float>(L.off_hs);
    if (L.planes > 1 && L.pack_weight) a.h.range = v.at<float2>(L.off_rh);
    const int64_t tail = L.vocab % kHeadTile;
    if (L.pack_weight) a.w = pack_weight(c, v, backward, 0, std::min(L.piece, L.vocab));
    else if (!L.stream_weight && tail != 0) a.w = pack_weight(c, v, backward, L.vocab - tail, tail);
    if (coef != nullptr) a.coef = *coef;
    HEAD_TRY(launch_head_prepare(a, c.stream));
    return DMUON_OK;
}

// vocab rows [v0, v0 + rows) of W as the products' P operand: in place, with
// the last partial tile copied, or packed (the first piece by gather_rows).
dmuon_status weight_piece(const Call& c, const Views& v, bool backward, int64_t v0, int64_t rows, HeadGemmArgs& a) {
    const HeadLayout& L = v.L;
    const int64_t left = std::min(rows, L.vocab - v0);  // real rows
    a.tail_row = INT_MAX;
    a.p_rows = left;
    if (L.pack_weight) {
        if (v0 > 0) {
            HeadPrepareArgs p{};
            p.esize = L.esize;
            p.w = pack_weight(c, v, backward, v0, left);
            HEAD_TRY(launch_head_prepare(p, c.stream));
        }
        a.p = v.ws + L.off_w;
        a.p_plane = 2 * L.piece * L.d_pad;
        a.p_ld = (int32_t)L.d_pad;
        return DMUON_OK;
    }
    a.p = static_cast<const char*>(c.weight) + v0 * L.hidden * L.esize;
    a.p_ld = (int32_t)L.hidden;
    if (!L.stream_weight && left % kHeadTile != 0) {
        a.tail_row = (int32_t)(left / kHeadTile * kHeadTile);
        a.p_tail = v.ws + L.off_w;
    }
    return DMUON_OK;
}

void logits_args(const Call& c, const Views& v, int64_t v0, int64_t rows, HeadGemmArgs& a) {
    const HeadLayout& L = v.L;
    a.count = v.count();
    a.q = v.ws + L.off_h;
    a.q_ld = (int32_t)L.d_pad;
    a.q_plane = 2 * L.t_pad * L.d_pad;
    a.parts = L.planes;
    a.k = (int32_t)L.d_pad;
    if (L.planes > 1 && !L.stream_weight) {
        a.p = v.ws + L.off_w2;
        a.q = v.ws + L.off_h2;
        a.p_ld = a.q_ld = a.k = (int32_t)(2 * L.d_pad);
        a.p_scale = v.at<float>(L.off_ws);
        a.q_scale = v.at<float>(L.off_hs);
    }
    a.tiles_i = (int32_t)ceil_div(std::min(rows, L.vocab - v0), L.s_tile.tp);
    a.v0 = v0;
    a.vocab = L.vocab;
    a.inv_temp = 1.f / c.temp;
    a.target = c.ids != nullptr ? nullptr : v.target();
    a.t_pad = L.t_pad;
    a.first_tile = (int32_t)(v0 / L.s_tile.tp);
}

// The logits of vocab rows v0 .. (a: logits_args') and what becomes of them.  fp32 rows in
// two fp16 parts: then once more from three bf16 parts, by a launch that returns at once
// unless some row's range is more than two parts hold.
hipError_t launch_logits(int mode, const Call& c, const Views& v, int64_t v0, int64_t rows, const HeadGemmArgs& a,
                         int64_t token_rows) {
    const HeadLayout& L = v.L;
    const int64_t tiles = a.tiles_i * ceil_div(token_rows, L.s_tile.tq);
    if (L.stream_weight) return launch_head_stream(mode, L.s_tile, a, tiles, c.stream);
    const hipError_t e = launch_head_gemm(mode, L.s_tile, a, tiles, c.stream);
    if (e != hipSuccess || L.planes == 1) return e;
    HeadGemmArgs b = a;
    b.p = static_cast<const char*>(c.weight) + v0 * L.hidden * L.esize;
    b.q = v.ws + L.off_h;
    b.p_ld = (int32_t)L.hidden;
    b.q_ld = b.k = (int32_t)L.d_pad;
    b.p_range = v.at<float2>(L.off_rw);
    b.p_ranges = head_range_blocks(round_up(std::min(rows, L.vocab - v0), kHeadTile));
    b.q_range = v.at<float2>(L.off_rh);
    b.q_ranges = head_range_blocks(L.t_pad);
    return launch_head_stream(mode, L.s_tile, b, a.tiles_i * ceil_div(token_rows, std::min(128, L.s_tile.tq)), c.stream);
}

dmuon_status forward(const Call& c, bool distill, float* losses, float* lse, float* student) {
    Buffers b;
    dmuon_status st = check_call(c, distill, b);
    if (st != DMUON_OK) return st;
    const dmuon_head_desc& d = *c.desc;
    b.add(losses, 4 * d.tokens, true);
    b.add(lse, 4 * d.tokens, true);
    if (distill) b.add(student, 4 * d.tokens * d.top_k, true);
    const HeadLayout L = head_layout_of(d, false);
    if (d.tokens == 0) return b.good() ? DMUON_OK : DMUON_ERR_INVALID_ARG;
    st = check_rest(c, L, b);
    if (st != DMUON_OK) return st;

    const Views v{static_cast<char*>(c.workspace), L};
    st = gather_rows(c, v, losses, lse, student, nullptr);
    if (st != DMUON_OK) return st;
    if (distill && !L.keep_logits) {
        HeadStudentArgs t{};
        t.count = v.count();
        t.src = v.src();
        t.t = teacher_of(c);
        t.hidden = c.hidden;
        t.weight = c.weight;
        t.esize = L.esize;
        t.cols = L.hidden;
        t.student = student;
        t.tokens = L.tokens;
        HEAD_TRY(launch_head_student(t, c.stream));
    }
    // read in place, the whole vocabulary is one launch
    const int64_t step = L.pack_weight ? L.piece : round_up(L.vocab, kHeadTile);
    for (int64_t v0 = 0; v0 < L.vocab; v0 += step) {
        HeadGemmArgs a{};
        st = weight_piece(c, v, false, v0, step, a);
        if (st != DMUON_OK) return st;
        logits_args(c, v, v0, step, a);
        a.part = v.at<float2>(L.off_part);
        a.target_logit = v.target_logit();
        if (L.keep_logits) a.logits = v.at<float>(L.off_logits);
        a.logits_ld = (int32_t)round_up(L.vocab, kHeadTile);
        HEAD_TRY(launch_logits(kHeadLse, c, v, v0, step, a, L.tokens));
    }
    HeadMergeArgs m{};
    m.count = v.count();
    m.src = v.src();
    m.part = v.at<float2>(L.off_part);
    m.t_pad = L.t_pad;
    m.parts = (int32_t)ceil_div(L.vocab, L.s_tile.tp) * head_wave_rows(L.s_tile.tp, L.s_tile.tq);
    m.tokens = L.tokens;
    m.inv_temp = 1.f / c.temp;
    m.temp = c.temp;
    m.target = distill ? nullptr : v.target();
    m.target_logit = v.target_logit();
    m.t = teacher_of(c);
    m.q = v.q();
    m.student = student;
    if (L.keep_logits) m.logits = v.at<float>(L.off_logits);
    m.logits_ld = round_up(L.vocab, kHeadTile);
    m.losses = losses;
    m.lse = lse;
    HEAD_TRY(launch_head_merge(m, c.stream));
    return DMUON_OK;
}

dmuon_status backward(const Call& c, bool distill, const float* lse, const float* student, const float* grad_losses,
                      const float* grad_lse, void* grad_hidden, void* grad_weight) {
    Buffers b;
    dmuon_status st = check_call(c, distill, b);
    if (st != DMUON_OK) return st;
    const dmuon_head_desc& d = *c.desc;
    const int64_t e = d.dtype == DMUON_BF16 ? 2 : 4;
    if (grad_hidden == nullptr && grad_weight == nullptr && (d.tokens > 0)) return DMUON_ERR_INVALID_ARG;
    b.add(lse, 4 * d.tokens, false);
    b.add(grad_losses, 4 * d.tokens, false);
    if (grad_lse != nullptr) b.add(grad_lse, 4 * d.tokens, false);
    if (distill) b.add(student, 4 * d.tokens * d.top_k, false);
    if (grad_hidden != nullptr) b.add(grad_hidden, d.tokens * d.hidden * e, true);
    if (grad_weight != nullptr) b.add(grad_weight, d.vocab * d.hidden * e, true);
    const HeadLayout L = head_layout_of(d, true);
    if (d.tokens == 0) {
        if (!b.good()) return DMUON_ERR_INVALID_ARG;
        if (grad_weight != nullptr) HEAD_TRY(launch_head_zero(grad_weight, d.vocab * d.hidden * e, c.stream));
        return DMUON_OK;
    }
    st = check_rest(c, L, b);
    if (st != DMUON_OK) return st;

    const Views v{static_cast<char*>(c.workspace), L};
    HeadCoefArgs k{};
    k.q = distill ? v.q() : nullptr;
    k.lse = lse;
    k.grad_losses = grad_losses;
    k.grad_lse = grad_lse;
    k.temp = c.temp;
    k.lse_c = v.lse();
    k.cp = v.cp();
    k.ct = v.ct();
    k.norm = v.norm();
    k.t_pad = L.t_pad;
    st = gather_rows(c, v, nullptr, nullptr, nullptr, &k);
    if (st != DMUON_OK) return st;
    const int64_t dh_tiles_j = ceil_div(L.low ? 2 * head_low_row((int)L.tokens) : L.tokens, L.dh_tile.tq);
    const int32_t dh_tiles_i = (int32_t)ceil_div(L.hidden, L.dh_tile.tp);
    for (int64_t v0 = 0; v0 < L.vocab; v0 += L.piece) {
        const int64_t left = std::min(L.piece, L.vocab - v0);
        HeadGemmArgs w{};
        st = weight_piece(c, v, true, v0, L.piece, w);
        if (st != DMUON_OK) return st;
        HeadGemmArgs a = w;
        logits_args(c, v, v0, L.piece, a);
        a.lse = v.lse();
        a.cp = v.cp();
        a.ct = v.ct();
        a.norm = v.norm();
        a.low = L.low;
        a.g = v.ws + L.off_g;
        a.g_plane = 2 * L.t_pad * L.piece;
        a.g_ld = (int32_t)L.piece;
        HEAD_TRY(launch_logits(kHeadGrad, c, v, v0, L.piece, a, round_up(L.tokens, kHeadSlab)));
        if (distill) {
            HeadFixArgs f{};
            f.count = v.count();
            f.src = v.src();
            f.t = teacher_of(c);
            f.q = v.q();
            f.student = student;
            f.lse_c = v.lse();
            f.cp = v.cp();
            f.norm = v.norm();
            f.low = L.low;
            f.g = v.at<uint16_t>(L.off_g);
            f.g_plane = L.t_pad * L.piece;
            f.g_ld = L.piece;
            f.planes = L.planes;
            f.v0 = v0;
            f.v1 = v0 + left;
            f.tokens = L.tokens;
            HEAD_TRY(launch_head_fix(f, c.stream));
        }
        if (grad_hidden != nullptr) {
            HeadGemmArgs h = w;
            h.count = v.count() + 1;
            h.q = v.ws + L.off_g;
            h.q_ld = (int32_t)L.piece;
            h.q_plane = 2 * L.t_pad * L.piece;
            h.parts = L.planes;
            h.k = (int32_t)round_up(left, kHeadSlab);
            h.split_k = (int32_t)L.split_k;
            h.splits = (int32_t)ceil_div(h.k, L.split_k);
            h.tiles_i = dh_tiles_i;
            h.sums = v.at<float>(L.off_dh);
            h.accumulate = v0 != 0;
            const auto launch = L.stream_weight ? launch_head_stream : launch_head_gemm;
            HEAD_TRY(launch(kHeadDh, L.dh_tile, h, h.splits * dh_tiles_i * dh_tiles_j, c.stream));
        }
        if (grad_weight != nullptr) {
            HeadGemmArgs g{};
            g.count = v.count() + 1;
            g.norm = v.norm();
            g.p = v.ws + L.off_h;
            g.p_ld = (int32_t)L.d_pad;
            g.p_plane = 2 * L.t_pad * L.d_pad;
            g.tail_row = INT_MAX;
            g.q = v.ws + L.off_g;
            g.q_ld = (int32_t)L.piece;
            g.q_plane = 2 * L.t_pad * L.piece;
            g.parts = L.planes;
            g.tiles_i = (int32_t)ceil_div(L.hidden, L.dw_tile.tp);
            g.tiles_j = (int32_t)ceil_div(left, L.dw_tile.tq);
            g.dw = static_cast<char*>(grad_weight) + v0 * L.hidden * L.esize;
            g.dw_rows = left;
            g.dw_ld = (int32_t)L.hidden;
            g.splits = L.dw_splits;
            g.sums = v.at<float>(L.off_dw);
            HEAD_TRY(launch_head_gemm(g.splits > 1 ? kHeadDwSum : kHeadDw, L.dw_tile, g, (int64_t)g.tiles_i * g.tiles_j * g.splits, c.stream));
            if (g.splits > 1) {
                HeadSumArgs d{};
                d.rows = left;
                d.norm = v.norm();
                d.sums = g.sums;
                d.splits = g.splits;
                d.tiles_i = g.tiles_i;
                d.tile = L.dw_tile;
                d.out = g.dw;
                d.esize = L.esize;
                d.cols = L.hidden;
                HEAD_TRY(launch_head_sum(d, c.stream));
            }
        }
    }
    if (grad_hidden != nullptr) {
        HeadSumArgs h{};
        h.count = v.count();
        h.rows = L.tokens;
        h.src = v.src();
        h.norm = v.norm();
        h.low = L.low;
        h.sums = v.at<float>(L.off_dh);
        h.splits = L.splits;
        h.tiles_i = dh_tiles_i;
        h.tile = L.dh_tile;
        h.out = grad_hidden;
        h.esize = L.esize;
        h.cols = L.hidden;
        HEAD_TRY(launch_head_sum(h, c.stream));
    }
    return DMUON_OK;
}

}  // namespace

extern "C" dmuon_status head_loss_workspace_bytes(const dmuon_head_desc* desc, int32_t backward, size_t* bytes) {
    if (bytes == nullptr) return DMUON_ERR_INVALID_ARG;
    const dmuon_status st = head_check_desc(desc);
    if (st != DMUON_OK) return st;
    // the cut depends on the number of tokens, so a shorter batch may need more:
    // the largest over all of them (tokens enter a layout in steps of the smallest
    // tile edge)
    dmuon_head_desc d = *desc;
    size_t most = 0;
    for (int64_t t = std::min<int64_t>(64, desc->tokens);; t = std::min(round_up(t + 1, 64), desc->tokens)) {
        d.tokens = t;
        most = std::max(most, head_layout_of(d, backward != 0).bytes);
        if (t == desc->tokens) break;
    }
    *bytes = most;
    return DMUON_OK;
}

extern "C" dmuon_status head_cross_entropy_forward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                                   const int64_t* targets, int64_t ignore_index, float* losses,
                                                   float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    try {
        const Call c{desc, hidden, weight, targets, ignore_index, nullptr, nullptr, 1.f, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream)};
        return forward(c, false, losses, lse, nullptr);
    } catch (...) {
        return DMUON_ERR_ALLOC;
    }
}

extern "C" dmuon_status head_cross_entropy_backward(const dmuon_head_desc* desc, const void* hidden,
                                                    const void* weight, const int64_t* targets, int64_t ignore_index,
                                                    const float* lse, const float* grad_losses, const float* grad_lse,
                                                    void* grad_hidden, void* grad_weight, void* workspace,
                                                    size_t workspace_bytes, void* stream) {
    try {
        const Call c{desc, hidden, weight, targets, ignore_index, nullptr, nullptr, 1.f, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream)};
        return backward(c, false, lse, nullptr, grad_losses, grad_lse, grad_hidden, grad_weight);
    } catch (...) {
        return DMUON_ERR_ALLOC;
    }
}

extern "C" dmuon_status head_distill_forward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                             const int64_t* teacher_ids, const float* teacher_logits,
                                             float temperature, float* losses, float* lse, float* student_logits,
                                             void* workspace, size_t workspace_bytes, void* stream) {
    try {
        const Call c{desc, hidden, weight, nullptr, 0, teacher_ids, teacher_logits, temperature, workspace,
                     workspace_bytes, static_cast<hipStream_t>(stream)};
        return forward(c, true, losses, lse, student_logits);
    } catch (...) {
        return DMUON_ERR_ALLOC;
    }
}

extern "C" dmuon_status head_distill_backward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                              const int64_t* teacher_ids, const float* teacher_logits,
                                              float temperature, const float* lse, const float* student_logits,
                                              const float* grad_losses, void* grad_hidden, void* grad_weight,
                                              void* workspace, size_t workspace_bytes, void* stream) {
    try {
        const Call c{desc, hidden, weight, nullptr, 0, teacher_ids, teacher_logits, temperature, workspace,
                     workspace_bytes, static_cast<hipStream_t>(stream)};
        return backward(c, true, lse, student_logits, grad_losses, nullptr, grad_hidden, grad_weight);
    } catch (...) {
        return DMUON_ERR_ALLOC;
    }
}
