// Row kernels of the output-head losses: which rows carry a loss, their hidden
// states packed together, the join of the softmax statistics, the coefficients
// of the gradient and the hidden states' gradient scattered back.
//
// All of them move bytes, and few: of 26 ms for 8192 tokens, hidden 4096 and
// vocabulary 128256, forward and backward, 0.2 ms.  The exceptions: the student's
// logits at the teacher's ids, a row of W each (4096 tokens of 64 entries, 2.1 GB of
// rows, half of them from the caches: 347 us of 13.5 ms), and the packing of W for fp32
// (32000 x 1536: 97 us forward, 143 backward).  For few tokens launches count: up to
// 1024 of them one launch finds the rows and packs them (8 us for 777 x 1536; two
// launches made scoring one token, 202 us in all, 13 us longer).
#include "head_internal.h"
#include "kcommon.h"

namespace dmuon {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float wave_sum(float v) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7fc00000u); }

// One wave per token: the teacher's softmax over its K entries, as the largest z
// and the log of the sum of exp((z - max) / T).  The difference is taken before the
// division: equal entries then differ by 0 however large they are, also where the
// compiler fuses the two (the type's lowest value stands in masks).  A row whose entries
// are all absent or -inf carries no loss; an id past the vocabulary marks the row NaN,
// unless its entry is -inf.
__global__ __launch_bounds__(kRowThreads) void head_teacher_kernel(HeadTeacher t, int64_t tokens, float2* q,
                                                                   int32_t* flag, float* student) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6);
    if (row >= tokens) return;
    const int64_t* ids = t.ids + row * t.k;
    const float* z = t.logits + row * t.k;
    float m = -INFINITY;
    bool bad = false, held = false;
    for (int k = lane; k < t.k; k += 64) {
        const int64_t id = ids[k];
        if (student != nullptr) student[row * t.k + k] = 0.f;
        if (id < 0) continue;
        const float y = z[k];
        if (y == -INFINITY) continue;  // no mass
        held = true;
        bad = bad || id >= t.vocab || y != y;
        m = fmaxf(m, y);
    }
    held = __builtin_amdgcn_ballot_w64(held) != 0;
    bad = __builtin_amdgcn_ballot_w64(bad) != 0;
    m = wave_max(m);
    float l = 0.f;
    if (held && !bad)
        for (int k = lane; k < t.k; k += 64)
            if (ids[k] >= 0) l += expf((z[k] - m) * t.inv_temp);
    l = wave_sum(l);
    if (lane == 0) {
        flag[row] = held;
        q[row] = bad ? make_float2(nan_f(), nan_f()) : make_float2(m, held ? logf(l) : 0.f);
    }
}

// The rows that carry a loss keep their order at the front of src, the others
// fill it from the back.  Run by a whole block; list (null: not) receives the
// front as well, and only a writer writes to memory.  Returns the rows' number.
template <int THREADS>
__device__ __forceinline__ int scan_rows(const HeadRowsArgs& a, bool writer, int* list) {
    __shared__ int wave_n[THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int n = 0;
    for (int t0 = 0; t0 < a.tokens; t0 += THREADS) {
        const int t = t0 + threadIdx.x;
        const bool in = t < a.tokens;
        const int64_t target = in && a.targets != nullptr ? a.targets[t] : 0;
        const bool live = in && (a.targets != nullptr ? target != a.ignore_index : a.flag == nullptr || a.flag[t] != 0);
        const uint64_t b = __builtin_amdgcn_ballot_w64(live);
        if (lane == 0) wave_n[wave] = __popcll(b);
        __syncthreads();
        int before = __popcll(b & ((1ull << lane) - 1)), all = 0;
        for (int w = 0; w < THREADS / 64; ++w) {
            before += w < wave ? wave_n[w] : 0;
            all += wave_n[w];
        }
        __syncthreads();
        const int c = n + before;
        if (live && list != nullptr) list[c] = t;
        if (live && writer) {
            a.src[c] = t;
            if (a.targets != nullptr) a.target[c] = target >= 0 && target < a.vocab ? (int)target : -2;
        } else if (in && writer) {
            a.src[a.tokens - 1 - (t - c)] = t;
            if (a.losses != nullptr) {
                a.losses[t] = 0.f;
                a.lse[t] = 0.f;
            }
        }
        n += all;
    }
    if (a.targets != nullptr && writer)
        for (int c = n + threadIdx.x; c < a.t_pad; c += THREADS) a.target[c] = -1;
    if (threadIdx.x == 0 && writer) {
        a.count[0] = n;
        a.count[1] = a.low ? 2 * head_low_row(n) : n;
    }
    return n;
}

constexpr int kScanThreads = 1024;
__global__ __launch_bounds__(kScanThreads) void head_rows_kernel(HeadRowsArgs a) {
    scan_rows<kScanThreads>(a, true, nullptr);
    if (threadIdx.x == 0) *a.norm = 0.f;
}

// Eight columns c .. c + 7 of a row, zeros past its end.
template <int ESIZE>
__device__ __forceinline__ void load_cols(const void* in, int64_t row, int64_t cols, int64_t c, bool vec, float (&x)[8]) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (ESIZE == 2) {
        const uint16_t* p = static_cast<const uint16_t*>(in) + row * cols + c;
        if (vec && c < cols) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            #pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = bf16_to_f32((uint16_t)(w[e / 2] >> (16 * (e & 1))));
        } else {
            #pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) x[e] = bf16_to_f32(p[e]);
        }
    } else {
        const float* p = static_cast<const float*>(in) + row * cols + c;
        if (vec && c < cols) {
            const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
            x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
        } else {
            #pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) x[e] = p[e];
        }
    }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&x)[8]) {
    uint32_t w[4];
    #pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)f32_to_bf16(x[2 * e]) | ((uint32_t)f32_to_bf16(x[2 * e + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One wave per output row, 8 columns a lane and step.
template <int ESIZE>
__device__ __forceinline__ void pack_rows(const HeadPackArgs& a, const int32_t* src, int64_t limit, int block,
                                          int blocks) {
    // rows past the last one: zeros up to a whole tile
    int64_t end = (limit + kHeadTile - 1) / kHeadTile * kHeadTile;
    if (end == 0) end = kHeadTile;
    if (end > a.out_rows) end = a.out_rows;
    const bool vec = a.cols % 8 == 0;
    const int64_t low_row = a.low ? head_low_row((int)limit) : end;
    const int lane = threadIdx.x & 63;
    constexpr int kWavesBlock = kRowThreads / 64;
    float2 range = make_float2(0.f, 0.f);
    for (int64_t r = (int64_t)block * kWavesBlock + (threadIdx.x >> 6); r < end; r += (int64_t)blocks * kWavesBlock) {
        const int64_t of = r < low_row ? r : r - low_row;
        const int64_t from = of < limit ? (src != nullptr ? (int64_t)src[of] : of) : -1;
        float scale = 1.f;
        if (ESIZE == 4 && a.half2 != nullptr) {
            // a power of two that puts the row's largest element in [2^14, 2^15)
            float m = 0.f, sum = 0.f;
            if (from >= 0)
                for (int64_t c = lane * 8; c < a.cols; c += 512) {
                    float x[8];
                    load_cols<ESIZE>(a.in, from, a.cols, c, vec, x);
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        m = fmaxf(m, fabsf(x[e]));
                        sum += fabsf(x[e]);
                    }
                }
            m = wave_max(m);
            // (a NaN counts for neither: it makes its logits NaN in any form)
            range = make_float2(fmaxf(range.x, m), fmaxf(range.y, wave_sum(sum)));
            // exponents below 2^-100 would need a scale past fp32's range
            const int e = min(max((int)(__float_as_uint(m) >> 23), 27), 254);
            scale = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
            if (lane == 0) a.scale[r] = 1.f / scale;
        }
        #pragma unroll 2
        for (int64_t c = lane * 8; c < a.ld; c += 512) {
            float x[8];
            if (from >= 0) {
                load_cols<ESIZE>(a.in, from, a.cols, c, vec, x);
            } else {
                #pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            }
            if (ESIZE == 2) {
                *reinterpret_cast<uint4*>(a.out + r * a.ld + c) = pack_bf16(x);
                continue;
            }
            if (a.half2 != nullptr) {
            uint16_t h[2][8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = x[e] * scale;
                const _Float16 hi = (_Float16)y;
                h[0][e] = __builtin_bit_cast(uint16_t, hi);
                h[1][e] = __builtin_bit_cast(uint16_t, (_Float16)(y - (float)hi));
            }
            uint16_t* o = a.half2 + r * 2 * a.ld + (c / 32) * 64 + c % 32;
            #pragma unroll
            for (int part = 0; part < 2; ++part) {
                uint32_t w[4];
                #pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = (uint32_t)h[part][2 * e] | ((uint32_t)h[part][2 * e + 1] << 16);
                *reinterpret_cast<uint4*>(o + 32 * part) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            }
            if (a.out != nullptr) {
                #pragma unroll
                for (int part = 0; part < kHeadMaxPlanes; ++part) {
                    *reinterpret_cast<uint4*>(a.out + part * a.plane + r * a.ld + c) = pack_bf16(x);
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] -= bf16_to_f32(f32_to_bf16(x[e]));
                }
            }
        }
    }
    if (ESIZE == 4 && a.range != nullptr) {
        __shared__ float2 of_wave[kWavesBlock];
        if (lane == 0) of_wave[threadIdx.x >> 6] = range;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWavesBlock; ++w)
                range = make_float2(fmaxf(range.x, of_wave[w].x), fmaxf(range.y, of_wave[w].y));
            a.range[block] = range;
        }
    }
}

// R rows by 256 / R groups of tiles a block: each thread joins its group's (max,
// sum) pairs of its row, then the groups are joined, all in a fixed order; the
// groups then share the row's teacher entries.  R = 16 reads whole 128-byte lines
// of the statistics; few tokens take fewer rows a block, so that more threads
// share a row.
template <int R>
__global__ __launch_bounds__(256) void head_merge_kernel(HeadMergeArgs a) {
    constexpr int kGroups = 256 / R;
    __shared__ float red[4][R];
    const int n = *a.count;
    const int r = threadIdx.x % R, g = threadIdx.x / R, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * R + r;
    const float scale = a.inv_temp;
    if ((int64_t)blockIdx.x * R >= n) return;
    const bool in = c < n;
    // over the row's groups: inside a wave, then the four waves in order
    auto over_groups = [&](float v, bool max) {
        #pragma unroll
        for (int off = 32; off >= R; off >>= 1) {
            const float o = __shfl_xor(v, off, 64);
            v = max ? fmaxf(v, o) : v + o;
        }
        __syncthreads();
        if ((threadIdx.x & 63) < R) red[wave][r] = v;
        __syncthreads();
        v = red[0][r];
        #pragma unroll
        for (int w = 1; w < 4; ++w) v = max ? fmaxf(v, red[w][r]) : v + red[w][r];
        return v;
    };
    const int per = (a.parts + kGroups - 1) / kGroups;
    const int p0 = g * per, mine = in ? min(a.parts, p0 + per) - p0 : 0;
    const float2* p = a.part + (int64_t)p0 * a.t_pad + c;
    // (a NaN does not survive fmaxf, but is in the sum too, and stays)
    float m = -INFINITY, l = 0.f;
    #pragma unroll 4
    for (int k = 0; k < mine; ++k) m = fmaxf(m, p[k * a.t_pad].x);
    m = over_groups(m, true);
    const float m0 = m == -INFINITY ? 0.f : m;
    #pragma unroll 4
    for (int k = 0; k < mine; ++k) {
        const float2 x = p[k * a.t_pad];
        l = fmaf(x.y, expf((x.x - m0) * scale), l);
    }
    l = over_groups(l, false);
    // A loss takes the largest logit's distance first: lse, rounded at its own size, would
    // leave a loss of large logits 2^-24 of those.
    const float log_l = logf(l), lse = fmaf(m, scale, log_l);
    const int t = in ? a.src[c] : 0;
    const bool writer = in && g == 0;
    if (writer) a.lse[t] = lse;
    if (a.target != nullptr) {
        if (writer) a.losses[t] = a.target[c] < 0 ? nan_f() : (m - a.target_logit[c]) + log_l;
        return;
    }
    // distillation: sum of q (log q - s / T + lse) over the row's entries
    float loss = 0.f;
    if (in) {
        const float2 q = a.q[t];
        for (int k = g; k < a.t.k; k += kGroups) {
            const int64_t at = (int64_t)t * a.t.k + k, id = a.t.ids[at];
            if (id < 0) continue;
            float s = 0.f;
            if (a.logits != nullptr) {
                if (id < a.t.vocab) s = a.logits[c * a.logits_ld + id];
                a.student[at] = s;
            } else {
                s = a.student[at];
            }
            const float logq = (a.t.logits[at] - q.x) * scale - q.y;
            if (logq == -INFINITY) continue;  // no mass
            loss = fmaf(expf(logq), logq + fmaf(m - s, scale, log_l), loss);
        }
    }
    loss = over_groups(loss, false);
    if (writer) a.losses[t] = a.temp * a.temp * loss;  // (q is NaN where an id is past the vocabulary)
}

// A wave per teacher entry of the rows with a loss: the student's logit.
template <int ESIZE>
__global__ __launch_bounds__(kRowThreads) void head_student_kernel(HeadStudentArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t entries = (int64_t)*a.count * a.t.k, step = (int64_t)gridDim.x * (kRowThreads / 64);
    const bool vec = a.cols % (16 / ESIZE) == 0;
    for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6); w < entries; w += step) {
        const int64_t c = w / a.t.k;
        const int64_t row = a.src[c], at = row * a.t.k + (w - c * a.t.k);
        const int64_t id = a.t.ids[at];
        if (id < 0 || id >= a.t.vocab) continue;
        float s = 0.f;
        if (ESIZE == 2) {
            const uint16_t* h = static_cast<const uint16_t*>(a.hidden) + row * a.cols;
            const uint16_t* x = static_cast<const uint16_t*>(a.weight) + id * a.cols;
            if (vec) {
                #pragma unroll 4
                for (int64_t d = lane * 8; d < a.cols; d += 512) {
                    const uint4 u = *reinterpret_cast<const uint4*>(h + d), v = *reinterpret_cast<const uint4*>(x + d);
                    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s = fmaf(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16), s);
                        s = fmaf(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(vs[e] & 0xffff0000u), s);
                    }
                }
            } else {
                #pragma unroll 4
                for (int64_t d = lane; d < a.cols; d += 64) s = fmaf(bf16_to_f32(h[d]), bf16_to_f32(x[d]), s);
            }
        } else {
            const float* h = static_cast<const float*>(a.hidden) + row * a.cols;
            const float* x = static_cast<const float*>(a.weight) + id * a.cols;
            if (vec) {
                #pragma unroll 4
                for (int64_t d = lane * 4; d < a.cols; d += 256) {
                    const float4 u = *reinterpret_cast<const float4*>(h + d), v = *reinterpret_cast<const float4*>(x + d);
                    s = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, s))));
                }
            } else {
                #pragma unroll 4
                for (int64_t d = lane; d < a.cols; d += 64) s = fmaf(h[d], x[d], s);
            }
        }
        s = wave_sum(s);
        if (lane == 0) a.student[at] = s;
    }
}

// The coefficients of compact row c < n, of token t; the larger one's magnitude, for
// the largest of all, by which ds is divided.
__device__ __forceinline__ float coefficients(const HeadCoefArgs& a, int64_t c, int t, bool bad) {
    const float ct = a.grad_losses != nullptr ? a.temp * a.grad_losses[t] : 0.f;
    float cp = a.grad_lse != nullptr ? ct + a.grad_lse[t] : ct;
    float m = fabsf(ct);
    if (a.grad_entropy != nullptr) {
        const float ce = a.temp * a.grad_entropy[t];
        cp = fmaf(ce, a.entropy[t], cp);
        a.ce[c] = ce;
        m = fmaxf(m, fabsf(ce));
    }
    a.lse_c[c] = a.lse[t];
    a.cp[c] = bad ? nan_f() : cp;
    a.ct[c] = ct;
    m = fmaxf(fabsf(cp), m);
    // (within 2^100 either way, so that its inverse is a normal number)
    return m > 0.f && m < INFINITY ? fminf(fmaxf(m, 0x1p-100f), 0x1p100f) : 0.f;
}
__device__ __forceinline__ void no_coefficients(const HeadCoefArgs& a, int64_t c) {
    a.lse_c[c] = 0.f;
    a.cp[c] = 0.f;
    a.ct[c] = 0.f;
    if (a.grad_entropy != nullptr) a.ce[c] = 0.f;
}

// After head_rows_kernel.
template <int ESIZE>
__global__ __launch_bounds__(kRowThreads) void head_prepare_kernel(HeadPrepareArgs a) {
    int block = (int)blockIdx.x;
    if (block < a.h_blocks) {
        pack_rows<ESIZE>(a.h, a.rows.src, *a.rows.count, block, a.h_blocks);
        return;
    }
    block -= a.h_blocks;
    if (block < a.w_blocks) {
        pack_rows<ESIZE>(a.w, nullptr, a.w.rows, block, a.w_blocks);
        return;
    }
    const HeadCoefArgs& k = a.coef;
    const int64_t c = (int64_t)(block - a.w_blocks) * kRowThreads + threadIdx.x;
    if (c >= k.t_pad) return;
    if (c >= *a.rows.count) {
        no_coefficients(k, c);
        return;
    }
    const int t = a.rows.src[c];
    const float m = coefficients(k, c, t, k.q != nullptr ? k.q[t].x != k.q[t].x : a.rows.targets != nullptr && a.rows.target[c] < 0);
    // (integer order is float order for these bits; the maximum does not depend on the order)
    atomicMax(reinterpret_cast<unsigned int*>(k.norm), __float_as_uint(m));
}

// The same with the rows found here, by every block for itself (at most
// kScanTokens tokens): one launch less.
template <int ESIZE>
__global__ __launch_bounds__(kRowThreads) void head_scan_prepare_kernel(HeadPrepareArgs a) {
    __shared__ int list[kScanTokens];
    __shared__ float largest[kRowThreads / 64];
    int block = (int)blockIdx.x;
    if (block >= a.h_blocks && block < a.h_blocks + a.w_blocks) {
        pack_rows<ESIZE>(a.w, nullptr, a.w.rows, block - a.h_blocks, a.w_blocks);
        return;
    }
    const int n = scan_rows<kRowThreads>(a.rows, block == 0, list);
    __syncthreads();
    if (block < a.h_blocks) {
        pack_rows<ESIZE>(a.h, list, n, block, a.h_blocks);
        return;
    }
    const HeadCoefArgs& k = a.coef;  // one block
    float m = 0.f;
    for (int c = threadIdx.x; c < k.t_pad; c += kRowThreads) {
        if (c >= n) {
            no_coefficients(k, c);
            continue;
        }
        const int t = list[c];
        bool bad;
        if (k.q != nullptr) {
            bad = k.q[t].x != k.q[t].x;
        } else {
            const int64_t target = a.rows.targets != nullptr ? a.rows.targets[t] : 0;
            bad = target < 0 || target >= a.rows.vocab;
        }
        m = fmaxf(m, coefficients(k, c, t, bad));
    }
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) largest[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kRowThreads / 64; ++w) m = fmaxf(m, largest[w]);
        *k.norm = m;
    }
}

// One wave per row with a loss: ds at each teacher id of the piece; an id held
// twice takes the sum of its entries' q.  bf16: from the student logit of the
// forward call, so that p - q is rounded once.  fp32: the tile's own cp p, whole in
// its three parts, less cp q (its p and lse come from one and the same logit).
__global__ __launch_bounds__(kRowThreads) void head_fix_kernel(HeadFixArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6);
    if (c >= *a.count) return;
    const int64_t row = a.src[c];
    const int64_t* ids = a.t.ids + row * a.t.k;
    const float* z = a.t.logits + row * a.t.k;
    const float2 qs = a.q[row];
    const float norm = *a.norm;
    const float cp = a.cp[c] * (1.f / (norm > 0.f ? norm : 1.f)), lse = a.lse_c[c];
    const int64_t low_step = a.low ? (int64_t)head_low_row(*a.count) * a.g_ld : a.g_plane;
    for (int k0 = 0; k0 < a.t.k; k0 += 64) {
        const int k = k0 + lane;
        const int64_t id = k < a.t.k ? ids[k] : -1;
        const bool here = id >= a.v0 && id < a.v1;
        if (!__builtin_amdgcn_ballot_w64(here)) continue;
        const int mine = here ? (int)(id - a.v0) : -1;  // (a piece has fewer than 2^31 rows)
        float q = 0.f;
        bool first = true;  // of the entries with this id
        for (int j0 = 0; j0 < a.t.k; j0 += 64) {
            const int j = j0 + lane;
            const int64_t other = j < a.t.k ? ids[j] : -1;
            const int off = other >= a.v0 && other < a.v1 ? (int)(other - a.v0) : -2;
            const float qj = off >= 0 ? expf((z[j] - qs.x) * a.t.inv_temp - qs.y) : 0.f;
            const int last = min(64, a.t.k - j0);
            for (int i = 0; i < last; ++i) {
                const int o = __builtin_amdgcn_readlane(off, i);
                const float x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(qj), i));
                q += o == mine ? x : 0.f;
                first = first && !(o == mine && j0 + i < k);
            }
        }
        if (!here || !first) continue;
        uint16_t* out = a.g + c * a.g_ld + mine;
        float g;
        if (a.planes > 1) {
            float cpp = 0.f;
            for (int part = a.planes - 1; part >= 0; --part) cpp += bf16_to_f32(out[part * a.g_plane]);
            g = fmaf(-cp, q, cpp);
        } else {
            g = cp * (expf(fmaf(a.student[row * a.t.k + k], a.t.inv_temp, -lse)) - q);
        }
        for (int part = 0; part < (a.low ? 2 : a.planes); ++part) {
            const uint16_t b = f32_to_bf16(g);
            out[part * low_step] = b;
            g -= bf16_to_f32(b);
        }
    }
}

// A wave per 64 float4 of a tile's sums, in the product kernel's own order (a
// lane's four values are 4 consecutive columns of one row).
__global__ __launch_bounds__(kRowThreads) void head_sum_kernel(HeadSumArgs a) {
    const int TP = a.tile.tp, TQ = a.tile.tq;
    const int WR = head_wave_rows(TP, TQ), NW = head_waves(TP), RW = TP / WR, CW = TQ / (NW / WR);
    const int FI = RW / 32, FJ = CW / 32;
    const int kGroups = NW * FI * FJ * 4;
    const int n = a.count != nullptr ? *a.count : (int)a.rows;
    const int low_row = a.low ? head_low_row(n) : 0;
    const int tiles_j = (n + TQ - 1) / TQ;  // of the rows themselves
    const int64_t per_split = (int64_t)((a.low ? 2 * low_row : n) + TQ - 1) / TQ * a.tiles_i * (TP * TQ);
    int splits = a.splits;
    if (a.room != 0) {
        const int slabs = a.first_k / kHeadSlab, s = head_dh_splits(tiles_j * a.tiles_i, slabs, a.room);
        const int per = (slabs + s - 1) / s;
        splits = (slabs + per - 1) / per;
    }
    const int lane = threadIdx.x & 63;
    const float norm = *a.norm > 0.f ? *a.norm : 1.f;
    const int64_t groups = (int64_t)tiles_j * a.tiles_i * kGroups;
    const int64_t step = (int64_t)gridDim.x * (kRowThreads / 64);
    for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6); w < groups; w += step) {
        const int64_t tile = w / kGroups;
        int g = (int)(w % kGroups);
        const int v4 = g % 4; g /= 4;
        const int j = g % FJ; g /= FJ;
        const int i = g % FI; g /= FI;
        const int wr = g % WR, wc = g / WR;
        const int64_t J = tile / a.tiles_i, I = tile % a.tiles_i;
        const int64_t c0 = J * TQ + wc * CW + 32 * j, c = c0 + (lane & 31);
        const int64_t col = I * TP + wr * RW + 32 * i + 8 * v4 + 4 * (lane >> 5);
        if (c >= n || col >= a.cols) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](int64_t group) {
            const float* p = a.sums + group * 256 + lane * 4;
            #pragma unroll 4
            for (int k = 0; k < splits; ++k) {
                const float4 u = *reinterpret_cast<const float4*>(p + k * per_split);
                s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
            }
        };
        if (low_row != 0 && c0 < low_row) {  // the 32 rows of the low parts first
            const int64_t cl = c0 + low_row, Jl = cl / TQ;
            const int in = (int)(cl - Jl * TQ), wl = in / CW * WR + wr, jl = in % CW / 32;
            add((Jl * a.tiles_i + I) * kGroups + ((wl * FI + i) * FJ + jl) * 4 + v4);
        }
        add(w);
        s.x *= norm, s.y *= norm, s.z *= norm, s.w *= norm;
        const int64_t at = (a.src != nullptr ? (int64_t)a.src[c] : c) * a.cols + col;
        const float x[4] = {s.x, s.y, s.z, s.w};
        if (a.esize == 2) {
            uint16_t* o = static_cast<uint16_t*>(a.out) + at;
            if ((a.cols & 3) == 0) {
                *reinterpret_cast<uint2*>(o) = make_uint2((uint32_t)f32_to_bf16(x[0]) | ((uint32_t)f32_to_bf16(x[1]) << 16),
                                                          (uint32_t)f32_to_bf16(x[2]) | ((uint32_t)f32_to_bf16(x[3]) << 16));
            } else {
                for (int e = 0; e < 4; ++e)
                    if (col + e < a.cols) o[e] = f32_to_bf16(x[e]);
            }
        } else {
            float* o = static_cast<float*>(a.out) + at;
            if ((a.cols & 3) == 0) {
                *reinterpret_cast<float4*>(o) = s;
            } else {
                for (int e = 0; e < 4; ++e)
                    if (col + e < a.cols) o[e] = x[e];
            }
        }
    }
    // rows without a loss
    const int64_t idle = a.rows - n;  // (src is given where there may be any)
    for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6); w < idle; w += step) {
        const int64_t at = (int64_t)a.src[n + w] * a.cols;
        for (int64_t d = lane; d < a.cols; d += 64) {
            if (a.esize == 2) static_cast<uint16_t*>(a.out)[at + d] = 0;
            else static_cast<float*>(a.out)[at + d] = 0.f;
        }
    }
}

__global__ __launch_bounds__(kRowThreads) void head_zero_kernel(char* p, int64_t bytes) {
    const int64_t step = (int64_t)gridDim.x * kRowThreads * 2;
    for (int64_t i = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) * 2; i < bytes; i += step)
        *reinterpret_cast<uint16_t*>(p + i) = 0;  // elements are 2 or 4 bytes
}

unsigned blocks_for(int64_t items, int64_t per_block, int64_t most) {
    const int64_t b = (items + per_block - 1) / per_block;
    return (unsigned)(b < 1 ? 1 : b > most ? most : b);
}

}  // namespace

hipError_t launch_head_teacher(const HeadTeacher& t, int64_t tokens, float2* q, int32_t* flag, float* student,
                               hipStream_t stream) {
    const unsigned grid = blocks_for(tokens, kRowThreads / 64, INT32_MAX);
    hipLaunchKernelGGL(head_teacher_kernel, dim3(grid), dim3(kRowThreads), 0, stream, t, tokens, q, flag, student);
    return hipGetLastError();
}

hipError_t launch_head_prepare(const HeadPrepareArgs& args, hipStream_t stream) {
    HeadPrepareArgs a = args;
    const int64_t per = kRowThreads / 64;
    const bool scan = a.rows.tokens > 0 && a.rows.tokens <= kScanTokens;
    if (a.rows.tokens > kScanTokens) {
        hipLaunchKernelGGL(head_rows_kernel, dim3(1), dim3(kScanThreads), 0, stream, a.rows);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    auto blocks_of = [&](const HeadPackArgs& p) {
        if (p.out_rows <= 0) return 0;
        return p.range != nullptr ? head_range_blocks(p.out_rows) : (int32_t)blocks_for(p.out_rows, per, 8192);
    };
    a.h_blocks = blocks_of(a.h);
    a.w_blocks = blocks_of(a.w);
    a.coef_blocks = scan ? (a.coef.t_pad > 0) : (int32_t)((a.coef.t_pad + kRowThreads - 1) / kRowThreads);
    const dim3 grid(a.h_blocks + a.w_blocks + a.coef_blocks), block(kRowThreads);
    if (a.esize == 2) {
        if (scan) hipLaunchKernelGGL((head_scan_prepare_kernel<2>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((head_prepare_kernel<2>), grid, block, 0, stream, a);
    } else {
        if (scan) hipLaunchKernelGGL((head_scan_prepare_kernel<4>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((head_prepare_kernel<4>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_head_merge(const HeadMergeArgs& a, hipStream_t stream) {
    const dim3 block(256);
    if (a.tokens > 1024)
        hipLaunchKernelGGL((head_merge_kernel<16>), dim3(blocks_for(a.tokens, 16, INT32_MAX)), block, 0, stream, a);
    else if (a.tokens > 128)
        hipLaunchKernelGGL((head_merge_kernel<4>), dim3(blocks_for(a.tokens, 4, INT32_MAX)), block, 0, stream, a);
    else
        hipLaunchKernelGGL((head_merge_kernel<1>), dim3(blocks_for(a.tokens, 1, INT32_MAX)), block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_head_student(const HeadStudentArgs& a, hipStream_t stream) {
    const dim3 grid(blocks_for(a.tokens * a.t.k, kRowThreads / 64, 1 << 20)), block(kRowThreads);
    if (a.esize == 2) hipLaunchKernelGGL((head_student_kernel<2>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((head_student_kernel<4>), grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_head_fix(const HeadFixArgs& a, hipStream_t stream) {
    const unsigned grid = blocks_for(a.tokens, kRowThreads / 64, INT32_MAX);
    hipLaunchKernelGGL(head_fix_kernel, dim3(grid), dim3(kRowThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_head_sum(const HeadSumArgs& a, hipStream_t stream) {
    const int64_t rows = (a.rows + a.tile.tq - 1) / a.tile.tq * a.tile.tq;
    const dim3 grid(blocks_for(rows * a.tiles_i * (a.tile.tp / 4), kRowThreads, 8192)), block(kRowThreads);
    hipLaunchKernelGGL(head_sum_kernel, grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_head_zero(void* p, int64_t bytes, hipStream_t stream) {
    const unsigned grid = blocks_for(bytes, kRowThreads * 2, 8192);
    hipLaunchKernelGGL(head_zero_kernel, dim3(grid), dim3(kRowThreads), 0, stream, static_cast<char*>(p), bytes);
    return hipGetLastError();
}

}  // namespace dmuon
