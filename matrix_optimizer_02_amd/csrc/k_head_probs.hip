// Row kernels of the output head's log probabilities (gfx950): one workgroup a
// token joins the statistics that the logits' products left, and finds the
// alternatives.
//
// A part is the words whose softmax statistics one wave formed (32 to 128 of them,
// one after the other); a group is 16 words of one lane: of the block of 32 words
// b, group 2 b + h holds words 32 b + 8 q + 4 h + r (q, r < 4) as its elements
// 4 q + r, so a group's elements are in the order of their ids.  Of each group the
// products' epilogue shows the largest logit, its place and the size of the second.
//
// The K alternatives lie in the K parts with the largest maxima (equal maxima: the
// earlier part): were one in another part, each of those K parts would hold a word
// before it.  Of those parts' groups, in the same way, only the K with the largest shown
// logits can hold alternatives.  A group whose second logit comes before the K-th
// shown one is opened: its other 15 logits are formed again from H and W.  A row's K spread
// over V / 16 groups share one 8 K^2 / V times: 0.02 times for K = 20 of 128256
// words, once for K = 128.
//
// What bounds it: latency.  The largest of n values are found by counting how many reach
// a threshold, two bits of it a round, with the values in registers.
#include "head_internal.h"
#include "kcommon.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kK = kHeadMaxAlternatives;

__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7fc00000u); }

// Floats as integers of the same order (-0 as +0; 0: nothing, as -inf is), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f), o = u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
    return o > 0x007fffffu ? o : 0;
}
__device__ __forceinline__ float from_order(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}

// What is sorted: a logit and its place, the larger logit and then the lower place
// first.  No two are the same.
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t place) {
    return order != 0 ? ((uint64_t)order << 32) | (uint32_t)~place : 0;
}
__device__ __forceinline__ uint32_t place_of(uint64_t key) { return ~(uint32_t)key; }
__device__ __forceinline__ uint32_t order_in(uint64_t key) { return (uint32_t)(key >> 32); }

// Joins over the block, the same in every thread, in a fixed order.
struct Joins {
    float f[kWaves];
    int4 counts[2][kWaves];
};
__device__ __forceinline__ float wave_max(float v) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ __forceinline__ float wave_add(float v) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ float block_max(float v, Joins& red) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red.f[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(red.f[0], red.f[1]), fmaxf(red.f[2], red.f[3]));
}
__device__ __forceinline__ float block_add(float v, Joins& red) {
    v = wave_add(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red.f[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red.f[0] + red.f[1]) + (red.f[2] + red.f[3]);
}

// The k largest of up to PER values a thread (orders o, 0 where there is none, at places
// p), in any order; returns their number (fewer than k where there are not as many).
template <int PER, typename P>
__device__ __forceinline__ int largest(const uint32_t (&o)[PER], P&& place, int k, uint64_t* out, int* taken,
                                       Joins& red) {
    int turn = 0;
    // how many of the values are at least a, b and c, by `at`
    auto count = [&](auto&& at, uint32_t a, uint32_t b, uint32_t c) {
        int4 n = make_int4(0, 0, 0, 0);
        #pragma unroll
        for (int u = 0; u < PER; ++u) {
            const uint32_t x = at(u);
            n.x += __popcll(__builtin_amdgcn_ballot_w64(x >= a));
            n.y += __popcll(__builtin_amdgcn_ballot_w64(x >= b));
            n.z += __popcll(__builtin_amdgcn_ballot_w64(x >= c));
        }
        turn ^= 1;  // (the counts of the round before may still be read)
        if ((threadIdx.x & 63) == 0) red.counts[turn][threadIdx.x >> 6] = n;
        __syncthreads();
        n = red.counts[turn][0];
        #pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            const int4 m = red.counts[turn][w];
            n.x += m.x, n.y += m.y, n.z += m.z;
        }
        return n;
    };
    // The largest threshold that k values reach: two bits a round.
    auto threshold = [&](auto&& at, int top, int want, int& reach) {
        uint32_t least = 0;
        for (int bit = top; bit >= 0 && reach != want; bit -= 2) {
            const uint32_t a = least | 1u << bit, b = least | 2u << bit, c = least | 3u << bit;
            const int4 n = count(at, a, b, c);
            if (n.z >= want) least = c, reach = n.z;
            else if (n.y >= want) least = b, reach = n.y;
            else if (n.x >= want) least = a, reach = n.x;
        }
        return least;
    };
    __syncthreads();
    const int held = count([&](int u) { return o[u]; }, 1u, 1u, 1u).x;
    if (threadIdx.x == 0) *taken = 0;
    if (k > held) k = held;
    int reach = held;
    const uint32_t least = threshold([&](int u) { return o[u]; }, 30, k, reach);
    // of values equal to the least one, those at the lowest places
    uint32_t low = 0;
    if (reach > k) {
        const int above = least == 0xffffffffu ? 0 : count([&](int u) { return o[u]; }, least + 1, 1u, 1u).x;
        int equal = reach - above;
        low = threshold([&](int u) { return o[u] == least ? ~place(u) : 0u; }, 30, k - above, equal);
    }
    __syncthreads();
    if (k > 0) {
        #pragma unroll
        for (int u = 0; u < PER; ++u)
            if (o[u] != 0 && (o[u] > least || (o[u] == least && ~place(u) >= low)))
                out[atomicAdd(taken, 1)] = key_of(o[u], place(u));  // (places in a list that is sorted next)
    }
    __syncthreads();
    return k;
}

// The same of n keys in LDS.
template <int PER>
__device__ __forceinline__ int largest_keys(const uint64_t* keys, int n, int k, uint64_t* out, int* taken, Joins& red) {
    uint32_t o[PER], p[PER];
    #pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int i = u * kThreads + (int)threadIdx.x;
        const uint64_t x = i < n ? keys[i] : 0;
        o[u] = order_in(x);
        p[u] = place_of(x);
    }
    return largest<PER>(o, [&](int u) { return p[u]; }, k, out, taken, red);
}

// n different keys in descending order.
__device__ __forceinline__ void sort_keys(const uint64_t* keys, int n, uint64_t* sorted) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t mine = keys[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += keys[j] > mine ? 1 : 0;
        sorted[rank] = mine;
    }
    __syncthreads();
}

// A token that takes no part.
__device__ __forceinline__ void idle_row(const HeadProbsArgs& a, int64_t t, int thread, int threads) {
    if (thread == 0) {
        if (a.logprobs != nullptr) a.logprobs[t] = 0.f;
        if (a.entropy != nullptr) a.entropy[t] = 0.f;
        a.lse[t] = 0.f;
    }
    for (int i = thread; i < a.k; i += threads) {
        a.top_ids[t * a.k + i] = -1;
        a.top_logprobs[t * a.k + i] = 0.f;
    }
}

struct Row {
    float m, log_l;
    bool fine;  // has a distribution
};

// The row's outputs by m, its largest logit, l = sum of exp((s - m) / T) and e = the sum
// of that times (s - m) / T.
__device__ __forceinline__ Row row_of(const HeadProbsArgs& a, int64_t c, int64_t t, float m, float l, float e,
                                      bool writer) {
    Row r{m, nan_f(), l > 0.f && l < INFINITY};
    if (r.fine) r.log_l = logf(l);
    if (writer) {
        a.lse[t] = r.fine ? fmaf(m, a.inv_temp, r.log_l) : nan_f();
        if (a.entropy != nullptr) a.entropy[t] = r.log_l - e / l;
        if (a.logprobs != nullptr)
            a.logprobs[t] = a.target[c] < 0 ? nan_f() : fmaf(a.target_logit[c] - m, a.inv_temp, -r.log_l);
    }
    return r;
}
// One part's share of l and e.  (A NaN does not survive fmaxf, but is in the sum too, and
// stays; a part whose exponential is 0 may have an infinite distance.)
__device__ __forceinline__ void add_part(const HeadProbsArgs& a, float m, const float2& p, float pe, float& l, float& e) {
    const float x = (p.x - m) * a.inv_temp, f = expf(x);
    l = fmaf(p.y, f, l);
    if (f > 0.f) e = fmaf(f, fmaf(pe, 0.693147181f, p.y * x), e);
}

__device__ __forceinline__ void write_top(const HeadProbsArgs& a, int64_t t, const uint64_t* sorted, int held,
                                          const Row& r) {
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        a.top_ids[t * a.k + i] = i < held ? (int64_t)place_of(sorted[i]) : -1;
        a.top_logprobs[t * a.k + i] = !r.fine     ? nan_f()
                                      : i < held ? fmaf(from_order(order_in(sorted[i])) - r.m, a.inv_temp, -r.log_l)
                                                 : -INFINITY;
    }
}

// The parts' statistics in registers, PER a thread (more parts: joined as they are read).
template <int PER>
struct Parts {
    uint32_t order[PER];  // of the parts' maxima
};
template <int PER>
__device__ __forceinline__ Row join_parts(const HeadProbsArgs& a, int64_t c, int64_t t, Parts<PER>& parts, Joins& red) {
    const float2* const part = a.part + c;
    const float* const part_e = a.part_e + c;
    float2 p[PER];
    float pe[PER];
    #pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int i = u * kThreads + (int)threadIdx.x;
        const bool in = i < a.parts;
        p[u] = in ? part[i * a.t_pad] : make_float2(-INFINITY, 0.f);
        pe[u] = in ? part_e[i * a.t_pad] : 0.f;
    }
    float m = -INFINITY;
    #pragma unroll
    for (int u = 0; u < PER; ++u) m = fmaxf(m, p[u].x);
    for (int i = PER * kThreads + (int)threadIdx.x; i < a.parts; i += kThreads) m = fmaxf(m, part[i * a.t_pad].x);
    m = block_max(m, red);
    float l = 0.f, e = 0.f;
    #pragma unroll
    for (int u = 0; u < PER; ++u) {
        add_part(a, m, p[u], pe[u], l, e);
        parts.order[u] = order_of(p[u].x);
    }
    for (int i = PER * kThreads + (int)threadIdx.x; i < a.parts; i += kThreads)
        add_part(a, m, part[i * a.t_pad], part_e[i * a.t_pad], l, e);
    l = block_add(l, red);
    e = block_add(e, red);
    return row_of(a, c, t, m, l, e, threadIdx.x == 0);
}

// Statistics alone, of many rows: 16 rows by 16 threads a block, so that the rows' parts,
// which lie side by side, are read in whole lines.  The sums are added as join_parts adds
// them (a thread stands for 16 of its 256): outputs do not depend on K or on the number
// of tokens.
constexpr int kJoinRows = 16;
__global__ __launch_bounds__(kThreads) void probs_join_kernel(HeadProbsArgs a) {
    const int n = *a.count;
    const int r = threadIdx.x / 16, g = threadIdx.x % 16;
    const int64_t c = (int64_t)blockIdx.x * kJoinRows + r;
    if (c >= a.tokens) return;
    const int64_t t = a.src[c];
    if (c >= n) {
        idle_row(a, t, g, 16);
        return;
    }
    const float2* const part = a.part + c;
    const float* const part_e = a.part_e + c;
    float m = -INFINITY;
    #pragma unroll 4
    for (int i = g; i < a.parts; i += 16) m = fmaxf(m, part[i * a.t_pad].x);
    #pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 16));
    float l[kWaves], e[kWaves];
    #pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        float pl[4] = {0.f, 0.f, 0.f, 0.f}, pe[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = 64 * w + g; i < a.parts; i += kThreads) {
            #pragma unroll
            for (int b = 0; b < 4; ++b)
                if (i + 16 * b < a.parts) add_part(a, m, part[(i + 16 * b) * a.t_pad], part_e[(i + 16 * b) * a.t_pad], pl[b], pe[b]);
        }
        l[w] = (pl[0] + pl[2]) + (pl[1] + pl[3]);
        e[w] = (pe[0] + pe[2]) + (pe[1] + pe[3]);
        #pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
            l[w] += __shfl_xor(l[w], off, 16);
            e[w] += __shfl_xor(e[w], off, 16);
        }
    }
    row_of(a, c, t, m, (l[0] + l[1]) + (l[2] + l[3]), (e[0] + e[1]) + (e[2] + e[3]), g == 0);
}

// Statistics alone, of few rows.
__global__ __launch_bounds__(kThreads) void probs_row_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t, threadIdx.x, kThreads);
        return;
    }
    Parts<8> parts;
    join_parts<8>(a, c, t, parts, red);
}

// Alternatives from the row's kept logits (at most 64 kK words).
constexpr int kKeptPer = 64 * kK / kThreads;
__global__ __launch_bounds__(kThreads) void probs_logits_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint64_t keys[kK], sorted[kK];
    __shared__ int taken;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t, threadIdx.x, kThreads);
        return;
    }
    Parts<1> parts;
    const Row r = join_parts<1>(a, c, t, parts, red);
    int held = 0;
    if (r.fine) {
        const float* const row = a.logits + c * a.logits_ld;
        uint32_t o[kKeptPer];
        #pragma unroll
        for (int u = 0; u < kKeptPer; ++u) {
            const int i = u * kThreads + (int)threadIdx.x;
            o[u] = i < a.vocab ? order_of(row[i]) : 0;
        }
        held = largest<kKeptPer>(o, [&](int u) { return (uint32_t)(u * kThreads + (int)threadIdx.x); }, a.k, keys, &taken, red);
        sort_keys(keys, held, sorted);
    }
    write_top(a, t, sorted, held, r);
}

// One wave: the logits of a row of H and four rows of W.
template <int ESIZE>
__device__ __forceinline__ void dots(const HeadProbsArgs& a, int64_t t, const uint32_t (&word)[4], float (&s)[4]) {
    const int lane = threadIdx.x & 63;
    #pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = 0.f;
    if (ESIZE == 2) {
        const uint16_t* h = static_cast<const uint16_t*>(a.hidden) + t * a.cols;
        const uint16_t* w = static_cast<const uint16_t*>(a.weight);
        if (a.cols % 8 == 0) {
            #pragma unroll 2
            for (int64_t d = lane * 8; d < a.cols; d += 512) {
                const uint4 u = *reinterpret_cast<const uint4*>(h + d);
                const uint32_t us[4] = {u.x, u.y, u.z, u.w};
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 v = *reinterpret_cast<const uint4*>(w + word[q] * a.cols + d);
                    const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[q] = fmaf(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16), s[q]);
                        s[q] = fmaf(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(vs[e] & 0xffff0000u), s[q]);
                    }
                }
            }
        } else {
            for (int64_t d = lane; d < a.cols; d += 64) {
                const float x = bf16_to_f32(h[d]);
                #pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = fmaf(x, bf16_to_f32(w[word[q] * a.cols + d]), s[q]);
            }
        }
    } else {
        const float* h = static_cast<const float*>(a.hidden) + t * a.cols;
        const float* w = static_cast<const float*>(a.weight);
        if (a.cols % 4 == 0) {
            #pragma unroll 2
            for (int64_t d = lane * 4; d < a.cols; d += 256) {
                const float4 u = *reinterpret_cast<const float4*>(h + d);
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v = *reinterpret_cast<const float4*>(w + word[q] * a.cols + d);
                    s[q] = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, s[q]))));
                }
            }
        } else {
            for (int64_t d = lane; d < a.cols; d += 64) {
                #pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = fmaf(h[d], w[word[q] * a.cols + d], s[q]);
            }
        }
    }
    #pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = wave_add(s[q]);
}

__device__ __forceinline__ uint32_t group_of(uint32_t word) { return word / 32 * 2 + ((word >> 2) & 1); }
__device__ __forceinline__ uint32_t word_of(uint32_t group, int at) {
    return group / 2 * 32 + 8 * (at / 4) + 4 * (group & 1) + at % 4;
}
// The order of a group's second logit, or up to 15 more: its last four bits hold a place.
__device__ __forceinline__ uint32_t second_order(float shown) {
    const uint32_t u = __float_as_uint(shown);
    return order_of(__uint_as_float(u >> 31 ? u & ~15u : u | 15u));
}

constexpr int kShown = kK * 8;                // largest logits of the groups of kK parts of 128 words
constexpr int kPool = kK + kK * 16;           // ... and after groups are opened
constexpr int kPoolPer = (kPool + kThreads - 1) / kThreads;

// Statistics, and alternatives from the parts' groups.  PER: parts a thread.
template <int ESIZE, int PER>
__global__ __launch_bounds__(kThreads) void probs_groups_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint64_t pool[kPool], keys[kK], sorted[kK];
    __shared__ uint32_t open[kK];
    __shared__ int taken, opened;
    static_assert(kShown <= kPool, "the groups' logits fit");
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t, threadIdx.x, kThreads);
        return;
    }
    Parts<PER> p;
    const Row r = join_parts<PER>(a, c, t, p, red);
    if (!r.fine) {
        write_top(a, t, sorted, 0, r);
        return;
    }
    int parts = largest<PER>(p.order, [&](int u) { return (uint32_t)(u * kThreads + (int)threadIdx.x); }, a.k, keys, &taken, red);
    // more parts: the best of those before and the next ones
    for (int first = PER * kThreads; first < a.parts; first += PER * kThreads - kK) {
        uint32_t o[PER], at[PER];
        #pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int i = u * kThreads + (int)threadIdx.x, next = first + i - kK;
            const uint64_t before = i < parts ? keys[i] : 0;
            const bool in = i >= kK && next < a.parts;
            o[u] = i < kK ? order_in(before) : in ? order_of(a.part[next * a.t_pad + c].x) : 0;
            at[u] = i < kK ? place_of(before) : (uint32_t)next;
        }
        parts = largest<PER>(o, [&](int u) { return at[u]; }, a.k, keys, &taken, red);
    }
    // the logits that those parts' groups show; the K largest
    const int groups = a.part_rows / 16;
    for (int i = threadIdx.x; i < parts * groups; i += kThreads) {
        const uint32_t g = place_of(keys[i / groups]) * groups + i % groups;
        const float2 x = a.top[g * a.t_pad + c];
        pool[i] = key_of(order_of(x.x), word_of(g, (int)(__float_as_uint(x.y) & 15u)));
    }
    if (threadIdx.x == 0) opened = 0;
    __syncthreads();
    int held = largest_keys<kShown / kThreads>(pool, parts * groups, a.k, keys, &taken, red);
    sort_keys(keys, held, sorted);
    // Groups that may hide one before the last of them (whose own comes after it; fewer than
    // K: any that hides one).
    const uint64_t last = held == a.k ? sorted[held - 1] : 0;
    for (int i = threadIdx.x; i < (held == a.k ? held - 1 : held); i += kThreads) {
        const uint32_t g = group_of(place_of(sorted[i]));
        const uint32_t second = second_order(a.top[g * a.t_pad + c].y);
        if (key_of(second, word_of(g, 0)) > last) open[atomicAdd(&opened, 1)] = i;  // (in any order: they are sorted again)
    }
    __syncthreads();
    if (opened > 0) {
        for (int i = threadIdx.x; i < held; i += kThreads) pool[i] = sorted[i];
        for (int i = threadIdx.x >> 6; i < 4 * opened; i += kWaves) {
            const uint32_t shown = place_of(sorted[open[i / 4]]), g = group_of(shown);
            uint32_t word[4], from[4];
            #pragma unroll
            for (int q = 0; q < 4; ++q) {
                word[q] = word_of(g, 4 * (i % 4) + q);
                from[q] = word[q] < a.vocab ? word[q] : shown;
            }
            float s[4];
            dots<ESIZE>(a, t, from, s);
            if ((threadIdx.x & 63) == 0) {
                #pragma unroll
                for (int q = 0; q < 4; ++q)
                    pool[held + 4 * i + q] = word[q] < a.vocab && word[q] != shown ? key_of(order_of(s[q]), word[q]) : 0;
            }
        }
        __syncthreads();
        held = largest_keys<kPoolPer>(pool, held + 16 * opened, a.k, keys, &taken, red);
        sort_keys(keys, held, sorted);
    }
    write_top(a, t, sorted, held, r);
}

template <int ESIZE>
void launch_groups(const HeadProbsArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.tokens), block(kThreads);
    if (a.parts <= 4 * kThreads) hipLaunchKernelGGL((probs_groups_kernel<ESIZE, 4>), grid, block, 0, stream, a);
    else if (a.parts <= 8 * kThreads) hipLaunchKernelGGL((probs_groups_kernel<ESIZE, 8>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((probs_groups_kernel<ESIZE, 24>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_head_probs(const HeadProbsArgs& a, hipStream_t stream) {
    const dim3 block(kThreads);
    if (a.k == 0) {
        // (8192 rows of 1002 parts: 169 us a block a row)
        if (a.tokens > 1024)
            hipLaunchKernelGGL(probs_join_kernel, dim3((unsigned)((a.tokens + kJoinRows - 1) / kJoinRows)), block, 0, stream, a);
        else
            hipLaunchKernelGGL(probs_row_kernel, dim3((unsigned)a.tokens), block, 0, stream, a);
    } else if (a.logits != nullptr) {
        hipLaunchKernelGGL(probs_logits_kernel, dim3((unsigned)a.tokens), block, 0, stream, a);
    } else if (a.esize == 2) {
        launch_groups<2>(a, stream);
    } else {
        launch_groups<4>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace dmuon
