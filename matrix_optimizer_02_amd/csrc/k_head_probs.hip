// Row kernels of the output head's log probabilities (gfx950): one workgroup a
// token joins the statistics that the logits' products left, and finds the
// alternatives.
//
// A part is the words whose softmax statistics one wave formed: 32 F of them, one after
// the other (F 1, 2 or 4).  A group is 16 words of one lane: group h F + i of a part (h <
// 2, i < F) holds its words 32 i + 8 q + 4 h + r (q, r < 4) as its elements 4 q + r,
// in the order of their ids.  Of each group the products' epilogue shows the largest logit,
// its place and the size of the second.
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
// a threshold, two bits of it a round.  A row of 128256 words, 20 alternatives: 15 us (5 of
// them the statistics), 27 where a group is opened; 2048 rows with 5 49 us, 4096 with 64 120.
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

// At least the k largest and at most `most` (>= k) of n values in LDS (n <= PER kThreads;
// orders o, 0 where there is none; at places p, or INDEX: at their own), equal ones by the
// lower place, in any order; returns their number (fewer than k where there are not as
// many).  Counting how many reach a threshold, two bits of it a round: a few rounds leave few
// enough of them.  Then, of too many that equal the threshold, the same with their places,
// from the last on.
template <int PER, bool INDEX = false>
__device__ __forceinline__ int largest(const uint32_t* o, const uint32_t* p, int n, int k, int most, uint64_t* out,
                                       int* taken, Joins& red) {
    __syncthreads();  // the values are there, and the last call's number has been read
    if (threadIdx.x == 0) *taken = 0;
    uint32_t x[PER];
    #pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int i = u * kThreads + (int)threadIdx.x;
        x[u] = i < n ? o[i] : 0;
    }
    uint32_t least = 0, low = 0, at = 0;
    int reach = n, above = 0, bit = 30, turn = 0;
    enum { kOrders, kAbove, kPlaces } pass = kOrders;
    #pragma unroll 1
    while (reach > most) {
        // thresholds of this round (no order is the largest integer)
        const uint32_t a = pass == kAbove ? least + 1 : at | 1u << bit, b = at | 2u << bit, c = at | 3u << bit;
        int4 s = make_int4(0, 0, 0, 0);
        #pragma unroll
        for (int u = 0; u < PER; ++u) {
            if (u > 0 && u * kThreads >= n) break;
            s.x += __popcll(__builtin_amdgcn_ballot_w64(x[u] >= a));
            s.y += __popcll(__builtin_amdgcn_ballot_w64(x[u] >= b));
            s.z += __popcll(__builtin_amdgcn_ballot_w64(x[u] >= c));
        }
        turn ^= 1;  // (the counts of the round before may still be read)
        if ((threadIdx.x & 63) == 0) red.counts[turn][threadIdx.x >> 6] = s;
        __syncthreads();
        s = red.counts[turn][0];
        #pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            const int4 m = red.counts[turn][w];
            s.x += m.x, s.y += m.y, s.z += m.z;
        }
        if (pass == kAbove) {
            above = s.x;
            #pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int i = u * kThreads + (int)threadIdx.x;
                x[u] = x[u] == least ? ~(INDEX ? (uint32_t)i : p[i]) : 0;  // (least > 0: i < n)
            }
            pass = kPlaces;
            at = 0;
            bit = 30;
            continue;
        }
        if (above + s.z >= k) at = c, reach = above + s.z;
        else if (above + s.y >= k) at = b, reach = above + s.y;
        else if (above + s.x >= k) at = a, reach = above + s.x;
        (pass == kOrders ? least : low) = at;
        bit -= 2;
        if (bit < 0) {
            if (least == 0 || pass == kPlaces) break;  // (fewer than k: all of them)
            pass = kAbove;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t y = o[i], place = INDEX ? (uint32_t)i : p[i];
        if (y != 0 && (y > least || (y == least && ~place >= low)))
            out[atomicAdd(taken, 1)] = key_of(y, place);  // (places in a list that is sorted)
    }
    __syncthreads();
    return *taken;
}

// The k first of n different keys in descending order.
__device__ __forceinline__ int sort_keys(const uint64_t* keys, int n, int k, uint64_t* sorted) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t mine = keys[i];
        int rank = 0;
        #pragma unroll 16
        for (int j = 0; j < n; ++j) rank += keys[j] > mine ? 1 : 0;
        if (rank < k) sorted[rank] = mine;
    }
    __syncthreads();
    return n < k ? n : k;
}

// A token that takes no part.
__device__ __forceinline__ void idle_row(const HeadProbsArgs& a, int64_t t) {
    if (threadIdx.x == 0) {
        if (a.logprobs != nullptr) a.logprobs[t] = 0.f;
        if (a.entropy != nullptr) a.entropy[t] = 0.f;
        a.lse[t] = 0.f;
    }
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
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
__device__ __forceinline__ Row row_of(const HeadProbsArgs& a, int64_t c, int64_t t, float m, float l, float e) {
    Row r{m, nan_f(), l > 0.f && l < INFINITY};
    if (r.fine) r.log_l = logf(l);
    if (threadIdx.x == 0) {
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

// Parts a thread takes, one after the other.
__device__ __forceinline__ int share_of_parts(const HeadProbsArgs& a) { return (a.parts + kThreads - 1) / kThreads; }

// The row's outputs from its parts; orders (null: not) receives those of each thread's
// largest maximum.
__device__ __forceinline__ Row join_parts(const HeadProbsArgs& a, int64_t c, int64_t t, uint32_t* orders, Joins& red) {
    const int per = share_of_parts(a), first = (int)threadIdx.x * per;
    const int mine = max(0, min(per, a.parts - first));
    const float2* const part = a.part + c * a.row_parts + first;
    const float* const part_e = a.part_e + c * a.row_parts + first;
    constexpr int kAhead = 8;  // loads on their way at once; the first ones' results are kept
    float2 x[kAhead];
    float y[kAhead];
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        x[u] = u < mine ? part[u] : make_float2(-INFINITY, 0.f);
        y[u] = u < mine ? part_e[u] : 0.f;
    }
    float m = -INFINITY;
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) m = fmaxf(m, x[u].x);
    #pragma unroll 1
    for (int i = kAhead; i < mine; i += kAhead) {
        float z[kAhead];
        #pragma unroll
        for (int u = 0; u < kAhead; ++u) z[u] = part[min(i + u, mine - 1)].x;
        #pragma unroll
        for (int u = 0; u < kAhead; ++u) m = fmaxf(m, z[u]);
    }
    if (orders != nullptr) orders[threadIdx.x] = order_of(m);
    m = block_max(m, red);
    float l = 0.f, e = 0.f;
    #pragma unroll 1
    for (int i = 0;;) {
        #pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i + u < mine) add_part(a, m, x[u], y[u], l, e);
        i += kAhead;
        if (i >= mine) break;
        #pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int at = min(i + u, mine - 1);
            x[u] = part[at];
            y[u] = part_e[at];
        }
    }
    l = block_add(l, red);
    e = block_add(e, red);
    return row_of(a, c, t, m, l, e);
}

// Statistics alone.  8192 rows of 1002 parts, 5734 of them live: 19 us, for 48 a wave a row.
__global__ __launch_bounds__(kThreads) void probs_row_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t);
        return;
    }
    join_parts(a, c, t, nullptr, red);
}

// Alternatives from the row's kept logits.
constexpr int kKept = 64 * kK;
__global__ __launch_bounds__(kThreads) void probs_logits_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint32_t orders[kKept];
    __shared__ uint64_t keys[kK], sorted[kK];
    __shared__ int taken;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t);
        return;
    }
    const Row r = join_parts(a, c, t, nullptr, red);
    int held = 0;
    if (r.fine) {
        const float* const row = a.logits + c * a.logits_ld;
        const int n = (int)a.vocab;  // at most kKept (head_layout.cpp)
        #pragma unroll 8
        for (int i = threadIdx.x; i < n; i += kThreads) orders[i] = order_of(row[i]);
        held = sort_keys(keys, largest<kKept / kThreads, true>(orders, nullptr, n, a.k, kK, keys, &taken, red), a.k, sorted);
    }
    write_top(a, t, sorted, held, r);
}

// One wave: the logits of a row of H and four rows of W, kDeep loads of each on their way.
constexpr int kDeep = 4;
template <int ESIZE>
__device__ __forceinline__ void dots(const HeadProbsArgs& a, int64_t t, const uint32_t (&word)[4], float (&s)[4]) {
    const int lane = threadIdx.x & 63;
    #pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = 0.f;
    if (ESIZE == 2) {
        const uint16_t* h = static_cast<const uint16_t*>(a.hidden) + t * a.cols;
        const uint16_t* w = static_cast<const uint16_t*>(a.weight);
        if (a.cols % 8 == 0) {
            #pragma unroll 1
            for (int64_t d0 = lane * 8; d0 < a.cols; d0 += 512 * kDeep) {
                uint4 u[kDeep], v[kDeep][4];
                #pragma unroll
                for (int i = 0; i < kDeep; ++i) {
                    const int64_t d = min(d0 + 512 * i, a.cols - 8);
                    u[i] = *reinterpret_cast<const uint4*>(h + d);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = *reinterpret_cast<const uint4*>(w + word[q] * a.cols + d);
                }
                #pragma unroll
                for (int i = 0; i < kDeep; ++i) {
                    if (d0 + 512 * i >= a.cols) break;
                    const uint32_t us[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t vs[4] = {v[i][q].x, v[i][q].y, v[i][q].z, v[i][q].w};
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[q] = fmaf(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16), s[q]);
                            s[q] = fmaf(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(vs[e] & 0xffff0000u), s[q]);
                        }
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
            #pragma unroll 1
            for (int64_t d0 = lane * 4; d0 < a.cols; d0 += 256 * kDeep) {
                float4 u[kDeep], v[kDeep][4];
                #pragma unroll
                for (int i = 0; i < kDeep; ++i) {
                    const int64_t d = min(d0 + 256 * i, a.cols - 4);
                    u[i] = *reinterpret_cast<const float4*>(h + d);
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = *reinterpret_cast<const float4*>(w + word[q] * a.cols + d);
                }
                #pragma unroll
                for (int i = 0; i < kDeep; ++i) {
                    if (d0 + 256 * i >= a.cols) break;
                    #pragma unroll
                    for (int q = 0; q < 4; ++q)
                        s[q] = fmaf(u[i].x, v[i][q].x, fmaf(u[i].y, v[i][q].y, fmaf(u[i].z, v[i][q].z, fmaf(u[i].w, v[i][q].w, s[q]))));
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

// Groups and their words, for parts of 32 << f words.
__device__ __forceinline__ uint32_t group_of(uint32_t word, int f) {
    const uint32_t part = word >> (5 + f), i = (word >> 5) & ((1 << f) - 1), h = (word >> 2) & 1;
    return (((part << 1) + h) << f) + i;
}
__device__ __forceinline__ uint32_t word_of(uint32_t group, int at, int f) {
    const uint32_t i = group & ((1 << f) - 1), h = (group >> f) & 1, part = group >> (f + 1);
    return (part << (5 + f)) + 32 * i + 8 * (at / 4) + 4 * h + at % 4;
}
// The order of a group's second logit, or up to 15 more: its last four bits hold a place.
__device__ __forceinline__ uint32_t second_order(float shown) {
    const uint32_t u = __float_as_uint(shown);
    return order_of(__uint_as_float(u >> 31 ? u & ~15u : u | 15u));
}

constexpr int kFew = 2;              // a round leaves up to kFew K candidates: fewer take more steps to find
constexpr int kList = 512;           // of threads, then parts, that may hold alternatives
constexpr int kPool = kK + kK * 16;  // candidates after groups are opened
constexpr int kPoolPer = (kPool + kThreads - 1) / kThreads;

// Statistics, and alternatives from the parts' groups.
template <int ESIZE>
__global__ __launch_bounds__(kThreads) void probs_groups_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint32_t orders[kPool], places[kPool];
    __shared__ uint64_t keys[kList], sorted[kK];
    __shared__ uint32_t list[kThreads], open[kK];
    __shared__ int taken, opened;
    static_assert(kK * 8 <= kPool && kK <= kPool / 8, "the groups of kK parts of 128 words fit");
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t);
        return;
    }
    const Row r = join_parts(a, c, t, orders, red);
    if (!r.fine) {
        write_top(a, t, sorted, 0, r);
        return;
    }
    // Of the threads' largest maxima the K largest and as many more as the next round holds, of
    // those threads' parts in the same way (a thread's parts follow one another), of those
    // parts' groups, and of the words of groups that are opened.  One loop, so that the code is
    // fetched once.
    enum { kOfThreads, kOfParts, kOfGroups, kOfWords } stage = kOfThreads;
    places[threadIdx.x] = list[threadIdx.x] = threadIdx.x;
    const int per = share_of_parts(a), groups = a.part_rows / 16, f = groups / 4;  // (groups 2, 4 or 8)
    int n = kThreads, threads = 0, first = 0, held = 0;
    #pragma unroll 1
    for (;;) {
        const int most = stage == kOfThreads ? min(kThreads, max(a.k, min(kFew * a.k, kPool / per)))
                         : stage == kOfParts ? min(kList, max(a.k, min(kFew * a.k, kPool / groups))) : kK;
        // (all threads' parts may fit the next round as they are)
        const bool all = stage == kOfThreads && most == kThreads && kThreads * per <= kPool;
        const int got = all ? kThreads : largest<kPoolPer>(orders, places, n, a.k, most, keys, &taken, red);
        if (stage >= kOfGroups) {
            held = sort_keys(keys, got, a.k, sorted);
            if (stage == kOfWords) break;
            // Groups that may hide one before the last of them (whose own comes after it; fewer
            // than K: any that hides one).
            const uint64_t last = held == a.k ? sorted[held - 1] : 0;
            for (int i = threadIdx.x; i < (held == a.k ? held - 1 : held); i += kThreads) {
                const uint32_t g = group_of(place_of(sorted[i]), f);
                const uint32_t second = second_order(a.top[c * a.row_groups + g].y);
                if (key_of(second, word_of(g, 0, f)) > last) open[atomicAdd(&opened, 1)] = i;  // (in any order, too)
            }
            __syncthreads();
            if (opened == 0) break;
            for (int i = threadIdx.x; i < held; i += kThreads) {
                orders[i] = order_in(sorted[i]);
                places[i] = place_of(sorted[i]);
            }
            for (int i = threadIdx.x >> 6; i < 4 * opened; i += kWaves) {
                const uint32_t shown = place_of(sorted[open[i / 4]]), g = group_of(shown, f);
                uint32_t word[4], from[4];
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    word[q] = word_of(g, 4 * (i % 4) + q, f);
                    from[q] = word[q] < a.vocab ? word[q] : shown;
                }
                float s[4];
                dots<ESIZE>(a, t, from, s);
                if ((threadIdx.x & 63) == 0) {
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int at = held + 4 * i + q;
                        orders[at] = word[q] < a.vocab && word[q] != shown ? order_of(s[q]) : 0;
                        places[at] = word[q];
                    }
                }
            }
            n = held + 16 * opened;
            stage = kOfWords;
            continue;
        }
        int parts = got;
        if (stage == kOfThreads) {
            if (!all && (int)threadIdx.x < got) list[threadIdx.x] = place_of(keys[threadIdx.x]);
            if (threadIdx.x == 0) opened = 0;
            __syncthreads();
            threads = got;
            parts = 0;
            stage = kOfParts;
        }
        if (first < threads * per) {
            // (more than the pool holds: the best of those before and the next ones)
            const int next = min(threads * per - first, kPool - parts);
            for (int i = threadIdx.x; i < parts + next; i += kThreads) {
                const int at = first + i - parts;
                const int part = i < parts ? (int)place_of(keys[i]) : (int)list[at / per] * per + at % per;
                orders[i] = i < parts ? order_in(keys[i]) : part < a.parts ? order_of(a.part[c * a.row_parts + part].x) : 0;
                places[i] = (uint32_t)part;
            }
            first += next;
            n = parts + next;
            continue;
        }
        // what those parts' groups show
        for (int i = threadIdx.x; i < parts * groups; i += kThreads) {
            const uint32_t g = place_of(keys[i / groups]) * groups + i % groups;
            const float2 x = a.top[c * a.row_groups + g];
            orders[i] = order_of(x.x);
            places[i] = word_of(g, (int)(__float_as_uint(x.y) & 15u), f);
        }
        n = parts * groups;
        stage = kOfGroups;
    }
    write_top(a, t, sorted, held, r);
}

}  // namespace

hipError_t launch_head_probs(const HeadProbsArgs& a, hipStream_t stream) {
    const dim3 block(kThreads), rows((unsigned)a.tokens);
    if (a.k == 0) hipLaunchKernelGGL(probs_row_kernel, rows, block, 0, stream, a);
    else if (a.logits != nullptr) hipLaunchKernelGGL(probs_logits_kernel, rows, block, 0, stream, a);
    else if (a.esize == 2) hipLaunchKernelGGL((probs_groups_kernel<2>), rows, block, 0, stream, a);
    else hipLaunchKernelGGL((probs_groups_kernel<4>), rows, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace dmuon
