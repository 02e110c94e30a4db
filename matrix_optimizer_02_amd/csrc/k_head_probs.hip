// Row kernels of the output head's log probabilities (gfx950): one workgroup a
// token joins the statistics that the logits' products left, and finds the
// alternatives.
//
// A part is the words whose softmax statistics one wave formed (32 to 128 of them,
// one after the other); a group is 16 words of one lane: of the block of 32 words
// b, group 2 b + h holds words 32 b + 8 q + 4 h + r (q, r < 4) as its elements
// 4 q + r, so a group's elements are in the order of their ids.  The products' epilogue
// leaves each group's two largest logits.
//
// The K alternatives lie in the K parts with the largest maxima (equal maxima: the
// earlier part): were one in another part, each of those K parts would hold a word
// before it.  So the K parts' groups hold all candidates, except that a group with
// both of its shown logits among the row's K may hide a third: the logits of such groups
// are formed again from H and W.  A row's K spread over V / 16 groups share
// one 8 K^2 / V times: 0.02 times for K = 20 of 128256 words, once for K = 128.
#include "head_internal.h"
#include "kcommon.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kK = kHeadMaxAlternatives;

__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7fc00000u); }

// Floats as integers of the same order (-0 as +0), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kOrderNegInf = 0x007fffffu;  // of -inf

// What is sorted: a logit and its place, the larger logit and then the lower place
// first.  No two are the same; 0: nothing (-inf too).
__device__ __forceinline__ uint64_t key_of(float x, uint32_t at) {
    const uint32_t o = order_of(x);
    return o > kOrderNegInf ? ((uint64_t)o << 32) | (uint32_t)~at : 0;
}
__device__ __forceinline__ uint32_t place_of(uint64_t key) { return ~(uint32_t)key; }
__device__ __forceinline__ float logit_of(uint64_t key) { return from_order((uint32_t)(key >> 32)); }

// Joins over the block, the same in every thread, in a fixed order.
struct Joins {
    float f[kWaves];
    int i[2][kWaves];
};
__device__ __forceinline__ float block_max(float v, Joins& red) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red.f[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red.f[0];
    #pragma unroll
    for (int w = 1; w < kWaves; ++w) v = fmaxf(v, red.f[w]);
    return v;
}
__device__ __forceinline__ float block_add(float v, Joins& red) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red.f[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red.f[0];
    #pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red.f[w];
    return v;
}

// The k largest of n different keys that are not 0, in any order; returns their
// number (fewer than k where there are not as many).  The k-th largest is found bit by
// bit, by counting the keys that are no smaller: 32 rounds at most unless it equals
// another logit.
template <typename F>
__device__ __forceinline__ int largest(int n, int k, F&& key, uint64_t* out, int* taken, Joins& red) {
    int turn = 0;
    auto count = [&](uint64_t least) {
        int c = 0;
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + (int)threadIdx.x;
            c += __popcll(__builtin_amdgcn_ballot_w64(i < n && key(i) >= least));
        }
        turn ^= 1;  // (the counts of the round before may still be read)
        if ((threadIdx.x & 63) == 0) red.i[turn][threadIdx.x >> 6] = c;
        __syncthreads();
        c = red.i[turn][0];
        #pragma unroll
        for (int w = 1; w < kWaves; ++w) c += red.i[turn][w];
        return c;
    };
    __syncthreads();
    const int held = count(1);
    if (k > held) k = held;
    if (threadIdx.x == 0) *taken = 0;
    uint64_t least = k == held ? 1 : 0;
    for (int bit = 63, reach = held; bit >= 0 && reach != k; --bit) {
        const uint64_t at = least | (1ull << bit);
        const int c = count(at);
        if (c >= k) least = at, reach = c;
    }
    __syncthreads();
    if (k > 0)
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t x = key(i);
            if (x >= least) out[atomicAdd(taken, 1)] = x;  // (places in a list that is sorted next)
        }
    __syncthreads();
    return k;
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

// The row's softmax from its parts: largest logit m, l = sum of exp((s - m) / T), e =
// the sum of that times (s - m) / T.
__device__ __forceinline__ Row join_parts(const HeadProbsArgs& a, int64_t c, int64_t t, Joins& red) {
    const float2* const part = a.part + c;
    const float* const part_e = a.part_e + c;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < a.parts; i += kThreads) m = fmaxf(m, part[i * a.t_pad].x);
    m = block_max(m, red);
    float l = 0.f, e = 0.f;
    // (a NaN does not survive fmaxf, but is in the sum too, and stays)
    for (int i = threadIdx.x; i < a.parts; i += kThreads) {
        const float2 p = part[i * a.t_pad];
        const float x = (p.x - m) * a.inv_temp, f = expf(x);
        l = fmaf(p.y, f, l);
        if (f > 0.f) e = fmaf(f, fmaf(part_e[i * a.t_pad], 0.693147181f, p.y * x), e);
    }
    l = block_add(l, red);
    e = block_add(e, red);
    Row r{m, nan_f(), l > 0.f && l < INFINITY};
    if (r.fine) r.log_l = logf(l);
    if (threadIdx.x == 0) {
        a.lse[t] = r.fine ? fmaf(m, a.inv_temp, r.log_l) : nan_f();
        if (a.entropy != nullptr) a.entropy[t] = r.log_l - e / l;
        if (a.logprobs != nullptr)
            a.logprobs[t] = a.target[c] < 0 ? nan_f() : fmaf(a.target_logit[c] - m, a.inv_temp, -r.log_l);
    }
    if (!r.fine)
        for (int i = threadIdx.x; i < a.k; i += kThreads) {
            a.top_ids[t * a.k + i] = -1;
            a.top_logprobs[t * a.k + i] = nan_f();
        }
    return r;
}

__device__ __forceinline__ void write_top(const HeadProbsArgs& a, int64_t t, const uint64_t* sorted, int held,
                                          const Row& r) {
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        a.top_ids[t * a.k + i] = i < held ? (int64_t)place_of(sorted[i]) : -1;
        a.top_logprobs[t * a.k + i] = i < held ? fmaf(logit_of(sorted[i]) - r.m, a.inv_temp, -r.log_l) : -INFINITY;
    }
}

// Statistics alone, or alternatives from the row's kept logits.
__global__ __launch_bounds__(kThreads) void probs_logits_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint64_t keys[kK], sorted[kK];
    __shared__ int taken;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t);
        return;
    }
    const Row r = join_parts(a, c, t, red);
    if (!r.fine || a.k == 0) return;
    const float* const row = a.logits + c * a.logits_ld;
    const int held = largest((int)a.vocab, a.k, [&](int i) { return key_of(row[i], i); }, keys, &taken, red);
    sort_keys(keys, held, sorted);
    write_top(a, t, sorted, held, r);
}

// One wave: the logit of a row of H and a row of W.
template <int ESIZE>
__device__ __forceinline__ float dot(const HeadProbsArgs& a, int64_t t, int64_t word) {
    const int lane = threadIdx.x & 63;
    float s = 0.f;
    if (ESIZE == 2) {
        const uint16_t* h = static_cast<const uint16_t*>(a.hidden) + t * a.cols;
        const uint16_t* w = static_cast<const uint16_t*>(a.weight) + word * a.cols;
        if (a.cols % 8 == 0) {
            #pragma unroll 4
            for (int64_t d = lane * 8; d < a.cols; d += 512) {
                const uint4 u = *reinterpret_cast<const uint4*>(h + d), v = *reinterpret_cast<const uint4*>(w + d);
                const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s = fmaf(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16), s);
                    s = fmaf(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(vs[e] & 0xffff0000u), s);
                }
            }
        } else {
            for (int64_t d = lane; d < a.cols; d += 64) s = fmaf(bf16_to_f32(h[d]), bf16_to_f32(w[d]), s);
        }
    } else {
        const float* h = static_cast<const float*>(a.hidden) + t * a.cols;
        const float* w = static_cast<const float*>(a.weight) + word * a.cols;
        if (a.cols % 4 == 0) {
            #pragma unroll 4
            for (int64_t d = lane * 4; d < a.cols; d += 256) {
                const float4 u = *reinterpret_cast<const float4*>(h + d), v = *reinterpret_cast<const float4*>(w + d);
                s = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, s))));
            }
        } else {
            for (int64_t d = lane; d < a.cols; d += 64) s = fmaf(h[d], w[d], s);
        }
    }
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
    return s;
}

__device__ __forceinline__ uint32_t group_of(uint32_t word) { return word / 32 * 2 + ((word >> 2) & 1); }
__device__ __forceinline__ uint32_t word_of(uint32_t group, int at) {
    return group / 2 * 32 + 8 * (at / 4) + 4 * (group & 1) + at % 4;
}

constexpr int kHidden = 14;  // words that a group does not show
constexpr int kPool = kK * 16;  // shown logits of kK parts of 128 words
static_assert(kK + kK / 2 * kHidden <= kPool, "the second round's candidates fit");

// Statistics, and alternatives from the parts' groups.
template <int ESIZE>
__global__ __launch_bounds__(kThreads) void probs_groups_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint64_t pool[kPool], keys[kK], sorted[kK];
    __shared__ uint32_t open[kK / 2];
    __shared__ int taken, opened;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t);
        return;
    }
    const Row r = join_parts(a, c, t, red);
    if (!r.fine) return;
    const float2* const part = a.part + c;
    const int parts = largest(a.parts, a.k, [&](int i) { return key_of(part[i * a.t_pad].x, i); }, keys, &taken, red);
    // the shown logits of those parts' groups
    const int groups = a.part_rows / 16;
    for (int i = threadIdx.x; i < parts * groups; i += kThreads) {
        const uint32_t g = place_of(keys[i / groups]) * groups + i % groups;
        const float2 x = a.top[g * a.t_pad + c];
        const int at = a.top_at[g * a.t_pad + c];
        pool[2 * i] = key_of(x.x, word_of(g, at & 15));
        pool[2 * i + 1] = key_of(x.y, word_of(g, at >> 4));
    }
    if (threadIdx.x == 0) opened = 0;
    __syncthreads();
    int held = largest(2 * parts * groups, a.k, [&](int i) { return pool[i]; }, keys, &taken, red);
    sort_keys(keys, held, sorted);
    // groups whose second logit is among them and not the last: what they hide may be too
    for (int i = threadIdx.x; i < a.k - 1 && i < held; i += kThreads) {
        const uint32_t g = group_of(place_of(sorted[i]));
        bool second = false;
        for (int j = 0; j < i; ++j) second = second || group_of(place_of(sorted[j])) == g;
        if (second) open[atomicAdd(&opened, 1)] = g;  // (the order of the candidates does not matter)
    }
    __syncthreads();
    if (opened > 0) {
        for (int i = threadIdx.x; i < held; i += kThreads) pool[i] = sorted[i];
        for (int i = threadIdx.x >> 6; i < 16 * opened; i += kWaves) {
            const uint32_t g = open[i / 16], word = word_of(g, i % 16);
            bool shown = word >= a.vocab;
            int before = 0;  // shown ones among the elements before
            for (int j = 0; j < held; ++j) {
                const uint32_t w = place_of(sorted[j]);
                shown = shown || w == word;
                before += group_of(w) == g && w < word ? 1 : 0;
            }
            const float s = word < a.vocab && !shown ? dot<ESIZE>(a, t, word) : 0.f;
            // (a group shows two words: the other 14 take its places in order)
            const bool listed = word < a.vocab && shown;
            if ((threadIdx.x & 63) == 0 && !listed) pool[held + i / 16 * kHidden + i % 16 - before] = shown ? 0 : key_of(s, word);
        }
        __syncthreads();
        held = largest(held + opened * kHidden, a.k, [&](int i) { return pool[i]; }, keys, &taken, red);
        sort_keys(keys, held, sorted);
    }
    write_top(a, t, sorted, held, r);
}

}  // namespace

hipError_t launch_head_probs(const HeadProbsArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.tokens), block(kThreads);
    if (a.k == 0 || a.logits != nullptr) hipLaunchKernelGGL(probs_logits_kernel, grid, block, 0, stream, a);
    else if (a.esize == 2) hipLaunchKernelGGL((probs_groups_kernel<2>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((probs_groups_kernel<4>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace dmuon
