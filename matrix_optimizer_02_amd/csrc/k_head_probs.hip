// Row kernels of the output head's log probabilities (gfx950): from a row's
// logits to its outputs.
#include "head_internal.h"
#include "kcommon.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

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

// Sums and maxima over the block, the same in every thread, in a fixed order.
struct Joins {
    float f[kWaves];
    int i[kWaves];
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
__device__ __forceinline__ int block_add(int v, Joins& red) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red.i[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red.i[0];
    #pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red.i[w];
    return v;
}

// The k largest of n values above -inf, equal ones by the lower index, in any
// order: (order, ~index) pairs in out; returns their number (fewer than k where
// there are not as many).  value(i): order_of the i-th.  The k-th largest is found
// bit by bit, by counting.
template <typename F>
__device__ __forceinline__ int largest(int n, int k, F&& value, uint64_t* out, int* taken, Joins& red) {
    auto count = [&](auto&& in) {
        int c = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) c += in(value(i), i) ? 1 : 0;
        return block_add(c, red);
    };
    const int held = count([](uint32_t v, int) { return v > kOrderNegInf; });
    if (k > held) k = held;
    if (k == 0) return 0;
    uint32_t least = 0;
    int reach = 0;  // values >= least
    for (int bit = 31; bit >= 0 && reach != k; --bit) {
        const uint32_t at = least | (1u << bit);
        const int c = count([at](uint32_t v, int) { return v >= at; });
        if (c >= k) least = at, reach = c;
    }
    // of the values that equal the least one, those below index `end`
    int end = n;
    if (reach > k) {
        int lo = 0;  // fewer than k with the equal ones below lo
        while (end - lo > 1) {
            const int mid = lo + (end - lo) / 2;
            const int c = count([=](uint32_t v, int i) { return v > least || (v == least && i < mid); });
            if (c >= k) end = mid; else lo = mid;
        }
    }
    if (threadIdx.x == 0) *taken = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t v = value(i);
        if (v > least || (v == least && i < end)) {
            const int at = atomicAdd(taken, 1);  // (places, not sums: they are sorted next)
            if (at < k) out[at] = ((uint64_t)v << 32) | (uint32_t)~i;
        }
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

// m: the row's largest logit, l: sum of exp((s - m) / T), e: the sum of that times
// (s - m) / T.  A row without a distribution has l neither positive nor finite.
__device__ __forceinline__ bool write_row(const HeadProbsArgs& a, int64_t c, int64_t t, float m, float l, float e,
                                          float target_logit, float& log_l) {
    const bool fine = l > 0.f && l < INFINITY;
    log_l = fine ? logf(l) : nan_f();
    if (threadIdx.x == 0) {
        a.lse[t] = fine ? fmaf(m, a.inv_temp, log_l) : nan_f();
        if (a.entropy != nullptr) a.entropy[t] = log_l - e / l;
        if (a.logprobs != nullptr)
            a.logprobs[t] = a.target[c] < 0 ? nan_f() : fmaf(target_logit - m, a.inv_temp, -log_l);
    }
    if (!fine)
        for (int i = threadIdx.x; i < a.k; i += kThreads) {
            a.top_ids[t * a.k + i] = -1;
            a.top_logprobs[t * a.k + i] = nan_f();
        }
    return fine;
}

__device__ __forceinline__ void write_top(const HeadProbsArgs& a, int64_t t, const uint64_t* sorted, int held, float m,
                                          float log_l) {
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        const uint64_t key = i < held ? sorted[i] : 0;
        a.top_ids[t * a.k + i] = i < held ? (int64_t)(uint32_t)~(uint32_t)key : -1;
        a.top_logprobs[t * a.k + i] = i < held ? fmaf(from_order((uint32_t)(key >> 32)) - m, a.inv_temp, -log_l) : -INFINITY;
    }
}

// One block per token, from its row of logits.
__global__ __launch_bounds__(kThreads) void probs_logits_kernel(HeadProbsArgs a) {
    __shared__ Joins red;
    __shared__ uint64_t keys[kHeadMaxAlternatives], sorted[kHeadMaxAlternatives];
    __shared__ int taken;
    const int64_t c = blockIdx.x;
    const int64_t t = a.src[c];
    if (c >= *a.count) {
        idle_row(a, t);
        return;
    }
    const float* const row = a.logits + c * a.logits_ld;
    const int n = (int)a.vocab;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kThreads) m = fmaxf(m, row[i]);
    m = block_max(m, red);
    float l = 0.f, e = 0.f;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const float x = (row[i] - m) * a.inv_temp, p = expf(x);
        l += p;
        e += p == 0.f ? 0.f : p * x;
    }
    l = block_add(l, red);
    e = block_add(e, red);
    const int target = a.target != nullptr ? a.target[c] : -1;
    float log_l;
    if (!write_row(a, c, t, m, l, e, target >= 0 ? row[target] : 0.f, log_l) || a.k == 0) return;
    const int held = largest(n, a.k, [&](int i) { return order_of(row[i]); }, keys, &taken, red);
    sort_keys(keys, held, sorted);
    write_top(a, t, sorted, held, m, log_l);
}

}  // namespace

hipError_t launch_head_probs(const HeadProbsArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(probs_logits_kernel, dim3((unsigned)a.tokens), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dmuon
