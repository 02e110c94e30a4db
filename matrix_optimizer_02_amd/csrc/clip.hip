// The global norm of many gradients and clipping by it (dmuon_clip.h): argument
// checks, launches and kernels (gfx950).
//
//   norm    one launch per kNormRecs tensors leaves a fp64 sum of squares per
//           workgroup, one workgroup adds them up in order
//   clip    one launch per kClipRecs tensors
//
// A tensor is cut into pieces of 32 KB at 16-byte addresses, so that every
// whole group of 16 bytes is one load whatever element the tensor begins at, and a
// thread has all its loads of a piece in flight; the groups that its ends cut are read
// an element a thread.  Workgroup b takes
// pieces b, b + grid, ...: the launch sweeps over the tensors.
//
// What bounds it: memory.  28 bf16 tensors of 1.75 GB: squares 280 us, 6.2 TB/s; clipping 641
// us, 5.5 TB/s, by reads and writes.  Of small tensors the launches, 4 and 2 us for 96 of 98 KB, and
// the host's time for them.
#include <hip/hip_runtime.h>

#include <cmath>
#include <new>
#include <vector>

#include "../../include/dmuon_clip.h"
#include "kcommon.h"
#include "spans.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 8;                            // 16-byte groups a thread has in flight
constexpr int kPiece = kThreads * kGroups * 16;       // bytes
constexpr int kMostBlocks = 2048;                     // of a launch: 8 workgroups on each of 256 CUs
constexpr int kNormRecs = 192, kClipRecs = 128;       // tensors of a launch: a table of 3.8 KB at most in its arguments
constexpr int64_t kMostBytes = int64_t(1) << 45;      // of a tensor
constexpr int64_t kMostPieces = int64_t(1) << 30;     // of a launch

struct NormRec {
    const char* in;
    int64_t bytes_bf16;  // 2 bytes + whether it is bf16
};
struct NormArgs {
    double* sums;   // one per workgroup
    int32_t count, pieces;
    int32_t first[kNormRecs];  // a tensor's first piece in the launch
    NormRec rec[kNormRecs];
};

struct ClipRec {
    const char* in;
    char* out;
    int64_t bytes_bf16;
};
struct ClipArgs {
    const float* norm;
    double max_norm, eps;
    int32_t count, pieces;
    int32_t first[kClipRecs];
    ClipRec rec[kClipRecs];
};

__device__ __forceinline__ int64_t low4(const void* p) { return (int64_t)(reinterpret_cast<uintptr_t>(p) & 15u); }

struct __attribute__((packed, aligned(2))) Any16 {  // 16 bytes at any element
    u32x4_t v;
};

__device__ __forceinline__ void add_square(double& s, float x) {
    const double y = (double)x;
    s = fma(y, y, s);
}
__device__ __forceinline__ void add_squares(double (&s)[2], const u32x4_t& u, bool bf16) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            add_square(s[0], __uint_as_float(u[i] << 16));
            add_square(s[1], __uint_as_float(u[i] & 0xffff0000u));
        } else {
            add_square(s[i & 1], __uint_as_float(u[i]));
        }
    }
}

// The record whose pieces hold piece c: the last whose first is at most c.  Every wave looks
// at all of them at once: a search by halves waits for eight loads, one after the other.
template <int RECS>
__device__ __forceinline__ int record_of(const int32_t* first, int count, int c) {
    static_assert(RECS % 64 == 0, "whole waves");
    const int lane = (int)(threadIdx.x & 63u);
    int at[RECS / 64], n = 0;
    #pragma unroll
    for (int k = 0; k < RECS / 64; ++k) at[k] = first[64 * k + lane];  // (what follows the records is not looked at)
    #pragma unroll
    for (int k = 0; k < RECS / 64; ++k) n += __popcll(__builtin_amdgcn_ballot_w64(64 * k + lane < count && at[k] <= c));
    return __builtin_amdgcn_readfirstlane(n) - 1;
}

// A piece's elements are bytes lo .. hi - 1 of it.  Of the 16-byte groups that lo and hi cut
// the workgroup's first 16 threads take an element each: this thread's place, or -1.
template <int E>
__device__ __forceinline__ int cut_element(int64_t lo, int64_t hi) {
    const int t = (int)threadIdx.x, each = 16 / E;
    const int begin = lo > 0 ? (int)lo : 0, end = hi < kPiece ? (int)hi : kPiece;
    if (t >= 2 * each) return -1;
    const int first = begin & ~15, last = (end - 1) & ~15;
    const int at = t < each ? first : last, e = at + t % each * E;
    const bool cut = at < begin || at + 16 > end;
    return cut && e >= begin && e < end && (t < each || last != first) ? e : -1;
}

// Squares in 64 bits: the conversion and the addition of an element take two
// instructions, which the loads hide, and no element is too large or too small
// to be squared.
template <bool BF16>
__device__ __forceinline__ void piece_squares(double (&s)[2], const char* base, int64_t lo, int64_t hi) {
    if (lo <= 0 && hi >= kPiece) {
        u32x4_t u[kGroups];
        #pragma unroll
        for (int j = 0; j < kGroups; ++j) u[j] = *reinterpret_cast<const u32x4_t*>(base + (j * kThreads + (int)threadIdx.x) * 16);
        #pragma unroll
        for (int j = 0; j < kGroups; ++j) add_squares(s, u[j], BF16);
        return;
    }
    u32x4_t u[kGroups];
    auto whole = [&](int j) {
        const int off = (j * kThreads + (int)threadIdx.x) * 16;
        return off >= lo && off + 16 <= hi;
    };
    #pragma unroll
    for (int j = 0; j < kGroups; ++j)
        if (whole(j)) u[j] = *reinterpret_cast<const u32x4_t*>(base + (j * kThreads + (int)threadIdx.x) * 16);
    const int e = cut_element<BF16 ? 2 : 4>(lo, hi);
    if (e >= 0) {
        if (BF16) add_square(s[0], bf16_to_f32(*reinterpret_cast<const uint16_t*>(base + e)));
        else add_square(s[0], *reinterpret_cast<const float*>(base + e));
    }
    #pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        if (whole(j)) add_squares(s, u[j], BF16);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int THREADS>
__device__ __forceinline__ double block_sum64(double v) {
    __shared__ double red[THREADS / 64];
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double total = 0.0;
    #pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) total += red[w];
    return total;
}

__global__ __launch_bounds__(kThreads) void norm_squares_kernel(NormArgs a) {
    double s[2] = {0.0, 0.0};
    for (int c = (int)blockIdx.x; c < a.pieces; c += (int)gridDim.x) {
        const int i = record_of<kNormRecs>(a.first, a.count, c);
        const char* const in = a.rec[i].in;
        const int64_t bytes = a.rec[i].bytes_bf16 >> 1;
        const int64_t at = (int64_t)(c - a.first[i]) * kPiece - low4(in);  // of the piece in the tensor
        if (a.rec[i].bytes_bf16 & 1) piece_squares<true>(s, in + at, -at, bytes - at);
        else piece_squares<false>(s, in + at, -at, bytes - at);
    }
    const double total = block_sum64<kThreads>(s[0] + s[1]);
    if (threadIdx.x == 0) a.sums[blockIdx.x] = total;
}

constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void norm_join_kernel(const double* sums, int n, float* norm) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kJoinThreads) s += sums[i];
    s = block_sum64<kJoinThreads>(s);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

template <bool BF16>
__device__ __forceinline__ u32x4_t scaled(const u32x4_t& u, float f) {
    u32x4_t o;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16)
            o[i] = (uint32_t)f32_to_bf16(__uint_as_float(u[i] << 16) * f) |
                   ((uint32_t)f32_to_bf16(__uint_as_float(u[i] & 0xffff0000u) * f) << 16);
        else
            o[i] = __float_as_uint(__uint_as_float(u[i]) * f);
    }
    return o;
}

// The piece's 16-byte groups lie at 16-byte addresses of the output; the input's
// are read at whatever element they begin.
template <bool BF16>
__device__ __forceinline__ void piece_scaled(const char* in, char* out, int64_t lo, int64_t hi, float f) {
    if (lo <= 0 && hi >= kPiece) {
        u32x4_t u[kGroups];
        #pragma unroll
        for (int j = 0; j < kGroups; ++j) u[j] = reinterpret_cast<const Any16*>(in + (j * kThreads + (int)threadIdx.x) * 16)->v;
        #pragma unroll
        for (int j = 0; j < kGroups; ++j)
            *reinterpret_cast<u32x4_t*>(out + (j * kThreads + (int)threadIdx.x) * 16) = scaled<BF16>(u[j], f);
        return;
    }
    u32x4_t u[kGroups];
    auto whole = [&](int j) {
        const int off = (j * kThreads + (int)threadIdx.x) * 16;
        return off >= lo && off + 16 <= hi;
    };
    #pragma unroll
    for (int j = 0; j < kGroups; ++j)
        if (whole(j)) u[j] = reinterpret_cast<const Any16*>(in + (j * kThreads + (int)threadIdx.x) * 16)->v;
    const int e = cut_element<BF16 ? 2 : 4>(lo, hi);
    if (e >= 0) {
        if (BF16) Elem<uint16_t>::store(reinterpret_cast<uint16_t*>(out + e), bf16_to_f32(*reinterpret_cast<const uint16_t*>(in + e)) * f);
        else *reinterpret_cast<float*>(out + e) = *reinterpret_cast<const float*>(in + e) * f;
    }
    #pragma unroll
    for (int j = 0; j < kGroups; ++j)
        if (whole(j)) *reinterpret_cast<u32x4_t*>(out + (j * kThreads + (int)threadIdx.x) * 16) = scaled<BF16>(u[j], f);
}

__global__ __launch_bounds__(kThreads) void clip_kernel(ClipArgs a) {
    const float norm = *a.norm;
    const double ratio = a.max_norm / ((double)norm + a.eps);
    // (a ratio that is NaN: both infinite, and nothing is to be clipped)
    const float f = norm != norm ? norm : ratio < 1.0 ? (float)ratio : 1.f;
    for (int c = a.pieces - 1 - (int)blockIdx.x; c >= 0; c -= (int)gridDim.x) {
        const int i = record_of<kClipRecs>(a.first, a.count, c);
        const char* const in = a.rec[i].in;
        char* const out = a.rec[i].out;
        if (in == out && f == 1.f) continue;
        const int64_t bytes = a.rec[i].bytes_bf16 >> 1;
        const int64_t at = (int64_t)(c - a.first[i]) * kPiece - low4(out);
        if (a.rec[i].bytes_bf16 & 1) piece_scaled<true>(in + at, out + at, -at, bytes - at, f);
        else piece_scaled<false>(in + at, out + at, -at, bytes - at, f);
    }
}

int64_t element_bytes(int32_t dtype) { return dtype == DMUON_BF16 ? 2 : 4; }

// Pieces of a tensor that begins `low` bytes past a 16-byte address.
int64_t pieces_of(int64_t bytes, int64_t low) { return (low + bytes + kPiece - 1) / kPiece; }

// Calls launch(first tensor, end, pieces) for runs of at most `most` tensors that
// are not empty; where(i) is the address whose 16-byte groups the pieces follow.
// UNSUPPORTED if a run's pieces do not fit.
template <typename Where, typename Launch>
dmuon_status for_runs(int32_t count, const int64_t* numels, const int32_t* dtypes, int most, Where where, Launch launch) {
    int32_t i = 0;
    while (i < count) {
        const int32_t begin = i;
        int64_t pieces = 0;
        for (int n = 0; i < count && n < most; ++i) {
            if (numels[i] == 0) continue;
            ++n;
            pieces += pieces_of(numels[i] * element_bytes(dtypes[i]), (int64_t)(where(i) & 15u));
        }
        if (pieces >= kMostPieces) return DMUON_ERR_UNSUPPORTED;
        if (pieces == 0) continue;
        const dmuon_status st = launch(begin, i, (int32_t)pieces);
        if (st != DMUON_OK) return st;
    }
    return DMUON_OK;
}

int blocks_of(int32_t pieces) { return pieces < kMostBlocks ? pieces : kMostBlocks; }

dmuon_status check_sizes(int32_t count, const int64_t* numels, const int32_t* dtypes) {
    if (count < 0 || (count > 0 && (numels == nullptr || dtypes == nullptr))) return DMUON_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i)
        if (numels[i] < 0 || (dtypes[i] != DMUON_F32 && dtypes[i] != DMUON_BF16)) return DMUON_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i)
        if (numels[i] >= kMostBytes / element_bytes(dtypes[i])) return DMUON_ERR_UNSUPPORTED;
    return DMUON_OK;
}

// Sums that a norm call leaves at most, whatever addresses its tensors have: a tensor that
// begins inside a 16-byte group may take one piece more.
dmuon_status most_sums(int32_t count, const int64_t* numels, const int32_t* dtypes, int64_t* sums) {
    *sums = 0;
    return for_runs(count, numels, dtypes, kNormRecs, [](int32_t) { return (uintptr_t)14; },
                    [&](int32_t, int32_t, int32_t pieces) {
                        *sums += blocks_of(pieces);
                        return *sums < INT32_MAX ? DMUON_OK : DMUON_ERR_UNSUPPORTED;
                    });
}

bool at_element(const void* p, int32_t dtype) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(element_bytes(dtype) - 1)) == 0;
}

Span span_of(const void* p, int64_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + (uintptr_t)bytes, written};
}

dmuon_status norm(int32_t count, const int64_t* numels, const int32_t* dtypes, const void* const* grads, float* out,
                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
    dmuon_status st = check_sizes(count, numels, dtypes);
    if (st != DMUON_OK) return st;
    if (!at_element(out, DMUON_F32) || (count > 0 && grads == nullptr)) return DMUON_ERR_INVALID_ARG;
    int64_t sums = 0;
    st = most_sums(count, numels, dtypes, &sums);
    if (st != DMUON_OK) return st;
    if (sums > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0 ||
                     workspace_bytes < align_up((size_t)sums * 8)))
        st = DMUON_ERR_WORKSPACE;
    // (the gradients are only read: each has to miss the two that are written)
    const Span to = span_of(out, 4, true), ws_span = span_of(sums > 0 ? workspace : nullptr, sums * 8, true);
    auto meet = [](const Span& x, const Span& y) { return x.lo < y.hi && y.lo < x.hi; };
    for (int32_t i = 0; i < count; ++i) {
        if (numels[i] == 0) continue;
        if (!at_element(grads[i], dtypes[i])) return DMUON_ERR_INVALID_ARG;
        const Span g = span_of(grads[i], numels[i] * element_bytes(dtypes[i]), false);
        if (meet(g, to) || (st == DMUON_OK && meet(g, ws_span))) return DMUON_ERR_INVALID_ARG;
    }
    if (st != DMUON_OK) return st;
    if (meet(to, ws_span)) return DMUON_ERR_INVALID_ARG;

    double* const ws = static_cast<double*>(workspace);
    int32_t used = 0;
    st = for_runs(count, numels, dtypes, kNormRecs, [&](int32_t i) { return reinterpret_cast<uintptr_t>(grads[i]); },
                  [&](int32_t begin, int32_t end, int32_t pieces) {
                      NormArgs a;
                      a.sums = ws + used;
                      a.count = 0;
                      a.pieces = pieces;
                      int32_t first = 0;
                      for (int32_t i = begin; i < end; ++i) {
                          if (numels[i] == 0) continue;
                          const int64_t bytes = numels[i] * element_bytes(dtypes[i]);
                          a.first[a.count] = first;
                          a.rec[a.count++] = NormRec{static_cast<const char*>(grads[i]), 2 * bytes + (dtypes[i] == DMUON_BF16)};
                          first += (int32_t)pieces_of(bytes, (int64_t)(reinterpret_cast<uintptr_t>(grads[i]) & 15u));
                      }
                      const int blocks = blocks_of(pieces);
                      hipLaunchKernelGGL(norm_squares_kernel, dim3(blocks), dim3(kThreads), 0, stream, a);
                      used += blocks;
                      return hipGetLastError() == hipSuccess ? DMUON_OK : DMUON_ERR_HIP;
                  });
    if (st != DMUON_OK) return st;
    hipLaunchKernelGGL(norm_join_kernel, dim3(1), dim3(kJoinThreads), 0, stream, ws, used, out);
    return hipGetLastError() == hipSuccess ? DMUON_OK : DMUON_ERR_HIP;
}

dmuon_status clip(int32_t count, const int64_t* numels, const int32_t* dtypes, const void* const* grads,
                  void* const* outs, const float* norm, double max_norm, double eps, hipStream_t stream) {
    dmuon_status st = check_sizes(count, numels, dtypes);
    if (st != DMUON_OK) return st;
    if (!(max_norm >= 0.0) || !(eps > 0.0) || !std::isfinite(eps)) return DMUON_ERR_INVALID_ARG;
    if (!at_element(norm, DMUON_F32) || (count > 0 && (grads == nullptr || outs == nullptr)))
        return DMUON_ERR_INVALID_ARG;
    std::vector<Span> spans;
    spans.reserve(2 * (size_t)count + 1);
    spans.push_back(span_of(norm, 4, false));
    for (int32_t i = 0; i < count; ++i) {
        if (numels[i] == 0) continue;
        if (!at_element(grads[i], dtypes[i]) || !at_element(outs[i], dtypes[i])) return DMUON_ERR_INVALID_ARG;
        const int64_t bytes = numels[i] * element_bytes(dtypes[i]);
        if (outs[i] != grads[i]) spans.push_back(span_of(grads[i], bytes, false));
        spans.push_back(span_of(outs[i], bytes, true));
    }
    if (!disjoint_where_written(spans)) return DMUON_ERR_INVALID_ARG;
    const auto where = [&](int32_t i) { return reinterpret_cast<uintptr_t>(outs[i]); };
    // every launch's pieces fit: checked before the first one
    st = for_runs(count, numels, dtypes, kClipRecs, where, [](int32_t, int32_t, int32_t) { return DMUON_OK; });
    if (st != DMUON_OK) return st;
    return for_runs(count, numels, dtypes, kClipRecs, where, [&](int32_t begin, int32_t end, int32_t pieces) {
        ClipArgs a;
        a.norm = norm;
        a.max_norm = max_norm;
        a.eps = eps;
        a.count = 0;
        a.pieces = pieces;
        int32_t first = 0;
        for (int32_t i = begin; i < end; ++i) {
            if (numels[i] == 0) continue;
            const int64_t bytes = numels[i] * element_bytes(dtypes[i]);
            a.first[a.count] = first;
            a.rec[a.count++] = ClipRec{static_cast<const char*>(grads[i]), static_cast<char*>(outs[i]),
                                       2 * bytes + (dtypes[i] == DMUON_BF16)};
            first += (int32_t)pieces_of(bytes, (int64_t)(where(i) & 15u));
        }
        hipLaunchKernelGGL(clip_kernel, dim3(blocks_of(pieces)), dim3(kThreads), 0, stream, a);
        return hipGetLastError() == hipSuccess ? DMUON_OK : DMUON_ERR_HIP;
    });
}

}  // namespace
}  // namespace dmuon

extern "C" dmuon_status grad_norm_workspace_bytes(int32_t count, const int64_t* numels, const int32_t* dtypes,
                                                  size_t* bytes) {
    if (bytes == nullptr) return DMUON_ERR_INVALID_ARG;
    dmuon_status st = dmuon::check_sizes(count, numels, dtypes);
    if (st != DMUON_OK) return st;
    int64_t sums = 0;
    st = dmuon::most_sums(count, numels, dtypes, &sums);
    if (st == DMUON_OK) *bytes = dmuon::align_up((size_t)sums * 8);
    return st;
}

extern "C" dmuon_status grad_norm_batched(int32_t count, const int64_t* numels, const int32_t* dtypes,
                                          const void* const* grads, float* norm, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    try {
        return dmuon::norm(count, numels, dtypes, grads, norm, workspace, workspace_bytes,
                           static_cast<hipStream_t>(stream));
    } catch (...) {
        return DMUON_ERR_ALLOC;
    }
}

extern "C" dmuon_status grad_clip_batched(int32_t count, const int64_t* numels, const int32_t* dtypes,
                                          const void* const* grads, void* const* outs, const float* norm,
                                          double max_norm, double eps, void* stream) {
    try {
        return dmuon::clip(count, numels, dtypes, grads, outs, norm, max_norm, eps, static_cast<hipStream_t>(stream));
    } catch (...) {
        return DMUON_ERR_ALLOC;
    }
}
