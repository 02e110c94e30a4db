// Tile products of the output-head losses that read W as it lies in memory:
// fp32 weights, and bf16 ones whose rows are not whole slabs (any width, rows
// at any 2- or 4-byte offset).  The modes are those of k_head_gemm.hip (Lse,
// Grad, dH); W is the P operand of all three.
//
// Batches of few tokens are bound by reading W once, and a padded copy of it
// would read it, write it and read the copy: here each lane loads 16 bytes of W
// into registers, some slabs ahead, and writes them to LDS, fp32 values split
// into three bf16 parts on the way (x = hi + mid + lo, exact to 24 bits).  All
// parts of a slab lie in LDS together, so the six products of an fp32 tile (hi
// hi, hi mid, mid hi, mid mid, hi lo, lo hi) read W once.
//
// A slab is 128 bytes of every row of W (Lse, Grad: 32 fp32 or 64 bf16 of K) or
// as many rows of it (dH).  Two LDS stages; the other operand (packed hidden
// states, or ds) goes through registers as well.
//
// It also multiplies the logits of larger fp32 calls in which a row's range is more
// than two fp16 parts hold (wide_range below).  Its launch follows the two-part one,
// whose results it writes over; in other calls it returns at once (5 us).
// 819 tokens, hidden 1536, vocabulary 32000 with such rows: forward 807 us for 369,
// backward 1721 for 1349.
//
// What bounds it: few tokens, the reads of W and the instructions that split it.
// 64 tokens, fp32, hidden 4090, vocabulary 50000: forward 303 us, 2.7 TB/s of W
// (a copy reaches 6.0), backward 1320 us.  From some hundred tokens on the split,
// repeated for every tile of tokens, costs more than a padded copy (head_layout.cpp
// has both sides measured).
#include "head_tile.h"

namespace dmuon {
namespace {

using namespace head;

// 16 bytes at any element boundary.
struct __attribute__((packed, aligned(2))) Raw2 {
    u32x4_t v;
};
struct __attribute__((packed, aligned(4))) Raw4 {
    u32x4_t v;
};

template <typename C_, bool F32_>
struct Stream {
    using C = C_;
    static constexpr bool F32 = F32_;
    static constexpr int kParts = F32 ? kHeadMaxPlanes : 1;
    static constexpr int kK = F32 ? 32 : 64;         // K of a slab
    static constexpr int kElems = F32 ? 4 : 8;       // W elements of a 16-byte chunk
    static constexpr int kRow = kK * 2;              // bytes of a K-contiguous bf16 row in LDS
    static constexpr int kRowChunks = kRow / 16;
    static constexpr int kSteps = kK / 16;           // MFMA k-steps
    static constexpr int kPPart = C::TP * kRow, kQPart = C::TQ * kRow;
    static constexpr int kStage = kParts * (kPPart + kQPart);
    static constexpr int kLds = 2 * kStage > C::TP * C::TQ * 2 ? 2 * kStage : C::TP * C::TQ * 2;
    static constexpr int kPItems = C::TP * 8 / C::NT;  // 16-byte chunks of W a lane loads per slab
    static constexpr int kQChunks = kParts * C::TQ * kRowChunks;
    static constexpr int kQItems = (kQChunks + C::NT - 1) / C::NT;
    // register sets: slabs on their way.  A 64 x 64 tile's are small, and its slabs
    // short: it needs more of them to cover a load's latency.
    static constexpr int kSets = C::TP == 64 ? 4 : C::TQ == 64 ? 3 : 2;
    // rows of 4 chunks: 16 rows at one chunk hit 16 bank groups
    __device__ static __forceinline__ int swz(int r) { return F32 ? (r >> 2) & 3 : swizzle(r); }
};

// Whether two fp16 parts, each row scaled by its largest element, leave a logit of
// these operands off by more than 2^-22 T beside what they leave out of each product:
// an element is then off by up to 2^-39 of its row's largest, a logit by
// 2^-39 (max |h| sum |w| + max |w| sum |h|).  Run by a whole block.
template <int NT>
__device__ __forceinline__ bool wide_range(const HeadGemmArgs& args, float4* red) {
    float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
    // eight loads on their way at once
    auto largest = [](const float2* range, int n, float& element, float& sum) {
        for (int i = threadIdx.x; i < n; i += 8 * NT) {
            float2 x[8];
            #pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = range[imin(i + u * NT, n - 1)];
            #pragma unroll
            for (int u = 0; u < 8; ++u) element = fmaxf(element, x[u].x), sum = fmaxf(sum, x[u].y);
        }
    };
    largest(args.q_range, args.q_ranges, m.x, m.y);
    largest(args.p_range, args.p_ranges, m.z, m.w);
    auto join = [&](const float4& o) {
        m = make_float4(fmaxf(m.x, o.x), fmaxf(m.y, o.y), fmaxf(m.z, o.z), fmaxf(m.w, o.w));
    };
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        join(make_float4(__shfl_xor(m.x, off, 64), __shfl_xor(m.y, off, 64), __shfl_xor(m.z, off, 64),
                         __shfl_xor(m.w, off, 64)));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < NT / 64; ++w) join(red[w]);
    __syncthreads();
    return !((m.x * m.w + m.z * m.y) * args.inv_temp <= 0x1p17f);
}

template <typename S, int MODE>
__global__ __launch_bounds__(S::C::NT, S::C::NT == 512 ? 1 : 2) void head_stream_kernel(HeadGemmArgs args) {
    using C = typename S::C;
    constexpr int TP = C::TP, TQ = C::TQ, NT = C::NT;
    constexpr bool PW = MODE == kHeadDh;
    using WP = Wide<TP>;
    __shared__ __attribute__((aligned(1024))) char smem[S::kLds];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % C::WR, wc = wave / C::WR;
    const int lrow = lane & 31, khalf = lane >> 5;
    if (S::F32 && !PW && args.q_range != nullptr && !wide_range<NT>(args, reinterpret_cast<float4*>(smem))) return;
    const int n = __builtin_amdgcn_readfirstlane(*args.count);
    const int n_k = n <= kBK ? kBK : (n + kBK - 1) / kBK * kBK;
    const Share sh = share_of<TQ, MODE>(args, n, n_k, args.splits);
    const int cols = args.p_ld;  // of W

    for (int kq = sh.at; kq < sh.count; kq += sh.step) {
        const Tile t = tile_at(args, sh, kq);
        const int k_first = MODE == kHeadDh ? t.split * args.split_k : 0;
        const int K = MODE == kHeadDh ? imin(args.split_k, args.k - k_first) : args.k;
        const int slabs = (K + S::kK - 1) / S::kK;

        // ---- W: chunk i of this lane is chunk (i NT + tid) of the slab ------------------
        // W's rows (dH: columns) of the tile and its slabs' columns (dH: rows) that exist:
        // a slab inside both is loaded without a look at its lanes.
        constexpr int kPRowChunks = PW ? TP / S::kElems : 8;
        constexpr int kSize = S::F32 ? 4 : 2;
        const int64_t left = args.p_rows - (PW ? k_first : (int64_t)t.I * TP);
        const int rows = left < INT_MAX ? (int)left : INT_MAX;  // from the tile's first row
        const int cols_left = cols - (PW ? t.I * TP : 0);
        const bool tile_full = PW ? cols_left >= TP : rows >= TP;
        const char* const p0 = args.p + ((PW ? (int64_t)k_first : (int64_t)t.I * TP) * cols + (PW ? t.I * TP : 0)) * kSize;
        const int64_t p_step = (PW ? (int64_t)S::kK * cols : S::kK) * kSize;  // bytes from slab to slab
        uint32_t p_off[S::kPItems];
        #pragma unroll
        for (int i = 0; i < S::kPItems; ++i) {
            const int item = i * NT + tid;
            p_off[i] = (uint32_t)(((item / kPRowChunks) * (int64_t)cols + (item % kPRowChunks) * S::kElems) * kSize);
        }
        auto load_p = [&](int s, u32x4_t (&r)[S::kPItems]) {
            const char* const base = p0 + s * p_step;
            if (tile_full && (PW ? (s + 1) * S::kK <= rows : (s + 1) * S::kK <= cols_left)) {
                #pragma unroll
                for (int i = 0; i < S::kPItems; ++i) {
                    if (S::F32) r[i] = reinterpret_cast<const Raw4*>(base + p_off[i])->v;
                    else r[i] = reinterpret_cast<const Raw2*>(base + p_off[i])->v;
                }
                return;
            }
            #pragma unroll
            for (int i = 0; i < S::kPItems; ++i) {
                const int item = i * NT + tid;
                const int row = item / kPRowChunks + (PW ? s * S::kK : 0);
                const int col = (item % kPRowChunks) * S::kElems + (PW ? 0 : s * S::kK);
                const char* p = base + p_off[i];
                r[i] = u32x4_t{0, 0, 0, 0};
                if (row >= rows || col >= cols_left) continue;
                if (col + S::kElems <= cols_left) {
                    if (S::F32) r[i] = reinterpret_cast<const Raw4*>(p)->v;
                    else r[i] = reinterpret_cast<const Raw2*>(p)->v;
                } else {  // the row ends inside the chunk
                    #pragma unroll
                    for (int e = 0; e < S::kElems; ++e)
                        if (col + e < cols_left) {
                            if (S::F32) r[i][e] = reinterpret_cast<const uint32_t*>(p)[e];
                            else r[i][e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
                        }
                }
            }
        };
        auto write_p = [&](char* base, const u32x4_t (&r)[S::kPItems]) {
            #pragma unroll
            for (int i = 0; i < S::kPItems; ++i) {
                const int item = i * NT + tid;
                const int row = item / kPRowChunks, ch = item % kPRowChunks;
                if (S::F32) {
                    const int lc = ch / 2;  // two chunks of W make one of a part
                    const int o = PW ? row * WP::kBytes + ((lc ^ WP::swz(row)) << 4) + (ch & 1) * 8
                                     : row * S::kRow + ((lc ^ S::swz(row)) << 4) + (ch & 1) * 8;
                    float x[4];
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[i][e]);
                    #pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        uint16_t b[4];
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            b[e] = f32_to_bf16(x[e]);
                            x[e] -= bf16_to_f32(b[e]);
                        }
                        *reinterpret_cast<uint2*>(base + part * S::kPPart + o) =
                            make_uint2((uint32_t)b[0] | ((uint32_t)b[1] << 16), (uint32_t)b[2] | ((uint32_t)b[3] << 16));
                    }
                } else {
                    const int o = PW ? row * WP::kBytes + ((ch ^ WP::swz(row)) << 4)
                                     : row * S::kRow + ((ch ^ S::swz(row)) << 4);
                    *reinterpret_cast<u32x4_t*>(base + o) = r[i];
                }
            }
        };
        // ---- the other operand: packed, K-contiguous rows -------------------------------
        const char* const q0 = args.q + 2 * ((int64_t)t.J * TQ * args.q_ld + k_first);
        auto load_q = [&](int s, u32x4_t (&r)[S::kQItems]) {
            #pragma unroll
            for (int i = 0; i < S::kQItems; ++i) {
                const int item = i * NT + tid;
                if (S::kQChunks % NT != 0 && item >= S::kQChunks) continue;
                const int part = item / (TQ * S::kRowChunks), rest = item % (TQ * S::kRowChunks);
                const uint32_t off = (uint32_t)(2 * ((rest / S::kRowChunks) * args.q_ld + (rest % S::kRowChunks) * 8));
                r[i] = *reinterpret_cast<const u32x4_t*>(q0 + part * args.q_plane + 2 * s * S::kK + off);
            }
        };
        auto write_q = [&](char* base, const u32x4_t (&r)[S::kQItems]) {
            #pragma unroll
            for (int i = 0; i < S::kQItems; ++i) {
                const int item = i * NT + tid;
                if (S::kQChunks % NT != 0 && item >= S::kQChunks) continue;
                const int part = item / (TQ * S::kRowChunks), rest = item % (TQ * S::kRowChunks);
                const int row = rest / S::kRowChunks, ch = rest % S::kRowChunks;
                *reinterpret_cast<u32x4_t*>(base + part * S::kQPart + row * S::kRow + ((ch ^ S::swz(row)) << 4)) = r[i];
            }
        };

        floatx16 acc[C::FI][C::FJ];
        #pragma unroll
        for (int i = 0; i < C::FI; ++i)
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j)
                #pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

        const int tr_g = lane >> 4, tr_s = lane & 15;
        const int tr_row = 8 * (tr_g >> 1) + (tr_s >> 2);
        const int tr_col = 16 * (tr_g & 1) + 4 * (tr_s & 3);
        auto read_rows = [&](const char* base, int row0, int ks) -> bf16x8 {
            return *reinterpret_cast<const bf16x8*>(base + (row0 + lrow) * S::kRow +
                                                    (((ks * 2 + khalf) ^ S::swz(lrow)) << 4));
        };
        auto read_p = [&](const char* base, int i, int ks) -> bf16x8 {
            const int row0 = wr * C::RW + 32 * i;
            if (!PW) return read_rows(base, row0, ks);
            shortx4 h[2];
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 16 * ks + 4 * u + tr_row, c = row0 + tr_col;
                const int o = r * WP::kBytes + (((c >> 3) ^ WP::swz(tr_s >> 2)) << 4) + (c & 7) * 2;
                h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_shortx4*)((__attribute__((address_space(3))) char*)base + o));
            }
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
        };
        auto multiply = [&](const char* pb) {
            const char* qb = pb + S::kParts * S::kPPart;
            #pragma unroll
            for (int ks = 0; ks < S::kSteps; ++ks) {
                bf16x8 fb[S::kParts][C::FJ];
                #pragma unroll
                for (int part = 0; part < S::kParts; ++part)
                    #pragma unroll
                    for (int j = 0; j < C::FJ; ++j)
                        fb[part][j] = read_rows(qb + part * S::kQPart, wc * C::CW + 32 * j, ks);
                #pragma unroll
                for (int i = 0; i < C::FI; ++i) {
                    bf16x8 fa[S::kParts];
                    #pragma unroll
                    for (int part = 0; part < S::kParts; ++part) fa[part] = read_p(pb + part * S::kPPart, i, ks);
                    // smallest products first
                    #pragma unroll
                    for (int sum = S::kParts - 1; sum >= 0; --sum)
                        #pragma unroll
                        for (int a = 0; a <= sum; ++a)
                            #pragma unroll
                            for (int j = 0; j < C::FJ; ++j)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a], fb[sum - a][j], acc[i][j], 0, 0, 0);
                }
            }
        };

        // ---- main loop -------------------------------------------------------------------
        // Slab s is multiplied out of stage s % 2 while slabs s + 1 .. s + kSets wait in, or
        // load into, the register sets.
        struct Set {
            u32x4_t p[S::kPItems], q[S::kQItems];
        } set[S::kSets];
        auto fetch = [&](int s, Set& r) {
            if (s >= slabs) return;
            load_q(s, r.q);
            load_p(s, r.p);
        };
        auto put = [&](int s, const Set& r) {
            char* const stage = smem + (s & 1) * S::kStage;
            write_p(stage, r.p);
            write_q(stage + S::kParts * S::kPPart, r.q);
        };
        #pragma unroll
        for (int i = 0; i < S::kSets; ++i) fetch(i, set[i]);
        __syncthreads();  // the previous tile's epilogue has left the buffers
        put(0, set[0]);
        fetch(S::kSets, set[0]);
        __syncthreads();
        for (int s0 = 0; s0 < slabs; s0 += S::kSets) {
            #pragma unroll
            for (int i = 0; i < S::kSets; ++i) {
                const int s = s0 + i;
                if (s < slabs) {
                    Set& next = set[(i + 1) % S::kSets];
                    multiply(smem + (s & 1) * S::kStage);
                    if (s + 1 < slabs) {
                        put(s + 1, next);
                        fetch(s + 1 + S::kSets, next);
                    }
                    __syncthreads();
                }
            }
        }
        write_tile<C, MODE, false, S::kParts>(args, t, sh.tiles_j, smem, acc, [] {});
    }
}

template <typename S, int MODE>
hipError_t launch(const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    const int64_t per_xcd = (max_tiles + kXcds - 1) / kXcds, most = head_slots(S::C::TP) / kXcds;
    const int wgs = kXcds * (int)(per_xcd < most ? per_xcd : most);
    hipLaunchKernelGGL((head_stream_kernel<S, MODE>), dim3(wgs), dim3(S::C::NT), 0, stream, a);
    return hipGetLastError();
}

template <typename C>
hipError_t launch_config(int mode, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    using F = Stream<C, true>;
    using B = Stream<C, false>;
    const bool f32 = a.parts > 1;
    switch (mode) {
        case kHeadLse:
            return f32 ? launch<F, kHeadLse>(a, max_tiles, stream) : launch<B, kHeadLse>(a, max_tiles, stream);
        case kHeadGrad:
            return f32 ? launch<F, kHeadGrad>(a, max_tiles, stream) : launch<B, kHeadGrad>(a, max_tiles, stream);
        case kHeadGradEntropy:
            return f32 ? launch<F, kHeadGradEntropy>(a, max_tiles, stream) : launch<B, kHeadGradEntropy>(a, max_tiles, stream);
        case kHeadProbs:
            return f32 ? launch<F, kHeadProbs>(a, max_tiles, stream) : launch<B, kHeadProbs>(a, max_tiles, stream);
        case kHeadTop:
            return f32 ? launch<F, kHeadTop>(a, max_tiles, stream) : launch<B, kHeadTop>(a, max_tiles, stream);
        case kHeadDh:
            return f32 ? launch<F, kHeadDh>(a, max_tiles, stream) : launch<B, kHeadDh>(a, max_tiles, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_head_stream(int mode, HeadTile tile, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    if (max_tiles <= 0) return hipSuccess;
    if (max_tiles > (int64_t)0x3fffffff) return hipErrorInvalidValue;
    if (tile.tq == 256) {
        // in the place of a 256 x 256 tile: half of one, its statistics laid out as the whole one's
        using F = Stream<Config<256, 128, 3, head_wave_rows(256, 256)>, true>;
        if (a.parts == 1) return hipErrorInvalidValue;
        switch (mode) {
            case kHeadLse: return launch<F, kHeadLse>(a, max_tiles, stream);
            case kHeadProbs: return launch<F, kHeadProbs>(a, max_tiles, stream);
            case kHeadTop: return launch<F, kHeadTop>(a, max_tiles, stream);
            case kHeadGrad: return launch<F, kHeadGrad>(a, max_tiles, stream);
            case kHeadGradEntropy: return launch<F, kHeadGradEntropy>(a, max_tiles, stream);
            default: return hipErrorInvalidValue;
        }
    }
    if (tile.tp == 64) return launch_config<Config<64, 64, 4>>(mode, a, max_tiles, stream);
    if (tile.tq == 64) return launch_config<Config<256, 64, 2>>(mode, a, max_tiles, stream);
    return launch_config<Config<256, 128, 3>>(mode, a, max_tiles, stream);
}

}  // namespace dmuon
