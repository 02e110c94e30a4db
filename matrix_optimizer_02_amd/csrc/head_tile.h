// Device code shared by the tile kernels of the output-head losses: tile shapes,
// LDS layouts, direct loads and the epilogues.
#pragma once

#include "head_internal.h"
#include "kcommon.h"
#include "tile_map.h"

#include <climits>

namespace dmuon {
namespace head {

typedef __attribute__((address_space(3))) void* lptr_t;
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef short shortx8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;

constexpr int kBK = kHeadSlab;
constexpr int kRowBytes = kBK * 2;  // a K-contiguous slab row
constexpr int kChunks = kRowBytes / 16;
constexpr int KS = kBK / 16;        // MFMA k-steps per slab
constexpr float kLog2e = 1.4426950408889634f;

typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

// A tile's wave grid: WR waves along P's rows, WC along Q's.
template <int TP_, int TQ_, int ST_, int WR_ = head_wave_rows(TP_, TQ_)>
struct Config {
    static constexpr int TP = TP_, TQ = TQ_, ST = ST_;
    static constexpr int WR = WR_;
    static constexpr int WC = head_waves(TP) / WR;
    static constexpr int NW = WR * WC, NT = 64 * NW;
    static constexpr int RW = TP / WR, CW = TQ / WC;
    static constexpr int FI = RW / 32, FJ = CW / 32;
    static constexpr int kPBytes = TP * kRowBytes, kQBytes = TQ * kRowBytes;
    static constexpr int kPLoads = kPBytes / 1024 / NW;  // 1 KB wave loads per wave per slab
    static constexpr int kQLoads = kQBytes / 1024 / NW;
    static constexpr int kLds = ST * (kPBytes + kQBytes);
    static_assert(TQ * TP * 2 <= kLds, "the staged output fits");
};

// A K-major slab of W columns: rows of one k.
template <int W>
struct Wide {
    static constexpr int kBytes = 2 * W, kChunksRow = W / 8, kRows = 1024 / kBytes;  // rows a 1 KB load fills
    // a transposing read takes 4 rows; their chunk offsets spread over the banks
    // (and keep the two chunks of 16 columns next to each other)
    __device__ static __forceinline__ int swz(int r) {
        return W >= 128 ? (0xEA40 >> ((r & 3) * 4)) & 15 : 2 * (r & 3);
    }
};

template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One wave-wide direct load: lane l's 16 bytes at base + voff go to LDS byte
// lds + 16 l (lds wave-uniform).  The compiler does not count these loads: the
// kernel waits for them itself.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

__device__ __forceinline__ uint32_t lds_offset(const void* p) { return (uint32_t)(uintptr_t)(lptr_t)p; }

// Chunk swizzles: rows of 8 chunks (K-contiguous slabs) are read 8 or 16 rows at
// one chunk; rows of the staged output along themselves.
__device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

struct Tile {
    int I, J, split;
};

// Wave-uniform bases and per-lane offsets of a tile's slab loads.
struct Loads {
    const char* p;
    const char* q;
    uint32_t voff_p[2], voff_q[2];
    int tail_k;  // dH: first k (from the tile's first) that lies in the tail copy
};

// Orders a region of M MFMAs and D fragment reads (of the next region): after
// each MFMA some of the reads, so that they are on their way under the MFMAs.
// Left alone, the compiler reads a fragment, waits for it and uses it.
template <int M, int D>
__device__ __forceinline__ void weave() {
    constexpr int kPer = (D + M - 1) / M;
    #pragma unroll
    for (int m = 0; m < M; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // MFMA
        if (m * kPer < D) __builtin_amdgcn_sched_group_barrier(0x100, kPer, 0);  // LDS reads
    }
    __builtin_amdgcn_sched_barrier(0);
}

constexpr bool is_dw(int mode) { return mode == kHeadDw || mode == kHeadDwSum; }

// The tiles of a launch and this workgroup's share of them: XCD x takes one
// contiguous run of the tiles (neighbours share operand rows in its L2), its
// workgroups in turn.
struct Share {
    int tiles_j, per_split, first, count, at, step;
};
template <int TQ, int MODE>
__device__ __forceinline__ Share share_of(const HeadGemmArgs& args, int n, int n_k) {
    Share s;
    s.tiles_j = is_dw(MODE) ? args.tiles_j : ((MODE == kHeadGrad ? n_k : n) + TQ - 1) / TQ;
    s.per_split = args.tiles_i * s.tiles_j;
    const int total = s.per_split * (MODE == kHeadDh || MODE == kHeadDwSum ? args.splits : 1);
    const int x = (int)(blockIdx.x % kXcds);
    s.step = ((int)gridDim.x - x + kXcds - 1) / kXcds;
    const int each = total / kXcds, rem = total % kXcds;
    s.first = x * each + imin(x, rem);
    s.count = each + (x < rem ? 1 : 0);
    s.at = (int)(blockIdx.x / kXcds);
    return s;
}
__device__ __forceinline__ Tile tile_at(const HeadGemmArgs& args, const Share& s, int kq) {
    Tile t;
    int local = s.first + kq;
    t.split = local / s.per_split;
    local -= t.split * s.per_split;
    bx_decode_banded(local, args.tiles_i, s.tiles_j, t.I, t.J);
    return t;
}

// What ds is divided by before it is rounded: the largest coefficient, so that
// equal weights of all tokens, the usual case, round no target's entry (1 - p
// instead of w (1 - p), whose rounding all tokens would share).
__device__ __forceinline__ float norm_of(const float* norm) {
    const float x = *norm;
    return x > 0.f ? x : 1.f;
}

// Which product tiles take the main loop that is not pipelined in registers: the
// softmax statistics of 256 x 256 bf16 tiles.  The compiler makes it 82 instructions
// and the loads, with the row numbers of the epilogue kept in registers, where the
// pipelined loop takes 300.  Forward, pipelined against plain, one card: 8192 x 4096 x
// 128256 7.55 / 7.38 ms, 3687 x 3584 x 128256 3.31 / 3.14, 4225 x 396 x 82304 470 / 447
// us; smaller tiles lose 1 to 2% by it (300 x 576 x 3904 19.3 / 19.6 us), and so do
// the backward modes (3687 x 3584 x 128256 9.06 / 9.25 ms).
template <typename C, int MODE>
constexpr bool plain_loop(bool scaled) {
    return MODE == kHeadLse && !scaled && C::TQ == 256;
}

// Writes a finished tile.  acc[i][j][v]: P row wr RW + 32 i + 8 (v / 4) + 4 khalf
// + v % 4, Q row wc CW + 32 j + lrow.  SCALED: fp32 logits of scaled rows.  PARTS:
// bf16 parts of the outputs (Grad) or an fp32 output (dW) where 3.
//
// The staged tile takes PIECES pieces of its Q rows one after the other, each in
// the first TQ / PIECES x 2 TP bytes of smem.  prefetch() is called once, when the
// waves are done with the slabs and what the epilogue itself loads has come: what
// it loads (into the rest of the LDS) is on its way while the tile is written.
template <typename C, int MODE, bool SCALED, int PARTS, int PIECES = 1, typename F>
__device__ __forceinline__ void write_tile(const HeadGemmArgs& args, const Tile& t, int tiles_j, char* smem,
                                           floatx16 (&acc)[C::FI][C::FJ], F&& prefetch) {
    constexpr int TP = C::TP, TQ = C::TQ;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % C::WR, wc = wave / C::WR;
    const int lrow = lane & 31;
    // Rows are compared as (constant) against (bound - 4 khalf), the lane's part on the one
    // side that is not a constant: 64 row numbers would otherwise be kept in registers.
    // (The plain loop leaves room for them, and is compiled to the shorter code with them.)
    constexpr bool kRowNumbers = plain_loop<C, MODE>(SCALED);
    int khalf = lane >> 5;
    if constexpr (!kRowNumbers) asm volatile("" : "+v"(khalf));
    if constexpr (SCALED) {
        // the rows' scales out again (powers of two)
        float sq[C::FJ];
        #pragma unroll
        for (int j = 0; j < C::FJ; ++j) sq[j] = args.q_scale[t.J * TQ + wc * C::CW + 32 * j + lrow];
        #pragma unroll
        for (int i = 0; i < C::FI; ++i) {
            #pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
                const float4 sp = *reinterpret_cast<const float4*>(args.p_scale + t.I * TP + wr * C::RW + 32 * i +
                                                                   8 * v4 + 4 * khalf);
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) {
                    acc[i][j][4 * v4 + 0] *= sp.x * sq[j];
                    acc[i][j][4 * v4 + 1] *= sp.y * sq[j];
                    acc[i][j][4 * v4 + 2] *= sp.z * sq[j];
                    acc[i][j][4 * v4 + 3] *= sp.w * sq[j];
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // no more of the scales in registers at once
        }
    }
    if constexpr (MODE == kHeadLse) {
        const int64_t v_base = args.v0 + (int64_t)t.I * TP + wr * C::RW;  // vocab row of the wave's row 0
        const int64_t left = args.vocab - v_base;
        const int limit = left < C::RW ? (int)(left < 0 ? 0 : left) : C::RW;  // rows inside the vocabulary
        const float scale = args.inv_temp * kLog2e;
        int target[C::FJ];
        #pragma unroll
        for (int j = 0; j < C::FJ; ++j) {
            target[j] = -1;
            if (args.target != nullptr) target[j] = args.target[t.J * TQ + wc * C::CW + 32 * j + lrow];
            asm volatile("" : "+v"(target[j]));
        }
        __syncthreads();
        prefetch();
        #pragma unroll
        for (int j = 0; j < C::FJ; ++j) {
            const int row = t.J * TQ + wc * C::CW + 32 * j + lrow;
            if (args.logits != nullptr) {
                float* out = args.logits + (int64_t)row * args.logits_ld + v_base + 4 * khalf;
                #pragma unroll
                for (int i = 0; i < C::FI; ++i)
                    #pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
                        *reinterpret_cast<float4*>(out + 32 * i + 8 * v4) =
                            make_float4(acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2], acc[i][j][4 * v4 + 3]);
            }
            if (limit < C::RW) {
                #pragma unroll
                for (int i = 0; i < C::FI; ++i)
                    #pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (kRowNumbers ? 32 * i + 8 * (v / 4) + 4 * khalf + v % 4 >= limit
                                        : 32 * i + 8 * (v / 4) + v % 4 >= limit - 4 * khalf)
                            acc[i][j][v] = -INFINITY;
            }
            if (args.target != nullptr) {
                const int64_t off = target[j] - v_base;
                const int at = off >= 0 && off < limit ? (int)off : -1;
                const bool mine = at >= 0 && ((at >> 2) & 1) == khalf;
                if (__builtin_amdgcn_ballot_w64(mine)) {
                    float s = 0.f;
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (kRowNumbers ? at == 32 * i + 8 * (v / 4) + 4 * khalf + v % 4
                                            : at - 4 * khalf == 32 * i + 8 * (v / 4) + v % 4)
                                s = acc[i][j][v];
                    if (mine) args.target_logit[row] = s;
                }
            }
            float m = -INFINITY;
            #pragma unroll
            for (int i = 0; i < C::FI; ++i)
                #pragma unroll
                for (int v = 0; v < 16; ++v) m = fmaxf(m, acc[i][j][v]);
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            const float m0 = m == -INFINITY ? 0.f : m;
            float ls[4] = {0.f, 0.f, 0.f, 0.f};  // four chains: an addition need not wait for the one before
            #pragma unroll
            for (int i = 0; i < C::FI; ++i) {
                #pragma unroll
                for (int v = 0; v < 16; ++v) ls[v & 3] += __builtin_amdgcn_exp2f((acc[i][j][v] - m0) * scale);
                if (!kRowNumbers) __builtin_amdgcn_sched_barrier(0);  // no more of the differences in registers at once
            }
            float l = (ls[0] + ls[1]) + (ls[2] + ls[3]);
            l += __shfl_xor(l, 32, 64);
            if (khalf == 0)
                args.part[((int64_t)(args.first_tile + t.I) * C::WR + wr) * args.t_pad + row] = make_float2(m, l);
        }
    } else if constexpr (MODE == kHeadDh || MODE == kHeadDwSum) {
        __syncthreads();
        prefetch();
        float4* d = reinterpret_cast<float4*>(
            args.sums + ((int64_t)(t.split * tiles_j + t.J) * args.tiles_i + t.I) * (TP * TQ));
        #pragma unroll
        for (int i = 0; i < C::FI; ++i)
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j)
                #pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    float4* p = d + (((wave * C::FI + i) * C::FJ + j) * 4 + v4) * 64 + lane;
                    float4 o = make_float4(acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2],
                                           acc[i][j][4 * v4 + 3]);
                    if (MODE == kHeadDh && args.accumulate) {
                        const float4 b = *p;
                        o = make_float4(o.x + b.x, o.y + b.y, o.z + b.z, o.w + b.w);
                    }
                    *p = o;
                }
    } else {
        if constexpr (MODE == kHeadGrad) {
            const float inv_norm = 1.f / norm_of(args.norm);
            float row_lse[C::FJ], row_cp[C::FJ], row_ct[C::FJ];
            int row_target[C::FJ];
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j) {
                const int row = t.J * TQ + wc * C::CW + 32 * j + lrow;
                row_lse[j] = args.lse[row];
                row_cp[j] = args.cp[row] * inv_norm;
                row_ct[j] = args.ct[row] * inv_norm;
                row_target[j] = -1;
                if (args.target != nullptr) row_target[j] = args.target[row];
                asm volatile("" : "+v"(row_lse[j]), "+v"(row_cp[j]), "+v"(row_ct[j]), "+v"(row_target[j]));
            }
            __syncthreads();
            prefetch();
            const int64_t v_base = args.v0 + (int64_t)t.I * TP + wr * C::RW;
            const int64_t left = args.vocab - v_base;
            const int limit = left < C::RW ? (int)(left < 0 ? 0 : left) : C::RW;
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j) {
                const float lse = row_lse[j], cp = row_cp[j], ct = row_ct[j];
                const int64_t off = row_target[j] - v_base;
                const int at = off >= 0 && off < limit ? (int)off : -1;
                #pragma unroll
                for (int i = 0; i < C::FI; ++i)
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int r = 32 * i + 8 * (v / 4) + v % 4;  // less 4 khalf
                        float g = cp * __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], args.inv_temp, -lse) * kLog2e);
                        if (r == at - 4 * khalf) g -= ct;
                        acc[i][j][v] = r < limit - 4 * khalf ? g : 0.f;
                    }
            }
        }
        if constexpr (MODE == kHeadDw) {
            float norm = norm_of(args.norm);
            asm volatile("" : "+v"(norm));
            __syncthreads();
            prefetch();
            #pragma unroll
            for (int i = 0; i < C::FI; ++i)
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j)
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) acc[i][j][v] *= norm;
        }
        if constexpr (MODE == kHeadDw && PARTS > 1) {
            float* dw = static_cast<float*>(args.dw);
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j) {
                const int64_t row = (int64_t)t.J * TQ + wc * C::CW + 32 * j + lrow;
                if (row < args.dw_rows) {
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int v4 = 0; v4 < 4; ++v4) {
                            const int col = t.I * TP + wr * C::RW + 32 * i + 8 * v4 + 4 * khalf;
                            float* p = dw + row * args.dw_ld + col;
                            if ((args.dw_ld & 3) == 0) {
                                if (col < args.dw_ld)
                                    *reinterpret_cast<float4*>(p) =
                                        make_float4(acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2],
                                                    acc[i][j][4 * v4 + 3]);
                            } else {
                                #pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (col + e < args.dw_ld) p[e] = acc[i][j][4 * v4 + e];
                            }
                        }
                }
            }
        } else {
            // bf16 rows: staged through LDS as E[c][r], stored in whole 16-byte chunks
            // (256 token rows: never in two parts)
            constexpr bool kSplit = MODE == kHeadGrad && (PARTS > 1 || TQ <= 128);
            const int kOut = !kSplit ? 1 : PARTS > 1 ? PARTS : args.low + 1;
            constexpr int kEBytes = 2 * TP, kEChunks = TP / 8, kRows = TQ / PIECES;
            const int low_row = kSplit && PARTS == 1 && args.low ? head_low_row(*args.count) : 0;
            #pragma unroll 1
            for (int turn = 0; turn < kOut * PIECES; ++turn) {
                const int part = turn / PIECES, first = turn % PIECES * kRows;
                if (turn > 0) __syncthreads();  // the piece before has been read
                if (PIECES == 1 || wc * C::CW / kRows * kRows == first) {
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int j = 0; j < C::FJ; ++j)
                            #pragma unroll
                            for (int v4 = 0; v4 < 4; ++v4) {
                                const int r = wr * C::RW + 32 * i + 8 * v4 + 4 * khalf;
                                const int c = wc * C::CW + 32 * j + lrow - first;
                                uint16_t b[4];
                                #pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    b[e] = f32_to_bf16(acc[i][j][4 * v4 + e]);
                                    if (kSplit) acc[i][j][4 * v4 + e] -= bf16_to_f32(b[e]);
                                }
                                uint2 o;
                                o.x = (uint32_t)b[0] | ((uint32_t)b[1] << 16);
                                o.y = (uint32_t)b[2] | ((uint32_t)b[3] << 16);
                                *reinterpret_cast<uint2*>(smem + c * kEBytes + (((r >> 3) ^ (c & (kEChunks - 1))) << 4) +
                                                          (r & 7) * 2) = o;
                            }
                }
                __syncthreads();
                for (int q = tid; q < kRows * kEChunks; q += C::NT) {
                    const int cp = q / kEChunks, ch = q % kEChunks, c = first + cp;
                    const uint4 v = *reinterpret_cast<const uint4*>(smem + cp * kEBytes +
                                                                    ((ch ^ (cp & (kEChunks - 1))) << 4));
                    if (MODE == kHeadGrad) {
                        // the low parts' rows begin where this tile's padding may reach
                        if (low_row != 0 && t.J * TQ + c >= low_row) continue;
                        const int64_t row = t.J * TQ + c + part * low_row;
                        char* g = args.g + (PARTS > 1 ? part * args.g_plane : 0) +
                                  2 * (row * args.g_ld + t.I * TP + ch * 8);
                        *reinterpret_cast<uint4*>(g) = v;
                    } else {
                        const int64_t row = (int64_t)t.J * TQ + c;
                        const int col = t.I * TP + ch * 8;
                        if (row < args.dw_rows && col < args.dw_ld) {
                            uint16_t* p = static_cast<uint16_t*>(args.dw) + row * args.dw_ld + col;
                            if ((args.dw_ld & 7) == 0) {
                                *reinterpret_cast<uint4*>(p) = v;
                            } else {
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                                #pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (col + e < args.dw_ld) p[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
                            }
                        }
                    }
                }
            }
        }
    }
}

}  // namespace head
}  // namespace dmuon
