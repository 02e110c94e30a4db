// The products of the output-head losses on bf16 MFMA (gfx950), one tile
// kernel in four modes, each C[r][c] = sum over k of P[r][k] Q[c][k]:
//   Lse   s^T = W H^T     softmax statistics of every 256-row vocab tile
//   Grad  s^T = W H^T     again, ds = cp exp(s / T - lse) - ct [target] out
//   dH    dH^T = W^T ds^T  k over the vocab rows of the piece, fp32 sums
//   dW    dW^T = H^T ds    k over the tokens
// s itself never leaves the registers.  With the vocabulary along the tile's P
// rows, a lane holds 32 x FI / 2 logits of each of its tokens, so the running
// maximum and sum of the softmax are formed inside a lane and joined across
// two lanes by one shuffle.
//
// fp32 operands come as three bf16 parts x = hi + mid + lo (24 bits); the six
// products hi hi, hi mid, mid hi, mid mid, hi lo, lo hi, accumulated in fp32,
// leave out only terms below 2^-25 of the whole.
//
// Tile: 256 P rows by TQ Q rows (256, or 64 for batches of at most 64 rows, where the
// call is bound by reading W and a 256-row tile would only add MFMAs), 8 waves,
// v_mfma_f32_32x32x16_bf16.  K is staged through LDS in 64-deep slabs by direct
// global->LDS loads, two buffers; 16-byte chunks are XOR-swizzled by row.
#include "head_internal.h"
#include "kcommon.h"
#include "tile_map.h"

#include <climits>

namespace dmuon {
namespace {

typedef __attribute__((address_space(3))) void* lptr_t;
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef short shortx8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kBK = kHeadSlab;
constexpr int kTP = kHeadTile;
constexpr int kRowBytes = kBK * 2;           // a K-contiguous slab row
constexpr int kChunks = kRowBytes / 16;
constexpr int kWideBytes = 2 * kTP;          // a K-major slab row: 256 values of one k
constexpr int kWideChunks = kWideBytes / 16;
constexpr int KS = kBK / 16;                 // MFMA k-steps per slab
constexpr float kLog2e = 1.4426950408889634f;

// Wave grid: WR waves along P's rows, WC along Q's.
template <int TQ>
struct Grid {
    static constexpr int WR = TQ == 256 ? 2 : 4;
    static constexpr int WC = kWaves / WR;
    static constexpr int RW = kTP / WR, CW = TQ / WC;
    static constexpr int FI = RW / 32, FJ = CW / 32;
    static constexpr int kPBytes = kTP * kRowBytes;
    static constexpr int kQBytes = TQ * kRowBytes;
    static constexpr int kPLoads = kPBytes / 1024 / kWaves;  // 1 KB wave loads per wave per slab
    static constexpr int kQLoads = kQBytes / 1024 / kWaves;
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

// Chunk swizzles: rows of 8 chunks (K-contiguous slabs) read 8 or 16 rows at
// one chunk; rows of 32 chunks (K-major slabs) are read 4 rows at a time by the
// transposing LDS read; rows of the staged output are read along themselves.
__device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swizzle_wide(int r) { return (0xEA40 >> ((r & 3) * 4)) & 15; }
__device__ __forceinline__ int swizzle_out(int r) { return r & 31; }

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

// PARTS: bf16 parts of the operands, 1 (bf16) or 3 (fp32).
template <int TQ, int MODE, int PARTS>
__global__ __launch_bounds__(kThreads, 1) void head_gemm_kernel(HeadGemmArgs args) {
    using C = Grid<TQ>;
    constexpr bool PW = MODE == kHeadDh || MODE == kHeadDw;  // P is K-major
    constexpr bool QW = MODE == kHeadDw;                     // Q is K-major
    static_assert(!QW || TQ == 256, "a K-major Q slab has 256 columns");
    __shared__ __attribute__((aligned(1024))) char smem[2 * (C::kPBytes + C::kQBytes)];
    static_assert(TQ * kWideBytes <= (int)sizeof(smem), "the staged output fits");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % C::WR, wc = wave / C::WR;
    const int lrow = lane & 31, khalf = lane >> 5;

    // ---- which tiles -----------------------------------------------------------------
    const int n = __builtin_amdgcn_readfirstlane(*args.count);
    const int n_k = n <= kHeadMinK ? kHeadMinK : (n + kHeadMinK - 1) / kHeadMinK * kHeadMinK;  // dW's K extent
    const int tiles_j = MODE == kHeadDw ? args.tiles_j : ((MODE == kHeadGrad ? n_k : n) + TQ - 1) / TQ;
    const int splits = MODE == kHeadDh ? args.splits : 1;
    const int per_split = args.tiles_i * tiles_j;
    const int total = per_split * splits;
    // XCD x takes one contiguous run of the tiles, its workgroups in turn
    const int x = (int)(blockIdx.x % kXcds);
    const int wgs_x = ((int)gridDim.x - x + kXcds - 1) / kXcds;
    const int share = total / kXcds, rem = total % kXcds;
    const int first = x * share + imin(x, rem), count_x = share + (x < rem ? 1 : 0);

    for (int kq = (int)(blockIdx.x / kXcds); kq < count_x; kq += wgs_x) {
        Tile t;
        {
            int local = first + kq;
            t.split = local / per_split;
            local -= t.split * per_split;
            bx_decode_banded(local, args.tiles_i, tiles_j, t.I, t.J);
        }
        // ---- operands ----------------------------------------------------------------
        int K;  // this tile's K extent, a multiple of kBK
        int k_first = 0;
        if (MODE == kHeadDh) {
            k_first = t.split * args.split_k;
            K = imin(args.split_k, args.k - k_first);
        } else {
            K = MODE == kHeadDw ? n_k : args.k;
        }
        Loads L;
        L.tail_k = INT_MAX;
        if (PW) {
            L.p = args.p + 2 * (int64_t)k_first * args.p_ld;
            if (MODE == kHeadDh && args.tail_row != INT_MAX) L.tail_k = args.tail_row - k_first;
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / kWideChunks;  // + 2 q
                const int lc = (lane % kWideChunks) ^ swizzle_wide(2 * par + row);
                // columns past the row's end repeat its last chunk (never stored)
                const int col = imin(t.I * kTP + lc * 8, args.p_ld - 8);
                L.voff_p[par] = (uint32_t)(2 * (row * args.p_ld + col));
            }
        } else {
            const int row0 = t.I * kTP;
            L.p = row0 >= args.tail_row ? args.p_tail + 2 * (int64_t)(row0 - args.tail_row) * args.p_ld
                                        : args.p + 2 * (int64_t)row0 * args.p_ld;
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / kChunks;  // + 8 q
                const int lc = (lane % kChunks) ^ swizzle(8 * par + row);
                L.voff_p[par] = (uint32_t)(2 * (row * args.p_ld + lc * 8));
            }
        }
        if (QW) {
            L.q = args.q;
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / kWideChunks;
                const int lc = (lane % kWideChunks) ^ swizzle_wide(2 * par + row);
                L.voff_q[par] = (uint32_t)(2 * (row * args.q_ld + t.J * kTP + lc * 8));
            }
        } else {
            L.q = args.q + 2 * ((int64_t)t.J * TQ * args.q_ld + k_first);
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / kChunks;
                const int lc = (lane % kChunks) ^ swizzle(8 * par + row);
                L.voff_q[par] = (uint32_t)(2 * (row * args.q_ld + lc * 8));
            }
        }
        // products of parts, in order: hi hi, hi mid, mid hi, mid mid, hi lo, lo hi
        auto p_part = [](int seg) { return (0x201100 >> (4 * seg)) & 15; };
        auto q_part = [](int seg) { return (0x021010 >> (4 * seg)) & 15; };
        auto load_slab = [&](int seg, int k0, int buf) {
            const char* pb = L.p + (PARTS > 1 ? p_part(seg) * args.p_plane : 0);
            if (PW) {
                if (MODE == kHeadDh && k0 >= L.tail_k)
                    pb = args.p_tail + 2 * (int64_t)(k0 - L.tail_k) * args.p_ld;
                else
                    pb += 2 * (int64_t)k0 * args.p_ld;
            } else {
                pb += 2 * k0;
            }
            char* pd = smem + buf * C::kPBytes;
            #pragma unroll
            for (int i = 0; i < C::kPLoads; ++i) {
                const int q = wave * C::kPLoads + i;
                dma16(pb + (int64_t)q * ((PW ? 4 : 16) * (int64_t)args.p_ld), L.voff_p[i & 1], lds_offset(pd + q * 1024));
            }
            const char* qb = L.q + (PARTS > 1 ? q_part(seg) * args.q_plane : 0) +
                             (QW ? 2 * (int64_t)k0 * args.q_ld : 2 * (int64_t)k0);
            char* qd = smem + 2 * C::kPBytes + buf * C::kQBytes;
            #pragma unroll
            for (int i = 0; i < C::kQLoads; ++i) {
                const int q = wave * C::kQLoads + i;
                const uint32_t vo = C::kQLoads % 2 == 0 ? L.voff_q[i & 1] : (q & 1 ? L.voff_q[1] : L.voff_q[0]);
                dma16(qb + (int64_t)q * ((QW ? 4 : 16) * (int64_t)args.q_ld), vo, lds_offset(qd + q * 1024));
            }
        };

        floatx16 acc[C::FI][C::FJ];
        #pragma unroll
        for (int i = 0; i < C::FI; ++i)
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j)
                #pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

        // ---- main loop ---------------------------------------------------------------
        const int slabs = K / kBK * (PARTS > 1 ? 6 : 1);
        const int swz = swizzle(lrow);
        // transposing read: lane 16 g + s addresses row s / 4 and columns 4 (s % 4) ..
        // of a 4 x 16 block and receives the block's column s: 4 consecutive k
        const int tr_g = lane >> 4, tr_s = lane & 15;
        const int tr_row = 8 * (tr_g >> 1) + (tr_s >> 2);
        const int tr_col = 16 * (tr_g & 1) + 4 * (tr_s & 3);
        const int tr_sw = swizzle_wide(tr_s >> 2);
        auto read_wide = [&](const char* base, int col0, int ks) -> bf16x8 {
            shortx4 h[2];
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 16 * ks + 4 * u + tr_row, c = col0 + tr_col;
                const int o = r * kWideBytes + (((c >> 3) ^ tr_sw) << 4) + (c & 7) * 2;
                h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_shortx4*)((__attribute__((address_space(3))) char*)base + o));
            }
            const shortx8 w = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, w);
        };
        auto read_rows = [&](const char* base, int row0, int ks) -> bf16x8 {
            return *reinterpret_cast<const bf16x8*>(base + (row0 + lrow) * kRowBytes + (((ks * 2 + khalf) ^ swz) << 4));
        };
        __syncthreads();  // the previous tile's epilogue has left the buffers
        load_slab(0, 0, 0);
        int seg = 0, k0 = 0;
        for (int s = 0; s < slabs; ++s) {
            k0 += kBK;
            if (k0 == K) {
                k0 = 0;
                ++seg;
            }
            wait_vm<0>();
            __syncthreads();  // slab s has landed, and every wave is done with slab s - 1
            if (s + 1 < slabs) load_slab(seg, k0, (s + 1) & 1);
            const char* pb = smem + (s & 1) * C::kPBytes;
            const char* qb = smem + 2 * C::kPBytes + (s & 1) * C::kQBytes;
            #pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 fa[C::FI], fb[C::FJ];
                #pragma unroll
                for (int i = 0; i < C::FI; ++i)
                    fa[i] = PW ? read_wide(pb, wr * C::RW + 32 * i, ks) : read_rows(pb, wr * C::RW + 32 * i, ks);
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j)
                    fb[j] = QW ? read_wide(qb, wc * C::CW + 32 * j, ks) : read_rows(qb, wc * C::CW + 32 * j, ks);
                #pragma unroll
                for (int i = 0; i < C::FI; ++i)
                    #pragma unroll
                    for (int j = 0; j < C::FJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
            }
        }

        // ---- epilogue ------------------------------------------------------------------
        // acc[i][j][v]: P row wr RW + 32 i + 8 (v / 4) + 4 khalf + v % 4, Q row wc CW + 32 j + lrow
        if constexpr (MODE == kHeadLse) {
            const int64_t v_base = args.v0 + (int64_t)t.I * kTP + wr * C::RW;  // vocab row of the wave's row 0
            const int64_t left = args.vocab - v_base;
            const int limit = left < C::RW ? (int)(left < 0 ? 0 : left) : C::RW;  // rows inside the vocabulary
            const float scale = args.inv_temp * kLog2e;
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j) {
                const int row = t.J * TQ + wc * C::CW + 32 * j + lrow;
                if (limit < C::RW) {
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (32 * i + 8 * (v / 4) + 4 * khalf + v % 4 >= limit) acc[i][j][v] = -INFINITY;
                }
                if (args.target != nullptr) {
                    const int64_t off = args.target[row] - v_base;
                    const int at = off >= 0 && off < limit ? (int)off : -1;
                    const bool mine = at >= 0 && ((at >> 2) & 1) == khalf;
                    if (__builtin_amdgcn_ballot_w64(mine)) {
                        float s = 0.f;
                        #pragma unroll
                        for (int i = 0; i < C::FI; ++i)
                            #pragma unroll
                            for (int v = 0; v < 16; ++v)
                                if (at == 32 * i + 8 * (v / 4) + 4 * khalf + v % 4) s = acc[i][j][v];
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
                float l = 0.f;
                #pragma unroll
                for (int i = 0; i < C::FI; ++i)
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) l += __builtin_amdgcn_exp2f((acc[i][j][v] - m0) * scale);
                l += __shfl_xor(l, 32, 64);
                if (khalf == 0)
                    args.part[((int64_t)(args.first_tile + t.I) * C::WR + wr) * args.t_pad + row] = make_float2(m, l);
            }
        } else if constexpr (MODE == kHeadDh) {
            float4* d = reinterpret_cast<float4*>(
                args.dh + ((int64_t)(t.split * tiles_j + t.J) * args.tiles_i + t.I) * (kTP * TQ));
            #pragma unroll
            for (int i = 0; i < C::FI; ++i)
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j)
                    #pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        float4* p = d + (((wave * C::FI + i) * C::FJ + j) * 4 + v4) * 64 + lane;
                        float4 o = make_float4(acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2],
                                               acc[i][j][4 * v4 + 3]);
                        if (args.accumulate) {
                            const float4 b = *p;
                            o = make_float4(o.x + b.x, o.y + b.y, o.z + b.z, o.w + b.w);
                        }
                        *p = o;
                    }
        } else {
            if constexpr (MODE == kHeadGrad) {
                const int64_t v_base = args.v0 + (int64_t)t.I * kTP + wr * C::RW;
                const int64_t left = args.vocab - v_base;
                const int limit = left < C::RW ? (int)(left < 0 ? 0 : left) : C::RW;
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) {
                    const int row = t.J * TQ + wc * C::CW + 32 * j + lrow;
                    const float lse = args.lse[row], cp = args.cp[row], ct = args.ct[row];
                    const int64_t off = args.target != nullptr ? args.target[row] - v_base : -1;
                    const int at = off >= 0 && off < limit ? (int)off : -1;
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const int r = 32 * i + 8 * (v / 4) + 4 * khalf + v % 4;
                            float g = cp * __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], args.inv_temp, -lse) * kLog2e);
                            if (r == at) g -= ct;
                            acc[i][j][v] = r < limit ? g : 0.f;
                        }
                }
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
                                const int col = t.I * kTP + wr * C::RW + 32 * i + 8 * v4 + 4 * khalf;
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
                constexpr int kOut = MODE == kHeadGrad ? PARTS : 1;
                #pragma unroll 1
                for (int part = 0; part < kOut; ++part) {
                    __syncthreads();
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int j = 0; j < C::FJ; ++j)
                            #pragma unroll
                            for (int v4 = 0; v4 < 4; ++v4) {
                                const int r = wr * C::RW + 32 * i + 8 * v4 + 4 * khalf;
                                const int c = wc * C::CW + 32 * j + lrow;
                                uint16_t b[4];
                                #pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    b[e] = f32_to_bf16(acc[i][j][4 * v4 + e]);
                                    if (kOut > 1) acc[i][j][4 * v4 + e] -= bf16_to_f32(b[e]);
                                }
                                uint2 o;
                                o.x = (uint32_t)b[0] | ((uint32_t)b[1] << 16);
                                o.y = (uint32_t)b[2] | ((uint32_t)b[3] << 16);
                                *reinterpret_cast<uint2*>(smem + c * kWideBytes + (((r >> 3) ^ swizzle_out(c)) << 4) +
                                                          (r & 7) * 2) = o;
                            }
                    __syncthreads();
                    for (int q = tid; q < TQ * kWideChunks; q += kThreads) {
                        const int c = q / kWideChunks, ch = q % kWideChunks;
                        const uint4 v = *reinterpret_cast<const uint4*>(smem + c * kWideBytes +
                                                                        ((ch ^ swizzle_out(c)) << 4));
                        if (MODE == kHeadGrad) {
                            char* g = args.g + part * args.g_plane +
                                      2 * ((int64_t)(t.J * TQ + c) * args.g_ld + t.I * kTP + ch * 8);
                            *reinterpret_cast<uint4*>(g) = v;
                        } else {
                            const int64_t row = (int64_t)t.J * TQ + c;
                            const int col = t.I * kTP + ch * 8;
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
}

template <int TQ, int MODE, int PARTS>
hipError_t launch(const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    constexpr int kCusPerXcd = 32;
    const int64_t per_xcd = (max_tiles + kXcds - 1) / kXcds;
    const int wgs = kXcds * (int)(per_xcd < kCusPerXcd ? per_xcd : kCusPerXcd);
    hipLaunchKernelGGL((head_gemm_kernel<TQ, MODE, PARTS>), dim3(wgs), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

template <int PARTS>
hipError_t launch_mode(int mode, int tq, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    const bool wide = tq == 256;
    switch (mode) {
        case kHeadLse:
            return wide ? launch<256, kHeadLse, PARTS>(a, max_tiles, stream)
                        : launch<64, kHeadLse, PARTS>(a, max_tiles, stream);
        case kHeadGrad:
            return wide ? launch<256, kHeadGrad, PARTS>(a, max_tiles, stream)
                        : launch<64, kHeadGrad, PARTS>(a, max_tiles, stream);
        case kHeadDh:
            return wide ? launch<256, kHeadDh, PARTS>(a, max_tiles, stream)
                        : launch<64, kHeadDh, PARTS>(a, max_tiles, stream);
        case kHeadDw: return launch<256, kHeadDw, PARTS>(a, max_tiles, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_head_gemm(int mode, int tq, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    if (max_tiles <= 0) return hipSuccess;
    if (max_tiles > (int64_t)0x3fffffff) return hipErrorInvalidValue;
    return a.parts > 1 ? launch_mode<kHeadMaxPlanes>(mode, tq, a, max_tiles, stream)
                       : launch_mode<1>(mode, tq, a, max_tiles, stream);
}

}  // namespace dmuon
