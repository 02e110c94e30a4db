// dH and dW of the output-head losses for fp32 operands (modes as in
// k_head_gemm.hip): every operand lies in memory as three bf16 parts, x = hi +
// mid + lo, exact to 24 bits, and a tile takes six products of them (hi hi, hi
// mid, mid hi, mid mid, hi lo, lo hi); what they leave out is below 2^-23 of a
// product.
//
// A slab holds all three parts of both operands for a few k, so each is loaded
// once for six products: half the LDS reads and a third of the loads per MFMA
// that one product after the other would take.  A k-step is 18 KB of fragment
// reads per 48 MFMAs of a 128 x 64 wave.  Slabs of 16 k for tiles of 256 P rows
// (48 KB), of 32 for 64 x 64 ones, in a ring of three.
//
// What bounds it: the MFMA, six products of fp32's one.  820 tokens, hidden 1536,
// vocabulary 32000: dH 507 us, dW 412 us, 954 and 1174 TFLOP/s of bf16 products
// (159 and 196 of fp32, counting the 820 of 1024 token rows that are not padding;
// a library's fp32 product reaches 153), the matrix cores busy for 53% of the cycles.  One product after the other, each with
// slabs of its own, took 618 and 527 us where this took 513 and 415 (one card).
// Fragments in two sets, as in k_head_gemm.hip, do not fit beside the 128
// accumulators of a 256 x 256 tile.
#include "head_tile.h"

namespace dmuon {
namespace {

using namespace head;

template <typename C_>
struct X3 {
    using C = C_;
    static constexpr int kParts = kHeadMaxPlanes, kStages = 3;
    static constexpr int kK = C::TP == 64 ? 32 : 16;  // K of a slab
    static constexpr int kSteps = kK / 16;
    static constexpr int kRow = 2 * kK;               // a K-contiguous row of a part
    static constexpr int kRowChunks = kRow / 16;
    static constexpr int kPPart = C::TP * kRow, kQPart = C::TQ * kRow;
    static constexpr int kStage = kParts * (kPPart + kQPart);
    static constexpr int kLds = kStages * kStage > C::TP * C::TQ * 2 ? kStages * kStage : C::TP * C::TQ * 2;
    // 1 KB loads of a part, and per wave of an operand (waves past the last one repeat it, so
    // that every wave has as many to wait for)
    static constexpr int kPPartLoads = kPPart / 1024, kQPartLoads = kQPart / 1024;
    static constexpr int kPWave = (kParts * kPPartLoads + C::NW - 1) / C::NW;
    static constexpr int kQWave = (kParts * kQPartLoads + C::NW - 1) / C::NW;
    // K-contiguous rows of 2 or 4 chunks: 16 rows at one chunk hit 16 bank groups
    __device__ static __forceinline__ int swz(int r) { return kRowChunks == 2 ? (r >> 3) & 1 : (r >> 2) & 3; }
};

template <typename S, int MODE>
__global__ __launch_bounds__(S::C::NT, S::C::NT == 512 ? 1 : 2) void head_x3_kernel(HeadGemmArgs args) {
    using C = typename S::C;
    constexpr int TP = C::TP, TQ = C::TQ;
    constexpr bool QW = is_dw(MODE);  // Q is K-major, as P always is
    using WP = Wide<TP>;
    using WQ = Wide<TQ>;
    __shared__ __attribute__((aligned(1024))) char smem[S::kLds];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % C::WR, wc = wave / C::WR;
    const int lrow = lane & 31, khalf = lane >> 5;
    const int n = __builtin_amdgcn_readfirstlane(*args.count);
    const int n_k = n <= kBK ? kBK : (n + kBK - 1) / kBK * kBK;
    const Share sh = share_of<TQ, MODE>(args, n, n_k);

    for (int kq = sh.at; kq < sh.count; kq += sh.step) {
        const Tile t = tile_at(args, sh, kq);
        int K = n_k, k_first = 0;
        if (MODE == kHeadDh) {
            k_first = t.split * args.split_k;
            K = imin(args.split_k, args.k - k_first);
        } else if (MODE == kHeadDwSum) {
            const int each = (n_k / kBK + args.splits - 1) / args.splits * kBK;
            k_first = imin(t.split * each, n_k);
            K = imin(each, n_k - k_first);
        }
        const int slabs = K / S::kK;
        // ---- loads: block q of an operand's slab is 1 KB of part q / (loads of a part) --------
        const char* const p0 = args.p + 2 * (int64_t)k_first * args.p_ld;
        uint32_t voff_p[2], voff_q[2];
        #pragma unroll
        for (int par = 0; par < 2; ++par) {
            const int row = lane / WP::kChunksRow;
            const int lc = (lane % WP::kChunksRow) ^ WP::swz(WP::kRows * par + row);
            // columns past the row's end repeat its last chunk (never stored)
            voff_p[par] = (uint32_t)(2 * (row * args.p_ld + imin(t.I * TP + lc * 8, args.p_ld - 8)));
        }
        const char* q0;
        if (QW) {
            q0 = args.q + 2 * (int64_t)k_first * args.q_ld;
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / WQ::kChunksRow;
                const int lc = (lane % WQ::kChunksRow) ^ WQ::swz(WQ::kRows * par + row);
                voff_q[par] = (uint32_t)(2 * (row * args.q_ld + t.J * TQ + lc * 8));
            }
        } else {
            q0 = args.q + 2 * ((int64_t)t.J * TQ * args.q_ld + k_first);
            // (a block's rows start at a multiple of 16: the swizzle does not depend on the block)
            const int row = lane / S::kRowChunks;
            voff_q[0] = voff_q[1] = (uint32_t)(2 * (row * args.q_ld + ((lane % S::kRowChunks) ^ S::swz(row)) * 8));
        }
        auto load_slab = [&](int s, int stage) {
            char* const base = smem + stage * S::kStage;
            const char* const pk = p0 + 2 * (int64_t)s * S::kK * args.p_ld;
            #pragma unroll
            for (int i = 0; i < S::kPWave; ++i) {
                const int q = imin(wave * S::kPWave + i, S::kParts * S::kPPartLoads - 1);
                const int part = q / S::kPPartLoads, b = q % S::kPPartLoads;
                dma16(pk + part * args.p_plane + (int64_t)b * (2 * WP::kRows * (int64_t)args.p_ld),
                      b & 1 ? voff_p[1] : voff_p[0], lds_offset(base + q * 1024));
            }
            const char* const qk = q0 + (QW ? 2 * (int64_t)s * S::kK * args.q_ld : 2 * (int64_t)s * S::kK);
            constexpr int kQRows = QW ? WQ::kRows : 1024 / S::kRow;
            #pragma unroll
            for (int i = 0; i < S::kQWave; ++i) {
                const int q = imin(wave * S::kQWave + i, S::kParts * S::kQPartLoads - 1);
                const int part = q / S::kQPartLoads, b = q % S::kQPartLoads;
                dma16(qk + part * args.q_plane + (int64_t)b * (2 * kQRows * (int64_t)args.q_ld),
                      b & 1 ? voff_q[1] : voff_q[0], lds_offset(base + S::kParts * S::kPPart + q * 1024));
            }
        };

        floatx16 acc[C::FI][C::FJ];
        #pragma unroll
        for (int i = 0; i < C::FI; ++i)
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j)
                #pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
        // ---- fragments: see k_head_gemm.hip -----------------------------------------------------
        const int tr_g = lane >> 4, tr_s = lane & 15;
        const int tr_row = 8 * (tr_g >> 1) + (tr_s >> 2);
        const int tr_col = 16 * (tr_g & 1) + 4 * (tr_s & 3);
        auto read_wide = [&](const char* base, int row_bytes, int sw, int col0, int ks) -> bf16x8 {
            shortx4 h[2];
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 16 * ks + 4 * u + tr_row, c = col0 + tr_col;
                h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_shortx4*)((__attribute__((address_space(3))) char*)base + r * row_bytes +
                                   (((c >> 3) ^ sw) << 4) + (c & 7) * 2));
            }
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
        };
        __syncthreads();  // the previous tile's epilogue has left the buffers
        #pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s)
            if (s < slabs) load_slab(s, s);
        int stage = 0;
        for (int s = 0; s < slabs; ++s) {
            // loads complete in order: slab s has landed when only the next slab's are in flight
            if (s + 1 < slabs) wait_vm<S::kPWave + S::kQWave>(); else wait_vm<0>();
            __syncthreads();  // ... for every wave, and every wave is done with slab s - 1
            if (s + 2 < slabs) load_slab(s + 2, stage == 0 ? 2 : stage - 1);
            const char* const pb = smem + stage * S::kStage;
            const char* const qb = pb + S::kParts * S::kPPart;
            stage = stage == 2 ? 0 : stage + 1;
            #pragma unroll
            for (int ks = 0; ks < S::kSteps; ++ks) {
                bf16x8 fb[S::kParts][C::FJ];
                #pragma unroll
                for (int part = 0; part < S::kParts; ++part)
                    #pragma unroll
                    for (int j = 0; j < C::FJ; ++j) {
                        const char* const b = qb + part * S::kQPart;
                        const int row0 = wc * C::CW + 32 * j;
                        fb[part][j] = QW ? read_wide(b, WQ::kBytes, WQ::swz(tr_s >> 2), row0, ks)
                                         : *reinterpret_cast<const bf16x8*>(b + (row0 + lrow) * S::kRow +
                                                                            (((ks * 2 + khalf) ^ S::swz(lrow)) << 4));
                    }
                #pragma unroll
                for (int i = 0; i < C::FI; ++i) {
                    bf16x8 fa[S::kParts];
                    #pragma unroll
                    for (int part = 0; part < S::kParts; ++part)
                        fa[part] = read_wide(pb + part * S::kPPart, WP::kBytes, WP::swz(tr_s >> 2), wr * C::RW + 32 * i, ks);
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
        }
        write_tile<C, MODE, false, kHeadMaxPlanes>(args, t, sh.tiles_j, smem, acc, [] {});
    }
}

template <typename S, int MODE>
hipError_t launch(const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    const int64_t per_xcd = (max_tiles + kXcds - 1) / kXcds, most = head_slots(S::C::TP) / kXcds;
    const int wgs = kXcds * (int)(per_xcd < most ? per_xcd : most);
    hipLaunchKernelGGL((head_x3_kernel<S, MODE>), dim3(wgs), dim3(S::C::NT), 0, stream, a);
    return hipGetLastError();
}

template <typename C>
hipError_t launch_config(int mode, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    switch (mode) {
        case kHeadDh: return launch<X3<C>, kHeadDh>(a, max_tiles, stream);
        case kHeadDw: return launch<X3<C>, kHeadDw>(a, max_tiles, stream);
        case kHeadDwSum: return launch<X3<C>, kHeadDwSum>(a, max_tiles, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_head_x3(int mode, HeadTile tile, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    if (tile.tp == 64) return launch_config<Config<64, 64, 4>>(mode, a, max_tiles, stream);
    if (tile.tq == 64) return launch_config<Config<256, 64, 2>>(mode, a, max_tiles, stream);
    if (tile.tq == 128) return launch_config<Config<256, 128, 3>>(mode, a, max_tiles, stream);
    return launch_config<Config<256, 256, 2>>(mode, a, max_tiles, stream);
}

}  // namespace dmuon
