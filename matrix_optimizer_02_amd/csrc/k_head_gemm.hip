// The products of the output-head losses on bf16 MFMA (gfx950), one tile
// kernel in five modes, each C[r][c] = sum over k of P[r][k] Q[c][k]:
//   Lse   s^T = W H^T     softmax statistics of every vocab tile
//   Grad  s^T = W H^T     again, ds = cp exp(s / T - lse) - ct [target] out
//   dH    dH^T = W^T ds^T  k over the vocab rows of the piece, fp32 sums
//   dW    dW^T = H^T ds    k over the tokens (DwSum: in splits of them, fp32 sums)
// s itself never leaves the registers.  With the vocabulary along the tile's P
// rows, a lane holds 32 x FI / 2 logits of each of its tokens, so the running
// maximum and sum of the softmax are formed inside a lane and joined across
// two lanes by one shuffle.
//
// fp32 operands.  The logits' come as two fp16 parts x = hi + lo, each row
// scaled by a power of two to put its largest element near 2^14: 22 bits, so a
// logit is off by at most 2^-21 of the sum of its products' magnitudes, less
// than fp32's own additions of more than 8 products may be (a logit's error
// counts absolutely: exp turns it into a relative one).  An element below 2^-17 of
// its row's largest has a low part among fp16's subnormals and is off by up to
// 2^-39 of that largest; calls in which this could move a logit by more than 2^-22 T
// take the three-part products of k_head_stream.hip instead, decided on the device
// from the rows' largest elements and sums (wide_range there).  A row's 32 hi and 32 lo
// values of a k-block lie next to each other, so a slab holds both and takes 6
// MFMA k-steps (hi hi, hi lo, lo hi).  The gradients of fp32 operands:
// k_head_x3.hip.
//
// Tiles.  256 x 256 outputs, 8 waves, for work that fills the chip; 256 x 128
// where 256 token rows would be mostly padding; 256 x 64 for batches of at most
// 64 rows, which are bound by reading W; 64 x 64, 4 waves, where the others
// would leave most CUs idle (pick_tile in head_layout.cpp has the rule, with the
// measured cost of each shape).  K goes through a ring of ST slabs of 64 in LDS, filled by
// direct global->LDS loads ST - 1 slabs ahead; 16-byte chunks are XOR-swizzled by row.
//
// What bounds it: the MFMA.  The main loop is pipelined in registers: while one set
// of fragments is multiplied the next is read from LDS, also across the barrier that
// lands the next slab, and the first slab of the next tile loads behind the epilogue.
// Against read, wait, multiply (8192 tokens, hidden 4096, vocabulary 128256, bf16):
// backward 21.4 ms for 21.8; 238 x 1792 x 16374 backward 92 us for 103.  The softmax
// statistics of 256 x 256 bf16 tiles keep the plain loop (plain_loop in head_tile.h
// has the figures).  At that first size Lse reaches 1148 TFLOP/s, Grad 1063, dH 1160
// and dW 1166 on one card (1234, 1153, 1221 and 1235 on another), where a library's plain
// products of the same operands, logits written, reach 1451 (logits), 1345 (dH) and 1124
// (dW).  The matrix cores are busy for 56 to 60% of the cycles, LDS conflicts take at most
// 2% of its own and memory is read and written at 1.0 to 1.2 TB/s: what is lost is lost
// at barriers and in epilogues.  What keeps Lse from more is its epilogue (an exponential a
// logit, with the MFMA idle: two tiles' accumulators do not fit in one wave's
// registers) and one workgroup a CU, so that no other covers the barriers.
#include "head_tile.h"

namespace dmuon {
namespace {

using namespace head;

// KIND: kHeadBf16, or kHeadHalf2 (logits of fp32 operands).
template <typename C, int MODE, int KIND>
__global__ __launch_bounds__(C::NT) __attribute__((
    amdgpu_waves_per_eu(2, plain_loop<C, MODE>(KIND == kHeadHalf2) ? 8 : 2))) void head_gemm_kernel(HeadGemmArgs args) {
    constexpr bool PW = MODE == kHeadDh || is_dw(MODE);  // P is K-major
    constexpr bool QW = is_dw(MODE);                     // Q is K-major
    constexpr int TP = C::TP, TQ = C::TQ;
    using WP = Wide<TP>;
    using WQ = Wide<TQ>;
    __shared__ __attribute__((aligned(1024))) char smem[C::kLds];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % C::WR, wc = wave / C::WR;
    const int lrow = lane & 31, khalf = lane >> 5;

    // ---- which tiles -----------------------------------------------------------------
    const int n = __builtin_amdgcn_readfirstlane(*args.count);
    const int n_k = n <= kBK ? kBK : (n + kBK - 1) / kBK * kBK;  // dW's K extent
    const Share sh = share_of<TQ, MODE>(args, n, n_k);
    // Where a tile's slabs come from, and its K extent (a multiple of kBK).
    struct Plan {
        Tile t;
        Loads L;
        int K;
        bool empty;
    };
    auto plan = [&](int kq, Plan& pl) {
        const Tile t = pl.t = tile_at(args, sh, kq);
        Loads& L = pl.L;
        int& K = pl.K;
        // ---- operands ----------------------------------------------------------------
        int k_first = 0;
        if (MODE == kHeadDh) {
            k_first = t.split * args.split_k;
            K = imin(args.split_k, args.k - k_first);
        } else if (MODE == kHeadDw) {
            K = n_k;
        } else if (MODE == kHeadDwSum) {
            const int each = (n_k / kBK + args.splits - 1) / args.splits * kBK;
            k_first = t.split * each;
            K = imin(each, n_k - k_first);
            pl.empty = K <= 0;  // a last split may have nothing: it multiplies a slab for nothing
            if (pl.empty) {
                k_first = 0;
                K = kBK;
            }
        } else {
            K = args.k;
        }
        L.tail_k = INT_MAX;
        if (PW) {
            L.p = args.p + 2 * (int64_t)k_first * args.p_ld;
            if (MODE == kHeadDh && args.tail_row != INT_MAX) L.tail_k = args.tail_row - k_first;
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / WP::kChunksRow;  // + kRows q
                const int lc = (lane % WP::kChunksRow) ^ WP::swz(WP::kRows * par + row);
                // columns past the row's end repeat its last chunk (never stored)
                const int col = imin(t.I * TP + lc * 8, args.p_ld - 8);
                L.voff_p[par] = (uint32_t)(2 * (row * args.p_ld + col));
            }
        } else {
            const int row0 = t.I * TP;
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
            L.q = args.q + 2 * (int64_t)k_first * args.q_ld;
            #pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int row = lane / WQ::kChunksRow;
                const int lc = (lane % WQ::kChunksRow) ^ WQ::swz(WQ::kRows * par + row);
                L.voff_q[par] = (uint32_t)(2 * (row * args.q_ld + t.J * TQ + lc * 8));
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
    };
    // the slab at k0 into a stage
    auto load_slab = [&](const Loads& L, int k0, int stage) {
        const char* pb = L.p;
        if (PW) {
            if (MODE == kHeadDh && k0 >= L.tail_k)
                pb = args.p_tail + 2 * (int64_t)(k0 - L.tail_k) * args.p_ld;
            else
                pb += 2 * (int64_t)k0 * args.p_ld;
        } else {
            pb += 2 * k0;
        }
        char* pd = smem + stage * (C::kPBytes + C::kQBytes);
        constexpr int kPStep = PW ? 2 * WP::kRows : 16;  // bytes per element of the row stride between 1 KB blocks
        #pragma unroll
        for (int i = 0; i < C::kPLoads; ++i) {
            const int q = wave * C::kPLoads + i;
            dma16(pb + (int64_t)q * (kPStep * (int64_t)args.p_ld), L.voff_p[i & 1], lds_offset(pd + q * 1024));
        }
        const char* qb = L.q + (QW ? 2 * (int64_t)k0 * args.q_ld : 2 * (int64_t)k0);
        char* qd = pd + C::kPBytes;
        constexpr int kQStep = QW ? 2 * WQ::kRows : 16;
        #pragma unroll
        for (int i = 0; i < C::kQLoads; ++i) {
            const int q = wave * C::kQLoads + i;
            const uint32_t vo = C::kQLoads % 2 == 0 ? L.voff_q[i & 1] : (q & 1 ? L.voff_q[1] : L.voff_q[0]);
            dma16(qb + (int64_t)q * (kQStep * (int64_t)args.q_ld), vo, lds_offset(qd + q * 1024));
        }
    };
    static_assert(C::kPLoads % 2 == 0, "load parity");

    if (sh.at >= sh.count) return;
    // The first slab of a tile goes to the last stage: the others hold the output of
    // the tile before, piece by piece, while it loads.
    constexpr int kRest = (C::ST - 1) * (C::kPBytes + C::kQBytes);
    constexpr int kPieces = (TQ * TP * 2 + kRest - 1) / kRest;
    static_assert(TQ % kPieces == 0 && TQ / kPieces % C::CW == 0, "a wave's columns lie in one piece");
    // Stores that every wave issues behind that slab's loads, at least: they need not
    // have completed for the slab to be there.
    constexpr int kStores = MODE == kHeadLse ? C::FJ
                            : MODE == kHeadGrad && TQ == 256 ? TQ * TP / 8 / C::NT
                            : MODE == kHeadDh ? C::FI * C::FJ * 4 : 0;
    bool behind = false;
    Plan pl;
    plan(sh.at, pl);
    load_slab(pl.L, 0, C::ST - 1);
    for (int kq = sh.at;;) {
        floatx16 acc[C::FI][C::FJ];
        #pragma unroll
        for (int i = 0; i < C::FI; ++i)
            #pragma unroll
            for (int j = 0; j < C::FJ; ++j)
                #pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

        constexpr bool kPlain = plain_loop<C, MODE>(KIND == kHeadHalf2);
        // ---- main loop ---------------------------------------------------------------
        const int slabs = pl.K / kBK;
        const int swz = swizzle(lrow);
        // transposing read: lane 16 g + s addresses row s / 4 and columns 4 (s % 4) ..
        // of a 4 x 16 block and receives the block's column s: 4 consecutive k
        const int tr_g = lane >> 4, tr_s = lane & 15;
        const int tr_row = 8 * (tr_g >> 1) + (tr_s >> 2);
        const int tr_col = 16 * (tr_g & 1) + 4 * (tr_s & 3);
        auto read_wide = [&](const char* base, int row_bytes, int sw, int col0, int ks) -> bf16x8 {
            shortx4 h[2];
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 16 * ks + 4 * u + tr_row, c = col0 + tr_col;
                const int o = r * row_bytes + (((c >> 3) ^ sw) << 4) + (c & 7) * 2;
                h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_shortx4*)((__attribute__((address_space(3))) char*)base + o));
            }
            const shortx8 w = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, w);
        };
        auto read_rows = [&](const char* base, int row0, int ks) -> bf16x8 {
            return *reinterpret_cast<const bf16x8*>(base + (row0 + lrow) * kRowBytes + (((ks * 2 + khalf) ^ swz) << 4));
        };
        auto read_p = [&](const char* pb, int i, int ks) -> bf16x8 {
            return PW ? read_wide(pb, WP::kBytes, WP::swz(tr_s >> 2), wr * C::RW + 32 * i, ks)
                      : read_rows(pb, wr * C::RW + 32 * i, ks);
        };
        auto read_q = [&](const char* qb, int j, int ks) -> bf16x8 {
            return QW ? read_wide(qb, WQ::kBytes, WQ::swz(tr_s >> 2), wc * C::CW + 32 * j, ks)
                      : read_rows(qb, wc * C::CW + 32 * j, ks);
        };
        __syncthreads();  // the previous tile's epilogue has left the buffers
        #pragma unroll
        for (int s = 1; s < C::ST - 1; ++s)
            if (!kPlain || s < slabs) load_slab(pl.L, imin(s, slabs - 1) * kBK, s - 1);
        int stage = C::ST - 1;
        // Loads complete in order: a slab has landed when only later slabs' may be in flight.
        // The barrier lands it for every wave; each is then done with the slab before.
        auto arrive = [&] {
            wait_vm<(C::ST - 2) * (C::kPLoads + C::kQLoads)>();
            __syncthreads();
        };
        auto first = [&] {
            if (C::ST == 2 && behind) {
                wait_vm<kStores>();
                __syncthreads();
            } else {
                arrive();
            }
        };
        // The slab ST - 1 further, into the stage that the slab before s has left.  Past the
        // tile's end the last slab again: no branch may part the loop's regions, or the
        // compiler moves the accumulators about.
        auto load_ahead = [&](int s) {
            load_slab(pl.L, imin(s + C::ST - 1, slabs - 1) * kBK, stage == 0 ? C::ST - 1 : stage - 1);
        };
        constexpr int kPReads = PW ? 2 : 1, kQReads = QW ? 2 : 1;  // LDS reads a fragment takes
        const char* pb = smem + stage * (C::kPBytes + C::kQBytes);
        const char* qb = pb + C::kPBytes;
        auto next_stage = [&] {
            stage = stage + 1 == C::ST ? 0 : stage + 1;
            pb = smem + stage * (C::kPBytes + C::kQBytes);
            qb = pb + C::kPBytes;
        };
        // Regions: MFMAs on one set of fragments while the next set is read.  The last
        // region of a slab runs behind the barrier that lands the next one.
        if constexpr (kPlain) {
            // read, wait, multiply: see plain_loop
            for (int s = 0; s < slabs; ++s) {
                if (C::ST > 2 && s + C::ST - 2 < slabs)
                    wait_vm<(C::ST - 2) * (C::kPLoads + C::kQLoads)>();
                else if (C::ST == 2 && s == 0 && behind)
                    wait_vm<kStores>();
                else
                    wait_vm<0>();
                __syncthreads();
                if (s + C::ST - 1 < slabs)
                    load_slab(pl.L, (s + C::ST - 1) * kBK, stage == 0 ? C::ST - 1 : stage - 1);
                const char* pb = smem + stage * (C::kPBytes + C::kQBytes);
                const char* qb = pb + C::kPBytes;
                stage = stage + 1 == C::ST ? 0 : stage + 1;
                #pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bf16x8 fa[C::FI], fb[C::FJ];
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i) fa[i] = read_p(pb, i, ks);
                    #pragma unroll
                    for (int j = 0; j < C::FJ; ++j) fb[j] = read_q(qb, j, ks);
                    #pragma unroll
                    for (int i = 0; i < C::FI; ++i)
                        #pragma unroll
                        for (int j = 0; j < C::FJ; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
                }
            }
        } else if constexpr (KIND == kHeadHalf2) {
            // k-steps 0, 1 of the slab hold hi, 2, 3 lo.  A region: one P fragment pair (i)
            // of one k-step, its three products with the Q pairs.
            bf16x8 ph[2], pl_[2], qh[2][C::FJ], ql[2][C::FJ];
            auto read_pair = [&](int set, int i, int ks) {
                ph[set] = read_p(pb, i, ks);
                pl_[set] = read_p(pb, i, ks + 2);
            };
            auto read_q_pairs = [&](int ks) {
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) {
                    qh[ks][j] = read_q(qb, j, ks);
                    ql[ks][j] = read_q(qb, j, ks + 2);
                }
            };
            auto mma = [&](floatx16& c, const bf16x8& x, const bf16x8& y) {
                c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, x),
                                                           __builtin_bit_cast(halfx8, y), c, 0, 0, 0);
            };
            auto multiply = [&](int set, int i, int ks) {
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) mma(acc[i][j], pl_[set], qh[ks][j]);
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) mma(acc[i][j], ph[set], ql[ks][j]);
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) mma(acc[i][j], ph[set], qh[ks][j]);
            };
            constexpr int U = 2 * C::FI;  // regions of a slab (even)
            first();
            load_ahead(0);
            read_q_pairs(0);
            read_pair(0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            for (int s = 0;;) {
                #pragma unroll
                for (int u = 0; u < U - 1; ++u) {
                    if ((u + 1) % C::FI == 0) read_q_pairs((u + 1) / C::FI);
                    read_pair((u + 1) & 1, (u + 1) % C::FI, (u + 1) / C::FI);
                    multiply(u & 1, u % C::FI, u / C::FI);
                    weave<3 * C::FJ, 2 + 2 * C::FJ>();
                }
                if (++s == slabs) break;
                arrive();
                next_stage();
                load_ahead(s);
                read_q_pairs(0);
                read_pair(0, 0, 0);
                multiply(1, C::FI - 1, 1);
                weave<3 * C::FJ, 2 + 2 * C::FJ>();
            }
            multiply(1, C::FI - 1, 1);
        } else {
            // A region: kI P fragments of one k-step.
            constexpr int kI = C::FI >= 2 ? C::FI / 2 : 1, kParts = C::FI / kI, U = KS * kParts;
            bf16x8 fa[2][kI], fb[2][C::FJ];
            auto read_a = [&](int set, int u) {
                #pragma unroll
                for (int i = 0; i < kI; ++i) fa[set][i] = read_p(pb, u % kParts * kI + i, u / kParts);
            };
            auto read_b = [&](int ks) {
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j) fb[ks & 1][j] = read_q(qb, j, ks);
            };
            auto multiply = [&](int u) {
                #pragma unroll
                for (int i = 0; i < kI; ++i)
                    #pragma unroll
                    for (int j = 0; j < C::FJ; ++j)
                        acc[u % kParts * kI + i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            fa[u & 1][i], fb[u / kParts & 1][j], acc[u % kParts * kI + i][j], 0, 0, 0);
            };
            constexpr int kAReads = kPReads * kI, kAllReads = kAReads + kQReads * C::FJ;
            static_assert(U % 2 == 0 && KS % 2 == 0, "a slab starts with the sets 0");
            first();
            load_ahead(0);
            read_b(0);
            read_a(0, 0);
            __builtin_amdgcn_sched_barrier(0);
            for (int s = 0;;) {
                #pragma unroll
                for (int u = 0; u < U - 1; ++u) {
                    const bool turn = (u + 1) % kParts == 0;
                    if (turn) read_b((u + 1) / kParts);
                    read_a((u + 1) & 1, u + 1);
                    multiply(u);
                    if (turn) weave<kI * C::FJ, kAllReads>(); else weave<kI * C::FJ, kAReads>();
                }
                if (++s == slabs) break;
                arrive();
                next_stage();
                load_ahead(s);
                read_b(0);
                read_a(0, 0);
                multiply(U - 1);
                weave<kI * C::FJ, kAllReads>();
            }
            multiply(U - 1);
        }

        wait_vm<0>();  // the loads past the end, before their stages hold the output
        if (MODE == kHeadDwSum && pl.empty) {
            #pragma unroll
            for (int i = 0; i < C::FI; ++i)
                #pragma unroll
                for (int j = 0; j < C::FJ; ++j)
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
        }
        const Tile t = pl.t;
        kq += sh.step;
        const bool more = kq < sh.count;
        if (more) plan(kq, pl);
        write_tile<C, MODE, KIND == kHeadHalf2, KIND == kHeadBf16 ? 1 : kHeadMaxPlanes, kPieces>(
            args, t, sh.tiles_j, smem, acc, [&] {
                if (more) load_slab(pl.L, 0, C::ST - 1);
            });
        if (!more) break;
        behind = true;
    }
}

template <typename C, int MODE, int KIND>
hipError_t launch(const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    const int64_t per_xcd = (max_tiles + kXcds - 1) / kXcds, most = head_slots(C::TP) / kXcds;
    const int wgs = kXcds * (int)(per_xcd < most ? per_xcd : most);
    hipLaunchKernelGGL((head_gemm_kernel<C, MODE, KIND>), dim3(wgs), dim3(C::NT), 0, stream, a);
    return hipGetLastError();
}

template <typename C>
hipError_t launch_config(int mode, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    const bool f32 = a.parts > 1;
    switch (mode) {
        case kHeadLse:
            return f32 ? launch<C, kHeadLse, kHeadHalf2>(a, max_tiles, stream)
                       : launch<C, kHeadLse, kHeadBf16>(a, max_tiles, stream);
        case kHeadGrad:
            return f32 ? launch<C, kHeadGrad, kHeadHalf2>(a, max_tiles, stream)
                       : launch<C, kHeadGrad, kHeadBf16>(a, max_tiles, stream);
        case kHeadDh:
            return launch<C, kHeadDh, kHeadBf16>(a, max_tiles, stream);
        case kHeadDw:
            return launch<C, kHeadDw, kHeadBf16>(a, max_tiles, stream);
        case kHeadDwSum:
            return launch<C, kHeadDwSum, kHeadBf16>(a, max_tiles, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_head_gemm(int mode, HeadTile tile, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    if (max_tiles <= 0) return hipSuccess;
    if (max_tiles > (int64_t)0x3fffffff) return hipErrorInvalidValue;
    if (a.parts > 1 && mode != kHeadLse && mode != kHeadGrad) return launch_head_x3(mode, tile, a, max_tiles, stream);
    if (tile.tp == 64) return launch_config<Config<64, 64, 4>>(mode, a, max_tiles, stream);
    if (tile.tq == 64) return launch_config<Config<256, 64, 2>>(mode, a, max_tiles, stream);
    if (tile.tq == 128) return launch_config<Config<256, 128, 3>>(mode, a, max_tiles, stream);
    return launch_config<Config<256, 256, 2>>(mode, a, max_tiles, stream);
}

}  // namespace dmuon
