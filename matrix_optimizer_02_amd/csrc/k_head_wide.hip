// Tile products of the output head for bf16 operands and work that fills the chip: 256 x
// 256 tiles by four waves of 128 x 128 (the modes of k_head_gemm.hip; the same sums in
// the same order, the same statistics as its other tiles).
//
// Eight waves of 128 x 64 read 192 KB of fragments from LDS for every 64 KB that a slab
// brings; four of 128 x 128 read 128 KB.  Their 256 accumulators a lane are all of the
// accumulation registers, which leaves the compiler none to move them about with: they
// are named here, and it learns only what each product writes (mma).  One wave a SIMD has nobody to
// cover for it, so everything is issued between its products: a slab's 32 fragments one k-step
// ahead, its 16 loads spread over three k-steps (they fill LDS against the fragments' reads: all in
// one they take 10% longer, 4 + 6 + 6 of them 4% than 8 + 6 + 2, which suits the gradients by 0.5%
// and the cross entropy's statistics, with 6 + 6 + 4, not by 2%), and its one barrier with a k-step's
// products on their way and fragments of the next slab behind it.  The sequence of slabs runs on
// over the tiles' ends, so the next tile's first two slabs load behind the epilogue.
//
// What bounds it: the matrix cores with the loads' way into LDS.  8192 tokens, hidden
// 4096, vocabulary 128256, statistics of softmax and entropy: 6.29 ms, 1368 TFLOP/s,
// where eight waves take 6.96 to 7.15 on the same cards; 5.8 without its loads.  5734
// tokens of that size, a piece of 16384 vocabulary rows: ds 627 us for 712, dH 772 for 829 (627
// with its splits cut by the rows that take part), dW 559 for 625.  Lines touched ahead of the loads cost 10%.
#include "head_tile.h"

#include <type_traits>
#include <utility>

namespace dmuon {
namespace {

using namespace head;

constexpr int kWT = 256;                      // tile edge
constexpr int kWThreads = 256;
constexpr int kHalf = kWT * kRowBytes;        // an operand's slab
constexpr int kWStage = 2 * kHalf;
constexpr int kWPiece = 32 * 256;             // 32 token rows of a wave's 128 words, bf16

typedef __attribute__((address_space(3))) const bf16x8 lds_frag;
__device__ __forceinline__ bf16x8 frag(uint32_t at) { return *reinterpret_cast<lds_frag*>(at); }

// ... of a K-major slab: two transposing reads, STEP bytes apart.
template <int AT, int STEP>
__device__ __forceinline__ bf16x8 frag_wide(uint32_t at) {
    const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_shortx4*>(at + AT));
    const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_shortx4*>(at + AT + STEP));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename F, int... M>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, M...>) {
    (f(std::integral_constant<int, M>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
    each(f, std::make_integer_sequence<int, N>{});
}

// The accumulators are AGPRs that the compiler does not allocate: tuple (i, j) is
// a[16 (4 i + j)] to the 15 after it.  (As operands they cannot be had: given 16 of them
// the compiler moves them about and keeps up to 160 words of them in memory.)  A product
// names the tuple that it writes, so that nothing of the compiler's own lives in one across
// the main loop; that it uses none between the products and acc_at either is checked on
// every build's assembly (check_accumulators in build.py).
template <int N>
__device__ __forceinline__ void mma(const bf16x8& a, const bf16x8& b);
template <int N>
__device__ __forceinline__ void mma_first(const bf16x8& a, const bf16x8& b);
#define HEAD_TUPLE(N, ...)                                                                                            \
    template <>                                                                                                       \
    __device__ __forceinline__ void mma<N>(const bf16x8& a, const bf16x8& b) {                                        \
        asm volatile("v_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]" ::"v"(a), "v"(b), "n"(16 * N), "n"(16 * N + 15) \
                     : __VA_ARGS__);                                                                                  \
    }                                                                                                                 \
    template <>                                                                                                       \
    __device__ __forceinline__ void mma_first<N>(const bf16x8& a, const bf16x8& b) {                                  \
        asm volatile("v_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, 0" ::"v"(a), "v"(b), "n"(16 * N), "n"(16 * N + 15)     \
                     : __VA_ARGS__);                                                                                  \
    }
HEAD_TUPLE(0, "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", "a10", "a11", "a12", "a13", "a14", "a15")
HEAD_TUPLE(1, "a16", "a17", "a18", "a19", "a20", "a21", "a22", "a23", "a24", "a25", "a26", "a27", "a28", "a29", "a30", "a31")
HEAD_TUPLE(2, "a32", "a33", "a34", "a35", "a36", "a37", "a38", "a39", "a40", "a41", "a42", "a43", "a44", "a45", "a46", "a47")
HEAD_TUPLE(3, "a48", "a49", "a50", "a51", "a52", "a53", "a54", "a55", "a56", "a57", "a58", "a59", "a60", "a61", "a62", "a63")
HEAD_TUPLE(4, "a64", "a65", "a66", "a67", "a68", "a69", "a70", "a71", "a72", "a73", "a74", "a75", "a76", "a77", "a78", "a79")
HEAD_TUPLE(5, "a80", "a81", "a82", "a83", "a84", "a85", "a86", "a87", "a88", "a89", "a90", "a91", "a92", "a93", "a94", "a95")
HEAD_TUPLE(6, "a96", "a97", "a98", "a99", "a100", "a101", "a102", "a103", "a104", "a105", "a106", "a107", "a108", "a109", "a110", "a111")
HEAD_TUPLE(7, "a112", "a113", "a114", "a115", "a116", "a117", "a118", "a119", "a120", "a121", "a122", "a123", "a124", "a125", "a126", "a127")
HEAD_TUPLE(8, "a128", "a129", "a130", "a131", "a132", "a133", "a134", "a135", "a136", "a137", "a138", "a139", "a140", "a141", "a142", "a143")
HEAD_TUPLE(9, "a144", "a145", "a146", "a147", "a148", "a149", "a150", "a151", "a152", "a153", "a154", "a155", "a156", "a157", "a158", "a159")
HEAD_TUPLE(10, "a160", "a161", "a162", "a163", "a164", "a165", "a166", "a167", "a168", "a169", "a170", "a171", "a172", "a173", "a174", "a175")
HEAD_TUPLE(11, "a176", "a177", "a178", "a179", "a180", "a181", "a182", "a183", "a184", "a185", "a186", "a187", "a188", "a189", "a190", "a191")
HEAD_TUPLE(12, "a192", "a193", "a194", "a195", "a196", "a197", "a198", "a199", "a200", "a201", "a202", "a203", "a204", "a205", "a206", "a207")
HEAD_TUPLE(13, "a208", "a209", "a210", "a211", "a212", "a213", "a214", "a215", "a216", "a217", "a218", "a219", "a220", "a221", "a222", "a223")
HEAD_TUPLE(14, "a224", "a225", "a226", "a227", "a228", "a229", "a230", "a231", "a232", "a233", "a234", "a235", "a236", "a237", "a238", "a239")
HEAD_TUPLE(15, "a240", "a241", "a242", "a243", "a244", "a245", "a246", "a247", "a248", "a249", "a250", "a251", "a252", "a253", "a254", "a255")
#undef HEAD_TUPLE
template <int N>
__device__ __forceinline__ float acc_at() {
    float x;
    asm volatile("v_accvgpr_read_b32 %0, a[%1]" : "=v"(x) : "n"(N));
    return x;
}

// dma16 to lds + AT.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int AT>
__device__ __forceinline__ void dma16_at(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base), "n"(AT)
                 : "m0", "scc", "memory");
}
#pragma clang diagnostic pop

// A wave's 32 rows of 128 bf16 in an LDS piece of its own: written by the columns that
// the accumulators hold, read by rows (chunk ch of row c).
__device__ __forceinline__ void to_piece(char* piece, const float (&x)[64], int lrow, int khalf) {
    #pragma unroll
    for (int q = 0; q < 16; ++q) {
        uint16_t b[4];
        #pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = f32_to_bf16(x[4 * q + e]);
        *reinterpret_cast<uint2*>(piece + lrow * 256 + ((q ^ (lrow & 15)) << 4) + khalf * 8) =
            make_uint2((uint32_t)b[0] | ((uint32_t)b[1] << 16), (uint32_t)b[2] | ((uint32_t)b[3] << 16));
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (only this wave's own: there is no barrier)
}
__device__ __forceinline__ uint4 from_piece(const char* piece, int c, int ch) {
    return *reinterpret_cast<const uint4*>(piece + c * 256 + ((ch ^ (c & 15)) << 4));
}

// ds and dW are written past the caches, which the operands' tiles are read from again (8192
// tokens, hidden 4096, vocabulary 128256, forward and backward 19.68 ms for 19.84), or, where the
// layout says so, through them (head_layout.cpp).
template <bool CACHED>
__device__ __forceinline__ void store(void* p, const uint4& v) {
    if (CACHED) *static_cast<uint4*>(p) = v;
    else __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, static_cast<u32x4_t*>(p));
}

template <int MODE, bool CACHED = false>
__global__ __launch_bounds__(kWThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void head_wide_kernel(HeadGemmArgs args) {
    __shared__ __attribute__((aligned(1024))) char smem[2 * kWStage + (is_grad(MODE) || MODE == kHeadDw ? kWPiece * 4 : 0)];
    // loads of a slab that k-step 3 of the slab before the last one issues, k-step 0, k-step 1
    constexpr int kLoads3 = is_stats(MODE) ? 6 : 8, kLoads0 = 6, kLoads1 = 16 - kLoads3 - kLoads0;
    constexpr bool PW = MODE == kHeadDh || is_dw(MODE), QW = is_dw(MODE);  // K-major operands
    using WP = Wide<kWT>;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave & 1, wc = wave >> 1;
    const int lrow = lane & 31;
    const int khalf = lane >> 5;

    const int n = __builtin_amdgcn_readfirstlane(*args.count);
    const int n_k = n <= kBK ? kBK : (n + kBK - 1) / kBK * kBK;
    int split_k = args.split_k, splits = args.splits;
    if (MODE == kHeadDh && args.room != 0) {
        const int slabs = args.first_k / kBK, s = head_dh_splits((n + kWT - 1) / kWT * args.tiles_i, slabs, args.room);
        split_k = (slabs + s - 1) / s * kBK;
        splits = (args.k + split_k - 1) / split_k;
    }
    const Share sh = share_of<kWT, MODE>(args, n, n_k, splits);
    if (sh.at >= sh.count) return;
    // K extent of a tile: its first k and its slabs (a last split may have none: it then
    // multiplies one for nothing)
    auto extent = [&](const Tile& t, int& first, bool& empty) {
        first = 0;
        int k = args.k;
        if (MODE == kHeadDh) {
            first = t.split * split_k;
            k = imin(split_k, args.k - first);
        } else if (MODE == kHeadDw) {
            k = n_k;
        } else if (MODE == kHeadDwSum) {
            const int per = (n_k / kBK + splits - 1) / splits * kBK;
            first = t.split * per;
            k = imin(per, n_k - first);
        }
        empty = k <= 0;
        if (empty) first = 0;
        return empty ? 1 : k / kBK;
    };

    // ---- loads: slab by slab, over the ends of tiles ------------------------------------
    // (a lane's offsets from the wave's first row: kept, or every load would take two scalar
    // additions and some of the scalar registers that the loop has too few of)
    uint32_t voff_p[8], voff_q[8];
    struct Cursor {
        const char *p, *q;
        int kq, left;  // slabs left in the tile
        int k;         // dH: of the piece's rows
    } cur;
    // K-contiguous: the wave's 64 rows; K-major: its 16 k
    const int p_step = PW ? kBK * args.p_ld : kBK, q_step = QW ? kBK * args.q_ld : kBK;
    auto open_tile = [&](int kq) {
        const Tile t = tile_at(args, sh, kq);
        int first;
        bool empty;
        cur.left = extent(t, first, empty);
        cur.kq = kq;
        if constexpr (PW) {
            cur.k = first;
            const bool tail = MODE == kHeadDh && first >= args.tail_row;
            cur.p = (tail ? args.p_tail + 2 * (int64_t)(first - args.tail_row) * args.p_ld
                          : args.p + 2 * (int64_t)first * args.p_ld) + 32 * (int64_t)wave * args.p_ld;
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int row = lane / WP::kChunksRow, lc = (lane % WP::kChunksRow) ^ WP::swz(2 * k + row);
                // columns past the row's end repeat its last chunk (never stored)
                voff_p[k] = (uint32_t)(2 * ((2 * k + row) * args.p_ld + imin(t.I * kWT + lc * 8, args.p_ld - 8)));
            }
        } else {
            const int row0 = t.I * kWT;
            cur.p = (row0 >= args.tail_row ? args.p_tail + 2 * (int64_t)(row0 - args.tail_row) * args.p_ld
                                           : args.p + 2 * (int64_t)row0 * args.p_ld) + 128 * (int64_t)wave * args.p_ld;
        }
        if constexpr (QW) cur.q = args.q + 2 * ((int64_t)(first + 16 * wave) * args.q_ld + (int64_t)t.J * kWT);
        else cur.q = args.q + 2 * ((int64_t)(t.J * kWT + 64 * wave) * args.q_ld + first);
    };
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int row = lane / kChunks, lc = (lane % kChunks) ^ swizzle(8 * k + row);
        if (!PW) voff_p[k] = (uint32_t)(2 * ((8 * k + row) * args.p_ld + lc * 8));
        if (!QW) {
            voff_q[k] = (uint32_t)(2 * ((8 * k + row) * args.q_ld + lc * 8));
        } else {
            const int wrow = lane / WP::kChunksRow, wlc = (lane % WP::kChunksRow) ^ WP::swz(2 * k + wrow);
            voff_q[k] = (uint32_t)(2 * ((2 * k + wrow) * args.q_ld + wlc * 8));
        }
    }
    // (past the last tile's end its last slab again, which nobody reads)
    auto next_slab = [&] {
        if (cur.left > 1) {
            --cur.left;
            cur.p += 2 * (int64_t)p_step;
            cur.q += 2 * (int64_t)q_step;
            if (MODE == kHeadDh) {
                cur.k += kBK;
                if (cur.k == args.tail_row) cur.p = args.p_tail + 32 * (int64_t)wave * args.p_ld;
            }
        } else if (cur.kq + sh.step < sh.count) {
            open_tile(cur.kq + sh.step);
        }
    };
    const uint32_t lds0 = lds_offset(smem), mine = lds0 + wave * 8 * 1024;
    // load i of 16: 1 KB of P (i < 8) or Q
    auto load = [&](auto i_, uint32_t stage) {
        constexpr int i = decltype(i_)::value;
        if constexpr (i < 8) dma16_at<i * 1024>(cur.p, voff_p[i], mine + stage);
        else dma16_at<kHalf + (i - 8) * 1024>(cur.q, voff_q[i - 8], mine + stage);
    };

    // ---- fragments -------------------------------------------------------------------------
    // K-contiguous rows: of k-step ks in stage 0; K-major: of rows or columns 32 i ...
    uint32_t pa[4], qa[4];
    const int tr_g = lane >> 4, tr_s = lane & 15;
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t o = (uint32_t)(lrow * kRowBytes + (((k * 2 + khalf) ^ swizzle(lrow)) << 4));
        pa[k] = lds0 + wr * 128 * kRowBytes + o;
        qa[k] = lds0 + kHalf + wc * 128 * kRowBytes + o;
        // transposing read: see k_head_gemm.hip
        const int row = 8 * (tr_g >> 1) + (tr_s >> 2), col = 32 * k + 16 * (tr_g & 1) + 4 * (tr_s & 3);
        auto wide = [&](int col0) {
            return (uint32_t)(row * WP::kBytes + ((((col0 + col) >> 3) ^ WP::swz(tr_s >> 2)) << 4) + (col & 7) * 2);
        };
        if (PW) pa[k] = lds0 + wide(wr * 128);
        if (QW) qa[k] = lds0 + kHalf + wide(wc * 128);
    }
    // fragment i of k-step ks, `from` a stage
    auto read_p = [&](auto i_, auto ks_, uint32_t from) {
        constexpr int i = decltype(i_)::value, ks = decltype(ks_)::value;
        if constexpr (PW) return frag_wide<ks * 16 * WP::kBytes, 4 * WP::kBytes>(pa[i] + from);
        else return frag(pa[ks] + from + i * 32 * kRowBytes);
    };
    auto read_q = [&](auto j_, auto ks_, uint32_t from) {
        constexpr int j = decltype(j_)::value, ks = decltype(ks_)::value;
        if constexpr (QW) return frag_wide<ks * 16 * WP::kBytes, 4 * WP::kBytes>(qa[j] + from);
        else return frag(qa[ks] + from + j * 32 * kRowBytes);
    };
    bf16x8 fa[2][4], fb[2][4];

    open_tile(sh.at);
    each<16>([&](auto i_) { load(i_, 0); });
    next_slab();
    each<kLoads3>([&](auto i_) { load(i_, kWStage); });
    wait_vm<kLoads3>();
    __builtin_amdgcn_s_barrier();
    each<4>([&](auto r_) {
        constexpr int r = decltype(r_)::value;
        fa[0][r] = read_p(r_, std::integral_constant<int, 0>{}, 0);
        fb[0][r] = read_q(r_, std::integral_constant<int, 0>{}, 0);
    });
    uint32_t stage = 0;
    for (int kq = sh.at; kq < sh.count; kq += sh.step) {
        const Tile t = tile_at(args, sh, kq);
        int k_first;
        bool empty;
        const int slabs = extent(t, k_first, empty);
        #pragma unroll 1
        for (int s = 0; s < slabs; ++s) {
            // Regions: 16 MFMAs on one set of fragments while the next is read.
            auto region = [&](auto ks_, auto first_) {
                constexpr int ks = decltype(ks_)::value, set = ks & 1;
                constexpr bool kFirst = decltype(first_)::value;
                const uint32_t from = ks + 1 < KS ? stage : stage ^ kWStage;
                constexpr std::integral_constant<int, (ks + 1) % KS> next{};
                each<16>([&](auto m_) {
                    constexpr int m = decltype(m_)::value, i = m / 4, j = m % 4;
                    if constexpr (kFirst) mma_first<m>(fa[set][i], fb[set][j]);
                    else mma<m>(fa[set][i], fb[set][j]);
                    if constexpr (m < 8) {
                        // in the order of their use
                        constexpr std::integral_constant<int, m == 0 ? 0 : m <= 4 ? m - 1 : m - 4> r{};
                        if constexpr (m == 0 || m > 4) fa[set ^ 1][r] = read_p(r, next, from);
                        else fb[set ^ 1][r] = read_q(r, next, from);
                    }
                    if constexpr (m % 2 == 1) {
                        if constexpr (ks == KS - 1) {
                            if constexpr (m / 2 < kLoads3) load(std::integral_constant<int, m / 2>{}, stage);
                        } else if constexpr (ks == 0) {
                            if constexpr (m / 2 < kLoads0) load(std::integral_constant<int, kLoads3 + m / 2>{}, stage ^ kWStage);
                        } else if constexpr (ks == 1) {
                            if constexpr (m / 2 < kLoads1) load(std::integral_constant<int, kLoads3 + kLoads0 + m / 2>{}, stage ^ kWStage);
                        }
                    }
                });
            };
            if (s == 0) region(std::integral_constant<int, 0>{}, std::true_type{});
            else region(std::integral_constant<int, 0>{}, std::false_type{});
            region(std::integral_constant<int, 1>{}, std::false_type{});
            next_slab();
            region(std::integral_constant<int, 2>{}, std::false_type{});
            // every fragment of this stage is in registers, and the next slab has landed
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            region(std::integral_constant<int, 3>{}, std::false_type{});
            stage ^= kWStage;
        }
        // ---- epilogue: see write_tile --------------------------------------------------------
        asm volatile("s_nop 15\n\ts_nop 15");  // the last products are in the accumulators
        // (read from the kernel's arguments here: held through the loop, they would take the scalar
        // registers that it needs)
        const auto* ka = (const __attribute__((address_space(4))) HeadGemmArgs*)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(ka));
        const int64_t v_base = ka->v0 + (int64_t)t.I * kWT + wr * 128;
        const int64_t left = ka->vocab - v_base;
        const int limit = left < 128 ? (int)(left < 0 ? 0 : left) : 128;
        const int row0 = t.J * kWT + wc * 128 + lrow;
        [[maybe_unused]] int target[4];
        #pragma unroll
        for (int j = 0; j < 4; ++j)
            if constexpr (is_stats(MODE) || is_grad(MODE)) target[j] = ka->target != nullptr ? ka->target[row0 + 32 * j] : -1;
        // where a lane's target is among its elements: 32 i + 8 q + r of 32 i + 8 q + 4 khalf + r, or -1
        auto place = [&](int j) {
            const int64_t off = target[j] - v_base;
            return off >= 0 && off < limit && (((int)off >> 2) & 1) == khalf ? (int)off - 4 * khalf : -1;
        };
        auto row_of = [](int e) { return 32 * (e / 16) + 8 * (e % 16 / 4) + e % 4; };
        if constexpr (is_stats(MODE)) {
            const float scale = ka->inv_temp * kLog2e;
            const int64_t part = (int64_t)(ka->first_tile + t.I) * 2 + wr;
            each<4>([&](auto j_) {
                constexpr int j = decltype(j_)::value;
                float x[64];
                each<64>([&](auto e_) {
                    constexpr int e = decltype(e_)::value;
                    x[e] = acc_at<16 * (4 * (e / 16) + j) + e % 16>();
                });
                __builtin_amdgcn_sched_barrier(0);
                const int row = row0 + 32 * j;
                if constexpr (MODE != kHeadTop) {
                    if (ka->logits != nullptr) {
                        float* const out = ka->logits + (int64_t)row * ka->logits_ld + v_base + 4 * khalf;
                        #pragma unroll
                        for (int q = 0; q < 16; ++q)
                            *reinterpret_cast<float4*>(out + 8 * q) = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                    }
                }
                if (limit < 128) {
                    #pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (row_of(e) >= limit - 4 * khalf) x[e] = -INFINITY;
                }
                const int at = place(j);
                if (__builtin_amdgcn_ballot_w64(at >= 0)) {
                    float s = 0.f;
                    #pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (at == row_of(e)) s = x[e];
                    if (at >= 0) ka->target_logit[row] = s;
                }
                float m = -INFINITY;
                #pragma unroll
                for (int e = 0; e < 64; ++e) m = fmaxf(m, x[e]);
                m = fmaxf(m, __shfl_xor(m, 32, 64));
                const float m0 = m == -INFINITY ? 0.f : m;
                if constexpr (MODE == kHeadTop) {
                    float shown[8];
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float m1 = -INFINITY, m2 = -INFINITY;
                        uint32_t at1 = 0;
                        #pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const float y = x[16 * i + v];
                            const bool larger = y > m1;
                            at1 = larger ? v : at1;
                            m2 = __builtin_amdgcn_fmed3f(m1, m2, y);
                            m1 = larger ? y : m1;
                        }
                        shown[2 * i] = m1;
                        shown[2 * i + 1] = __uint_as_float((__float_as_uint(m2) & ~15u) | at1);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    float4* const out = reinterpret_cast<float4*>(ka->top + row * ka->row_groups + part * 8 + khalf * 4);
                    out[0] = make_float4(shown[0], shown[1], shown[2], shown[3]);
                    out[1] = make_float4(shown[4], shown[5], shown[6], shown[7]);
                }
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
                [[maybe_unused]] float es[4] = {0.f, 0.f, 0.f, 0.f};
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p[16];
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) x[16 * i + v] = (x[16 * i + v] - m0) * scale;
                    __builtin_amdgcn_sched_barrier(0);
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) p[v] = __builtin_amdgcn_exp2f(x[16 * i + v]);
                    __builtin_amdgcn_sched_barrier(0);
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        ls[v & 3] += p[v];
                        if constexpr (is_probs(MODE)) es[v & 3] = fmaf(p[v], fmaxf(x[16 * i + v], -200.f), es[v & 3]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                float l = (ls[0] + ls[1]) + (ls[2] + ls[3]);
                l += __shfl_xor(l, 32, 64);
                if constexpr (is_probs(MODE)) {
                    float e = (es[0] + es[1]) + (es[2] + es[3]);
                    e += __shfl_xor(e, 32, 64);
                    if (khalf == 0) {
                        const int64_t to = row * ka->row_parts + part;
                        ka->part[to] = make_float2(m, l);
                        ka->part_e[to] = e;
                    }
                } else if (khalf == 0) {
                    ka->part[part * ka->t_pad + row] = make_float2(m, l);
                }
            });
        } else if constexpr (MODE == kHeadDh || MODE == kHeadDwSum) {
            // in the order in which eight waves of 128 x 64 hold them (launch_head_sum)
            float4* const d = reinterpret_cast<float4*>(ka->sums) +
                              ((int64_t)(t.split * sh.tiles_j + t.J) * ka->tiles_i + t.I) * (kWT * kWT / 4) + lane;
            const bool add = MODE == kHeadDh && ka->accumulate;
            each<4>([&](auto j_) {
                constexpr int j = decltype(j_)::value;
                float x[64];
                each<64>([&](auto e_) {
                    constexpr int e = decltype(e_)::value;
                    x[e] = acc_at<16 * (4 * (e / 16) + j) + e % 16>();
                });
                const int wave8 = 2 * (2 * wc + j / 2) + wr;
                float4* const p = d + (int64_t)wave8 * (4 * 2 * 4 * 64) + (j % 2) * (4 * 64);
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 b[8];
                    if (add) {
                        #pragma unroll
                        for (int q = 0; q < 8; ++q) b[q] = p[((2 * h + q / 4) * 2 * 4 + q % 4) * 64];
                    }
                    #pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int e = 32 * h + 4 * q;
                        float4 o = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                        if (MODE == kHeadDwSum && empty) o = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (add) o = make_float4(o.x + b[q].x, o.y + b[q].y, o.z + b[q].z, o.w + b[q].w);
                        p[((2 * h + q / 4) * 2 * 4 + q % 4) * 64] = o;
                    }
                }
            });
        } else if constexpr (MODE == kHeadDw) {
            const float norm = norm_of(ka->norm);
            const int dw_ld = ka->dw_ld, col = t.I * kWT + wr * 128 + (lane % 16) * 8;
            const int64_t dw_rows = ka->dw_rows;
            uint16_t* const dw = static_cast<uint16_t*>(ka->dw);
            char* const piece = smem + 2 * kWStage + wave * kWPiece;
            each<4>([&](auto j_) {
                constexpr int j = decltype(j_)::value;
                float x[64];
                each<64>([&](auto e_) {
                    constexpr int e = decltype(e_)::value;
                    x[e] = acc_at<16 * (4 * (e / 16) + j) + e % 16>() * norm;
                });
                to_piece(piece, x, lrow, khalf);
                #pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int c = 4 * u + lane / 16;
                    const int64_t row = (int64_t)t.J * kWT + wc * 128 + 32 * j + c;
                    const uint4 v = from_piece(piece, c, lane % 16);
                    if (row >= dw_rows || col >= dw_ld) continue;
                    uint16_t* const p = dw + row * dw_ld + col;
                    if ((dw_ld & 7) == 0) {
                        store<CACHED>(p, v);
                    } else {
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        #pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (col + e < dw_ld) p[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
                    }
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            });
        } else {
            const float inv_norm = 1.f / norm_of(ka->norm), inv_temp = ka->inv_temp;
            float lse[4], cp[4], ct[4];
            [[maybe_unused]] float ce[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                lse[j] = ka->lse[row0 + 32 * j];
                cp[j] = ka->cp[row0 + 32 * j] * inv_norm;
                ct[j] = ka->ct[row0 + 32 * j] * inv_norm;
                if constexpr (MODE == kHeadGradEntropy) ce[j] = ka->ce[row0 + 32 * j] * inv_norm;
            }
            // a wave's 32 rows at a time through an LDS piece of its own, as rows of 128 words
            char* const piece = smem + 2 * kWStage + wave * kWPiece;
            const int64_t g_ld = ka->g_ld;
            char* const g_out = ka->g + 2 * ((int64_t)(t.J * kWT + wc * 128) * g_ld + t.I * kWT + wr * 128);
            each<4>([&](auto j_) {
                constexpr int j = decltype(j_)::value;
                float x[64];
                each<64>([&](auto e_) {
                    constexpr int e = decltype(e_)::value;
                    x[e] = acc_at<16 * (4 * (e / 16) + j) + e % 16>();
                });
                __builtin_amdgcn_sched_barrier(0);
                auto weight = [&](float y) { return MODE == kHeadGradEntropy ? fmaf(ce[j], fmaxf(y, -200.f), cp[j]) : cp[j]; };
                const int at = place(j);
                float hit = 0.f;
                const bool any = __builtin_amdgcn_ballot_w64(at >= 0);
                if (any) {
                    #pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (at == row_of(e)) hit = x[e];
                    const float y = fmaf(hit, inv_temp, -lse[j]);
                    hit = fmaf(__builtin_amdgcn_exp2f(y * kLog2e), weight(y), -ct[j]);
                }
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p[16];
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) x[16 * i + v] = fmaf(x[16 * i + v], inv_temp, -lse[j]);
                    __builtin_amdgcn_sched_barrier(0);
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) p[v] = __builtin_amdgcn_exp2f(x[16 * i + v] * kLog2e);
                    __builtin_amdgcn_sched_barrier(0);
                    #pragma unroll
                    for (int v = 0; v < 16; ++v) x[16 * i + v] = p[v] * weight(x[16 * i + v]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (any) {
                    #pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (at == row_of(e)) x[e] = hit;
                }
                if (limit < 128) {
                    #pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (row_of(e) >= limit - 4 * khalf) x[e] = 0.f;
                }
                to_piece(piece, x, lrow, khalf);
                #pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int c = 4 * u + lane / 16, ch = lane % 16;
                    store<CACHED>(g_out + 2 * ((32 * j + c) * g_ld + ch * 8), from_piece(piece, c, ch));
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            });
        }
    }
    wait_vm<0>();  // no load may land when the workgroup has gone
}

}  // namespace

hipError_t launch_head_wide(int mode, const HeadGemmArgs& a, int64_t max_tiles, hipStream_t stream) {
    const int64_t per_xcd = (max_tiles + kXcds - 1) / kXcds, most = head_slots(kWT) / kXcds;
    const dim3 grid(kXcds * (int)(per_xcd < most ? per_xcd : most)), block(kWThreads);
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    switch (mode) {
        case kHeadLse: launch(head_wide_kernel<kHeadLse>); break;
        case kHeadProbs: launch(head_wide_kernel<kHeadProbs>); break;
        case kHeadTop: launch(head_wide_kernel<kHeadTop>); break;
        case kHeadGrad:
            if (a.cached) launch(head_wide_kernel<kHeadGrad, true>);
            else launch(head_wide_kernel<kHeadGrad>);
            break;
        case kHeadGradEntropy:
            if (a.cached) launch(head_wide_kernel<kHeadGradEntropy, true>);
            else launch(head_wide_kernel<kHeadGradEntropy>);
            break;
        case kHeadDh: launch(head_wide_kernel<kHeadDh>); break;
        case kHeadDw:
            if (a.cached) launch(head_wide_kernel<kHeadDw, true>);
            else launch(head_wide_kernel<kHeadDw>);
            break;
        case kHeadDwSum: launch(head_wide_kernel<kHeadDwSum>); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace dmuon
