// Decode and verify attention over a 4-bit paged cache.
//
// out = softmax(scale q . k) v over a sequence's cached positions, with
// k = e2m1(code) * e4m3(group scale) * k_scale (V alike); pa_fp4.cuh has the
// format.  Work list, partitions, partials and their merge are those of the
// 16-bit decode kernel; the block step differs.
//
// One warp handles one (sequence partition, kv head) item and streams its
// (block, kv head) tiles, 9 D bytes each for K and for V, two blocks a step.
//  * The warp copies the tiles into its own ring of shared-memory slots with
//    16-byte cp.async, all lanes at once, and waits for no other warp.
//  * The tensor-core fragments come from the tiles without a 16-bit copy.  For
//    S^T = K Q^T a lane (g, c) = (lane / 4, lane % 4) reads its quarter row of
//    dims for two tokens (one 16-byte load each at head_dim 128); the order of
//    the dims in the contraction is free, and Q^T is loaded in the same order.
//    For O^T = V^T P^T it reads 16 dims (one scale group) of tokens 4c .. 4c +
//    3; two masks and shifts per word pair the tokens of each dim, so that one
//    conversion gives an fp16 pair of consecutive tokens of one dim, which is
//    what the fragment holds.
//  * Codes are widened to fp16 and multiplied by their group's scale (exact,
//    see group_values), then fed to mma.sync m16n8k16 (fp32 accumulate).  P is
//    fp16 (at most 2^8, 11 significant bits).  bf16 queries enter as fp16
//    times a power of two per column, chosen so that the column's largest
//    magnitude lies in [2^8, 2^9): every element above 2^-22 of it is exact.
//  * Softmax: a column's reference maximum moves only when some score passes
//    it by more than 2^8, so most steps need one vote and no reduction.  P^T
//    reaches the second product's layout through movmatrix.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pa_fp4.cuh"

namespace pa {

namespace {

constexpr int kFp4Warps = 4;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLazyLog2 = 8.f;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// D = A B (m16n8k16, fp16 operands, fp32 result), without an accumulator to clear.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 bytes from memory (src + kSrc) to shared memory (dst + kDst), not kept in
// L1 (each tile is read once).
template <int kDst, int kSrc>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(kDst), "n"(kSrc)
                 : "memory");
}
// f(0), f(1) .. f(N - 1) with the index as a compile-time constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_for<N, I + 1>(f);
    }
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {   // until at most N groups are pending
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// W 32-bit words (and 8- or 16-bit ones) of shared memory at `addr` + kOff.
template <int W, int kOff>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
    if constexpr (W == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr), "n"(kOff));
    else if constexpr (W == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr), "n"(kOff));
    else
        asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(addr), "n"(kOff));
}
template <int kOff>
__device__ __forceinline__ uint16_t lds_u16(uint32_t addr) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(x) : "r"(addr), "n"(kOff));
    return x;
}
template <int kOff>
__device__ __forceinline__ uint16_t lds_u8x2(uint32_t addr) {   // one byte, twice
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(x) : "r"(addr), "n"(kOff));
    return static_cast<uint16_t>(x * 0x0101u);
}

// One block's tiles as this lane holds them.
template <int D>
struct Fp4K {
    static constexpr int KW = D / 32;    // 32-bit words of codes per token (a quarter row)
    uint32_t k[2][KW];                   // tokens ta, ta + 2
    uint16_t ks[2];                      // their scales (two groups at head_dim 128, one twice at 64)
};
template <int D>
struct Fp4V {
    static constexpr int VW = D / 64;    // 32-bit words of codes per token
    uint32_t v[4][VW];                   // tokens 4c .. 4c + 3 (pairs swapped: flip), dims of this lane
    uint32_t vs;                         // scales of tokens 4c .. 4c + 3
};

// Byte offsets of this lane's words within a tile.  The lanes of a V load read
// 64-byte rows: quarters c = 2, 3 take their token pairs in swapped order, so
// that a load touches even and odd rows alike (two wavefronts per half warp
// instead of four); S^T takes its rows in the same order.
template <int D>
struct Fp4Lane {
    using Tile = Fp4Tile<D>;
    int ta;              // rows g and g + 8 of S^T: tokens ta, ta + 2
    int k, ks, vs;
    int va, vb;          // first and second token of a pair
    uint32_t flip;       // byte order of a word of four scales: this quarter's pairs may be swapped
    __device__ __forceinline__ explicit Fp4Lane(int lane) {
        const int g = lane >> 2, c = lane & 3;
        ta = 4 * (g >> 1) + ((g & 1) ^ (g >> 2));
        flip = c >> 1 ? 0x2301u : 0x3210u;
        k = ta * Tile::kRow + c * (Tile::kRow / 4);
        ks = Tile::scale_off(false, ta, c * (D / 64));
        va = (4 * c + (c >> 1)) * Tile::kRow + g * (Tile::kRow / 8);
        vb = (4 * c + 1 - (c >> 1)) * Tile::kRow + g * (Tile::kRow / 8);
        vs = Tile::scale_off(true, 4 * c, D == 128 ? g : g >> 1);
    }
    // `slot`: shared address of a slot; kJ: which of its two blocks.
    template <int kJ>
    __device__ __forceinline__ void load_k(Fp4K<D>& f, uint32_t slot) const {
        constexpr int o = 2 * kJ * Tile::kBytes;
        lds_words<Fp4K<D>::KW, o>(slot + k, f.k[0]);
        lds_words<Fp4K<D>::KW, o + 2 * Tile::kRow>(slot + k, f.k[1]);
        if constexpr (D == 128) {
            f.ks[0] = lds_u16<o>(slot + ks);
            f.ks[1] = lds_u16<o + 2 * Tile::kGroups>(slot + ks);
        } else {
            f.ks[0] = lds_u8x2<o>(slot + ks);
            f.ks[1] = lds_u8x2<o + 2 * Tile::kGroups>(slot + ks);
        }
    }
    template <int kJ>
    __device__ __forceinline__ void load_v(Fp4V<D>& f, uint32_t slot) const {
        constexpr int o = (2 * kJ + 1) * Tile::kBytes;
        lds_words<Fp4V<D>::VW, o>(slot + va, f.v[0]);
        lds_words<Fp4V<D>::VW, o>(slot + vb, f.v[1]);
        lds_words<Fp4V<D>::VW, o + 2 * Tile::kRow>(slot + va, f.v[2]);
        lds_words<Fp4V<D>::VW, o + 2 * Tile::kRow>(slot + vb, f.v[3]);
        uint32_t x[1];
        lds_words<1, o>(slot + vs, x);
        f.vs = x[0];
    }
};

// The (at most 8) (query, head) columns of one item.  E = 1: only one column
// (single queries without grouped heads), so that a lane's second one is left out.
template <int D, int E>
struct Fp4State {
    static constexpr int KS = D / 16;
    uint32_t qb[KS][2];       // Q^T: k-step kk holds dims c * D/4 + 4 kk + {0, 1 | 2, 3}
    float o[KS][4];           // O^T: m-tile mt holds dims g * D/8 + 2 mt + {0 | 1}
    float m[2], l[2], mul[2];
    int lim[2];               // first token the column may not see

    // S^T = K Q^T of one block (raw products).
    __device__ __forceinline__ void scores(const Fp4K<D>& f, float (&s)[4]) const {
        uint32_t sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) sc[i] = e4m3x2_to_f16x2(f.ks[i]);
#pragma unroll
        for (int w = 0; w < Fp4K<D>::KW; ++w) {
            uint32_t x[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // words 0, 1 belong to the lane's first group, 2, 3 to its second
                const uint32_t b = __byte_perm(sc[i], 0u, w < 2 ? 0x1010u : 0x3232u);
                e2m1x8_to_f16x2(f.k[i][w], x[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = hmul2_bits(x[i][j], b);
            }
            const uint32_t a0[4] = {x[0][0], x[1][0], x[0][1], x[1][1]};
            const uint32_t a1[4] = {x[0][2], x[1][2], x[0][3], x[1][3]};
            if (w == 0) mma_first(s, a0, qb[0][0], qb[0][1]);
            else Mma<__half>::run(s, a0, qb[2 * w][0], qb[2 * w][1]);
            Mma<__half>::run(s, a1, qb[2 * w + 1][0], qb[2 * w + 1][1]);
        }
    }

    // Tokens at and past the columns' limits (all of them when !ok) get -inf.
    __device__ __forceinline__ void mask(float (&s)[4], int base, bool ok, int ta) const {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (!ok || base + ta >= lim[e]) s[e] = -INFINITY;
            if (!ok || base + ta + 2 >= lim[e]) s[2 + e] = -INFINITY;
        }
    }

    // Softmax weights of NB blocks' raw scores against the running reference,
    // as the B operand of the second product (b[block][2]).  mul > 0.
    template <int NB>
    __device__ __forceinline__ void weights(const float (&s)[NB][4], uint32_t (&b)[NB][2]) {
        auto largest = [&](int e) {
            float mx = fmaxf(s[0][e], s[0][2 + e]);
#pragma unroll
            for (int j = 1; j < NB; ++j) mx = fmaxf(mx, fmaxf(s[j][e], s[j][2 + e]));
            return mx;
        };
        bool grow = false;
#pragma unroll
        for (int e = 0; e < E; ++e) grow |= largest(e) * mul[e] > m[e] + kLazyLog2;
        if (__any_sync(kAll, grow)) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float mx = largest(e);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, off));
                mx *= mul[e];
                if (!(mx > m[e] + kLazyLog2)) continue;
                const float al = fast_exp2(m[e] - mx);   // 0 while the column saw no token yet
                m[e] = mx;
                l[e] *= al;
#pragma unroll
                for (int mt = 0; mt < KS; ++mt) {
                    o[mt][e] *= al;
                    o[mt][2 + e] *= al;
                }
            }
        }
        // a column without a visible token yet keeps m = -inf; its weights are 2^(-inf - 0) = 0
        float r[E];
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                w[e] = fast_exp2(fmaf(s[j][e], mul[e], -r[e]));
                w[2 + e] = fast_exp2(fmaf(s[j][2 + e], mul[e], -r[e]));
                l[e] += w[e] + w[2 + e];
            }
            // rows 2c, 2c + 1 of the two 8 x 8 pieces are tokens 4c, 4c + 1 and 4c + 2, 4c + 3 (flipped alike)
            b[j][0] = movmatrix_trans(Elem<__half>::pack(w[0], w[1]));
            b[j][1] = movmatrix_trans(Elem<__half>::pack(w[2], w[3]));
        }
    }

    // O^T += V^T P^T of one block.  Unless `full`, tokens at and past nvalid
    // count as 0.
    __device__ __forceinline__ void accumulate(const Fp4V<D>& f, const uint32_t (&b)[2], bool full, int nvalid, int c,
                                               uint32_t flip) {
        uint32_t vs = f.vs;
        if (!full) {
            // rows past the end may hold anything, a NaN scale too: their scale becomes 0
            const int keep = min(4, max(0, nvalid - 4 * c));
            vs = keep == 4 ? vs : vs & ((1u << (8 * keep)) - 1u);
        }
        vs = __byte_perm(vs, 0u, flip);
        const uint32_t s01 = e4m3x2_to_f16x2(static_cast<uint16_t>(vs & 0xffffu));
        const uint32_t s23 = e4m3x2_to_f16x2(static_cast<uint16_t>(vs >> 16));
#pragma unroll
        for (int w = 0; w < Fp4V<D>::VW; ++w) {
            constexpr uint32_t kLow = 0x0f0f0f0fu;
            // byte b: (first, second token) of dim 8w + 2b (even) or 8w + 2b + 1 (odd)
            uint32_t e01[4], o01[4], e23[4], o23[4];
            e2m1x8_to_f16x2((f.v[0][w] & kLow) | ((f.v[1][w] << 4) & ~kLow), e01);
            e2m1x8_to_f16x2(((f.v[0][w] >> 4) & kLow) | (f.v[1][w] & ~kLow), o01);
            e2m1x8_to_f16x2((f.v[2][w] & kLow) | ((f.v[3][w] << 4) & ~kLow), e23);
            e2m1x8_to_f16x2(((f.v[2][w] >> 4) & kLow) | (f.v[3][w] & ~kLow), o23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a[4] = {hmul2_bits(e01[i], s01), hmul2_bits(o01[i], s01), hmul2_bits(e23[i], s23),
                                       hmul2_bits(o23[i], s23)};
                Mma<__half>::run(o[4 * w + i], a, b[0], b[1]);
            }
        }
    }
};

// A warp's ring of slots; a slot holds the (K tile, V tile) of a step's blocks.
// Four blocks a step with two slots and 12 warps per SM: against two blocks
// (three slots, 12 or 16 warps) 132 us to 136 and 131-143 at B=64 with 32
// heads, 169 to 175 us at eight contexts of 32K-128K; more warps, or two-block
// fetches for 16 warps, were slower (137-147 us).
template <int D>
struct Fp4Shape {
    static constexpr int kTile = Fp4Tile<D>::kBytes;
    static constexpr int kBlocks = 4;
    static constexpr int kSlot = 2 * kBlocks * kTile;
    static constexpr int kSlots = 2;
    static constexpr int kMinCtas = 3;
    static constexpr int kSmem = kFp4Warps * kSlots * kSlot;
};

// Persistent and warp-granular: a warp takes its first item by its own index
// and the following ones from the plan's counter, claimed one item ahead.  It
// fetches kSlots steps ahead of the step being computed and on into its next
// items.  Each step commits one group of copies (an empty one past the last
// item), so the oldest of kSlots groups is always the one being waited for.
// kCols: columns of an item, 1 or 8.  Rows with more columns are cut into
// chunks of 8, each of which reads the tiles again: against a 16-column kernel
// that widened each tile once (221 registers, 8 warps per SM), verify rows of
// 1-4 queries of 4 heads took 66 us instead of 73 and of 1-8 queries 97
// instead of 120; 32 heads per kv head 49 instead of 48.
template <typename T, int D, int kCols>
__global__ void __launch_bounds__(kFp4Warps * 32, Fp4Shape<D>::kMinCtas) decode_fp4_kernel(const DecodeParams p) {
    using Shape = Fp4Shape<D>;
    constexpr int NB = Shape::kBlocks;
    constexpr int E = kCols == 1 ? 1 : 2;
    constexpr int kTile = Shape::kTile;
    constexpr int kSlots = Shape::kSlots;
    constexpr int kQueue = 8;   // items fetched (in part) and not yet computed: at most kSlots + 1
    static_assert(kSlots + 1 < kQueue, "the item queue");
    struct Item {
        int b, h, part, n, qlen, qrow0, col0, nblk;
    };
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(16) Item all_queue[kFp4Warps][kQueue];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int G = p.group, H = p.num_kv_heads, C = p.col_chunks, P = p.partition_tokens;
    const int warps = gridDim.x * kFp4Warps;
    const uint32_t ring = smem_addr(smem_raw) + warp * kSlots * Shape::kSlot;
    Item* queue = all_queue[warp];
    // the work list (and, through it, the KV write) is complete; with
    // p.overlap the list was built before the prefill kernel that this one
    // runs beside, and the wait moves to the exit
    if (!p.overlap) pdl_wait();
    pdl_trigger();   // the merge may be scheduled; it waits for this grid
    const int total = *p.unit_count * H * C;

    // ---- fetch cursor ----------------------------------------------------
    uint32_t q_tail = 0, q_head = 0;
    const int32_t* f_bt = nullptr;
    // the item's head in block 0, plus this lane's 16 bytes: K, V, and the
    // tiles' last chunks (lanes 0 .. kTail - 1 of K, the next kTail lanes of V)
    constexpr int kFull = kTile / 16 / 32, kTail = kTile / 16 % 32;   // 16-byte chunks per lane, and left over
    const uint8_t *f_k = nullptr, *f_v = nullptr, *f_t = nullptr;
    const int t_off = lane < kTail ? 0 : kTile - 16 * kTail;          // where a lane's last chunk goes
    int f_nblk = 0, f_i = 0, ids = -1;
    const uint32_t block_bytes = static_cast<uint32_t>(H) * kTile;   // below 2^27: H <= 65535
    // The item after the cursor's is looked up ahead, one dependent load a
    // step, so that taking it finds everything in registers: its index
    // (claimed by lane 0), its unit, then its sequence's length and rows.
    int n_claim = blockIdx.x * kFp4Warps + warp, n_stage = 0;
    int n_w = 0, n_h = 0, n_col0 = 0, n_len = 0, n_row0 = 0, n_row1 = 0;
    uint32_t n_unit = 0;
    auto look_ahead = [&]() {
        if (n_stage == 0) {
            n_w = __shfl_sync(kAll, n_claim, 0);
            if (n_w < total) {
                const int ug = C == 1 ? n_w : n_w / C;
                const int u = ug / H;
                n_h = ug - u * H;
                n_col0 = (n_w - ug * C) * kCols;
                // (a plain load, like row_base below: the plan may have
                // been writing the list when this kernel started)
                n_unit = static_cast<uint32_t>(p.units[u]);
            }
            n_stage = 1;
        } else if (n_stage == 1) {
            if (n_w < total) {
                const int b = static_cast<int>(n_unit >> 16);
                n_len = __ldg(p.seq_lens + b);
                n_row0 = b;
                n_row1 = b + 1;
                if (p.cu_q_lens) {
                    n_row0 = __ldg(p.cu_q_lens + b);
                    n_row1 = __ldg(p.cu_q_lens + b + 1);
                }
            }
            n_stage = 2;
        }
    };
    auto next_item = [&]() {
        f_nblk = f_i = 0;
        for (;;) {
            while (n_stage < 2) look_ahead();
            if (n_w >= total) return;
            Item it;
            it.h = n_h;
            it.b = static_cast<int>(n_unit >> 16);
            it.part = static_cast<int>(n_unit & 0xffffu);
            it.n = n_len;
            it.qrow0 = n_row0;
            it.qlen = n_row1 - n_row0;
            it.col0 = n_col0;
            if (lane == 0) n_claim = warps + atomicAdd(p.work_counter, 1);
            n_stage = 0;
            // (the plan lists valid sequences only; a column chunk past the
            // row's last (query, head) pair has nothing to do)
            const bool ok = it.col0 < it.qlen * G && it.n >= it.qlen && it.n <= p.max_seq_len &&
                            it.n <= p.max_blocks * 16 && it.qlen >= 1 && it.qlen <= p.max_q && it.qrow0 >= 0 &&
                            it.qrow0 + it.qlen <= p.num_rows;
            const int tok0 = it.part * P;
            it.nblk = ok ? ((min(it.n, tok0 + P) + 15) >> 4) - (tok0 >> 4) : 0;
            if (it.nblk <= 0) continue;
            if (lane == 0) queue[q_tail % kQueue] = it;
            ++q_tail;
            f_bt = p.block_tables + static_cast<int64_t>(it.b) * p.max_blocks + (tok0 >> 4);
            f_nblk = it.nblk;
            f_k = static_cast<const uint8_t*>(p.k_pool) + static_cast<int64_t>(it.h) * kTile + 16 * lane;
            f_v = static_cast<const uint8_t*>(p.v_pool) + static_cast<int64_t>(it.h) * kTile + 16 * lane;
            f_t = lane < kTail ? f_k : f_v - 16 * kTail;
            return;
        }
    };
    // NB bits per pending step (newest lowest): its blocks' ids were inside the pool
    uint32_t loaded = 0;
    static_assert(NB * kSlots <= 32 && 32 % NB == 0, "the pending steps' bits, the id window");
    auto fetch_step = [&](uint32_t slot) {
        loaded <<= NB;
        if (f_i < f_nblk) {
            if ((f_i & 31) == 0) {   // the next 32 blocks' ids, one per lane
                ids = -1;
                if (f_i + lane < f_nblk) {
                    ids = __ldg(f_bt + f_i + lane);
                    if (ids < 0 || ids >= p.num_blocks) {
                        record_error(p.err, PA_DEVERR_BLOCK_ID_);   // its tokens contribute nothing
                        ids = -1;
                    }
                }
            }
            const uint32_t dst = slot + 16 * lane, dst_t = dst + t_off;
            static_for<NB>([&](auto j) {
                constexpr int o = 2 * j * kTile;
                const int id = __shfl_sync(kAll, ids, (f_i + j) & 31);
                if (id >= 0) {
                    const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(id)) * block_bytes;
                    const uint8_t *k = f_k + off, *v = f_v + off;
                    static_for<kFull>([&](auto i) {
                        cp_async16<o + 512 * i, 512 * i>(dst, k);
                        cp_async16<o + kTile + 512 * i, 512 * i>(dst, v);
                    });
                    if (lane < 2 * kTail) cp_async16<o + 512 * kFull, 512 * kFull>(dst_t, f_t + off);
                    loaded |= 1u << j;
                }
            });
            f_i += NB;
            if (f_i >= f_nblk) next_item();
            else if (n_stage < 2) look_ahead();
        }
        cp_async_commit();
    };
    next_item();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) fetch_step(ring + i * Shape::kSlot);

    // ---- compute: the fetched items in order --------------------------------
    uint32_t slot = ring;
    const uint32_t ring_end = ring + kSlots * Shape::kSlot;
    const Fp4Lane<D> at(lane);
    auto run_item = [&](const Item& it) {
        const int tok0 = it.part * P, tok1 = min(it.n, tok0 + P);
        const int ncols = min(kCols, it.qlen * G - it.col0);
        // query index of a column (one division, skipped for single queries)
        auto query_of = [&](int col) { return it.qlen == 1 ? 0 : col / G; };
        const int lim_min = min(tok1, it.n - it.qlen + 1 + query_of(it.col0));
        const bool parts = it.n > P;
        const int64_t prow = parts ? p.row_base[it.b] : 0;
        Fp4State<D, E> st;
        {
            // this lane's quarter of column g's query
            const bool ok = g < ncols;
            const int col = it.col0 + (ok ? g : 0);
            const int qi = query_of(col);
            const uint16_t* qq =
                static_cast<const uint16_t*>(p.q) +
                (static_cast<int64_t>(it.qrow0 + qi) * p.num_q_heads + it.h * G + (col - qi * G)) * D + c * (D / 4);
            uint32_t w[D / 8];
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint4 x = ok ? *reinterpret_cast<const uint4*>(qq + 8 * j) : make_uint4(0, 0, 0, 0);
                w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
            }
            // the score scale's sign goes into the query, so that the column's
            // multiplier is positive (the largest raw score is the largest)
            float undo = 1.f;
            const bool neg = p.scale_log2 < 0.f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                float mx = 0.f;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const float2 x = Elem<T>::to_float2(w[j]);
                    mx = fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
                mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
                // 2^(8 - e) for mx in [2^e, 2^(e+1)), the exponent kept in fp32's range
                const int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
                const int up = mx > 0.f && mx < INFINITY ? min(8 - e, 120) : 0;
                const float f = __uint_as_float((neg ? 0x80000000u : 0u) | static_cast<uint32_t>(127 + up) << 23);
                undo = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const float2 x = Elem<T>::to_float2(w[j]);
                    w[j] = Elem<__half>::pack(x.x * f, x.y * f);
                }
            } else if (neg) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) w[j] ^= 0x80008000u;
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                st.qb[kk][0] = w[2 * kk];
                st.qb[kk][1] = w[2 * kk + 1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // the accumulators' columns: 2c + e
                // (at least fp32's smallest normal, so that a masked -inf stays -inf)
                st.mul[e] = fmaxf(fabsf(p.scale_log2) * __shfl_sync(kAll, undo, (2 * c + e) * 4), 1.17549435e-38f);
                st.m[e] = -INFINITY;
                st.l[e] = 0.f;
                const int ce = 2 * c + e;
                st.lim[e] = ce < ncols ? min(tok1, it.n - it.qlen + 1 + query_of(it.col0 + ce)) : 0;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) st.o[mt][e] = st.o[mt][2 + e] = 0.f;
            }
        }
        int base = tok0;
        for (int i = 0; i < it.nblk; i += NB, base += 16 * NB) {
            cp_async_wait<kSlots - 1>();
            __syncwarp();   // every lane's copies of this step are in place
            const uint32_t have = loaded >> (NB * (kSlots - 1));   // (older steps' bits lie above)
            float sc[NB][4];
            uint32_t pb[NB][2];
            static_for<NB>([&](auto j) {
                Fp4K<D> f;
                at.template load_k<j>(f, slot);
                st.scores(f, sc[j]);
            });
            // every column sees all the step's tokens
            const bool full = base + 16 * NB <= lim_min && (have & ((1u << NB) - 1u)) == (1u << NB) - 1u;
            if (!full) {
#pragma unroll
                for (int j = 0; j < NB; ++j) st.mask(sc[j], base + 16 * j, (have >> j) & 1u, at.ta);
            }
            st.weights(sc, pb);
            static_for<NB>([&](auto j) {
                Fp4V<D> f;
                at.template load_v<j>(f, slot);
                st.accumulate(f, pb[j], full, (have >> j) & 1u ? tok1 - base - 16 * j : 0, c, at.flip);
            });
            __syncwarp();   // every lane has read the slot: refill it
            fetch_step(slot);
            slot = slot + Shape::kSlot == ring_end ? ring : slot + Shape::kSlot;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float lh = st.l[e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) lh += __shfl_xor_sync(kAll, lh, off);
            const int ce = 2 * c + e;
            if (ce >= ncols) continue;
            const int qi = query_of(it.col0 + ce);
            const int hq = it.h * G + (it.col0 + ce - qi * G);
            // this lane holds dims g * D/8 .. of the column, in order
            if (!parts) {
                const float inv = lh > 0.f ? p.v_scale / lh : 0.f;
                uint32_t* dst = reinterpret_cast<uint32_t*>(
                    static_cast<uint16_t*>(p.out) +
                    (static_cast<int64_t>(it.qrow0 + qi) * p.num_q_heads + hq) * D + g * (D / 8));
#pragma unroll
                for (int mt = 0; mt < D / 16; mt += 4)
                    *reinterpret_cast<uint4*>(dst + mt) =
                        make_uint4(Elem<T>::pack(st.o[mt][e] * inv, st.o[mt][2 + e] * inv),
                                   Elem<T>::pack(st.o[mt + 1][e] * inv, st.o[mt + 1][2 + e] * inv),
                                   Elem<T>::pack(st.o[mt + 2][e] * inv, st.o[mt + 2][2 + e] * inv),
                                   Elem<T>::pack(st.o[mt + 3][e] * inv, st.o[mt + 3][2 + e] * inv));
            } else {
                const int64_t pi = ((prow + qi) * p.num_q_heads + hq) * p.max_parts + it.part;
                if (g == 0) {
                    p.ws_m[pi] = st.m[e];
                    p.ws_l[pi] = lh;
                }
                float* a = p.ws_acc + pi * D + g * (D / 8);
#pragma unroll
                for (int mt = 0; mt < D / 16; mt += 2)
                    *reinterpret_cast<float4*>(a + 2 * mt) =
                        make_float4(st.o[mt][e] * p.v_scale, st.o[mt][2 + e] * p.v_scale,
                                    st.o[mt + 1][e] * p.v_scale, st.o[mt + 1][2 + e] * p.v_scale);
            }
        }
    };

    while (q_head != q_tail) {
        __syncwarp();
        const Item it = queue[q_head % kQueue];
        ++q_head;
        run_item(it);
    }
    cp_async_wait<0>();
    // beside a prefill kernel this grid completes only after it (what the
    // stream runs next is ordered after this grid alone)
    if (p.overlap) pdl_wait();
}

template <typename T, int D, int kCols>
cudaError_t launch_kernel(const DecodeParams& p, cudaStream_t s) {
    constexpr int smem = Fp4Shape<D>::kSmem;
    auto kern = decode_fp4_kernel<T, D, kCols>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    static const int ctas_per_sm = [&] {   // once per kernel variant (thread-safe)
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kFp4Warps * 32, smem) != cudaSuccess || n < 1) n = 1;
        return n;
    }();
    const long long items = static_cast<long long>(p.num_seqs) * p.max_parts * p.num_kv_heads * p.col_chunks;
    const long long want = (items + kFp4Warps - 1) / kFp4Warps;
    const int grid = static_cast<int>(
        std::max<long long>(1, std::min<long long>(want, static_cast<long long>(ctas_per_sm) * sm_count())));
    return launch_pdl(kern, dim3(grid), dim3(kFp4Warps * 32), smem, s, p);
}

// Chunks' blocks of a 4-bit cache widened into the 16-bit copy that the
// prefill kernel reads (code times group scale, exact in fp16 and in bf16; the
// pool scales are folded into the softmax scale and the epilogue).  Copy block
// u belongs to the last listed chunk k with chunk_base[k] <= u.
constexpr int kWidenFp4Threads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kWidenFp4Threads) widen_chunk_blocks_fp4_kernel(const Fp8Copy c,
                                                                                  const int32_t* __restrict__ seq_lens,
                                                                                  int max_blocks, int num_kv_heads) {
    using Tile = Fp4Tile<D>;
    constexpr int kUnroll = 4;
    // Runs of 8 dims, one 16-byte store each: a warp stores whole rows (runs of
    // a scale group, two stores each, made a step of four chunks and 60 rows
    // take 297 us instead of 292; eight runs in flight 293).
    constexpr int kRuns = D / 8;
    pdl_wait();   // the plan (no early trigger, as in the FP8 kernel)
    const int nchunks = c.hdr[0];
    const int used = min(c.hdr[1], c.cap_blocks);
    const int runs = num_kv_heads * 16 * kRuns;   // per block and pool
    const bool v = blockIdx.y;
    const uint8_t* codes = static_cast<const uint8_t*>(v ? c.v_codes : c.k_codes);
    T* out16 = static_cast<T*>(v ? c.v16 : c.k16);
    for (int u = blockIdx.x; u < used && nchunks > 0; u += gridDim.x) {
        int lo = 0, hi = nchunks - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (c.chunk_base[mid] <= u) lo = mid;
            else hi = mid - 1;
        }
        const int b = c.chunk_seq[lo];
        const int i = u - c.chunk_base[lo];
        if (i < 0 || i >= ((seq_lens[b] + 15) >> 4)) continue;
        const int src = c.src_tables[static_cast<int64_t>(b) * max_blocks + i];
        const bool ok = src >= 0 && src < c.src_num_blocks;   // else the attention kernel flags and masks it
        if (threadIdx.x == 0 && !v) c.table[static_cast<int64_t>(b) * max_blocks + i] = ok ? u : -1;
        if (!ok) continue;
        const uint8_t* blk = codes + static_cast<int64_t>(src) * num_kv_heads * Tile::kBytes;
        T* out = out16 + static_cast<int64_t>(u) * 16 * num_kv_heads * D;
        for (int x0 = threadIdx.x; x0 < runs; x0 += kUnroll * kWidenFp4Threads) {
            uint32_t raw[kUnroll];
            uint8_t sc[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                // source order: head, token, run
                const int x = min(x0 + k * kWidenFp4Threads, runs - 1);
                const int run = x % kRuns, t = x / kRuns & 15, h = x / kRuns >> 4;
                const uint8_t* tile = blk + static_cast<int64_t>(h) * Tile::kBytes;
                raw[k] = __ldcs(reinterpret_cast<const uint32_t*>(tile + t * Tile::kRow + 4 * run));
                sc[k] = tile[Tile::scale_off(v, t, run / 2)];
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int x = x0 + k * kWidenFp4Threads;
                if (x >= runs) break;
                const int run = x % kRuns, t = x / kRuns & 15, h = x / kRuns >> 4;
                uint32_t w[4];
                half_group_values(raw[k], sc[k], w);
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = Elem<__half>::to_float2(w[j]);
                        w[j] = Elem<T>::pack(f.x, f.y);
                    }
                }
                *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(t) * num_kv_heads + h) * D + 8 * run) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_d(const DecodeParams& p, cudaStream_t s) {
    return p.max_q * p.group > 1 ? launch_kernel<T, D, 8>(p, s) : launch_kernel<T, D, 1>(p, s);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeParams& p, int head_dim, int dtype, cudaStream_t s) {
    if (p.num_seqs == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    if (!p.overlap) e = launch_decode_plan(p, s, true);
    if (e != cudaSuccess) return e;
    if (dtype == 0)
        e = head_dim == 128 ? launch_d<__half, 128>(p, s) : launch_d<__half, 64>(p, s);
    else
        e = head_dim == 128 ? launch_d<__nv_bfloat16, 128>(p, s) : launch_d<__nv_bfloat16, 64>(p, s);
    if (e != cudaSuccess) return e;
    return launch_decode_reduce(p, head_dim, dtype, s);
}

cudaError_t launch_widen_fp4(const Fp8Copy& c, const int32_t* seq_lens, int max_blocks, int num_kv_heads, int head_dim,
                             int dtype, cudaStream_t s) {
    const dim3 grid(std::max(1, std::min(c.cap_blocks, 8 * sm_count())), 2);   // K and V
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, dim3(kWidenFp4Threads), 0, s, c, seq_lens, max_blocks, num_kv_heads);
    };
    if (dtype == 0)
        return head_dim == 128 ? go(widen_chunk_blocks_fp4_kernel<__half, 128>) : go(widen_chunk_blocks_fp4_kernel<__half, 64>);
    return head_dim == 128 ? go(widen_chunk_blocks_fp4_kernel<__nv_bfloat16, 128>)
                           : go(widen_chunk_blocks_fp4_kernel<__nv_bfloat16, 64>);
}

}  // namespace pa
