// Decode and verify attention over a 4-bit paged cache.
//
// out = softmax(scale q . k) v over a sequence's cached positions, with
// k = e2m1(code) * e4m3(group scale) * k_scale (V alike); pa_fp4.cuh has the
// format.  Work list, partitions, partials and their merge are those of the
// 16-bit decode kernel; the block step differs.
//
// One warp handles one (sequence partition, kv head) item and streams its
// (block, kv head) tiles, 9 D bytes each for K and for V.
//  * The tiles go from memory straight to registers, in the layout of the
//    tensor-core fragments, one block ahead of the block being computed: no
//    shared memory, no barriers.  For S^T = K Q^T a lane (g, c) = (lane / 4,
//    lane % 4) reads its quarter row of dims for two tokens (one 16-byte load
//    each at head_dim 128); the order of the dims in the contraction is free,
//    and Q^T is loaded in the same order.  For O^T = V^T P^T it reads 16 dims
//    (one scale group) of tokens 4c .. 4c + 3; two masks and shifts per word
//    pair the tokens of each dim, so that one conversion gives an fp16 pair of
//    consecutive tokens of one dim, which is what the fragment holds.
//  * Codes are widened to fp16 and multiplied by their group's scale (exact,
//    see group_values), then fed to mma.sync m16n8k16 (fp32 accumulate).  P is
//    fp16 (at most 2^8, 11 significant bits).  bf16 queries enter as fp16
//    times a power of two per column, chosen so that the column's largest
//    magnitude lies in [2^8, 2^9): every element above 2^-22 of it is exact.
//  * Softmax: a column's reference maximum moves only when some score passes
//    it by more than 2^8, so most blocks need one vote and no reduction.  P^T
//    reaches the second product's layout through movmatrix.
//
// Bound: HBM, 4.5 bits per cached value.  A tile pair is 18 D bytes (2304 at
// head_dim 128), 98 SM clocks at the measured copy rate over 152 SMs; a block
// step issues about 220 instructions per warp (64 conversions on the 16-lane
// pipe), 55 clocks per SM when four warps issue side by side.
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

// One block's tile pair as this lane holds it.
template <int D>
struct Fp4Frag {
    static constexpr int KW = D / 32;    // 32-bit words of K codes per token (a quarter row)
    static constexpr int VW = D / 64;    // 32-bit words of V codes per token
    uint32_t k[2][KW];                   // tokens ta, ta + 2
    uint32_t ks[2];                      // their scales (D / 64 bytes each)
    uint32_t v[4][VW];                   // tokens 4c .. 4c + 3, dims of this lane
    uint32_t vs;                         // their four scales
};

template <int D>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[D]) {
    if constexpr (D == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (D == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
}

template <int D>
__device__ __forceinline__ void load_frag(Fp4Frag<D>& f, const uint8_t* kt, const uint8_t* vt, int lane) {
    using Tile = Fp4Tile<D>;
    const int g = lane >> 2, c = lane & 3;
    const int ta = 4 * (g >> 1) + (g & 1);            // rows g and g + 8 of S^T
    const int vg = D == 128 ? g : g >> 1;             // scale group of this lane's V dims
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = ta + 2 * i;
        load_words(kt + t * Tile::kRow + c * (Tile::kRow / 4), f.k[i]);
        const uint8_t* s = kt + Tile::scale_off(false, t, c * (D / 64));
        if constexpr (D == 128) f.ks[i] = __ldg(reinterpret_cast<const uint16_t*>(s));
        else f.ks[i] = __ldg(s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) load_words(vt + (4 * c + i) * Tile::kRow + g * (Tile::kRow / 8), f.v[i]);
    f.vs = __ldg(reinterpret_cast<const uint32_t*>(vt + Tile::scale_off(true, 4 * c, vg)));
}

// NT tiles of 8 (query, head) columns of one item.
template <int D, int NT>
struct Fp4State {
    static constexpr int KS = D / 16;
    uint32_t qb[KS][NT][2];   // Q^T: k-step kk holds dims c * D/4 + 4 kk + {0, 1 | 2, 3}
    float o[KS][NT][4];       // O^T: m-tile mt holds dims g * D/8 + 2 mt + {0 | 1}
    float m[NT][2], l[NT][2], mul[NT][2];
    int lim[NT][2];           // first token the column may not see

    __device__ __forceinline__ void step(Fp4Frag<D>& f, int base, int nvalid, bool masked, int lane) {
        const int g = lane >> 2, c = lane & 3;
        const int ta = 4 * (g >> 1) + (g & 1);
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
        // S^T = K Q^T, two accumulation chains
        {
            uint32_t sc[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sc[i] = e4m3x2_to_f16x2(static_cast<uint16_t>(D == 128 ? f.ks[i] : f.ks[i] * 0x0101u));
#pragma unroll
            for (int w = 0; w < Fp4Frag<D>::KW; ++w) {
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
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    Mma<__half>::run(s[nt], a0, qb[2 * w][nt][0], qb[2 * w][nt][1]);
                    Mma<__half>::run(s2[nt], a1, qb[2 * w + 1][nt][0], qb[2 * w + 1][nt][1]);
                }
            }
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[nt][e] = (s[nt][e] + s2[nt][e]) * mul[nt][e];
                s[nt][2 + e] = (s[nt][2 + e] + s2[nt][2 + e]) * mul[nt][e];
                if (masked) {
                    if (base + ta >= lim[nt][e]) s[nt][e] = -INFINITY;
                    if (base + ta + 2 >= lim[nt][e]) s[nt][2 + e] = -INFINITY;
                }
                grow |= fmaxf(s[nt][e], s[nt][2 + e]) > m[nt][e] + kLazyLog2;
            }
        }
        if (__any_sync(kAll, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[nt][e], s[nt][2 + e]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, off));
                    if (!(mx > m[nt][e] + kLazyLog2)) continue;
                    const float al = fast_exp2(m[nt][e] - mx);   // 0 while the column saw no token yet
                    m[nt][e] = mx;
                    l[nt][e] *= al;
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt) {
                        o[mt][nt][e] *= al;
                        o[mt][nt][2 + e] *= al;
                    }
                }
            }
        }
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // a column without a visible token yet keeps m = -inf; its weights are 2^(-inf - 0) = 0
            const float r0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
            const float r1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
            const float p0 = fast_exp2(s[nt][0] - r0), p1 = fast_exp2(s[nt][1] - r1);
            const float p2 = fast_exp2(s[nt][2] - r0), p3 = fast_exp2(s[nt][3] - r1);
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            // rows 2c, 2c + 1 of the two 8 x 8 pieces are tokens 4c, 4c + 1 and 4c + 2, 4c + 3
            b0[nt] = movmatrix_trans(Elem<__half>::pack(p0, p1));
            b1[nt] = movmatrix_trans(Elem<__half>::pack(p2, p3));
        }
        uint32_t vs = f.vs;
        if (nvalid < 16) {
            // rows past the end may hold anything, a NaN scale too: their scale becomes 0
            const int keep = min(4, max(0, nvalid - 4 * c));
            vs = keep == 4 ? vs : vs & ((1u << (8 * keep)) - 1u);
        }
        const uint32_t s01 = e4m3x2_to_f16x2(static_cast<uint16_t>(vs & 0xffffu));
        const uint32_t s23 = e4m3x2_to_f16x2(static_cast<uint16_t>(vs >> 16));
#pragma unroll
        for (int w = 0; w < Fp4Frag<D>::VW; ++w) {
            constexpr uint32_t kLow = 0x0f0f0f0fu;
            // byte b: (first, second token) of dim 8w + 2b (even) or 8w + 2b + 1 (odd)
            uint32_t e01[4], o01[4], e23[4], o23[4];
            e2m1x8_to_f16x2((f.v[0][w] & kLow) | ((f.v[1][w] << 4) & ~kLow), e01);
            e2m1x8_to_f16x2(((f.v[0][w] >> 4) & kLow) | (f.v[1][w] & ~kLow), o01);
            e2m1x8_to_f16x2((f.v[2][w] & kLow) | ((f.v[3][w] << 4) & ~kLow), e23);
            e2m1x8_to_f16x2(((f.v[2][w] >> 4) & kLow) | (f.v[3][w] & ~kLow), o23);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t a[4] = {hmul2_bits(e01[b], s01), hmul2_bits(o01[b], s01), hmul2_bits(e23[b], s23),
                                       hmul2_bits(o23[b], s23)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) Mma<__half>::run(o[4 * w + b][nt], a, b0[nt], b1[nt]);
            }
        }
    }
};

// Persistent and warp-granular: a warp takes its first item by its own index
// and the following ones from the plan's counter, claimed one item ahead.
template <typename T, int D, int kMaxNT>
__global__ void __launch_bounds__(kFp4Warps * 32, kMaxNT == 1 ? 4 : 2) decode_fp4_kernel(const DecodeParams p) {
    using Tile = Fp4Tile<D>;
    constexpr int kCols = 8 * kMaxNT;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int G = p.group, H = p.num_kv_heads, C = p.col_chunks, P = p.partition_tokens;
    const int warps = gridDim.x * kFp4Warps;
    // the work list (and, through it, the KV write) is complete; with
    // p.overlap the list was built before the prefill kernel that this one
    // runs beside, and the wait moves to the exit
    if (!p.overlap) pdl_wait();
    pdl_trigger();   // the merge may be scheduled; it waits for this grid
    const int total = *p.unit_count * H * C;

    auto run_item = [&](auto nt_tag, int b, int h, int part, int n, int qlen, int64_t qrow0, int col0, int ncols) {
        constexpr int NT = decltype(nt_tag)::value;
        const int tok0 = part * P, tok1 = min(n, tok0 + P);
        const int blk0 = tok0 >> 4, nblk = ((tok1 + 15) >> 4) - blk0;
        const int lim_min = min(tok1, n - qlen + 1 + col0 / G);
        const int32_t* bt = p.block_tables + static_cast<int64_t>(b) * p.max_blocks + blk0;
        const uint8_t* kp = static_cast<const uint8_t*>(p.k_pool) + static_cast<int64_t>(h) * Tile::kBytes;
        const uint8_t* vp = static_cast<const uint8_t*>(p.v_pool) + static_cast<int64_t>(h) * Tile::kBytes;
        const int64_t block_bytes = static_cast<int64_t>(H) * Tile::kBytes;
        // ids of 32 blocks at a time, one per lane
        int ids = lane < nblk ? __ldg(bt + lane) : 0;
        auto block_id = [&](int i) {
            if ((i & 31) == 0 && i > 0) ids = i + lane < nblk ? __ldg(bt + i + lane) : 0;
            return __shfl_sync(kAll, ids, i & 31);
        };
        Fp4Frag<D> cur, nxt;
        bool cur_ok, nxt_ok = false;
        auto fetch = [&](Fp4Frag<D>& f, int i) {
            const int id = block_id(i);
            const bool ok = id >= 0 && id < p.num_blocks;
            if (ok) load_frag<D>(f, kp + id * block_bytes, vp + id * block_bytes, lane);
            else if (lane == 0) record_error(p.err, PA_DEVERR_BLOCK_ID_);
            return ok;
        };
        cur_ok = fetch(cur, 0);
        Fp4State<D, NT> st;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // this lane's quarter of column nt * 8 + g's query
            const int cl = nt * 8 + g;
            const bool ok = cl < ncols;
            const int col = col0 + (ok ? cl : 0);
            const int qi = col / G;
            const uint16_t* qq = static_cast<const uint16_t*>(p.q) +
                                 ((qrow0 + qi) * p.num_q_heads + h * G + (col - qi * G)) * D + c * (D / 4);
            uint32_t w[D / 8];
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint4 x = ok ? *reinterpret_cast<const uint4*>(qq + 8 * j) : make_uint4(0, 0, 0, 0);
                w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
            }
            float undo = 1.f;
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
                const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                undo = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const float2 x = Elem<T>::to_float2(w[j]);
                    w[j] = Elem<__half>::pack(x.x * f, x.y * f);
                }
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                st.qb[kk][nt][0] = w[2 * kk];
                st.qb[kk][nt][1] = w[2 * kk + 1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // the accumulators' columns: 2c + e
                st.mul[nt][e] = p.scale_log2 * __shfl_sync(kAll, undo, (2 * c + e) * 4);
                st.m[nt][e] = -INFINITY;
                st.l[nt][e] = 0.f;
                const int ce = nt * 8 + 2 * c + e;
                st.lim[nt][e] = ce < ncols ? min(tok1, n - qlen + 1 + (col0 + ce) / G) : 0;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) st.o[mt][nt][e] = st.o[mt][nt][2 + e] = 0.f;
            }
        }
        for (int i = 0; i < nblk; ++i) {
            if (i + 1 < nblk) nxt_ok = fetch(nxt, i + 1);
            if (cur_ok) {
                const int base = tok0 + 16 * i;
                st.step(cur, base, min(16, tok1 - base), base + 16 > lim_min, lane);
            }
            cur = nxt;
            cur_ok = nxt_ok;
        }
        const bool parts = n > P;
        const int64_t prow = parts ? p.row_base[b] : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float lh = st.l[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) lh += __shfl_xor_sync(kAll, lh, off);
                const int ce = nt * 8 + 2 * c + e;
                if (ce >= ncols) continue;
                const int qi = (col0 + ce) / G;
                const int hq = h * G + (col0 + ce - qi * G);
                // this lane holds dims g * D/8 .. of the column, in order
                if (!parts) {
                    const float inv = lh > 0.f ? p.v_scale / lh : 0.f;
                    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                                ((qrow0 + qi) * p.num_q_heads + hq) * D + g * (D / 8));
#pragma unroll
                    for (int mt = 0; mt < D / 16; mt += 4)
                        *reinterpret_cast<uint4*>(dst + mt) =
                            make_uint4(Elem<T>::pack(st.o[mt][nt][e] * inv, st.o[mt][nt][2 + e] * inv),
                                       Elem<T>::pack(st.o[mt + 1][nt][e] * inv, st.o[mt + 1][nt][2 + e] * inv),
                                       Elem<T>::pack(st.o[mt + 2][nt][e] * inv, st.o[mt + 2][nt][2 + e] * inv),
                                       Elem<T>::pack(st.o[mt + 3][nt][e] * inv, st.o[mt + 3][nt][2 + e] * inv));
                } else {
                    const int64_t pi = ((prow + qi) * p.num_q_heads + hq) * p.max_parts + part;
                    if (g == 0) {
                        p.ws_m[pi] = st.m[nt][e];
                        p.ws_l[pi] = lh;
                    }
                    float* a = p.ws_acc + pi * D + g * (D / 8);
#pragma unroll
                    for (int mt = 0; mt < D / 16; mt += 2)
                        *reinterpret_cast<float4*>(a + 2 * mt) =
                            make_float4(st.o[mt][nt][e] * p.v_scale, st.o[mt][nt][2 + e] * p.v_scale,
                                        st.o[mt + 1][nt][e] * p.v_scale, st.o[mt + 1][nt][2 + e] * p.v_scale);
                }
            }
        }
    };

    int w = blockIdx.x * kFp4Warps + (threadIdx.x >> 5);
    while (w < total) {
        int claim = 0;
        if (lane == 0) claim = atomicAdd(p.work_counter, 1);
        const int ug = w / C;
        const uint32_t unit = static_cast<uint32_t>(p.units[ug / H]);
        const int h = ug % H;
        const int b = static_cast<int>(unit >> 16), part = static_cast<int>(unit & 0xffffu);
        int qlen = 1;
        int64_t qrow0 = b;
        if (p.cu_q_lens) {
            qrow0 = p.cu_q_lens[b];
            qlen = p.cu_q_lens[b + 1] - static_cast<int>(qrow0);
        }
        const int n = p.seq_lens[b];
        const int col0 = (w % C) * kCols;
        const int ncols = min(kCols, qlen * G - col0);
        // (the plan lists valid sequences only; a column chunk past the row's last pair has nothing to do)
        if (ncols > 0 && n >= qlen && n <= p.max_seq_len && n <= p.max_blocks * 16 && qlen >= 1 && qlen <= p.max_q &&
            qrow0 >= 0 && qrow0 + qlen <= p.num_rows) {
            if (kMaxNT == 1 || ncols <= 8)
                run_item(std::integral_constant<int, 1>{}, b, h, part, n, qlen, qrow0, col0, ncols);
            else
                run_item(std::integral_constant<int, kMaxNT>{}, b, h, part, n, qlen, qrow0, col0, ncols);
        }
        w = warps + __shfl_sync(kAll, claim, 0);
    }
    // beside a prefill kernel this grid completes only after it (what the
    // stream runs next is ordered after this grid alone)
    if (p.overlap) pdl_wait();
}

template <typename T, int D, int kMaxNT>
cudaError_t launch_kernel(const DecodeParams& p, cudaStream_t s) {
    auto kern = decode_fp4_kernel<T, D, kMaxNT>;
    static const int ctas_per_sm = [&] {   // once per kernel variant (thread-safe)
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kFp4Warps * 32, 0) != cudaSuccess || n < 1) n = 1;
        return n;
    }();
    const long long items = static_cast<long long>(p.num_seqs) * p.max_parts * p.num_kv_heads * p.col_chunks;
    const long long want = (items + kFp4Warps - 1) / kFp4Warps;
    const int grid = static_cast<int>(
        std::max<long long>(1, std::min<long long>(want, static_cast<long long>(ctas_per_sm) * sm_count())));
    return launch_pdl(kern, dim3(grid), dim3(kFp4Warps * 32), 0, s, p);
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
    const int nchunks = c.hdr[0];
    const int used = min(c.hdr[1], c.cap_blocks);
    const int groups = num_kv_heads * 16 * Tile::kGroups;    // groups per block and pool
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
        if (threadIdx.x == 0) c.table[static_cast<int64_t>(b) * max_blocks + i] = ok ? u : -1;
        if (!ok) continue;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint8_t* blk = static_cast<const uint8_t*>(v ? c.v_codes : c.k_codes) +
                                 static_cast<int64_t>(src) * num_kv_heads * Tile::kBytes;
            T* out = static_cast<T*>(v ? c.v16 : c.k16) + static_cast<int64_t>(u) * 16 * num_kv_heads * D;
            for (int x = threadIdx.x; x < groups; x += kWidenFp4Threads) {
                // source order: head, token, group
                const int grp = x % Tile::kGroups, row = x / Tile::kGroups;
                const int h = row >> 4, t = row & 15;
                const uint8_t* tile = blk + static_cast<int64_t>(h) * Tile::kBytes;
                const uint2 codes = *reinterpret_cast<const uint2*>(tile + t * Tile::kRow + 8 * grp);
                uint32_t w[8];
                group_values(codes.x, codes.y, tile[Tile::scale_off(v, t, grp)], w);
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = Elem<__half>::to_float2(w[j]);
                        w[j] = Elem<T>::pack(f.x, f.y);
                    }
                }
                uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<int64_t>(t) * num_kv_heads + h) * D + 16 * grp);
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_d(const DecodeParams& p, cudaStream_t s) {
    return p.max_q * p.group > 8 ? launch_kernel<T, D, 2>(p, s) : launch_kernel<T, D, 1>(p, s);
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
    const int grid = std::max(1, std::min(c.cap_blocks, 8 * sm_count()));
    auto go = [&](auto kern) { kern<<<grid, kWidenFp4Threads, 0, s>>>(c, seq_lens, max_blocks, num_kv_heads); };
    if (dtype == 0) {
        if (head_dim == 128) go(widen_chunk_blocks_fp4_kernel<__half, 128>);
        else go(widen_chunk_blocks_fp4_kernel<__half, 64>);
    } else {
        if (head_dim == 128) go(widen_chunk_blocks_fp4_kernel<__nv_bfloat16, 128>);
        else go(widen_chunk_blocks_fp4_kernel<__nv_bfloat16, 64>);
    }
    return cudaGetLastError();
}

}  // namespace pa
