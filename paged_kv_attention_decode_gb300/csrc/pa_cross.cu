// Cross attention of short rows (decoder steps, beams) over an encoder's states
// in the paged cache.
//
// Sequence b has n encoder states (keys) and c query rows, and every row sees
// every state: out[r, h] = sum_t softmax_t(scale q[r, h] . k_t) v_t, t < n.  The
// beams of one request are rows of one sequence.  Rows and query heads of a KV
// head together are columns of two products, S^T = K Q^T and O^T += V^T P^T
// (mma.sync m16n8k16: 16 states, one block, are the M dimension and 8 or 16 columns
// the N; with so few columns the work is bound by the states' bytes).  The states
// are read once for 16 columns; with more, every 16 are another CTA's, next to one
// another in the grid: 64 requests over 512 to 4096 states, 32/8 heads, 4 rows (16
// columns) 96 us, 8 rows 125; 32 requests of 8 rows, 64/1 heads (512 columns) 128,
// by the products.  Longer chunks take the tcgen05 kernel.
//
// One launch, no plan and no second kernel: a CTA, or a cluster of `splits` CTAs,
// takes one (sequence, KV head, chunk of columns); its warps take the blocks in
// turn, each with its own ring of TMA tiles and its own running maximum, sum and
// accumulator.  The warps of a CTA join theirs in shared memory, the CTAs of a
// cluster through distributed shared memory, each CTA writing its share of the
// output.  Measured: 128 rows over 128 to 2048 states, 32/32 heads of 128, fp16, 350
// us (7.1 TB/s of states, at the copy rate and above); 64 requests of 4 beams over
// 512 to 4096 states, 32/8 heads, bf16, 95 us (6.4 TB/s, 0.94 of the copy rate); 1
// request of 4 beams, 1200 states, 12 heads of 64, 5.3 us (launch, four dependent
// loads, a step and a half a warp, the join).
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kMaxSplits = 8;         // CTAs of a cluster (the portable limit)
// Sequences that a CTA orders by length, one a thread (4 rows over 512 to 4096 states,
// 32/8 heads: 128 sequences 1.034 of the bytes' time, in order; 129, as they come, 1.049).
constexpr int kSortMax = 128;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLazyRescaleLog2 = 8.f;   // a column's reference maximum moves only when it has grown by this much

// kWarps: 8, one CTA an SM, for as few items as there are SMs; else 4.
template <int D, int NT, int kWarps>
struct CrossShape {
    static constexpr int kCols = 8 * NT;
    static constexpr int kTileBytes = 16 * D * 2;
    // blocks of a step: 8 KB of K and V either way, so that a step's latency and its
    // reductions are spent on as many bytes
    static constexpr int kBlocks = 128 / D;
    static constexpr int kStageBytes = 2 * kBlocks * kTileBytes;   // the K tiles, then the V tiles
    static constexpr int kMinCtas = kWarps == 8 ? 1 : NT > 1 ? 2 : 3;   // an SM holds, by registers
    static constexpr int kStages = NT > 1 ? 3 : 2;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    // the join: one fp32 accumulator [column][D] per warp, over the rings
    static constexpr int kPitch = D + 4;
    static constexpr int kAccBytes = kCols * kPitch * 4;
    static_assert(kWarps * kAccBytes <= kRingBytes, "the accumulators are joined where the rings were");
    static constexpr int kSmemBytes = kRingBytes + 1024;
};

// One warp's columns: the fragments of S^T and O^T share column ownership (lane
// l: columns 8 nt + 2 (l % 4) + {0, 1}), so rescaling moves no data.
template <typename T, int D, int NT>
struct CrossState {
    static constexpr int KS = D / 16;
    uint32_t qb[KS][NT][2];   // Q^T as the B operand
    float o[KS][NT][4];       // O^T
    float m[NT][2], l[NT][2];

    // kBlocks tiles of 16 states, of which the first valid[b] are the sequence's.
    static constexpr int NB = 128 / D, kTile = 16 * D * 2;
    __device__ __forceinline__ void step(uint8_t* stage, uint32_t valid, int lane, float scale_log2) {
        const uint32_t ka = smem_addr(stage), va = ka + NB * kTile;
        float c[NB][NT][4];
        {
            const int tok = (lane & 7) + ((lane >> 3) & 1) * 8, dsub = ((lane >> 4) & 1) * 8;
            float c2[NB][NT][4];   // two chains: even and odd k-steps
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[b][nt][e] = c2[b][nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t a[4];
                    ldsm_x4(ka + b * kTile + tile_off<D>(tok, kk * 16 + dsub), a[0], a[1], a[2], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) Mma<T>::run(kk & 1 ? c2[b][nt] : c[b][nt], a, qb[kk][nt][0], qb[kk][nt][1]);
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[b][nt][e] = (c[b][nt][e] + c2[b][nt][e]) * scale_log2;
        }
        const bool full = valid == (NB == 2 ? 0x1010u : 0x10u);
        if (!full) {
            const int r0 = lane >> 2;   // this lane's states: r0 and r0 + 8
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (r0 + (e >> 1) * 8 >= static_cast<int>(valid >> (8 * b) & 0xffu)) c[b][nt][e] = -INFINITY;
        }
        float mx[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(c[0][nt][e], c[0][nt][2 + e]);
                if constexpr (NB == 2) x = fmaxf(x, fmaxf(c[1][nt][e], c[1][nt][2 + e]));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
                mx[nt][e] = x;
                grow |= x > m[nt][e] + kLazyRescaleLog2;
            }
        }
        if (__any_sync(kFull, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!(mx[nt][e] > m[nt][e] + kLazyRescaleLog2)) continue;
                    const float al = fast_exp2(m[nt][e] - mx[nt][e]);   // (0 at first: m = -inf)
                    m[nt][e] = mx[nt][e];
                    l[nt][e] *= al;
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt) {
                        o[mt][nt][e] *= al;
                        o[mt][nt][2 + e] *= al;
                    }
                }
        }
        // P, rounded to T for the product with V (weights of 0 to 2^8), its sum kept in
        // fp32: matrix operands have 16 bits, and this rounding weighs as much as the
        // output's own (both together 1.4 times that alone: against 64 bits 2.3e-3 of
        // the norm in bf16, 2.9e-4 in fp16)
        uint32_t b0[NB][NT], b1[NB][NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // (a column whose scores are all -inf, or NaN, has no reference yet)
            const float mu0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], mu1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float p0 = fast_exp2(c[b][nt][0] - mu0), p1 = fast_exp2(c[b][nt][1] - mu1);
                const float p2 = fast_exp2(c[b][nt][2] - mu0), p3 = fast_exp2(c[b][nt][3] - mu1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                // the B operand wants P[state 2 (l % 4) + e (+ 8)][column l / 4]
                const uint32_t lo = Elem<T>::pack(p0, p1), hi = Elem<T>::pack(p2, p3);
                const int src = ((lane & 3) << 3) + (lane >> 3);
                const uint32_t x0 = __shfl_sync(kFull, lo, src), x1 = __shfl_sync(kFull, lo, src + 4);
                const uint32_t y0 = __shfl_sync(kFull, hi, src), y1 = __shfl_sync(kFull, hi, src + 4);
                const uint32_t sel = ((lane >> 2) & 1) ? 0x7632u : 0x5410u;
                b0[b][nt] = __byte_perm(x0, x1, sel);
                b1[b][nt] = __byte_perm(y0, y1, sel);
            }
        }
        if (!full) {
            // rows behind the last state (and tiles not loaded) may hold anything:
            // 0 * NaN must not reach O
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int v = static_cast<int>(valid >> (8 * b) & 0xffu), n16 = (16 - v) * 8;
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    uint4* z = reinterpret_cast<uint4*>(stage + (NB + b) * kTile + h * TileGeom<D>::kHalfBytes + v * 128);
                    for (int i = lane; i < n16; i += 32) z[i] = make_uint4(0, 0, 0, 0);
                }
            }
            // (these stores come before the copy that refills the slot; a step with a
            // block outside the pool need not be the warp's last)
            fence_proxy_async_smem();
            __syncwarp();
        }
        const int tok = (lane & 7) + ((lane >> 4) & 1) * 8, dsub = ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                uint32_t a[4];
                ldsm_x4_t(va + b * kTile + tile_off<D>(tok, mt * 16 + dsub), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) Mma<T>::run(o[mt][nt], a, b0[b][nt], b1[b][nt]);
            }
        }
    }
};

template <typename T, int D, int NT, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, CrossShape<D, NT, kWarps>::kMinCtas)
    cross_step_kernel(const CrossParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using Sh = CrossShape<D, NT, kWarps>;
    constexpr int kStages = Sh::kStages;
    constexpr int kCols = Sh::kCols;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ __align__(16) int s_len[kWarps == 4 ? kSortMax : 4];
    __shared__ int s_seq;
    __shared__ uint32_t s_valid[kWarps][kStages];   // states of a stage's tiles, a byte each
    __shared__ float s_m[kWarps][kCols];   // the warps' maxima, then [0]: the CTA's
    __shared__ float s_l[kWarps][kCols];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    // (the same offset in every CTA of the cluster: the accumulators are read across it)
    uint8_t* smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
    uint8_t* ring = smem + warp * kStages * Sh::kStageBytes;
    uint64_t* bar = bars[warp];
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&bar[s], 1);
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    __syncwarp();

    const int S = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int G = p.group;
    int item = static_cast<int>(blockIdx.x) / S;
    const int chunk = item % p.col_chunks;
    item /= p.col_chunks;
    const int g = item % p.num_kv_heads;
    int b = item / p.num_kv_heads;
    if (!p.overlap) pdl_wait();
    if (kWarps == 4 && p.longest_first) {
        // the b-th longest sequence: the CTAs that start last are the short ones
        // (negative lengths, which are refused below, rank before the threads without one)
        const int mine = tid < p.num_seqs ? max(p.seq_lens[tid], -1) : -2;
        s_len[tid] = mine;
        __syncthreads();
        int longer = 0;
#pragma unroll 4
        for (int i = 0; i < p.num_seqs; i += 4) {   // (behind the last one: shorter than any)
            const int4 o = *reinterpret_cast<const int4*>(s_len + i);
            longer += o.x > mine || (o.x == mine && i < tid);
            longer += o.y > mine || (o.y == mine && i + 1 < tid);
            longer += o.z > mine || (o.z == mine && i + 2 < tid);
            longer += o.w > mine || (o.w == mine && i + 3 < tid);
        }
        if (tid < p.num_seqs && longer == b) s_seq = tid;
        __syncthreads();
        b = s_seq;
    }

    // The length, the rows and this warp's first block ids are asked for together
    // (entries of the sequence's table row, used only if the length reaches them).
    constexpr int NB = Sh::kBlocks;
    const int first = rank * kWarps + warp, stride = S * kWarps;   // this warp's steps: first, first + stride, ...
    const int32_t* table = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    int n = p.seq_lens[b], ids[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t blk = (static_cast<int64_t>(first) + static_cast<int64_t>(lane) * stride) * NB + i;
        ids[i] = blk < p.max_blocks ? table[blk] : 0;
    }
    int row0 = b * p.q_per_seq, qlen = p.q_per_seq;
    if (p.cu_q_lens) {
        row0 = p.cu_q_lens[b];
        qlen = p.cu_q_lens[b + 1] - row0;
    }
    const int col0 = chunk * kCols;
    const int ncols = min(kCols, qlen * G - col0);
    const bool rows_ok = qlen >= 0 && row0 >= 0 && row0 <= p.num_rows - qlen;
    // none of the chunk's rows is here: longer chunks are another kernel's
    // (the same for the whole cluster)
    if (!rows_ok || qlen > p.max_q || ncols <= 0) {
        const bool theirs = qlen > PA_VERIFY_MAX_Q_ && p.chunks_follow;
        if ((!rows_ok || qlen > p.max_q) && !theirs && g == 0 && chunk == 0 && rank == 0 && tid == 0)
            record_error(p.err, PA_DEVERR_SEQ_LEN_);
        if (p.overlap) pdl_wait();
        return;
    }
    if (n < 0 || n > p.max_len || n > p.max_blocks * 16) {   // rows of zeros, as for no states
        if (g == 0 && chunk == 0 && rank == 0 && tid == 0) record_error(p.err, PA_DEVERR_SEQ_LEN_);
        n = 0;
    }
    const int nblk = (n + 15) >> 4;

    const int steps = (nblk + NB - 1) / NB;
    const int count = steps > first ? (steps - first + stride - 1) / stride : 0;
    int at = 0, issued = 0, next = 0;   // steps looked at and issued, the ring's next slot
    auto fetch = [&]() {    // the next step with a block in the pool (others contribute nothing)
        while (at < count) {
            if ((at & 31) == 0 && at > 0) {
                const int blk = (first + (at + lane) * stride) * NB;
#pragma unroll
                for (int i = 0; i < NB; ++i) ids[i] = at + lane < count && blk + i < nblk ? table[blk + i] : 0;
            }
            const int blk = (first + at * stride) * NB;
            uint32_t valid = 0;
            int id[NB], live = 0;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                id[i] = __shfl_sync(kFull, ids[i], at & 31);
                if (blk + i >= nblk) continue;
                if (id[i] < 0 || id[i] >= p.num_blocks) {
                    if (lane == 0) record_error(p.err, PA_DEVERR_BLOCK_ID_);
                    continue;
                }
                valid |= static_cast<uint32_t>(min(16, n - (blk + i) * 16)) << (8 * i);
                ++live;
            }
            ++at;
            if (live == 0) continue;
            if (lane == 0) {
                const int slot = next;
                uint8_t* dst = ring + slot * Sh::kStageBytes;
                s_valid[warp][slot] = valid;
                mbar_arrive_expect_tx(&bar[slot], live * 2 * Sh::kTileBytes);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (!(valid >> (8 * i) & 0xffu)) continue;
                    tma_load_4d(dst + i * Sh::kTileBytes, &kmap, &bar[slot], 0, id[i] * 16, 0, g);
                    tma_load_4d(dst + (NB + i) * Sh::kTileBytes, &vmap, &bar[slot], 0, id[i] * 16, 0, g);
                }
            }
            ++issued;
            next = next + 1 < kStages ? next + 1 : 0;
            return;
        }
    };
    for (int s = 0; s < kStages; ++s) fetch();

    CrossState<T, D, NT> st;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int cl = nt * 8 + (lane >> 2);
        const bool live = cl < ncols;
        const int c = col0 + (live ? cl : 0);
        const int qi = c / G, h = c - qi * G;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                            (static_cast<int64_t>(row0 + qi) * p.num_q_heads + g * G + h) * D + 2 * (lane & 3);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            st.qb[kk][nt][0] = live ? *reinterpret_cast<const uint32_t*>(q + kk * 16) : 0u;
            st.qb[kk][nt][1] = live ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 8) : 0u;
        }
        st.m[nt][0] = st.m[nt][1] = -INFINITY;
        st.l[nt][0] = st.l[nt][1] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[mt][nt][e] = 0.f;

    int done = 0, slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto pass = [&]() {
        ++done;
        if (++slot == kStages) {
            slot = 0;
            phase ^= 1u;
        }
    };
    while (done < issued) {
        ok = __all_sync(kFull, mbar_wait(&bar[slot], phase));
        if (!ok) break;
        st.step(ring + slot * Sh::kStageBytes, s_valid[warp][slot], lane, p.scale_log2);
        pass();
        __syncwarp();
        fetch();
    }
    if (!ok) {
        // give up: the copies still in flight first (another bounded wait each)
        if (lane == 0) {
            record_error(p.err, PA_DEVERR_TIMEOUT_);
            for (; done < issued; pass()) (void)mbar_wait(&bar[slot], phase);
        }
        __syncwarp();
    }

    // the CTA's warps: every accumulator relative to the CTA's maximum, summed in warp order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = st.l[nt][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
            st.l[nt][e] = l;
            if (lane < 4) s_m[warp][nt * 8 + 2 * lane + e] = st.m[nt][e];
        }
    __syncthreads();   // (and every ring is read)
    float* acc = reinterpret_cast<float*>(smem);
    float mc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * (lane & 3) + e;
            float m = s_m[0][col];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_m[w][col]);
            mc[nt][e] = m;
            const float f = st.m[nt][e] == -INFINITY ? 0.f : fast_exp2(st.m[nt][e] - m);
            if (lane < 4) s_l[warp][col] = st.l[nt][e] * f;
            float* dst = acc + warp * (Sh::kAccBytes / 4) + col * Sh::kPitch + (lane >> 2);
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                dst[mt * 16] = st.o[mt][nt][e] * f;
                dst[mt * 16 + 8] = st.o[mt][nt][2 + e] * f;
            }
        }
    __syncthreads();
    if (warp == 0 && lane < 4) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * lane + e;
                s_m[0][col] = mc[nt][e];
                float l = s_l[0][col];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) l += s_l[w][col];
                s_l[0][col] = l;
            }
    }
    for (int i = tid; i < ncols * (D / 4); i += kWarps * 32) {
        float4* x = reinterpret_cast<float4*>(acc + (i / (D / 4)) * Sh::kPitch) + i % (D / 4);
        float4 sum = *x;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 y = x[w * (Sh::kAccBytes / 16)];
            sum.x += y.x; sum.y += y.y; sum.z += y.z; sum.w += y.w;
        }
        *x = sum;
    }
    // the cluster's CTAs: each joins a share of the columns' 8-dim pieces
    if (S > 1) cluster_sync();
    else __syncthreads();
    const uint32_t a_acc = smem_addr(acc), a_m = smem_addr(&s_m[0][0]), a_l = smem_addr(&s_l[0][0]);
    for (int i = rank * kWarps * 32 + tid; i < ncols * (D / 8); i += S * kWarps * 32) {
        const int col = i / (D / 8), piece = i % (D / 8);
        const uint32_t off = static_cast<uint32_t>((col * Sh::kPitch + piece * 8) * 4);
        float m = -INFINITY;
        for (int r = 0; r < S; ++r) m = fmaxf(m, ld_cluster(map_rank(a_m + col * 4, r)));
        float l = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < S; ++r) {
            const float mr = ld_cluster(map_rank(a_m + col * 4, r));
            const float f = mr == -INFINITY ? 0.f : fast_exp2(mr - m);
            const uint32_t base = map_rank(a_acc + off, r);
            const float4 u = ld_cluster4(base), v = ld_cluster4(base + 16);
            l += f * ld_cluster(map_rank(a_l + col * 4, r));
            x[0] += f * u.x; x[1] += f * u.y; x[2] += f * u.z; x[3] += f * u.w;
            x[4] += f * v.x; x[5] += f * v.y; x[6] += f * v.z; x[7] += f * v.w;
        }
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // (a NaN stays)
        const int c = col0 + col, qi = c / G, h = c - qi * G;
        uint4 o;
        o.x = Elem<T>::pack(x[0] * inv, x[1] * inv);
        o.y = Elem<T>::pack(x[2] * inv, x[3] * inv);
        o.z = Elem<T>::pack(x[4] * inv, x[5] * inv);
        o.w = Elem<T>::pack(x[6] * inv, x[7] * inv);
        reinterpret_cast<uint4*>(static_cast<T*>(p.out) +
                                 (static_cast<int64_t>(row0 + qi) * p.num_q_heads + g * G + h) * D)[piece] = o;
    }
    if (S > 1) cluster_sync();   // no CTA leaves while its accumulators are read
    if (p.overlap) pdl_wait();
}

template <typename T, int D, int NT, int kWarps>
cudaError_t launch_t(const CrossParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int splits,
                     cudaStream_t s) {
    constexpr int smem = CrossShape<D, NT, kWarps>::kSmemBytes;
    auto kern = cross_step_kernel<T, D, NT, kWarps>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * p.num_kv_heads * p.col_chunks * splits);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, kmap, vmap);
}

__global__ void __launch_bounds__(256) uniform_rows_kernel(int32_t* cu, int num_seqs, int per) {
    pdl_trigger();
    pdl_wait();
    for (int i = blockIdx.x * 256 + threadIdx.x; i <= num_seqs; i += gridDim.x * 256) cu[i] = i * per;
}

}  // namespace

cudaError_t launch_uniform_rows(int32_t* cu, int num_seqs, int per, cudaStream_t s) {
    return launch_pdl(uniform_rows_kernel, dim3(std::min(num_seqs / 256 + 1, 64)), dim3(256), 0, s, cu, num_seqs, per);
}

cudaError_t launch_cross(CrossParams p, const CUtensorMap& kmap, const CUtensorMap& vmap, int head_dim, int dtype,
                         cudaStream_t s) {
    // An SM needs 8 warps to keep up with its share of the memory: two or three CTAs
    // of 4 where there are more items than SMs, else one CTA of 8, and for still
    // fewer items a cluster of 2, 4 or 8 of these, while all run at once (a cluster
    // lies within a GPC: 32 clusters of 4 do, 16 of 8 do not) and every warp still
    // has a block or two.  1000 to 2000 states, 32/8 heads of 128, 4 rows, us with
    // 1, 2, 4, 8 CTAs of 8 warps: 16 items 14.9, 11.3, 9.5, 17.3; 32 items 15.2,
    // 12.4, 11.8, 27.7; 64 items 18.3, 15.0, 22.2, 46.3; 128 items 22.5, 28.9, 41.0,
    // 82.9 (one of 4 warps: 29.0); 192 items 36.6 (one of 4 warps: 33.3).
    const long long items = static_cast<long long>(p.num_seqs) * p.num_kv_heads * p.col_chunks;
    const int blocks = p.max_len / 16 + (p.max_len % 16 != 0);   // (a bound up to the largest int)
    const bool few = items <= sm_count();
    int splits = 1;
    while (few && splits < kMaxSplits && 2 * splits * items <= (splits < 4 ? 128 : 96) && blocks >= splits * 16) splits *= 2;
    const bool wide = p.max_q * p.group > 8;
    // more CTAs than run at once: in order of length (64 requests of 512 to 4096
    // states, 512 items: 96 us instead of 112; the step of prompts beside beams 38
    // instead of 45)
    p.longest_first = p.num_seqs > 1 && p.num_seqs <= kSortMax && items * splits > 2LL * sm_count();
    auto go = [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        if (few) return wide ? launch_t<T, D, 2, 8>(p, kmap, vmap, splits, s) : launch_t<T, D, 1, 8>(p, kmap, vmap, splits, s);
        return wide ? launch_t<T, D, 2, 4>(p, kmap, vmap, splits, s) : launch_t<T, D, 1, 4>(p, kmap, vmap, splits, s);
    };
    auto of = [&](auto t) {
        return head_dim == 128 ? go(t, std::integral_constant<int, 128>{}) : go(t, std::integral_constant<int, 64>{});
    };
    return dtype == 0 ? of(__half{}) : of(__nv_bfloat16{});
}

}  // namespace pa
