// Beam search over a paged cache: selection of the best continuations over
// beams and vocabulary, and the reordering of tables and caches that follows.
#include <cfloat>

#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
// Candidate (beam w, token v) of a request scores score[w] + x[w, v] - lse(x[w]);
// the k best of its W * V candidates are wanted, ties to the lowest w * V + v.
// Two kernels.  The first reads every logit once: a CTA holds 16 KB of a row in
// registers, sums its exponentials and lists its k largest logits in order.
// The second joins a row's pieces and a request's rows.
//
// Within a row the order of scores is the order of logits, so the first kernel
// needs no sum.  A candidate is a 64-bit key, the logit's bits in an order-
// preserving form above the complement of its index: keys are distinct, larger
// is better, and ties go to the lower index.  Across rows, scores are compared
// in 64 bits: a sum of fp32 exponentials is good to about 2^-27 (the terms'
// errors are independent), but a score of magnitude 16 rounded to fp32 only to
// 2^-21, and the k best lie close together.
//
// -inf (and NaN, which counts as -inf) never enters a list: a request with
// fewer than k finite candidates fills up with the lowest other indices.
constexpr int kSelThreads = 256;
constexpr int kSelVecs = 4;                     // 16-byte pieces of a row per thread
constexpr int kSelGroups = 64;                  // groups of 4 threads, >= kMaxBeamOut
constexpr int kSelCap = 512;                    // candidates ranked at once
static_assert(kSelGroups >= kMaxBeamOut && kSelThreads == 4 * kSelGroups, "k groups give k candidates");

using u64 = unsigned long long;

// Bits of a float in an order-preserving form, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ u64 key_of(float x, int index) {
    // (-0 and +0 are one value)
    return static_cast<u64>(ordered(x + 0.f)) << 32 | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ u64 shfl_xor64(u64 x, int off) { return __shfl_xor_sync(kFull, x, off); }

// A 16-byte piece of a row: values as fp32, NaN as -inf, +inf as the type's largest.
template <typename T> struct Logits;
template <> struct Logits<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ uint4 clean(uint4 v) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __float_as_uint(fminf(fmaxf(__uint_as_float(w[i]), -INFINITY), FLT_MAX));
        return v;
    }
    static __device__ __forceinline__ float most(const uint4& v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ float get(const uint4& v, int i) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
        return __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ void put(uint4& v, int i, const float* src) {
        reinterpret_cast<uint32_t*>(&v)[i] = src ? __float_as_uint(*src) : 0xff800000u;
    }
};
template <typename T2, typename T> struct Logits16 {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ T2 two(uint32_t w) { return *reinterpret_cast<T2*>(&w); }
    static __device__ __forceinline__ uint4 clean(uint4 v) {
        constexpr uint32_t kLow = std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
        constexpr uint32_t kTop = std::is_same<T, __half>::value ? 0x7bff7bffu : 0x7f7f7f7fu;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T2 x = __hmin2(__hmax2(two(w[i]), two(kLow)), two(kTop));   // (max drops a NaN)
            w[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        return v;
    }
    static __device__ __forceinline__ float most(const uint4& v) {
        const T2 x = __hmax2(__hmax2(two(v.x), two(v.y)), __hmax2(two(v.z), two(v.w)));
        const float2 f = Elem<T>::to_float2(*reinterpret_cast<const uint32_t*>(&x));
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ float get(const uint4& v, int i) {
        const float2 f = Elem<T>::to_float2(reinterpret_cast<const uint32_t*>(&v)[i >> 1]);
        return i & 1 ? f.y : f.x;
    }
    static __device__ __forceinline__ void put(uint4& v, int i, const T* src) {
        constexpr uint16_t kLow = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
        reinterpret_cast<uint16_t*>(&v)[i] = src ? *reinterpret_cast<const uint16_t*>(src) : kLow;
    }
};
template <> struct Logits<__half> : Logits16<__half2, __half> {};
template <> struct Logits<__nv_bfloat16> : Logits16<__nv_bfloat162, __nv_bfloat16> {};

// Bytes `from` .. `from` + 15 of two words (0 < from < 16, the same for the CTA).
__device__ __forceinline__ uint4 bytes_from(const uint4& a, const uint4& b, uint32_t from) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (from & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (from & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (from & 3u) * 8u;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether row `row` of the logits has candidates (a dead beam's are all -inf, an
// ended one has its single one).
__device__ __forceinline__ bool reads_row(const BeamSelectParams& p, int row) {
    if (p.finished && p.finished[row]) return false;
    const float s = p.scores[row];
    return s > -INFINITY;   // (NaN counts as -inf)
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads) beam_pieces_kernel(const BeamSelectParams p) {
    using L = Logits<T>;
    constexpr int kPer = L::kPer;
    __shared__ float s_group[kSelGroups];
    __shared__ float s_m[kSelThreads / 32], s_s[kSelThreads / 32];
    __shared__ float s_tau;
    __shared__ int s_count;
    __shared__ u64 s_key[kSelCap];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = static_cast<int>(blockIdx.x) / p.chunks, piece = static_cast<int>(blockIdx.x) - row * p.chunks;
    if (tid == 0) s_count = 0;
    pdl_trigger();
    pdl_wait();
    if (!reads_row(p, row)) return;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // Pieces count from the row's first element, wherever that lies, so that equal
    // rows have equal sums: off a 16-byte boundary a thread takes its 16 bytes from
    // the two aligned words that hold them.
    const uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15u);
    const int before = static_cast<int>(lead / sizeof(T));   // elements of the first word in front of a piece
    const int k = p.k;

    uint4 v[kSelVecs];
    int at[kSelVecs];   // index of a piece's first element
#pragma unroll
    for (int j = 0; j < kSelVecs; ++j) at[j] = ((piece * kSelVecs + j) * kSelThreads + tid) * kPer;
    auto one_by_one = [&](int j) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) L::put(v[j], i, at[j] + i < p.vocab ? x + at[j] + i : nullptr);
    };
    if (lead == 0) {
#pragma unroll
        for (int j = 0; j < kSelVecs; ++j) {
            if (at[j] <= p.vocab - kPer) v[j] = __ldcs(reinterpret_cast<const uint4*>(x + at[j]));
            else one_by_one(j);
        }
    } else {
        uint4 next[kSelVecs];
        auto inside = [&](int j) { return at[j] >= before && at[j] - before + 2 * kPer <= p.vocab; };
#pragma unroll
        for (int j = 0; j < kSelVecs; ++j) {
            if (inside(j)) {
                const uint4* w = reinterpret_cast<const uint4*>(x + at[j] - before);
                v[j] = w[0];
                next[j] = w[1];
            }
        }
#pragma unroll
        for (int j = 0; j < kSelVecs; ++j) {
            if (inside(j)) v[j] = bytes_from(v[j], next[j], lead);
            else one_by_one(j);
        }
    }
    float tm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kSelVecs; ++j) {
        v[j] = L::clean(v[j]);
        tm = fmaxf(tm, L::most(v[j]));
    }
    float gm = fmaxf(tm, __shfl_xor_sync(kFull, tm, 1));
    gm = fmaxf(gm, __shfl_xor_sync(kFull, gm, 2));
    if ((lane & 3) == 0) s_group[tid >> 2] = gm;
    float wm = gm;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) wm = fmaxf(wm, __shfl_xor_sync(kFull, wm, off));
    // the warp's sum of 2^((x - wm) log2 e)
    float sum = 0.f;
    if (wm > -INFINITY) {
#pragma unroll
        for (int j = 0; j < kSelVecs; ++j)
#pragma unroll
            for (int i = 0; i < kPer; ++i) sum += fast_exp2((L::get(v[j], i) - wm) * kLog2e);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
    if (lane == 0) {
        s_m[warp] = wm;
        s_s[warp] = sum;
    }
    __syncthreads();
    // tau: the k-th largest of the groups' maxima.  k groups hold an element at
    // least as large, so the k best are not below it; with 64 groups they are few.
    if (tid < kSelGroups) {
        const float mine = s_group[tid];
        int better = 0;
#pragma unroll 8
        for (int i = 0; i < kSelGroups; ++i) {
            const float o = s_group[i];
            better += o > mine || (o == mine && i < tid);
        }
        if (better == k - 1) s_tau = mine;
    }
    __syncthreads();
    const float tau = s_tau;
    if (tm >= tau && tm > -INFINITY) {
#pragma unroll
        for (int j = 0; j < kSelVecs; ++j) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float f = L::get(v[j], i);
                if (f >= tau && f > -INFINITY) {
                    const int c = atomicAdd(&s_count, 1);
                    if (c < kSelCap) s_key[c] = key_of(f, at[j] + i);
                }
            }
        }
    }
    __syncthreads();
    const int found = s_count;
    const int64_t slot = static_cast<int64_t>(row) * p.chunks + piece;
    u64* best = p.best + slot * k;
    int listed = min(found, k);
    if (found <= kSelCap) {
        // rank them against one another
        for (int i = tid; i < found; i += kSelThreads) {
            const u64 mine = s_key[i];
            int better = 0;
            for (int o = 0; o < found; ++o) better += s_key[o] > mine;
            if (better < k) best[better] = mine;
        }
    } else {
        // many equal logits: the largest key below the last one, k times
        u64 last = ~0ull;
        for (int r = 0; r < k; ++r) {
            u64 top = 0;
#pragma unroll
            for (int j = 0; j < kSelVecs; ++j) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float f = L::get(v[j], i);
                    const u64 key = f > -INFINITY ? key_of(f, at[j] + i) : 0;
                    if (key < last && key > top) top = key;
                }
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) top = max(top, shfl_xor64(top, off));
            __syncthreads();
            if (lane == 0) s_key[warp] = top;
            __syncthreads();
            top = s_key[0];
#pragma unroll
            for (int w = 1; w < kSelThreads / 32; ++w) top = max(top, s_key[w]);
            if (tid == 0) best[r] = top;
            last = top;
        }
    }
    if (tid == 0) {
        float m = s_m[0];
#pragma unroll
        for (int w = 1; w < kSelThreads / 32; ++w) m = fmaxf(m, s_m[w]);
        float s = 0.f;
        if (m > -INFINITY) {
#pragma unroll
            for (int w = 0; w < kSelThreads / 32; ++w) s += s_s[w] * fast_exp2((s_m[w] - m) * kLog2e);
        }
        p.piece[slot] = make_uint4(__float_as_uint(m), __float_as_uint(s), static_cast<uint32_t>(listed), 0u);
    }
}

// A 64-bit maximum over the warp's lanes, in two 32-bit steps.
__device__ __forceinline__ u64 warp_max64(u64 x) {
    const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(x >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, static_cast<uint32_t>(x >> 32) == hi ? static_cast<uint32_t>(x) : 0u);
    return static_cast<u64>(hi) << 32 | lo;
}
__device__ __forceinline__ u64 ordered64(double x) {
    const u64 b = static_cast<u64>(__double_as_longlong(x));
    return b ^ (b >> 63 ? ~0ull : 1ull << 63);
}

constexpr int kJoinWarps = 8;
constexpr int kMaxPieces = 256;   // of a row (vocabularies of 2^20)

// One CTA per request.  A warp merges the ordered lists of a row's pieces (one
// head a lane, the largest leaves k times), then one warp merges the rows' by
// their scores (one beam a lane).
__global__ void __launch_bounds__(kJoinWarps * 32) beam_join_kernel(const BeamSelectParams p) {
    __shared__ u64 s_best[kMaxBeams][kMaxBeamOut];
    __shared__ int s_n[kMaxBeams];
    // score, the row's largest logit and the logarithm of its sum: a candidate is
    // score + ((x - largest) - logarithm), in this order, as the largest may be huge
    __shared__ float s_score[kMaxBeams], s_most[kMaxBeams];
    __shared__ double s_log[kMaxBeams];
    __shared__ uint8_t s_pos[kJoinWarps][kMaxPieces];
    __shared__ int s_flat[kMaxBeamOut];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = static_cast<int>(blockIdx.x);
    const int W = p.beams, k = p.k, C = p.chunks;
    pdl_trigger();
    pdl_wait();
    for (int w = warp; w < W; w += kJoinWarps) {
        const int row = s * W + w;
        const float score = fminf(p.scores[row], FLT_MAX);
        if (!reads_row(p, row)) {
            if (lane == 0) {
                // an ended beam goes on as it is, with its one candidate
                const bool ended = p.finished && p.finished[row] && p.scores[row] > -INFINITY;
                s_n[w] = ended ? 1 : 0;
                s_score[w] = score;
                s_most[w] = 0.f;
                s_log[w] = 0.0;
                s_best[w][0] = key_of(0.f, p.end_token);
            }
            continue;
        }
        const int64_t slot = static_cast<int64_t>(row) * C;
        float m = -INFINITY;
        for (int c = lane; c < C; c += 32) m = fmaxf(m, __uint_as_float(p.piece[slot + c].x));
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        // this lane's lists: c = lane, lane + 32, ...; its best head
        float sum = 0.f;
        u64 head = 0;
        int mine = 0;
        for (int c = lane; c < C; c += 32) {
            const uint4 d = p.piece[slot + c];
            if (m > -INFINITY) sum += __uint_as_float(d.y) * fast_exp2((__uint_as_float(d.x) - m) * kLog2e);
            s_pos[warp][c] = 0;
            const u64 h = d.z > 0 ? p.best[(slot + c) * k] : 0;
            if (h > head) {
                head = h;
                mine = c;
            }
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
        if (lane == 0) {
            s_score[w] = score;
            s_most[w] = m;
            s_log[w] = log(static_cast<double>(sum));
        }
        int n = 0;
        for (; n < k; ++n) {
            const u64 top = warp_max64(head);
            if (top == 0) break;
            if (lane == 0) s_best[w][n] = top;
            if (head == top) {   // (keys are distinct: one lane)
                ++s_pos[warp][mine];
                head = 0;
                for (int c = lane; c < C; c += 32) {
                    const int at = s_pos[warp][c];
                    const u64 h = at < static_cast<int>(p.piece[slot + c].z) ? p.best[(slot + c) * k + at] : 0;
                    if (h > head) {
                        head = h;
                        mine = c;
                    }
                }
            }
        }
        if (lane == 0) s_n[w] = n;
        __syncwarp();
    }
    __syncthreads();
    if (warp > 0) return;

    // beams: a lane each, heads compared by score, ties to the lower beam
    const int n = lane < W ? s_n[lane] : 0;
    const double cum = n > 0 ? s_score[lane] : 0.0, most = n > 0 ? s_most[lane] : 0.0, lg = n > 0 ? s_log[lane] : 0.0;
    int at = 0;
    double score = 0.0;
    u64 key = 0;
    auto load = [&]() {
        if (at < n) {
            score = cum + ((static_cast<double>(unordered(static_cast<uint32_t>(s_best[lane][at] >> 32))) - most) - lg);
            key = ordered64(score);
        } else {
            key = 0;
        }
    };
    load();
    const int64_t o = static_cast<int64_t>(s) * k;
    int r = 0;
    for (; r < k; ++r) {
        const u64 top = warp_max64(key);
        if (top == 0) break;
        const int win = __ffs(__ballot_sync(kFull, key == top)) - 1;
        if (lane == win) {
            const int token = static_cast<int>(~static_cast<uint32_t>(s_best[lane][at]));
            p.out_scores[o + r] = static_cast<float>(score);
            p.out_parents[o + r] = lane;
            p.out_tokens[o + r] = token;
            s_flat[r] = lane * p.vocab + token;
            if (p.out_finished)
                p.out_finished[o + r] = (p.finished && p.finished[s * W + lane]) || token == p.end_token;
            ++at;
            load();
        }
    }
    __syncwarp();
    // fewer than k finite candidates: the lowest others, all of score -inf
    const int found = r;
    for (int flat = 0; r < k; ++flat) {
        const bool taken = (lane < found && s_flat[lane] == flat) || (lane + 32 < found && s_flat[lane + 32] == flat);
        if (__any_sync(kFull, taken)) continue;
        if (lane == 0) {
            const int w = flat / p.vocab, token = flat - w * p.vocab;
            p.out_scores[o + r] = -INFINITY;
            p.out_parents[o + r] = w;
            p.out_tokens[o + r] = token;
            if (p.out_finished)
                p.out_finished[o + r] = (p.finished && p.finished[s * W + w]) || token == p.end_token;
        }
        ++r;
    }
}

// ---------------------------------------------------------------------------
// reordering
// ---------------------------------------------------------------------------
// A request's W rows hold n = 16 f + t tokens each; row j goes on from row
// parent[j].  Whole blocks are shared by reference.  The last block, of t > 0
// tokens, is written to in the next step, so every row needs its own: the
// lowest child of a parent takes the parent's block over, and the others take
// the blocks of the rows without a child, into which the parent's t tokens are
// copied.  There are as many of these as of those (W less the number of
// different parents), so no block is allocated, and no block is both read and
// written.  Table entries behind the last token stay with their row.
struct Family {
    bool ok;
    int f, t;
    int parent;      // lane j: of row j
    int tail;        // the block that row j goes on with (t > 0)
    int src;         // the block it is copied from, or -1
};

// Lane j works out row j (every lane of one warp calls).
__device__ __forceinline__ Family family_of(const BeamReorderParams& p, int s, int lane, bool report) {
    const int W = p.beams, row = s * W + lane;
    const bool live = lane < W;
    const uint32_t all = W == 32 ? kFull : (1u << W) - 1u;
    Family x{};
    const int n = live ? p.seq_lens[row] : 0;
    const int n0 = __shfl_sync(kFull, n, 0);
    x.parent = live ? p.parents[row] : 0;
    const bool len_ok = n0 >= 0 && n0 <= p.max_blocks * 16;
    uint32_t bad = __any_sync(kFull, live && (n != n0 || !len_ok || x.parent < 0 || x.parent >= W))
                       ? PA_DEVERR_BEAM_ : 0u;
    x.f = n0 >> 4;
    x.t = n0 & 15;
    int tail = -1 - lane;
    if (!bad && x.t > 0 && live) tail = p.tables[static_cast<int64_t>(row) * p.max_blocks + x.f];
    if (!bad && x.t > 0) {
        if (__any_sync(kFull, live && (tail < 0 || tail >= p.num_blocks))) bad = PA_DEVERR_BLOCK_ID_;
        // two rows that would write into one block
        const uint32_t twins = __match_any_sync(kFull, live ? tail : -1 - lane);
        if (!bad && __any_sync(kFull, live && (twins & (twins - 1)))) bad = PA_DEVERR_BEAM_;
    }
    if (bad && report && lane == 0) record_error(p.err, bad);
    x.ok = !bad;
    const uint32_t siblings = __match_any_sync(kFull, live && x.ok ? x.parent : 64 + lane);
    const bool moves = live && x.ok && x.t > 0 && (__ffs(siblings) - 1) != lane;
    const uint32_t movers = __ballot_sync(kFull, moves);
    const uint32_t parents = __reduce_or_sync(kFull, live && x.ok ? 1u << x.parent : 0u);
    const uint32_t childless = all & ~parents;
    const int rank = __popc(movers & ((1u << lane) - 1u));
    const int from = moves ? static_cast<int>(__fns(childless, 0, rank + 1)) : x.parent;
    const int mine = __shfl_sync(kFull, tail, from & 31), theirs = __shfl_sync(kFull, tail, x.parent & 31);
    x.tail = mine;
    x.src = moves ? theirs : -1;
    return x;
}

constexpr int kCopyThreads = 256;

// blockIdx: (slice, layer, request).  Every CTA works the request's family out
// for itself; slices and layers share its copies.
__global__ void __launch_bounds__(kCopyThreads) beam_copy_kernel(const __grid_constant__ BeamReorderParams p) {
    __shared__ int s_src[kMaxBeams], s_dst[kMaxBeams], s_parent[kMaxBeams], s_tail[kMaxBeams];
    __shared__ int s_pairs, s_f, s_t, s_ok;
    const int tid = threadIdx.x;
    const int s = static_cast<int>(blockIdx.z), layer = static_cast<int>(blockIdx.y);
    pdl_trigger();
    pdl_wait();
    if (tid < 32) {
        const Family x = family_of(p, s, tid, p.first && blockIdx.x == 0 && layer == 0);
        const uint32_t movers = __ballot_sync(kFull, x.src >= 0);
        if (x.src >= 0) {
            const int i = __popc(movers & ((1u << tid) - 1u));
            s_src[i] = x.src;
            s_dst[i] = x.tail;
        }
        if (tid < p.beams) {
            s_parent[tid] = x.parent;
            s_tail[tid] = x.tail;
        }
        if (tid == 0) {
            s_pairs = __popc(movers);
            s_f = x.f;
            s_t = x.t;
            s_ok = x.ok;
        }
    }
    __syncthreads();
    if (p.first && p.tables_out != p.tables) {
        // the request's table entries, shared by its CTAs
        const int W = p.beams, f = s_f;
        const bool ok = s_ok, tail = ok && s_t > 0;
        const int64_t base = static_cast<int64_t>(s) * W * p.max_blocks;
        const int total = W * p.max_blocks;
        const int cta = layer * gridDim.x + blockIdx.x, ctas = gridDim.x * gridDim.y;
        for (int i = cta * kCopyThreads + tid; i < total; i += ctas * kCopyThreads) {
            const int j = i / p.max_blocks, c = i - j * p.max_blocks;
            int v;
            if (ok && c < f) v = p.tables[base + static_cast<int64_t>(s_parent[j]) * p.max_blocks + c];
            else if (tail && c == f) v = s_tail[j];
            else v = p.tables[base + i];
            p.tables_out[base + i] = v;
        }
    }
    const int pairs = s_pairs;
    if (pairs == 0 || layer >= p.layers) return;
    // 16-byte pieces of one block: `per` in each of `runs` runs
    const uint32_t per = static_cast<uint32_t>(p.token_bytes ? s_t * p.token_bytes : p.block_bytes) / 16u;
    const uint32_t runs = p.token_bytes ? p.runs : 1, each = per * runs;
    const uint32_t total = each * 2u * pairs;
    const int64_t block16 = p.block_bytes / 16;
    const uint32_t run16 = p.run_stride / 16;
    const uint32_t step = gridDim.x * kCopyThreads;
    uint4* kp = static_cast<uint4*>(p.k[layer]);
    uint4* vp = static_cast<uint4*>(p.v[layer]);
    constexpr int kFly = 4;
    for (uint32_t i0 = blockIdx.x * kCopyThreads + tid; i0 < total; i0 += kFly * step) {
        uint4 x[kFly];
        uint4* to[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            const uint32_t i = i0 + u * step;
            to[u] = nullptr;
            if (i < total) {
                const uint32_t pk = i / each, c = i - pk * each;   // (pair, pool)
                const uint32_t run = c / per, off = c - run * per;
                uint4* pool = pk & 1u ? vp : kp;
                const int64_t in = static_cast<int64_t>(run) * run16 + off;
                x[u] = pool[static_cast<int64_t>(s_src[pk >> 1]) * block16 + in];
                to[u] = pool + static_cast<int64_t>(s_dst[pk >> 1]) * block16 + in;
            }
        }
#pragma unroll
        for (int u = 0; u < kFly; ++u)
            if (to[u]) *to[u] = x[u];
    }
}

// In place: one CTA per request, a column of its table rows per thread.  Runs
// behind the copies, which read the tables as they were.
__global__ void __launch_bounds__(kCopyThreads) beam_tables_kernel(const __grid_constant__ BeamReorderParams p) {
    __shared__ int s_parent[kMaxBeams], s_tail[kMaxBeams];
    __shared__ int s_f, s_t, s_ok;
    const int tid = threadIdx.x, s = static_cast<int>(blockIdx.x), W = p.beams;
    pdl_trigger();
    pdl_wait();
    if (tid < 32) {
        const Family x = family_of(p, s, tid, false);
        if (tid < W) {
            s_parent[tid] = x.parent;
            s_tail[tid] = x.tail;
        }
        if (tid == 0) {
            s_f = x.f;
            s_t = x.t;
            s_ok = x.ok;
        }
    }
    __syncthreads();
    if (!s_ok) return;
    int32_t* rows = p.tables_out + static_cast<int64_t>(s) * W * p.max_blocks;
    const int last = s_t > 0 ? s_f : s_f - 1;
    for (int c = tid; c <= last; c += kCopyThreads) {
        int old[kMaxBeams];
#pragma unroll
        for (int j = 0; j < kMaxBeams; ++j)
            if (j < W) old[j] = c < s_f ? rows[static_cast<int64_t>(s_parent[j]) * p.max_blocks + c] : s_tail[j];
#pragma unroll
        for (int j = 0; j < kMaxBeams; ++j)
            if (j < W) rows[static_cast<int64_t>(j) * p.max_blocks + c] = old[j];
    }
}

}  // namespace

int beam_chunk_elems(int dtype) { return kSelThreads * kSelVecs * (dtype == 2 ? 4 : 8); }

cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.chunks) * p.num_seqs * p.beams);
    auto kern = dtype == 0 ? beam_pieces_kernel<__half> : dtype == 1 ? beam_pieces_kernel<__nv_bfloat16>
                                                                     : beam_pieces_kernel<float>;
    cudaError_t e = launch_pdl(kern, grid, dim3(kSelThreads), 0, s, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_join_kernel, dim3(p.num_seqs), dim3(kJoinWarps * 32), 0, s, p);
}

cudaError_t launch_beam_copy(const BeamReorderParams& p, cudaStream_t s) {
    // a few CTAs per SM; a third of a request's beams move on average, 8 tokens each
    const long long bytes = 2LL * std::max(1, p.beams / 3) * (p.block_bytes / 2);
    const long long per_cta = 16LL * kCopyThreads * 4;
    const long long others = static_cast<long long>(p.num_seqs) * std::max(1, p.layers);
    const long long want = (4LL * sm_count() + others - 1) / others;
    const int slices = static_cast<int>(std::max(1LL, std::min(want, (bytes + per_cta - 1) / per_cta)));
    return launch_pdl(beam_copy_kernel, dim3(slices, std::max(1, p.layers), p.num_seqs), dim3(kCopyThreads), 0, s, p);
}

cudaError_t launch_beam_tables(const BeamReorderParams& p, cudaStream_t s) {
    return launch_pdl(beam_tables_kernel, dim3(p.num_seqs), dim3(kCopyThreads), 0, s, p);
}

}  // namespace pa
