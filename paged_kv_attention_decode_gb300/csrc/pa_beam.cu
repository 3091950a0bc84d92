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
// Two kernels.  The first reads every logit once and keeps almost nothing: a warp
// takes 4 KB of a row in registers and leaves the sum of its exponentials and the
// largest logit of every 512 bytes (a group).  The second, a CTA per request, joins
// the sums and looks for the k best groups: the k best candidates lie in them, as
// the groups' largest are k candidates that are not worse than any outside.  Their
// logits are read again, k * 512 bytes.  (Few requests take both steps in one launch,
// a cluster each.)
// Bound by the logits' bytes; each logit costs a conversion, a 2^x, and half of two
// additions, a product and a maximum.  (Listing the k best of every 16 KB in
// the first kernel took three times as many instructions.)  64 requests of 8 beams,
// 131072 tokens, 16 bits: 28.5 us, of which the first kernel takes 21 (134 MB at 6.4
// TB/s, 0.94 of the copy rate) and the second, whose chain of loads and meetings one
// request cannot shorten, 7.5; with lists it was 49.  The first kernel runs 16 CTAs an
// SM, at 64 registers a thread, and spills for it (bytes stored and loaded a thread:
// bf16 78 and 100, fp16 44 and 44, fp32 36 and 40): with 14, 12 and 10 CTAs, where
// less spills, and with 10 nothing, the call takes 29.5, 30.6 and 31.9 us, not 28.7.
//
// Within a row the order of scores is the order of logits, and the logarithm of the
// row's sum cancels, so that a beam's own candidates are in their order whatever the
// sum's error.  Across rows, scores are compared as sums of two fp32 numbers, as a
// score of magnitude 16 rounded to fp32 is good to 2^-21 only, and the k best lie close
// together.  The logarithm in them is less exact than their 48 bits: fp32 exponentials
// and sums leave it off by about 2^-24 (64 rows each of 1000 to 2^20 normal logits of
// deviations 0.1 to 3, the three types: mean 0 to 0.9, deviation 0.5 to 1.1, at most
// 5, in 2^-24; log2 e rounded to fp32 alone moves every exponent by 1.3e-8 of itself
// in one direction).  Candidates of different beams closer than that may come in
// either order.
//
// -inf (and NaN, which counts as -inf) is no candidate: a request with fewer than k
// finite ones fills up with the lowest other indices.
constexpr int kSelThreads = 64;
constexpr int kSelVecs = 8;                     // 16-byte words per thread

using u64 = unsigned long long;

// Bits of a float in an order-preserving form, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
// Order of a row's logits: larger first, then the lower index.
__device__ __forceinline__ u64 key_of(float x, int index) {
    // (-0 and +0 are one value)
    return static_cast<u64>(ordered(x + 0.f)) << 32 | static_cast<uint32_t>(~index);
}

// (x, y) <- (x + a, y + b) and (x * f, y * f), one instruction each
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 p, q, d;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 d, p, q;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void mul_pair(float& x, float& y, float f) {
    asm("{\n\t.reg .b64 p, q, d;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\t"
        "mul.rn.f32x2 d, p, q;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(f));
}

// Register words of a row: one fp32 logit, or two of 16 bits.  `clean` takes NaN to
// -inf and +inf to the type's largest; a maximum drops a NaN.
template <typename T> struct Logits;
template <> struct Logits<float> {
    static constexpr int kPer = 4;   // logits of 16 bytes
    static constexpr float kTop = FLT_MAX;
    static constexpr uint32_t kLow = 0xff800000u;
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return __float_as_uint(fminf(__uint_as_float(larger(w, kLow)), kTop));
    }
    static __device__ __forceinline__ float most(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ float value(const float* x) { return *x; }
    static __device__ __forceinline__ void put(uint32_t* w, int i, const float* src) {
        w[i] = src ? __float_as_uint(*src) : kLow;
    }
};
template <typename T2, typename T> struct Logits16 {
    static constexpr int kPer = 8;
    static constexpr bool kHalf = std::is_same<T, __half>::value;
    static constexpr float kTop = kHalf ? 65504.f : 3.3895313892515355e38f;
    static constexpr uint32_t kLow = kHalf ? 0xfc00fc00u : 0xff80ff80u;   // -inf twice
    static constexpr uint32_t kTop2 = kHalf ? 0x7bff7bffu : 0x7f7f7f7fu;
    static __device__ __forceinline__ T2 two(uint32_t w) { return *reinterpret_cast<T2*>(&w); }
    static __device__ __forceinline__ uint32_t bits(T2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return bits(__hmax2(two(a), two(b))); }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return bits(__hmin2(two(larger(w, kLow)), two(kTop2)));
    }
    static __device__ __forceinline__ float most(uint32_t w) {
        const float2 f = Elem<T>::to_float2(w);
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ float value(const T* x) {
        return Elem<T>::to_float2(*reinterpret_cast<const uint16_t*>(x)).x;
    }
    static __device__ __forceinline__ void put(uint32_t* w, int i, const T* src) {
        const uint32_t h = src ? *reinterpret_cast<const uint16_t*>(src) : kLow & 0xffffu;
        w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | h << 16 : h;
    }
};
template <> struct Logits<__half> : Logits16<__half2, __half> {};
template <> struct Logits<__nv_bfloat16> : Logits16<__nv_bfloat162, __nv_bfloat16> {};

// Two fp32 values of a pair of register words: words a and b of fp32, or the
// halves of word a.
template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<T, float>::value) return make_float2(__uint_as_float(a), __uint_as_float(b));
    else return Elem<T>::to_float2(a);
}

// Bytes `from` .. `from` + 15 of two words (0 < from < 16, the same for the warp).
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

// 16 bytes that are not soon read again (volatile: not ahead of the wait for the
// kernel that writes them).
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Whether row `row` of the logits has candidates (a dead beam's are all -inf, an
// ended one has its single one).
__device__ __forceinline__ bool reads_row(const BeamSelectParams& p, int row) {
    if (p.finished && p.finished[row]) return false;
    const float s = p.scores[row];
    return s > -INFINITY;   // (NaN counts as -inf)
}

// One warp's piece of a row, kSelVecs * 512 bytes: lane l leaves with the largest
// logit of group l % kSelVecs, and every lane with the piece's and its sum.
template <typename T>
__device__ __forceinline__ void sum_piece(const BeamSelectParams& p, int row, int piece, int lane, float& gm, float& wm,
                                          float& sum) {
    using L = Logits<T>;
    constexpr int kPer = L::kPer, kVecs = kSelVecs, kWords = kVecs * 4;
    constexpr bool kWide = std::is_same<T, float>::value;   // one logit a word
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // index of the first logit of this lane's word j
    auto at = [&](int j) { return ((piece * kVecs + j) * 32 + lane) * kPer; };

    // Words count from the row's first logit, wherever that lies, so that equal rows
    // have equal sums: off a 16-byte boundary a lane takes its 16 bytes from the two
    // aligned words that hold them.
    uint32_t v[kWords];
    const uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15u);
    const int before = static_cast<int>(lead / sizeof(T));   // logits of the first of them in front of ours
    auto one_by_one = [&](int j) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) L::put(v + 4 * j, i, at(j) + i < p.vocab ? x + at(j) + i : nullptr);
    };
    auto keep = [&](int j, const uint4& w) {
        v[4 * j] = w.x;
        v[4 * j + 1] = w.y;
        v[4 * j + 2] = w.z;
        v[4 * j + 3] = w.w;
    };
    if (lead == 0 && (piece + 1) * kVecs * 32 * kPer <= p.vocab) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) keep(j, load_once(x + at(j)));
    } else if (lead == 0) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (at(j) <= p.vocab - kPer) keep(j, load_once(x + at(j)));
            else one_by_one(j);
        }
    } else {
        auto inside = [&](int j) { return at(j) >= before && at(j) - before + 2 * kPer <= p.vocab; };
#pragma unroll
        for (int half = 0; half < kVecs; half += kVecs / 2) {   // (all of a half's loads in flight)
            uint4 a[kVecs / 2], b[kVecs / 2];
#pragma unroll
            for (int j = 0; j < kVecs / 2; ++j) {
                const uint4* w = reinterpret_cast<const uint4*>(x + at(half + j) - before);
                a[j] = b[j] = make_uint4(0u, 0u, 0u, 0u);
                if (inside(half + j)) {
                    a[j] = w[0];
                    b[j] = w[1];
                }
            }
#pragma unroll
            for (int j = 0; j < kVecs / 2; ++j) keep(half + j, bytes_from(a[j], b[j], lead));
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            if (!inside(j)) one_by_one(j);
    }

    // The groups' largest: lane l ends with that of every lane's word l % 8 (three
    // exchanges halve the words in hand, two more join the quarters), the warp's,
    // and the warp's sum of 2^((x - wm) log2 e): the largest counts as 1 exactly, so
    // that a beam with one candidate left keeps its score.  A NaN or +inf makes the
    // sum NaN: only then are the words cleaned and the sum taken again.
    auto largest = [&]() {
        static_assert(kVecs == 8, "eight words over eight lanes");
        uint32_t m[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            // (kLow first: of two NaN a maximum keeps one)
            m[j] = L::larger(L::larger(L::larger(v[4 * j], L::kLow), v[4 * j + 1]), L::larger(L::larger(v[4 * j + 2], L::kLow), v[4 * j + 3]));
        }
#pragma unroll
        for (int n = 4; n > 0; n >>= 1) {
            const bool upper = lane & n;
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const uint32_t send = upper ? m[j] : m[j + n], mine = upper ? m[j + n] : m[j];
                m[j] = L::larger(mine, __shfl_xor_sync(kFull, send, n));
            }
        }
        m[0] = L::larger(m[0], __shfl_xor_sync(kFull, m[0], 8));
        m[0] = L::larger(m[0], __shfl_xor_sync(kFull, m[0], 16));
        gm = L::most(m[0]);
        wm = unordered(__reduce_max_sync(kFull, ordered(gm)));
    };
    largest();
    {
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int i = 0; i < kWords; i += 2) {
            float2 a;
            if constexpr (kWide) {
                a = pair_of<T>(v[i], v[i + 1]);
            } else {
                a = pair_of<T>(v[i], 0u);
                float2 b = pair_of<T>(v[i + 1], 0u);
                add_pair(b.x, b.y, -wm, -wm);
                mul_pair(b.x, b.y, kLog2e);
                add_pair(s2, s3, fast_exp2(b.x), fast_exp2(b.y));
            }
            add_pair(a.x, a.y, -wm, -wm);
            mul_pair(a.x, a.y, kLog2e);
            add_pair(s0, s1, fast_exp2(a.x), fast_exp2(a.y));
        }
        sum = (s0 + s1) + (s2 + s3);
    }
    if (__any_sync(kFull, !(sum < INFINITY))) {   // (also where all of the warp's are -inf)
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = L::clean(v[i]);
        largest();
        sum = 0.f;
        if (wm > -INFINITY) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const float2 f = pair_of<T>(v[i], v[i]);
                sum += fast_exp2((f.x - wm) * kLog2e);
                if constexpr (!kWide) sum += fast_exp2((f.y - wm) * kLog2e);
            }
        }
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads, 16) beam_pieces_kernel(const BeamSelectParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t all = static_cast<int64_t>(p.num_seqs) * p.beams * p.pieces;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * (kSelThreads / 32) + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (slot >= all) return;
    const int row = static_cast<int>(slot / p.pieces), piece = static_cast<int>(slot - static_cast<int64_t>(row) * p.pieces);
    if (!reads_row(p, row)) return;
    float gm, wm, sum;
    sum_piece<T>(p, row, piece, lane, gm, wm, sum);
    if (lane < kSelVecs) p.groups[slot * kSelVecs + lane] = gm;
    if (lane == 0) p.sums[slot] = make_float2(wm, sum);
}

// Sums of two fp32 numbers, about 48 bits: fp64 runs at a small fraction of their
// rate here (with it the second kernel took 23 us under ncu, 64 requests of 8 beams,
// where it now takes 11).
struct Two {
    float hi, lo;   // |lo| at most half a unit of hi's last place
};
// a + b and its rounding error (Knuth)
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi);
    const float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), h = __fadd_rn(s.hi, e);
    return {h, __fadd_rn(e, -__fadd_rn(h, -s.hi))};
}
// In the numbers' order, to compare: hi's bits, then lo's.
__device__ __forceinline__ u64 order_of(Two x) {
    return static_cast<u64>(ordered(x.hi + 0.f)) << 32 | ordered(x.lo + 0.f);
}

// log((65 + 2 i) / 64), as sums of two
__device__ const float kLogTable[32][2] = {
    {0.015504186972975731f, -4.3701048335620385e-10f}, {0.045809537172317505f, -1.1410232758635175e-09f}, {0.0752234235405922f, -2.303004675852094e-09f}, {0.10379679501056671f, -1.328923193710807e-09f},
    {0.13157635927200317f, -1.4832839401179854e-09f}, {0.15860502421855927f, 5.9580793632108e-09f}, {0.18492233753204346f, 9.619685048534166e-10f}, {0.2105647623538971f, 6.753452463925669e-09f},
    {0.23556606471538544f, 6.597381307926753e-09f}, {0.25995752215385437f, 2.283071731667974e-09f}, {0.2837681770324707f, -3.9018259734291405e-09f}, {0.3070250451564789f, -9.86156667437399e-09f},
    {0.3297532796859741f, 6.686494025132106e-09f}, {0.3519764244556427f, -1.2984644470748208e-09f}, {0.37371641397476196f, -4.181178070439273e-09f}, {0.3949938118457794f, -3.604910370214043e-09f},
    {0.4158279001712799f, -5.027569027760137e-09f}, {0.43623676896095276f, -2.1860346866020564e-09f}, {0.45623743534088135f, -1.8592938300088235e-09f}, {0.47584590315818787f, 1.7117760542362248e-09f},
    {0.4950772523880005f, 1.4409851090135817e-08f}, {0.5139457583427429f, -7.2405086370963545e-09f}, {0.5324648022651672f, -3.395695280516975e-09f}, {0.5506471395492554f, -2.1596592958417204e-08f},
    {0.5685047507286072f, -1.5375938744455198e-08f}, {0.5860490202903748f, 2.4713203927717586e-08f}, {0.603290855884552f, -4.446467638530294e-09f}, {0.6202403903007507f, 1.9451107391432743e-08f},
    {0.6369074583053589f, 3.931710068627581e-09f}, {0.6533012986183167f, -2.660557107958539e-08f}, {0.669430673122406f, -1.9179775989641712e-08f}, {0.6853039860725403f, 1.702637852929456e-08f},
};
// The logarithm of a positive normal x, to 2^-29 absolute: x = 2^e m, m in [1, 2) near
// c = (65 + 2 i) / 64, log m = log c + log(1 + (m - c) / c), from a table of log c and
// the series of log(1 + u) (a table-driven logarithm as in P. T. P. Tang, ACM
// Transactions on Mathematical Software 16, 1990, with the midpoints of 32 intervals,
// Taylor coefficients and sums of two fp32 numbers).  Near 1 itself, c = 1: a beam with one
// candidate left scores what it scored.
__device__ __forceinline__ Two two_log(float x, const Two* table) {
    const uint32_t b = __float_as_uint(x);
    const bool near_one = x > 0.984375f && x < 1.03125f;
    const float e = near_one ? 0.f : static_cast<float>(static_cast<int>(b >> 23) - 127);
    const int i = static_cast<int>(b >> 18) & 31;
    const float m = near_one ? x : __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
    const float c = near_one ? 1.f : (65 + 2 * i) * 0.015625f;
    const float u = (m - c) / c;   // |u| <= 1 / 32
    // u - u^2 / 2 + ... : the next term, u^6 / 6, is below 2^-32
    const float v = u * u * fmaf(u, fmaf(u, fmaf(u, 0.2f, -0.25f), 0.33333333f), -0.5f);
    Two r = near_one ? Two{0.f, 0.f} : table[i];
    r = two_add(r, two_sum(u, v));
    return two_add(r, {e * 0.693115234375f, e * 3.194618329871446e-05f});   // (the first product is exact)
}

constexpr int kJoinThreads = 512;
constexpr int kJoinSets = kJoinThreads / 4;   // sets of groups, of four threads each
constexpr int kFewPieces = 256;                // of a request that one cluster takes
constexpr int kHeld = 8;                      // groups that a thread holds on to
constexpr int kJoinCap = 512;                 // groups, and candidates, ranked at once
static_assert(kJoinSets >= kMaxBeamOut, "k sets give k groups");

// A candidate, or a group by its best one: the score, then the lower beam, then the
// order within the row (key 0: none).
struct Cand {
    u64 score, key;
    int beam;
};
__device__ __forceinline__ bool better_than(const Cand& a, const Cand& b) {
    if (a.score != b.score) return a.score > b.score;
    return a.beam != b.beam ? a.beam < b.beam : a.key > b.key;
}

// One CTA per request, after its pieces: `all_sums` and `groups` are the request's.
// The k best groups are found by scores in fp32 (x plus a term of its beam), with
// room for their roundings; the candidates that come through are ranked by the exact
// ones.  Where too many come through (equal scores), groups and candidates are taken
// one by one.  `ready` comes between what needs no piece and the rest.
template <typename T, typename Ready>
__device__ __forceinline__ void join_request(const BeamSelectParams& p, int s, const float2* all_sums,
                                             const float* groups, Ready ready) {
    using L = Logits<T>;
    constexpr int kGroup = 32 * L::kPer;   // logits of a group
    constexpr int kWarps = kJoinThreads / 32;
    // score, the row's largest logit and the logarithm of its sum: a candidate is
    // score + ((x - largest) - logarithm), in this order, as the largest may be huge
    __shared__ float s_score[kMaxBeams], s_most[kMaxBeams];
    __shared__ Two s_log[kMaxBeams], s_table[32];
    __shared__ float s_add[kMaxBeams];                // score - largest - logarithm; -inf: no row of candidates
    __shared__ int8_t s_kind[kMaxBeams];              // 0: no candidates, 1: a row of logits, 2: ended
    __shared__ bool s_over[kMaxBeams];                // (as given: the results may take the inputs' place)
    __shared__ __align__(16) uint32_t s_set[kJoinSets];
    __shared__ float s_tau;
    __shared__ uint32_t s_room;                       // (bits of a float, 0 or more)
    __shared__ int s_groups, s_count;
    __shared__ bool s_far;                            // some s_add is past fp32's range
    __shared__ u64 s_cs[kJoinCap], s_ck[kJoinCap];
    __shared__ int s_cb[kJoinCap], s_list[kJoinCap];
    __shared__ int s_flat[kMaxBeamOut];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int W = p.beams, k = p.k, C = p.pieces;
    const int per_row = C * kSelVecs, total = W * per_row;   // groups (those past the row are -inf)
    if (tid < 32) s_table[tid] = {kLogTable[tid][0], kLogTable[tid][1]};
    if (tid == 0) {
        s_groups = s_count = 0;
        s_far = false;
        s_room = 0u;
    }
    ready();
    // This thread's groups: every 512th, so that the first 128 lie in different sets.
    // The first ones are asked for before the rows' sums are needed (a row that was
    // not read has whatever the workspace held).
    const int mine0 = (tid >> 2) + (tid & 3) * kJoinSets;
    float held[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
        const int g = mine0 + u * kJoinThreads;
        held[u] = g < total ? groups[g] : -INFINITY;
    }
    for (int w = warp; w < W; w += kWarps) {
        const int row = s * W + w;
        const float2* sums = all_sums + w * C;
        const float2 none = make_float2(-INFINITY, 0.f);
        const float2 a = lane < C ? sums[lane] : none, b = lane + 32 < C ? sums[lane + 32] : none;
        const float given = p.scores[row];
        const bool over = p.finished && p.finished[row], alive = given > -INFINITY;
        const float score = fminf(given, FLT_MAX);
        float m = fmaxf(a.x, b.x), sum = 0.f;
        if (!over && alive) {
            for (int c = lane + 64; c < C; c += 32) m = fmaxf(m, sums[c].x);
            m = unordered(__reduce_max_sync(kFull, ordered(m)));
            if (m > -INFINITY) {
                sum = a.y * fast_exp2((a.x - m) * kLog2e) + b.y * fast_exp2((b.x - m) * kLog2e);
                for (int c = lane + 64; c < C; c += 32) sum += sums[c].y * fast_exp2((sums[c].x - m) * kLog2e);
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
        }
        if (lane == 0) {
            // an ended beam goes on as it is, with its one candidate
            const int kind = !alive ? 0 : over ? 2 : m > -INFINITY ? 1 : 0;
            const Two lg = kind == 1 ? two_log(sum, s_table) : Two{0.f, 0.f};   // (the sum is 1 at least, but for its rounding)
            s_kind[w] = static_cast<int8_t>(kind);
            s_over[w] = over;
            s_score[w] = score;
            s_most[w] = kind == 1 ? m : 0.f;
            s_log[w] = lg;
            s_add[w] = kind == 1 ? (score - lg.hi) - m : -INFINITY;
            if (kind == 1 && !(fabsf(s_add[w]) <= FLT_MAX)) s_far = true;
            if (kind == 1) atomicMax(&s_room, __float_as_uint(fabsf(score) + fabsf(m) + fabsf(lg.hi)));
        }
    }
    __syncthreads();
    // the beam of group g: the quotient's error, 2^-18 at most, is below half a group
    const float inv_row = 1.f / static_cast<float>(per_row);
    auto beam_of = [&](int g) { return static_cast<int>((static_cast<float>(g) + 0.5f) * inv_row); };
    auto cand_of = [&](int beam, u64 key) {
        const float x = unordered(static_cast<uint32_t>(key >> 32));
        const Two lg = s_log[beam], less{-lg.hi, -lg.lo};
        const float most = s_most[beam], score = s_score[beam];
        Two t;
        if (x - most >= -FLT_MAX) {
            t = two_add({score, 0.f}, two_add(two_sum(x, -most), less));
        } else {   // (this difference alone is below the range: the large numbers of opposite signs first)
            t = two_add(two_add(two_sum(score, -most), {x, 0.f}), less);
        }
        // (below fp32's range: -inf, and no candidate)
        return t.hi >= -FLT_MAX ? Cand{order_of({fminf(t.hi, FLT_MAX), t.lo}), key, beam} : Cand{0, 0, 0};
    };
    auto ended = [&](int beam) { return cand_of(beam, key_of(0.f, p.end_token)); };
    auto row_of = [&](int beam) { return static_cast<const T*>(p.logits) + (s * W + beam) * p.stride; };

    // tau: the k-th best of the sets' best: k groups, or ended beams, are not below
    // it.  A set's number in the lowest bits tells equal ones apart; what it takes
    // off is part of the room.  With fewer groups than twice k the logits themselves
    // are shared out instead (at most 2^15 of them).
    const bool direct = W * ((p.vocab + kGroup - 1) / kGroup) < 2 * k;
    auto direct_logit = [&](int i, int& beam, int& e) {   // -inf: no candidate
        beam = i / p.vocab;
        e = i - beam * p.vocab;
        const float f = s_kind[beam] == 1 ? L::value(row_of(beam) + e) : -INFINITY;
        return f >= -L::kTop ? fminf(f, L::kTop) : -INFINITY;   // (not a NaN)
    };
    float best = -INFINITY;
    if (direct) {
        for (int i = tid; i < W * p.vocab; i += kJoinThreads) {
            int beam, e;
            const float f = direct_logit(i, beam, e);
            best = fmaxf(best, f + s_add[beam]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int g = mine0 + u * kJoinThreads;
            held[u] = g < total ? held[u] + s_add[beam_of(g)] : -INFINITY;
            best = fmaxf(best, held[u]);
        }
        for (int g = mine0 + kHeld * kJoinThreads; g < total; g += kJoinThreads) best = fmaxf(best, groups[g] + s_add[beam_of(g)]);
    }
    if (tid < W && s_kind[tid] == 2) best = fmaxf(best, s_score[tid]);
    best = fmaxf(best, __shfl_xor_sync(kFull, best, 1));
    best = fmaxf(best, __shfl_xor_sync(kFull, best, 2));
    const uint32_t mine = (ordered(best) & ~(kJoinSets - 1u)) | static_cast<uint32_t>(tid >> 2);
    if ((lane & 3) == 0) s_set[tid >> 2] = mine;
    __syncthreads();
    {
        int better = 0;
#pragma unroll
        for (int i = 0; i < kJoinSets / 4; i += 4) {   // (a fourth of the sets a thread)
            const uint4 o = *reinterpret_cast<const uint4*>(s_set + 4 * i + 4 * (tid & 3));
            better += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        }
        better += __shfl_xor_sync(kFull, better, 1);
        better += __shfl_xor_sync(kFull, better, 2);
        if (better == k - 1) s_tau = unordered(mine);
    }
    __syncthreads();
    // A score in fp32 is off by less than 2^-21 of `room` and itself (four roundings,
    // of numbers up to these), the number in the low bits is 2^-16 of tau (beside a
    // score of 0 less than the smallest normal number), and both sides are.  (tau of
    // no group: the lowest number; -inf is never a candidate.)
    const float t0 = s_tau;
    const float room = 9.5367431640625e-7f * __uint_as_float(s_room) + 3.0517578125e-5f * fabsf(t0) + FLT_MIN;
    const float tau = t0 > -FLT_MAX ? fmaxf(t0 - room, -FLT_MAX) : -FLT_MAX;
    auto push = [&](const Cand& c) {
        const int i = atomicAdd(&s_count, 1);
        if (i < kJoinCap) {
            s_cs[i] = c.score;
            s_ck[i] = c.key;
            s_cb[i] = c.beam;
        }
    };
    if (direct) {
        for (int i = tid; i < W * p.vocab; i += kJoinThreads) {
            int beam, e;
            const float f = direct_logit(i, beam, e);
            if (f + s_add[beam] >= tau) {
                const Cand c = cand_of(beam, key_of(f, e));
                if (c.key) push(c);
            }
        }
    } else if (best >= tau) {
        auto list = [&](int g) {
            const int i = atomicAdd(&s_groups, 1);
            if (i < kJoinCap) s_list[i] = g;
        };
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
            if (held[u] >= tau) list(mine0 + u * kJoinThreads);
        for (int g = mine0 + kHeld * kJoinThreads; g < total; g += kJoinThreads)
            if (groups[g] + s_add[beam_of(g)] >= tau) list(g);
    }
    if (tid < W && s_kind[tid] == 2 && s_score[tid] >= tau) push(ended(tid));
    __syncthreads();
    const int listed = s_groups;
    // their logits that reach it, a warp for each group and 16 bytes a lane, two
    // groups' loads in flight (NaN, as -inf, does not reach it)
    const int looked = min(listed, kJoinCap);
    for (int i = warp; i < looked; i += 2 * kWarps) {
        uint32_t v[2][4];
        float add[2];
        int beam[2], e0[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int g = s_list[min(i + u * kWarps, looked - 1)];
            beam[u] = beam_of(g);
            e0[u] = (g - beam[u] * per_row) * kGroup + lane * L::kPer;
            add[u] = i + u * kWarps < looked ? s_add[beam[u]] : -INFINITY;
            const T* x = row_of(beam[u]) + e0[u];
            if ((reinterpret_cast<uintptr_t>(x) & 15u) == 0 && e0[u] <= p.vocab - L::kPer) {
                const uint4 w = *reinterpret_cast<const uint4*>(x);
                v[u][0] = w.x;
                v[u][1] = w.y;
                v[u][2] = w.z;
                v[u][3] = w.w;
            } else {
#pragma unroll
                for (int c = 0; c < L::kPer; ++c) L::put(v[u], c, e0[u] + c < p.vocab ? x + c : nullptr);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            auto look = [&](float f, int e) {
                if (!(f + add[u] >= tau)) return;
                const Cand c = cand_of(beam[u], key_of(fminf(f, L::kTop), e));
                if (c.key) push(c);
            };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 f = pair_of<T>(v[u][c], v[u][c]);
                if constexpr (std::is_same<T, float>::value) {
                    look(f.x, e0[u] + c);
                } else {
                    look(f.x, e0[u] + 2 * c);
                    look(f.y, e0[u] + 2 * c + 1);
                }
            }
        }
    }
    __syncthreads();
    const int64_t o = static_cast<int64_t>(s) * k;
    auto put = [&](int r, const Cand& c) {
        const int token = static_cast<int>(~static_cast<uint32_t>(c.key));
        p.out_scores[o + r] = unordered(static_cast<uint32_t>(c.score >> 32));
        p.out_parents[o + r] = c.beam;
        p.out_tokens[o + r] = token;
        s_flat[r] = c.beam * p.vocab + token;
        if (p.out_finished) p.out_finished[o + r] = s_kind[c.beam] == 2 || token == p.end_token;
    };
    int found = s_count;
    if (listed <= kJoinCap && found <= kJoinCap && !s_far) {
        // rank them against one another: a warp for each, or a few lanes for each
        // when they are few
        if (found <= kJoinThreads / 16) {
            const int i = tid >> 4, sub = tid & 15;
            if (i < found) {
                const Cand c{s_cs[i], s_ck[i], s_cb[i]};
                int better = 0;
                for (int j = sub; j < found; j += 16) better += better_than({s_cs[j], s_ck[j], s_cb[j]}, c);
                const uint32_t half = lane < 16 ? 0xffffu : 0xffff0000u;
                better = __reduce_add_sync(half, better);
                if (sub == 0 && better < k) put(better, c);
            }
        } else {
            for (int i = warp; i < found; i += kWarps) {
                const Cand c{s_cs[i], s_ck[i], s_cb[i]};
                int better = 0;
                for (int j = lane; j < found; j += 32) better += better_than({s_cs[j], s_ck[j], s_cb[j]}, c);
                better = __reduce_add_sync(kFull, better);
                if (lane == 0 && better < k) put(better, c);
            }
        }
        found = min(found, k);
    } else {
        // Many equal scores, or huge ones.  The best of all threads' `mine`:
        auto best_of_all = [&](const Cand& mine) {
            Cand top = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const Cand c{__shfl_xor_sync(kFull, top.score, off), __shfl_xor_sync(kFull, top.key, off),
                             __shfl_xor_sync(kFull, top.beam, off)};
                if (better_than(c, top)) top = c;
            }
            __syncthreads();
            if (lane == 0) {
                s_cs[warp] = top.score;
                s_ck[warp] = top.key;
                s_cb[warp] = top.beam;
            }
            __syncthreads();
            top = {s_cs[0], s_ck[0], s_cb[0]};
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const Cand c{s_cs[w], s_ck[w], s_cb[w]};
                if (better_than(c, top)) top = c;
            }
            return top;
        };
        // the k best groups by their exact scores, one after another (a group's key
        // holds its number, whose order is that of its logits' indices) ...
        Cand last{~0ull, ~0ull, -1};
        int n = 0;
        for (; n < k; ++n) {
            Cand top{0, 0, 0};
            for (int g = tid; g < total; g += kJoinThreads) {
                const int beam = beam_of(g);
                if (s_kind[beam] != 1 || !(groups[g] > -INFINITY)) continue;
                const Cand c = cand_of(beam, key_of(groups[g], g - beam * per_row));
                if (c.key && better_than(last, c) && better_than(c, top)) top = c;
            }
            last = best_of_all(top);
            if (last.key == 0) break;
            if (tid == 0) s_list[n] = last.beam * per_row + static_cast<int>(~static_cast<uint32_t>(last.key));
        }
        __syncthreads();
        // ... and the k best candidates of these
        last = {~0ull, ~0ull, -1};
        for (found = 0; found < k; ++found) {
            Cand top{0, 0, 0};
            for (int i = tid; i < n * kGroup; i += kJoinThreads) {
                const int g = s_list[i / kGroup], beam = beam_of(g), e = (g - beam * per_row) * kGroup + i % kGroup;
                const float f = e < p.vocab ? L::value(row_of(beam) + e) : -INFINITY;
                if (!(f >= -L::kTop)) continue;
                const Cand c = cand_of(beam, key_of(fminf(f, L::kTop), e));
                if (c.key && better_than(last, c) && better_than(c, top)) top = c;
            }
            if (tid < W && s_kind[tid] == 2) {
                const Cand c = ended(tid);
                if (better_than(last, c) && better_than(c, top)) top = c;
            }
            last = best_of_all(top);
            if (last.key == 0) break;
            if (tid == 0) put(found, last);
        }
    }
    __syncthreads();
    // fewer than k finite candidates: the lowest others, all of score -inf
    if (warp > 0) return;
    for (int r = found, flat = 0; r < k; ++flat) {
        const bool taken = (lane < found && s_flat[lane] == flat) || (lane + 32 < found && s_flat[lane + 32] == flat);
        if (__any_sync(kFull, taken)) continue;
        if (lane == 0) {
            const int w = flat / p.vocab, token = flat - w * p.vocab;
            p.out_scores[o + r] = -INFINITY;
            p.out_parents[o + r] = w;
            p.out_tokens[o + r] = token;
            if (p.out_finished)
                p.out_finished[o + r] = s_over[w] || token == p.end_token;
        }
        ++r;
    }
}

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamSelectParams p) {
    const int s = static_cast<int>(blockIdx.x);
    const int64_t first = static_cast<int64_t>(s) * p.beams * p.pieces;
    join_request<T>(p, s, p.sums + first, p.groups + first * kSelVecs, [] {
        __syncthreads();
        pdl_trigger();
        pdl_wait();
    });
}

// Few requests: both in one launch.  A cluster takes a request; its warps leave
// their pieces' sums and groups in the first CTA's shared memory, which then joins
// them.  No workspace.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads, 1) beam_few_kernel(const BeamSelectParams p) {
    extern __shared__ __align__(16) uint8_t few_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int s = static_cast<int>(blockIdx.x / ctas), all = p.beams * p.pieces;
    float2* sums = reinterpret_cast<float2*>(few_smem);                       // [all]
    float* groups = reinterpret_cast<float*>(few_smem + kFewPieces * sizeof(float2));   // [all, kSelVecs]
    const uint32_t sums0 = map_rank(smem_addr(sums), 0), groups0 = map_rank(smem_addr(groups), 0);
    pdl_trigger();
    cluster_sync();   // (the first CTA runs: its shared memory may be written)
    pdl_wait();
    for (int i = static_cast<int>(rank) * (kJoinThreads / 32) + warp; i < all; i += static_cast<int>(ctas) * (kJoinThreads / 32)) {
        const int w = i / p.pieces, row = s * p.beams + w;
        if (!reads_row(p, row)) continue;
        float gm, wm, sum;
        sum_piece<T>(p, row, i - w * p.pieces, lane, gm, wm, sum);
        if (lane < kSelVecs) st_cluster(groups0 + (i * kSelVecs + lane) * 4, gm);
        if (lane == 0) {
            st_cluster(sums0 + i * 8, wm);
            st_cluster(sums0 + i * 8 + 4, sum);
        }
    }
    cluster_sync();
    if (rank > 0) return;
    join_request<T>(p, s, sums, groups, [] { __syncthreads(); });
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

// Lane j works out row j (every lane of one warp calls; `free`: shared memory).
__device__ __forceinline__ Family family_of(const BeamReorderParams& p, int s, int lane, bool report, int* free) {
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
    const uint32_t childless = all & ~parents, before = (1u << lane) - 1u;
    if (childless >> lane & 1u) free[__popc(childless & before)] = tail;
    __syncwarp();
    const int theirs = __shfl_sync(kFull, tail, x.parent & 31);
    const int mine = moves ? free[__popc(movers & before)] : theirs;
    x.tail = mine;
    x.src = moves ? theirs : -1;
    return x;
}

constexpr int kCopyThreads = 256;

// blockIdx: (slice, layer, request).  Every CTA works the request's family out
// for itself; slices and layers share its copies.
__global__ void __launch_bounds__(kCopyThreads) beam_copy_kernel(const __grid_constant__ BeamReorderParams p) {
    __shared__ int s_src[kMaxBeams], s_dst[kMaxBeams], s_parent[kMaxBeams], s_tail[kMaxBeams], s_free[kMaxBeams];
    __shared__ int s_pairs, s_f, s_t, s_ok;
    const int tid = threadIdx.x;
    const int s = static_cast<int>(blockIdx.z), layer = static_cast<int>(blockIdx.y);
    pdl_trigger();
    pdl_wait();
    if (tid < 32) {
        const Family x = family_of(p, s, tid, p.first && blockIdx.x == 0 && layer == 0, s_free);
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
    __shared__ int s_parent[kMaxBeams], s_tail[kMaxBeams], s_free[kMaxBeams];
    __shared__ int s_f, s_t, s_ok;
    const int tid = threadIdx.x, s = static_cast<int>(blockIdx.x), W = p.beams;
    pdl_trigger();
    pdl_wait();
    if (tid < 32) {
        const Family x = family_of(p, s, tid, false, s_free);
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

int beam_pieces(int vocab, int dtype) {
    const int per = 32 * kSelVecs * (dtype == 2 ? 4 : 8);
    return (vocab + per - 1) / per;
}

// A request in one cluster while all clusters run at once (see launch_cross) and a
// warp has a piece of it, or two: the second launch's gap then costs about what the
// fewer warps do, and the host, which sets the pace of calls this short, saves a
// launch and a workspace (4 to 5 us).  us of one cluster of 8, 4, 2, 1 CTAs and of
// two launches: 1 request of 4 beams, 32000 tokens (64 pieces) 6.8, 6.8, 8.1, 10.5
// and 6.5; 32 of them 12.5, 7.3, 8.8, 11.4 and 8.8; 64 of 2 beams, 8000 tokens 18.4,
// 12.9, 7.1, 6.8 and 7.6; 1 of 8 beams, 131072 tokens (512 pieces) 11.5, 16.3, 25.3,
// 43.4 and 7.5.  Two pieces a warp (8, 4, 4, 2, 1 CTAs) and two launches: 1 request
// of 8 beams, 50001 tokens 10.4 and 8.3; 16 of 5, 40000 8.6 and 8.5; 32 of 8, 32000
// 10.1 and 10.4; 64 of 4 10.3 and 11.0; 128 of 2 10.1 and 11.0.
int beam_cluster(int num_seqs, int beams, int vocab, int dtype) {
    constexpr int kWarps = kJoinThreads / 32;
    const long long pieces = static_cast<long long>(beams) * beam_pieces(vocab, dtype);
    const int most = num_seqs <= 8 ? 8 : num_seqs <= 32 ? 4 : num_seqs <= 64 ? 2 : num_seqs <= 128 ? 1 : 0;
    if (pieces > 2 * kWarps * most) return 0;
    int ctas = 1;
    while (ctas < most && pieces > kWarps * ctas) ctas *= 2;
    return ctas;
}
static_assert(kFewPieces == 2 * (kJoinThreads / 32) * 8, "two pieces a warp of the largest cluster");

cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, cudaStream_t s) {
    const int ctas = beam_cluster(p.num_seqs, p.beams, p.vocab, dtype);
    const long long warps = static_cast<long long>(p.num_seqs) * p.beams * p.pieces;
    const dim3 grid(static_cast<unsigned>((warps + kSelThreads / 32 - 1) / (kSelThreads / 32)));
    auto go = [&](auto t) {
        using T = decltype(t);
        if (ctas) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * ctas);
            cfg.blockDim = dim3(kJoinThreads);
            cfg.dynamicSmemBytes = kFewPieces * (sizeof(float2) + kSelVecs * sizeof(float));
            cfg.stream = s;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = ctas;
            attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            return cudaLaunchKernelEx(&cfg, beam_few_kernel<T>, p);
        }
        const cudaError_t e = launch_pdl(beam_pieces_kernel<T>, grid, dim3(kSelThreads), 0, s, p);
        if (e != cudaSuccess) return e;
        return launch_pdl(beam_join_kernel<T>, dim3(p.num_seqs), dim3(kJoinThreads), 0, s, p);
    };
    return dtype == 0 ? go(__half{}) : dtype == 1 ? go(__nv_bfloat16{}) : go(0.f);
}

cudaError_t launch_beam_copy(const BeamReorderParams& p, cudaStream_t s) {
    // 16 KB a CTA or, with many requests and layers, about 16 CTAs an SM (a third of a
    // request's beams move on average, 8 tokens each): 64 requests of 8 beams, 4
    // layers of 16 heads, with 4, 8, 16, 32 an SM: 27, 20.7, 18.2, 18.4 us
    const long long bytes = 2LL * std::max(1, p.beams / 3) * (p.block_bytes / 2);
    const long long per_cta = 16LL * kCopyThreads * 4;
    const long long others = static_cast<long long>(p.num_seqs) * std::max(1, p.layers);
    const long long want = (16LL * sm_count() + others - 1) / others;
    const int slices = static_cast<int>(std::max(1LL, std::min(want, (bytes + per_cta - 1) / per_cta)));
    return launch_pdl(beam_copy_kernel, dim3(slices, std::max(1, p.layers), p.num_seqs), dim3(kCopyThreads), 0, s, p);
}

cudaError_t launch_beam_tables(const BeamReorderParams& p, cudaStream_t s) {
    return launch_pdl(beam_tables_kernel, dim3(p.num_seqs), dim3(kCopyThreads), 0, s, p);
}

}  // namespace pa
