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
// Two kernels.  The first reads every logit once: a CTA holds 16 or 32 KB of a row
// in registers, sums its exponentials and lists its k largest logits in order.
// The second joins a row's pieces and a request's rows.
//
// Within a row the order of scores is the order of logits, so the first kernel
// needs no sum.  A candidate is a 64-bit key, the logit's bits in an order-
// preserving form above the complement of its index: keys are distinct, larger
// is better, and ties go to the lower index.  Across rows, scores are compared
// as sums of two fp32 numbers: a sum of fp32 exponentials is good to 2^-24 (the
// terms' errors are independent), but a score of magnitude 16 rounded to fp32 only
// to 2^-21, and the k best lie close together.
//
// -inf (and NaN, which counts as -inf) never enters a list: a request with
// fewer than k finite candidates fills up with the lowest other indices.
constexpr int kSelThreads = 256;
constexpr int kSelGroups = kSelThreads / 4;     // groups of 4 threads
constexpr int kSelCap = 512;                    // candidates ranked at once
static_assert(kSelGroups >= kMaxBeamOut, "k groups give k candidates");

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

// (x, y) <- (x + a, y + b) and (x * f + a, y * f + a), one instruction each
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 p, q, d;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 d, p, q;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void fma_pair(float& x, float& y, float f, float a) {
    asm("{\n\t.reg .b64 p, q, r, d;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
        "fma.rn.f32x2 d, p, q, r;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(f), "f"(a));
}

// 16-byte words of a row.
template <typename T> struct Logits;
template <> struct Logits<float> {
    static constexpr int kPer = 4;
    static constexpr float kTop = FLT_MAX;
    // NaN as -inf, +inf as the type's largest
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return __float_as_uint(fminf(fmaxf(__uint_as_float(w), -INFINITY), FLT_MAX));
    }
    struct Most {
        float m = -INFINITY;
        __device__ __forceinline__ void take(uint32_t w) { m = fmaxf(m, __uint_as_float(w)); }
        __device__ __forceinline__ float get() const { return m; }
    };
    static __device__ __forceinline__ float value(const float* x) { return *x; }
    static __device__ __forceinline__ void put(uint32_t* w, int i, const float* src) {
        w[i] = src ? __float_as_uint(*src) : 0xff800000u;
    }
};
template <typename T2, typename T> struct Logits16 {
    static constexpr int kPer = 8;
    static constexpr bool kHalf = std::is_same<T, __half>::value;
    static constexpr float kTop = kHalf ? 65504.f : 3.3895313892515355e38f;
    static constexpr uint32_t kLow2 = kHalf ? 0xfc00fc00u : 0xff80ff80u;   // -inf twice
    static constexpr uint32_t kTop2 = kHalf ? 0x7bff7bffu : 0x7f7f7f7fu;
    static __device__ __forceinline__ T2 two(uint32_t w) { return *reinterpret_cast<T2*>(&w); }
    static __device__ __forceinline__ uint32_t bits(T2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return bits(__hmin2(__hmax2(two(w), two(kLow2)), two(kTop2)));   // (a maximum drops a NaN)
    }
    struct Most {
        uint32_t m = kLow2;
        __device__ __forceinline__ void take(uint32_t w) { m = bits(__hmax2(two(m), two(w))); }
        __device__ __forceinline__ float get() const {
            const float2 f = Elem<T>::to_float2(m);
            return fmaxf(f.x, f.y);
        }
    };
    static __device__ __forceinline__ float value(const T* x) {
        return Elem<T>::to_float2(*reinterpret_cast<const uint16_t*>(x)).x;
    }
    static __device__ __forceinline__ void put(uint32_t* w, int i, const T* src) {
        const uint32_t h = src ? *reinterpret_cast<const uint16_t*>(src) : kLow2 & 0xffffu;
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

// kVecs: 16-byte words per thread.
template <typename T, int kVecs>
__global__ void __launch_bounds__(kSelThreads, kVecs > 4 ? 4 : 6) beam_pieces_kernel(const BeamSelectParams p) {
    using L = Logits<T>;
    constexpr int kPer = L::kPer, kWords = kVecs * 4;
    constexpr bool kWide = std::is_same<T, float>::value;   // one logit a word
    __shared__ __align__(16) uint32_t s_group[kSelGroups];
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
    const int k = p.k;
    // index of the first element of this thread's word j
    auto at = [&](int j) { return ((piece * kVecs + j) * kSelThreads + tid) * kPer; };

    // Words count from the row's first element, wherever that lies, so that equal
    // rows have equal sums: off a 16-byte boundary a thread takes its 16 bytes from
    // the two aligned words that hold them.
    uint32_t v[kWords];
    const uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15u);
    const int before = static_cast<int>(lead / sizeof(T));   // elements of the first of them in front of ours
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
    const int end = (piece + 1) * kVecs * kSelThreads * kPer;   // of the CTA's piece
    if (lead == 0 && end <= p.vocab) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) keep(j, __ldcs(reinterpret_cast<const uint4*>(x + at(j))));
    } else if (lead == 0) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (at(j) <= p.vocab - kPer) keep(j, __ldcs(reinterpret_cast<const uint4*>(x + at(j))));
            else one_by_one(j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (at(j) >= before && at(j) - before + 2 * kPer <= p.vocab) {
                const uint4* w = reinterpret_cast<const uint4*>(x + at(j) - before);
                keep(j, bytes_from(w[0], w[1], lead));
            } else {
                one_by_one(j);
            }
        }
    }

    // This thread's, its group's and its warp's largest, and the warp's sum of
    // 2^((x - wm) log2 e), as 2^(x log2 e - c) with c = wm log2 e rounded, and that
    // rounding taken back from the sum.  A NaN or +inf makes the sum NaN, and from
    // logits of some 100,000 on c is too coarse: only then are the words cleaned and
    // the sum taken from the differences.
    float tm, gm, wm, sum;
    auto largest = [&]() {
        typename L::Most most;
#pragma unroll
        for (int i = 0; i < kWords; ++i) most.take(v[i]);
        tm = most.get();
        gm = fmaxf(tm, __shfl_xor_sync(kFull, tm, 1));
        gm = fmaxf(gm, __shfl_xor_sync(kFull, gm, 2));
        wm = unordered(__reduce_max_sync(kFull, ordered(gm)));
    };
    largest();
    {
        const float c = wm * kLog2e;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int i = 0; i < kWords; i += 2) {
            float2 a;
            if constexpr (kWide) {
                a = pair_of<T>(v[i], v[i + 1]);
            } else {
                a = pair_of<T>(v[i], 0u);
                float2 b = pair_of<T>(v[i + 1], 0u);
                fma_pair(b.x, b.y, kLog2e, -c);
                add_pair(s2, s3, fast_exp2(b.x), fast_exp2(b.y));
            }
            fma_pair(a.x, a.y, kLog2e, -c);
            add_pair(s0, s1, fast_exp2(a.x), fast_exp2(a.y));
        }
        sum = (s0 + s1) + (s2 + s3);
        const float e = 0.6931471805599453f * fmaf(wm, kLog2e, -c);   // times 1 - e + e^2 / 2
        sum = fmaf(sum, fmaf(0.5f * e, e, -e), sum);
        if (!(fabsf(e) < 0.0078125f)) sum = INFINITY;
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
    // (a group's number in the lowest bits makes its maximum distinct; a tau that is
    // lower by them is one as well)
    const uint32_t gkey = (ordered(gm) & ~(kSelGroups - 1u)) | static_cast<uint32_t>(tid >> 2);
    if ((lane & 3) == 0) s_group[tid >> 2] = gkey;
    if (lane == 0) {
        s_m[warp] = wm;
        s_s[warp] = sum;
    }
    __syncthreads();
    // tau: the k-th largest of the groups' maxima.  k groups hold an element at
    // least as large, so the k best are not below it; with 64 groups they are few
    // (8 of 8192 logits: 8 or 9 pass; 64: about 300).  A group's four threads
    // count a quarter of the others each.
    {
        int better = 0;
#pragma unroll
        for (int i = 0; i < kSelGroups / 4; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(s_group + (tid & 3) * (kSelGroups / 4) + i);
            better += (o.x > gkey) + (o.y > gkey) + (o.z > gkey) + (o.w > gkey);
        }
        better += __shfl_xor_sync(kFull, better, 1);
        better += __shfl_xor_sync(kFull, better, 2);
        if (better == k - 1) s_tau = unordered(gkey & ~(kSelGroups - 1u));
    }
    __syncthreads();
    const float tau = fmaxf(s_tau, -L::kTop);   // (-inf is no candidate)
    if (tm >= tau) {
        // a bit for each logit that passes; their values come from memory again
        // (registers have no index): few of a thread's do
        constexpr int kMasks = kWide ? (kWords + 31) / 32 : (kWords + 15) / 16;
        uint32_t mask[kMasks];
#pragma unroll
        for (int b = 0; b < kMasks; ++b) mask[b] = 0u;
        if constexpr (kWide) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) mask[i >> 5] |= __uint_as_float(v[i]) >= tau ? 1u << (i & 31) : 0u;
        } else {
            const uint32_t t2 = Elem<T>::pack(tau, tau);
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                mask[i >> 4] |= __hge2_mask(L::two(v[i]), L::two(t2)) & (0x00010001u << (i & 15));
        }
#pragma unroll
        for (int b = 0; b < kMasks; ++b) {
            while (mask[b]) {
                const int bit = __ffs(mask[b]) - 1;
                mask[b] &= mask[b] - 1u;
                const int i = kWide ? 32 * b + bit : 16 * b + (bit & 15);
                const int e = at(i >> 2) + (kWide ? i & 3 : (i & 3) * 2 + (bit >> 4));
                const int c = atomicAdd(&s_count, 1);
                if (c < kSelCap) s_key[c] = key_of(fminf(L::value(x + e), L::kTop), e);
            }
        }
    }
    __syncthreads();
    const int found = s_count;
    const int64_t slot = static_cast<int64_t>(row) * p.chunks + piece;
    u64* best = p.best + slot * k;
    if (found <= kSelCap) {
        // rank them against one another
        for (int i = tid; i < found; i += kSelThreads) {
            const u64 mine = s_key[i];
            int better = 0;
            for (int o = 0; o < found; ++o) better += s_key[o] > mine;
            if (better < k) best[better] = mine;
        }
    } else {
        // many equal logits: the largest key below the last one, k times (read again:
        // kept in registers as keys they would not fit)
        u64 last = ~0ull;
        for (int r = 0; r < k; ++r) {
            u64 top = 0;
#pragma unroll 1
            for (int j = 0; j < kVecs; ++j) {
                const int stop = min(at(j) + kPer, p.vocab);
#pragma unroll 1
                for (int e = at(j); e < stop; ++e) {
                    const float f = L::value(x + e);   // (NaN and -inf pass by)
                    const u64 key = f >= -L::kTop ? key_of(fminf(f, L::kTop), e) : 0;
                    if (key < last && key > top) top = key;
                }
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) top = max(top, __shfl_xor_sync(kFull, top, off));
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
        p.piece[slot] = make_uint4(__float_as_uint(m), __float_as_uint(s), static_cast<uint32_t>(min(found, k)), 0u);
    }
}

// Sums of two fp32 numbers, about 48 bits: fp64 runs at a small fraction of their
// rate here (the join took 23 us with it, 64 requests of 8 beams).
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
// The logarithm of a positive normal x, to about 2^-30 absolute: x = 2^e m, m in [1, 2)
// near c = (65 + 2 i) / 64, log m = log c + log(1 + (m - c) / c).
__device__ __forceinline__ Two two_log(float x) {
    const uint32_t b = __float_as_uint(x);
    const float e = static_cast<float>(static_cast<int>(b >> 23) - 127);
    const int i = static_cast<int>(b >> 18) & 31;
    const float m = __uint_as_float((b & 0x7fffffu) | 0x3f800000u), c = (65 + 2 * i) * 0.015625f;
    const float u = (m - c) / c;   // |u| <= 1 / 65
    // u - u^2 / 2 + ... : the next term, u^6 / 6, is below 2^-38
    const float v = u * u * fmaf(u, fmaf(u, fmaf(u, 0.2f, -0.25f), 0.33333333f), -0.5f);
    Two r = {kLogTable[i][0], kLogTable[i][1]};
    r = two_add(r, two_sum(u, v));
    return two_add(r, {e * 0.693115234375f, e * 3.194618329871446e-05f});   // (the first product is exact)
}

constexpr int kJoinThreads = 256;
constexpr int kMaxPieces = 256;   // of a row
constexpr int kJoinCap = 512;     // candidates ranked at once

// A candidate: its score, then the lower beam, then its row's order (key 0: none).
struct Cand {
    u64 score, key;
    int beam;
};
__device__ __forceinline__ bool better_than(const Cand& a, const Cand& b) {
    if (a.score != b.score) return a.score > b.score;
    return a.beam != b.beam ? a.beam < b.beam : a.key > b.key;
}

// One CTA per request: the sums of its rows' pieces, then, of the ordered lists of
// all pieces, the entries that can be among the k best, ranked against one another.
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamSelectParams p) {
    // score, the row's largest logit and the logarithm of its sum: a candidate is
    // score + ((x - largest) - logarithm), in this order, as the largest may be huge
    __shared__ float s_score[kMaxBeams], s_most[kMaxBeams];
    __shared__ Two s_log[kMaxBeams];
    __shared__ int8_t s_kind[kMaxBeams];              // 0: no candidates, 1: a row of logits, 2: ended
    __shared__ __align__(16) uint32_t s_probe[kJoinThreads];
    __shared__ uint32_t s_tau;
    __shared__ int s_count;
    __shared__ u64 s_cs[kJoinCap], s_ck[kJoinCap];
    __shared__ int s_cb[kJoinCap];
    __shared__ uint8_t s_pos[kMaxBeams * kMaxPieces];
    __shared__ int s_flat[kMaxBeamOut];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = static_cast<int>(blockIdx.x);
    const int W = p.beams, k = p.k, C = p.chunks, lists = W * C;
    // Every list gives its d-th entry, d the smallest with lists * d >= k.  The
    // ceil(k / d)-th largest of these (of a thread's, the largest) has k entries
    // not below it.
    const int d = (k + lists - 1) / lists, q = (k + d - 1) / d;
    if (tid == 0) s_count = 0;
    pdl_trigger();
    pdl_wait();
    const int64_t slot0 = static_cast<int64_t>(s) * lists;
    // this thread's first list: asked for before the rows' sums are needed
    // (a row that was not read has whatever the workspace holds)
    const bool has = tid < lists;
    const int n_first = has ? static_cast<int>(p.piece[slot0 + tid].z) : 0;
    const u64 k_first = has ? p.best[(slot0 + tid) * k] : 0, k_probe = has && d > 1 ? p.best[(slot0 + tid) * k + d - 1] : k_first;
    for (int w = warp; w < W; w += kJoinThreads / 32) {
        const int row = s * W + w;
        const float score = fminf(p.scores[row], FLT_MAX);
        const int64_t slot = slot0 + w * C;
        uint4 mine = lane < C ? p.piece[slot + lane] : make_uint4(0xff800000u, 0u, 0u, 0u);
        if (!reads_row(p, row)) {
            // an ended beam goes on as it is, with its one candidate
            const bool ended = p.finished && p.finished[row] && p.scores[row] > -INFINITY;
            if (lane == 0) {
                s_kind[w] = ended ? 2 : 0;
                s_score[w] = score;
                s_most[w] = 0.f;
                s_log[w] = {0.f, 0.f};
            }
            continue;
        }
        float m = __uint_as_float(mine.x);
        for (int c = lane + 32; c < C; c += 32) m = fmaxf(m, __uint_as_float(p.piece[slot + c].x));
        m = unordered(__reduce_max_sync(kFull, ordered(m)));
        float sum = 0.f;
        if (m > -INFINITY)
            for (int c = lane; c < C; c += 32) {
                if (c != lane) mine = p.piece[slot + c];
                sum += __uint_as_float(mine.y) * fast_exp2((__uint_as_float(mine.x) - m) * kLog2e);
            }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
        if (lane == 0) {
            s_kind[w] = 1;
            s_score[w] = score;
            s_most[w] = m;
            s_log[w] = two_log(sum);   // (at least 1, where the row has candidates)
        }
    }
    __syncthreads();
    auto count_of = [&](int l, int n) -> int {   // entries of list l, n those of its piece
        const int kind = s_kind[l / C];
        return kind == 1 ? n : kind == 2 && l % C == 0 ? 1 : 0;
    };
    auto cand_of = [&](int l, u64 key) {
        Cand c;
        c.beam = l / C;
        c.key = s_kind[c.beam] == 2 ? key_of(0.f, p.end_token) : key;
        const float x = unordered(static_cast<uint32_t>(c.key >> 32));
        const Two lg = s_log[c.beam];
        const Two lp = two_add(two_sum(x, -s_most[c.beam]), {-lg.hi, -lg.lo});
        Two t = two_add({s_score[c.beam], 0.f}, lp);
        if (!(t.hi >= -FLT_MAX && t.hi <= FLT_MAX)) t = {__fadd_rn(s_score[c.beam], lp.hi >= -FLT_MAX ? lp.hi : -FLT_MAX), 0.f};
        c.score = order_of(t);
        return c;
    };
    auto entry = [&](int l, int i) { return cand_of(l, p.best[(slot0 + l) * k + i]); };
    // (scores are compared by hi alone here: the order of both is never the other way)
    uint32_t probe = 0;
    const int n0 = has ? count_of(tid, n_first) : 0;
    const Cand first = n0 > 0 ? cand_of(tid, k_first) : Cand{0, 0, 0};
    if (n0 >= d) probe = static_cast<uint32_t>((d > 1 ? cand_of(tid, k_probe) : first).score >> 32);
    for (int l = tid + kJoinThreads; l < lists; l += kJoinThreads)
        if (count_of(l, static_cast<int>(p.piece[slot0 + l].z)) >= d)
            probe = max(probe, static_cast<uint32_t>(entry(l, d - 1).score >> 32));
    s_probe[tid] = probe;
    __syncthreads();
    if (tid < lists) {
        const int n = min(lists, kJoinThreads);
        int better = 0;
        for (int i = 0; i < n; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(s_probe + i);   // (0 behind the last)
            better += o.x > probe || (o.x == probe && i < tid);
            better += o.y > probe || (o.y == probe && i + 1 < tid);
            better += o.z > probe || (o.z == probe && i + 2 < tid);
            better += o.w > probe || (o.w == probe && i + 3 < tid);
        }
        if (better == q - 1) s_tau = probe;
    }
    __syncthreads();
    const uint32_t tau = s_tau;
    for (int l = tid; l < lists; l += kJoinThreads) {
        const int n = l == tid ? n0 : count_of(l, static_cast<int>(p.piece[slot0 + l].z));
        for (int i = 0; i < n; ++i) {
            const Cand c = l == tid && i == 0 ? first : entry(l, i);
            if (static_cast<uint32_t>(c.score >> 32) < tau) break;
            const int at = atomicAdd(&s_count, 1);
            if (at < kJoinCap) {
                s_cs[at] = c.score;
                s_ck[at] = c.key;
                s_cb[at] = c.beam;
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
    if (found <= kJoinCap) {
        for (int i = tid; i < found; i += kJoinThreads) {
            const Cand mine{s_cs[i], s_ck[i], s_cb[i]};
            int better = 0;
            for (int j = 0; j < found; ++j) {
                const u64 other = s_cs[j];
                better += other > mine.score || (other == mine.score && better_than({other, s_ck[j], s_cb[j]}, mine));
            }
            if (better < k) put(better, mine);
        }
        found = min(found, k);
    } else {
        // many equal scores: the best of the lists' heads, k times
        for (int l = tid; l < lists; l += kJoinThreads) s_pos[l] = 0;
        for (found = 0; found < k; ++found) {
            Cand top{0, 0, 0};
            int from = -1;
            for (int l = tid; l < lists; l += kJoinThreads) {
                if (s_pos[l] >= count_of(l, static_cast<int>(p.piece[slot0 + l].z))) continue;
                const Cand c = entry(l, s_pos[l]);
                if (better_than(c, top)) {
                    top = c;
                    from = l;
                }
            }
            const Cand mine = top;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                Cand c;
                c.score = __shfl_xor_sync(kFull, top.score, off);
                c.key = __shfl_xor_sync(kFull, top.key, off);
                c.beam = __shfl_xor_sync(kFull, top.beam, off);
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
            for (int w = 1; w < kJoinThreads / 32; ++w) {
                const Cand c{s_cs[w], s_ck[w], s_cb[w]};
                if (better_than(c, top)) top = c;
            }
            // (candidates are distinct: one thread)
            if (from >= 0 && mine.score == top.score && mine.key == top.key && mine.beam == top.beam) {
                put(found, mine);
                ++s_pos[from];
            }
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

// 16-byte words per thread
static int select_vecs(int rows, int vocab, int dtype) {
    const long long bytes = static_cast<long long>(vocab) * (dtype == 2 ? 4 : 2);
    return rows * ((bytes + 32767) / 32768) >= 4LL * 152 ? 8 : 4;
}

int beam_pieces(int rows, int vocab, int dtype) {
    const int per = kSelThreads * select_vecs(rows, vocab, dtype) * (dtype == 2 ? 4 : 8);
    return (vocab + per - 1) / per;
}

cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, cudaStream_t s) {
    const int rows = p.num_seqs * p.beams;
    const dim3 grid(static_cast<unsigned>(p.chunks) * rows);
    const bool wide = select_vecs(rows, p.vocab, dtype) == 8;
    auto go = [&](auto t) {
        using T = decltype(t);
        return launch_pdl(wide ? beam_pieces_kernel<T, 8> : beam_pieces_kernel<T, 4>, grid, dim3(kSelThreads), 0, s, p);
    };
    const cudaError_t e = dtype == 0 ? go(__half{}) : dtype == 1 ? go(__nv_bfloat16{}) : go(0.f);
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_join_kernel, dim3(p.num_seqs), dim3(kJoinThreads), 0, s, p);
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
