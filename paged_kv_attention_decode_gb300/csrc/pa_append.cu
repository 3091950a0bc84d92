// Appending new tokens to a paged cache with the position rotation applied on
// the way, the 4-bit cache's write, and reading a 4-bit cache back.
//
// Rotation: with (cos_i, sin_i) = row `position` of the caller's table, the
// pair (a, b) of a query or key row becomes
//   a' = a cos_i - b sin_i,   b' = b cos_i + a sin_i
// in fp32, each product and each sum rounded separately (so that a quantised
// cache's codes do not depend on how a compiler fuses them).  Pair i is dims
// (i, i + rot / 2), or (2i, 2i + 1) when interleaved; dims at and past rot are
// copied.  The rotated query is rounded to its 16-bit type once; the rotated
// key is rounded (16-bit cache) or quantised (FP8, 4-bit cache) once, from
// fp32.
//
// Bound: HBM.  Every q, k and v value is read once and written once, with six
// operations per pair between; the table rows (512 bytes per token at head_dim
// 128) are shared by a token's heads.  A CTA takes one token at a time (or a
// share of its head rows when there are few tokens), eight CTAs per SM stride
// over the tokens (as many as are resident for 16-bit and FP8 caches; the 4-bit
// kernel's 80 registers let six be resident, and the others follow); eight threads of 16 dims share a head row
// at head_dim 128.  Measured at 8192 tokens, 32/8 heads of 128, bf16: 35 us for
// 206 MB (5.9 TB/s, 0.87 of the measured copy rate); one CTA per token 37 us.
// Several rows' loads at once cost occupancy and were slower (two rows 36.2
// us, four 40.3), as were 64 or 256 threads (36.2, 43.7); the next row's loads
// in flight during this one's stores: 35.1.
#include <algorithm>

#include "pa_fp4.cuh"

namespace pa {

namespace {

constexpr int kAppendThreads = 128;
enum { kSame = 0, kFp8 = 1, kFp4 = 2 };

// Eight 16-bit values.  (Not through the read-only path: q may be rotated in place.)
template <typename T>
__device__ __forceinline__ uint4 raw8(const T* p) {
    return *reinterpret_cast<const uint4*>(p);
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = Elem<T>::to_float2(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]),
                                              Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7]));
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = f32x2_to_e4m3x2(__fmul_rn(x[2 * j], inv), __fmul_rn(x[2 * j + 1], inv));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// A thread's 16 dims of a head row are two runs of 8: d0.. and d1...  Rotated
// halves: run u of each half of the rotated part (the pairs are within the
// thread); interleaved or past the rotated part: 16 consecutive dims.  The
// 4-bit cache needs 16 consecutive dims (one scale group) whatever the pairs,
// so there a thread of a key row also reads its dims' partners.
template <typename T, int D, int kCache>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
    pdl_trigger();   // a following kernel that only reads inputs may overlap this one
    constexpr int U = D / 16;                       // threads per head row
    constexpr int kRows = kAppendThreads / U;       // head rows per pass
    const int u = threadIdx.x % U;
    const int half = p.rot / 2;
    const T* q = static_cast<const T*>(p.q);
    const T* key = static_cast<const T*>(p.key);
    const T* value = static_cast<const T*>(p.value);
    T* q_out = static_cast<T*>(p.q_out);
    const bool rotated = 16 * u < p.rot;            // this thread's dims are rotated
    const bool split = rotated && !p.interleaved;   // its pairs are half a rotated part apart
    const int d0 = split ? 8 * u : 16 * u;
    // head rows of a token: queries, then keys, then values
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int step = gridDim.y * kRows;
    const int d1 = split ? half + 8 * u : 16 * u + 8;
    for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
        for (int r = blockIdx.y * kRows + threadIdx.x / U; r < rows; r += step) {
            // the row's loads first: they do not wait for the token's position,
            // slot and table row
            const bool is_q = r < p.num_q_heads, is_v = r >= p.num_q_heads + p.num_kv_heads;
            const int h = is_q ? r : r - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
            const T* src = (is_q   ? q + static_cast<int64_t>(t) * p.q_stride
                            : is_v ? value + static_cast<int64_t>(t) * p.value_stride
                                   : key + static_cast<int64_t>(t) * p.key_stride) +
                           h * D;
            // a quantised group is 16 consecutive dims whatever the pairs
            const bool whole = kCache == kFp4 && !is_q;
            const uint4 w0 = raw8(src + (whole ? 16 * u : d0));
            const uint4 w1 = raw8(src + (whole ? 16 * u + 8 : d1));
            int64_t pos = 0;
            if (p.rot) {
                pos = __ldg(p.positions + t);
                if (pos < 0 || pos >= p.max_positions) {
                    // neither the query row nor the cache row is written
                    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(p.err, PA_DEVERR_POSITION_);
                    break;
                }
            }
            const int64_t slot = __ldg(p.slots + t);
            const bool in_pool = slot >= 0 && slot < p.num_slots;
            if (slot >= p.num_slots && threadIdx.x == 0 && blockIdx.y == 0) record_error(p.err, PA_DEVERR_SLOT_);
            float cs[8], sn[8];                         // of this thread's 8 pairs
            if (rotated) {
                const float* row = p.cos_sin + pos * p.rot + 8 * u;
                const float4 c0 = __ldg(reinterpret_cast<const float4*>(row));
                const float4 c1 = __ldg(reinterpret_cast<const float4*>(row + 4));
                const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + half));
                const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + half + 4));
                cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
                cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
                sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
                sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
            }
            auto rotate = [&](float (&a)[8], float (&b)[8]) {
                if (!p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) rotate_pair(a[j], b[j], cs[j], sn[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        rotate_pair(a[2 * j], a[2 * j + 1], cs[j], sn[j]);
                        rotate_pair(b[2 * j], b[2 * j + 1], cs[4 + j], sn[4 + j]);
                    }
                }
            };
            float a[8], b[8];
            widen8<T>(w0, a);
            widen8<T>(w1, b);
            if (is_q) {
                if (rotated) rotate(a, b);
                T* dst = q_out + static_cast<int64_t>(t) * p.q_out_stride + h * D;
                store8(dst + d0, a);
                store8(dst + d1, b);
                continue;
            }
            if (!in_pool) continue;
            void* pool = is_v ? p.v_cache : p.k_cache;
            const int64_t blk = slot >> 4;
            const int off = static_cast<int>(slot & 15);
            if constexpr (kCache != kFp4) {
                if (rotated && !is_v) rotate(a, b);
                if constexpr (kCache == kSame) {
                    T* dst = static_cast<T*>(pool) + (slot * p.num_kv_heads + h) * D;
                    store8(dst + d0, a);
                    store8(dst + d1, b);
                } else {
                    const float inv = is_v ? p.v_inv : p.k_inv;
                    uint8_t* dst = static_cast<uint8_t*>(pool) + ((blk * p.num_kv_heads + h) * 16 + off) * D;
                    *reinterpret_cast<uint2*>(dst + d0) = codes8(a, inv);
                    *reinterpret_cast<uint2*>(dst + d1) = codes8(b, inv);
                }
            } else {
                if (rotated && !is_v) {
                    if (p.interleaved) {
                        rotate(a, b);
                    } else {
                        // the partners of a split pair lie half a rotated part away
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int d = 16 * u + 8 * x;
                            const bool first = d < half;      // a' = a c - b s, else b' = b c + a s
                            const float* row = p.cos_sin + pos * p.rot + (first ? d : d - half);
                            float o[8];
                            widen8<T>(raw8(src + (first ? d + half : d - half)), o);
                            float(&y)[8] = x ? b : a;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float c = __ldg(row + j), s = __ldg(row + half + j);
                                const float yc = __fmul_rn(y[j], c), os = __fmul_rn(o[j], s);
                                y[j] = first ? __fsub_rn(yc, os) : __fadd_rn(yc, os);
                            }
                        }
                    }
                }
                const float inv = is_v ? p.v_inv : p.k_inv;
                float y[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = __fmul_rn(a[j], inv);
                    y[8 + j] = __fmul_rn(b[j], inv);
                }
                uint32_t lo, hi;
                uint8_t sc;
                quantise_group(y, lo, hi, sc);
                using Tile = Fp4Tile<D>;
                uint8_t* tile = static_cast<uint8_t*>(pool) + (blk * p.num_kv_heads + h) * Tile::kBytes;
                *reinterpret_cast<uint2*>(tile + off * Tile::kRow + 8 * u) = make_uint2(lo, hi);
                tile[Tile::scale_off(is_v, off, u)] = sc;
            }
        }
    }
}

// Whole blocks of a 4-bit cache as 16-bit rows [blocks, 16, Hkv, D]: code *
// group scale (exact) * pool scale, rounded to T.  One thread per group of 16
// dims, K and V in turn.
template <typename T, int D>
__global__ void __launch_bounds__(256) unpack_fp4_kernel(T* __restrict__ k_out, T* __restrict__ v_out,
                                                         const uint8_t* __restrict__ k_cache,
                                                         const uint8_t* __restrict__ v_cache, int64_t groups,
                                                         int num_kv_heads, float k_scale, float v_scale) {
    pdl_trigger();
    using Tile = Fp4Tile<D>;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < groups;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int u = static_cast<int>(i % Tile::kGroups);
        const int64_t row = i / Tile::kGroups;                 // (block, token, head)
        const int h = static_cast<int>(row % num_kv_heads);
        const int64_t bt = row / num_kv_heads;
        const int t = static_cast<int>(bt & 15);
        const int64_t off = ((bt >> 4) * num_kv_heads + h) * Tile::kBytes;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint8_t* tile = (v ? v_cache : k_cache) + off;
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(tile + t * Tile::kRow + 8 * u));
            uint32_t w[8];
            group_values(c.x, c.y, __ldg(tile + Tile::scale_off(v, t, u)), w);
            const float scale = v ? v_scale : k_scale;
            uint4* dst = reinterpret_cast<uint4*>((v ? v_out : k_out) + i * 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = Elem<__half>::to_float2(w[j]);
                w[j] = Elem<T>::pack(f.x * scale, f.y * scale);
            }
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

template <typename T, int D>
void append_t(const AppendParams& p, int cache, dim3 grid, cudaStream_t s) {
    if (cache == kSame) append_kernel<T, D, kSame><<<grid, kAppendThreads, 0, s>>>(p);
    else if (cache == kFp8) append_kernel<T, D, kFp8><<<grid, kAppendThreads, 0, s>>>(p);
    else append_kernel<T, D, kFp4><<<grid, kAppendThreads, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int head_dim, int dtype, int cache, cudaStream_t s) {
    if (p.num_tokens == 0) return cudaSuccess;
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int per_pass = kAppendThreads / (head_dim / 16);
    const int passes = (rows + per_pass - 1) / per_pass;
    const int gx = std::min(p.num_tokens, 8 * sm_count());   // (six of eight are resident over a 4-bit cache)
    // few tokens: a token's head rows are shared out over CTAs
    const int gy = std::max(1, std::min(passes, 8 * sm_count() / gx));
    const dim3 grid(gx, gy);
    if (dtype == 0) {
        if (head_dim == 128) append_t<__half, 128>(p, cache, grid, s);
        else append_t<__half, 64>(p, cache, grid, s);
    } else {
        if (head_dim == 128) append_t<__nv_bfloat16, 128>(p, cache, grid, s);
        else append_t<__nv_bfloat16, 64>(p, cache, grid, s);
    }
    return cudaGetLastError();
}

cudaError_t launch_unpack_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache, int num_blocks,
                              int num_kv_heads, int head_dim, int dtype, float k_scale, float v_scale,
                              cudaStream_t s) {
    const int64_t groups = static_cast<int64_t>(num_blocks) * 16 * num_kv_heads * (head_dim / 16);
    const int grid = static_cast<int>(std::min<int64_t>((groups + 255) / 256, 8LL * sm_count()));
    auto go = [&](auto tag, auto kern) {
        using T = decltype(tag);
        kern<<<grid, 256, 0, s>>>(static_cast<T*>(k_out), static_cast<T*>(v_out), static_cast<const uint8_t*>(k_cache),
                                  static_cast<const uint8_t*>(v_cache), groups, num_kv_heads, k_scale, v_scale);
    };
    if (dtype == 0) {
        if (head_dim == 128) go(__half{}, unpack_fp4_kernel<__half, 128>);
        else go(__half{}, unpack_fp4_kernel<__half, 64>);
    } else {
        if (head_dim == 128) go(__nv_bfloat16{}, unpack_fp4_kernel<__nv_bfloat16, 128>);
        else go(__nv_bfloat16{}, unpack_fp4_kernel<__nv_bfloat16, 64>);
    }
    return cudaGetLastError();
}

}  // namespace pa
