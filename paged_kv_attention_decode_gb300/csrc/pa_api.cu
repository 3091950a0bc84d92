// C ABI of libpagedattn.so: argument validation, tensor-map set-up, launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "pa_internal.h"
#include "pagedattn.h"

namespace {

// Device error word: kernels OR PA_DEVERR_* bits into it.
__device__ unsigned int g_pa_device_error;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
unsigned int* g_err_addr[kMaxDevices] = {};

unsigned int* error_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_err_addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_pa_device_error) != cudaSuccess) return nullptr;
        g_err_addr[dev] = static_cast<unsigned int*>(p);
    }
    return g_err_addr[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Tensor map over one pool [num_blocks * 16 token rows, Hkv, D] viewed as 4-D
// (64-element row piece, D/64 pieces, head, token slot); one box = one 64-dim
// half of the 16 rows of one (block, head), 128-byte swizzled.
bool make_kv_map(CUtensorMap* map, const void* base, int num_blocks, int num_kv_heads, int head_dim, int dtype) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(head_dim / 64), static_cast<cuuint64_t>(num_kv_heads),
                                static_cast<cuuint64_t>(num_blocks) * 16};
    const cuuint64_t strides[3] = {128, static_cast<cuuint64_t>(head_dim) * 2,
                                   static_cast<cuuint64_t>(num_kv_heads) * head_dim * 2};
    const cuuint32_t box[4] = {64, 1, 1, 16};   // one 64-dim half of a (block, head) tile
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                    const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Tensor map over one pool whose box is a whole (16-token block, head) tile:
// dims (64-element row piece, token slot, D/64 pieces, head) with strides
// Hkv*D*2, 128 B and D*2 bytes; one box {64, 16, D/64, 1} lands as
// [piece][token][128 B], 128-byte swizzled -- byte for byte what D/64 boxes
// of make_kv_map would write, in one TMA operation.
bool make_kv_map_block(CUtensorMap* map, const void* base, int num_blocks, int num_kv_heads, int head_dim,
                       int dtype) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(num_blocks) * 16, static_cast<cuuint64_t>(head_dim / 64),
                                static_cast<cuuint64_t>(num_kv_heads)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(num_kv_heads) * head_dim * 2, 128,
                                   static_cast<cuuint64_t>(head_dim) * 2};
    const cuuint32_t box[4] = {64, 16, static_cast<cuuint32_t>(head_dim / 64), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                    const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Tensor map over the query rows [T, Hq, D] viewed as 4-D (64-element row
// piece, D/64 pieces, q head, token); one box = one 64-dim half of the `group`
// heads of `q_per_tile` consecutive tokens, i.e. q_per_tile * group <= 128
// rows of 128 bytes whose row index is token * group + head.
bool make_q_map(CUtensorMap* map, const void* q, int num_tokens, int num_q_heads, int head_dim, int group,
                int q_per_tile, int dtype) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(head_dim / 64), static_cast<cuuint64_t>(num_q_heads),
                                static_cast<cuuint64_t>(num_tokens)};
    const cuuint64_t strides[3] = {128, static_cast<cuuint64_t>(head_dim) * 2,
                                   static_cast<cuuint64_t>(num_q_heads) * head_dim * 2};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(q_per_tile)};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                    const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Tensor map over a head-major FP8 pool [num_blocks, Hkv, 16 token rows, 128
// codes]: one box = the 16 rows of one (block, head), a contiguous 2 KB run,
// landing as 16 rows of 128 bytes, 128-byte swizzled.
bool make_kv_map_fp8(CUtensorMap* map, const void* base, int num_blocks, int num_kv_heads) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {128, 16, static_cast<cuuint64_t>(num_kv_heads), static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t strides[3] = {128, 16 * 128, static_cast<cuuint64_t>(num_kv_heads) * 16 * 128};
    const cuuint32_t box[4] = {128, 16, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
size_t align256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

constexpr int kMaxGrid = 65535;
static_assert(PA_MAX_BEAMS == pa::kMaxBeams && PA_MAX_BEAM_OUT == pa::kMaxBeamOut, "one limit");
// Share of the SMs the tcgen05 prefill keeps while decode rows run beside it.
#ifndef PA_OVERLAP_NUM
#define PA_OVERLAP_NUM 1
#endif
#ifndef PA_OVERLAP_DEN
#define PA_OVERLAP_DEN 4
#endif
constexpr int kOverlapPrefillNum = PA_OVERLAP_NUM;
constexpr int kOverlapPrefillDen = PA_OVERLAP_DEN;
// Over an FP8 cache the decode rows cost less (half the bytes) while the
// chunks cost the same (the kernel reads their 16-bit copy).
#ifndef PA_OVERLAP_NUM_FP8
#define PA_OVERLAP_NUM_FP8 1
#endif
#ifndef PA_OVERLAP_DEN_FP8
#define PA_OVERLAP_DEN_FP8 4
#endif
constexpr int kOverlapPrefillNumFp8 = PA_OVERLAP_NUM_FP8;
constexpr int kOverlapPrefillDenFp8 = PA_OVERLAP_DEN_FP8;
constexpr int kMaxPoolBlocks = (1 << 27) - 1;  // token-row coordinate stays below 2^31

int check_shape(int num_q_heads, int num_kv_heads, int head_dim, int block_size, int dtype, int num_blocks) {
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (block_size != PA_BLOCK_SIZE) return PA_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > kMaxGrid) return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads) return PA_ERR_INVALID_ARG;
    if (num_q_heads / num_kv_heads > PA_MAX_GROUP) return PA_ERR_UNSUPPORTED;
    if (num_blocks <= 0 || num_blocks > kMaxPoolBlocks) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

int parts_for(int max_seq_len, int partition) {
    return max_seq_len > 0 ? (max_seq_len + partition - 1) / partition : 1;
}

// partition_size 0: PA_DEFAULT_PARTITION tokens, doubled (up to
// PA_MAX_AUTO_PARTITION) while a sequence of max_seq_len tokens would have more
// than PA_AUTO_MAX_PARTS partitions: long contexts then merge fewer partials
int effective_partition(int max_seq_len, int partition_size) {
    if (partition_size) return partition_size;
    int part = PA_DEFAULT_PARTITION;
    while (part < PA_MAX_AUTO_PARTITION && parts_for(max_seq_len, part) > PA_AUTO_MAX_PARTS) part *= 2;
    return part;
}

size_t partials_bytes(int num_seqs, int num_q_heads, int head_dim, int parts) {
    const size_t n = static_cast<size_t>(num_seqs) * num_q_heads * parts;
    return 2 * align256(n * sizeof(float)) + align256(n * head_dim * sizeof(float));
}

// Decode workspace:
//   [header 256 B: unit count @0, partials row count @64, work counter @128,
//    chunk CTAs of a varlen call @192]
//   [unit list: num_seqs * parts int32]
//   when parts > 1: [row_base: num_seqs int32][rows: max_rows int32][partials of max_rows rows]
size_t decode_ws_bytes(int num_seqs, int max_rows, int num_q_heads, int head_dim, int parts) {
    size_t b = 256 + align256(static_cast<size_t>(num_seqs) * parts * sizeof(int32_t));
    if (parts > 1)
        b += align256(static_cast<size_t>(num_seqs) * sizeof(int32_t)) +
             align256(static_cast<size_t>(max_rows) * sizeof(int32_t)) +
             partials_bytes(max_rows, num_q_heads, head_dim, parts);
    return b;
}

void carve_workspace(pa::DecodeParams& p, void* ws) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    p.unit_count = reinterpret_cast<int32_t*>(base);
    p.row_count = reinterpret_cast<int32_t*>(base + 64);
    p.work_counter = reinterpret_cast<int32_t*>(base + 128);
    p.split = reinterpret_cast<int32_t*>(base + 192);
    p.units = reinterpret_cast<int32_t*>(base + 256);
    base += 256 + align256(static_cast<size_t>(p.num_seqs) * p.max_parts * sizeof(int32_t));
    if (p.max_parts > 1) {
        p.row_base = reinterpret_cast<int32_t*>(base);
        base += align256(static_cast<size_t>(p.num_seqs) * sizeof(int32_t));
        p.rows = reinterpret_cast<int32_t*>(base);
        base += align256(static_cast<size_t>(p.max_rows) * sizeof(int32_t));
        const size_t n = static_cast<size_t>(p.max_rows) * p.num_q_heads * p.max_parts;
        p.ws_m = reinterpret_cast<float*>(base);
        p.ws_l = reinterpret_cast<float*>(base + align256(n * sizeof(float)));
        p.ws_acc = reinterpret_cast<float*>(base + 2 * align256(n * sizeof(float)));
    }
}

// Query rows of a varlen call that can need split-context partials: only
// chunks of at most PA_VERIFY_MAX_Q queries run in the decode kernel.
int verify_rows_bound(int num_seqs, int num_tokens) {
    const long long r = std::min<long long>(num_tokens, static_cast<long long>(num_seqs) * PA_VERIFY_MAX_Q);
    return static_cast<int>(r);
}

float scale_log2(float scale) { return scale * 1.4426950408889634f; }

// What the pools hold.
enum class Cache { k16, kFp8, kFp4 };

// Bytes of one 4-bit (block, kv head) tile: 16 rows of head_dim / 2 code bytes
// and head_dim / 16 group scales.
int fp4_tile_bytes(int head_dim) { return PA_BLOCK_SIZE * (head_dim / 2 + head_dim / 16); }

bool softcapped(const pa::ScoreMod& m) { return m.cap_log2 > 0.f; }

bool score_mod(pa::ScoreMod& m, float scale, float softcap, int window, const float* slopes) {
    if (!std::isfinite(softcap) || softcap < 0.f || window < 0) return false;
    m = pa::ScoreMod{};
    if (softcap > PA_SOFTCAP_MAX) return false;
    if (softcap > 0.f) {
        m.cap_in = 2.f * scale_log2(scale) / softcap;
        m.cap_log2 = scale_log2(softcap);
        // a cap so small that these leave fp32's normal range
        if (!std::isfinite(m.cap_in) || !std::isnormal(m.cap_log2)) return false;
    }
    m.window = window;
    m.slopes = slopes;
    return true;
}

}  // namespace

extern "C" {

int pa_version(void) { return 100; }

const char* pa_status_string(int status) {
    switch (status) {
        case PA_OK: return "PA_OK";
        case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
        case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
        case PA_ERR_WORKSPACE_TOO_SMALL: return "PA_ERR_WORKSPACE_TOO_SMALL";
        case PA_ERR_CUDA: return "PA_ERR_CUDA";
        default: return "PA_ERR_UNKNOWN";
    }
}

int pa_slot_mapping(int64_t* slot_mapping, const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* seq_lens, const int32_t* cu_q_lens, int num_seqs, int num_tokens,
                    int num_blocks, int block_size, void* stream) {
    if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
    if (block_size != PA_BLOCK_SIZE) return PA_ERR_UNSUPPORTED;
    if (num_blocks <= 0 || num_blocks > kMaxPoolBlocks) return PA_ERR_INVALID_ARG;
    if (!cu_q_lens && num_tokens != num_seqs) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!slot_mapping || !block_tables || !seq_lens) return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    cudaError_t e = pa::launch_slot_mapping(slot_mapping, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                                            num_seqs, num_tokens, num_blocks, err,
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_paged_kv_write(const void* key, const void* value, void* k_cache, void* v_cache,
                      const int64_t* slot_mapping, int num_tokens, int num_blocks, int num_kv_heads,
                      int head_dim, int block_size, int dtype, void* stream) {
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (block_size != PA_BLOCK_SIZE) return PA_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0 || num_blocks > kMaxPoolBlocks)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    cudaError_t e = pa::launch_kv_write(key, value, k_cache, v_cache, slot_mapping, num_tokens, num_blocks,
                                        num_kv_heads, head_dim, err, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_decode_partition(int max_seq_len, int partition_size) {
    if (max_seq_len < 0 || partition_size < 0 || partition_size % PA_BLOCK_SIZE) return -1;
    return effective_partition(max_seq_len, partition_size);
}

int pa_decode_partition_for(int num_seqs, int num_q_heads, int num_kv_heads, int max_seq_len) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_seq_len < 0 || num_q_heads % num_kv_heads)
        return -1;
    int part = effective_partition(max_seq_len, 0);
    if (max_seq_len <= 2 * PA_MIN_PARTITION) return part;   // one partition: no merge
    const int group = num_q_heads / num_kv_heads;
    const long long per_part = static_cast<long long>(num_seqs) * num_kv_heads * ((group + 15) / 16);
    // measured on the device, one partition length to the next: one sequence of
    // 4096 tokens, 32 heads, 4-bit: 128 tokens 16 us, 64 tokens 20 us; one of
    // 32768, 8 kv heads: 256 tokens 27 us, 128 tokens 38 us; eight of 32K-128K,
    // 8 kv heads: 1024 tokens 169 us, 2048 186 us, 512 183 us
    while (part > PA_MIN_PARTITION && per_part * parts_for(max_seq_len, part) < PA_PARTITION_ITEMS &&
           static_cast<long long>(part / 2) * (part / 2) >= 2LL * max_seq_len)
        part /= 2;
    return part;
}

size_t pa_decode_workspace_bytes(int num_seqs, int num_q_heads, int head_dim, int max_seq_len,
                                 int partition_size) {
    if (num_seqs <= 0 || num_q_heads <= 0 || head_dim <= 0 || max_seq_len < 0 || partition_size < 0) return 0;
    const int part = effective_partition(max_seq_len, partition_size);
    return decode_ws_bytes(num_seqs, num_seqs, num_q_heads, head_dim, parts_for(max_seq_len, part));
}

// Everything a decode launch needs, prepared and validated on the host.
struct DecodeCall {
    pa::DecodeParams p;
    CUtensorMap kmap, vmap;
    int head_dim, dtype;
    Cache cache;
    bool modified;
};

static int decode_prepare(DecodeCall& c, void* out, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                          const int32_t* cu_q_lens, int num_seqs, int max_seq_len, int num_blocks, float scale,
                          int num_q_heads, int num_kv_heads, int head_dim, int partition_size, void* workspace,
                          size_t workspace_bytes, int dtype, int max_q, int max_rows, int num_rows,
                          Cache cache = Cache::k16, float k_scale = 1.f, float v_scale = 1.f,
                          const pa::ScoreMod* mod = nullptr) {
    const int part = effective_partition(max_seq_len, partition_size);
    const int parts = parts_for(max_seq_len, part);
    if (parts > 65535) return PA_ERR_INVALID_ARG;   // partition index is a 16-bit field of the work list
    // (query, head) columns per work item: 8, or 16 once a row can have more
    // (8 over a 4-bit cache)
    const int cols = max_q * (num_q_heads / num_kv_heads);
    const int chunk = cols > 8 && cache != Cache::kFp4 ? 16 : 8;
    const int col_chunks = (cols + chunk - 1) / chunk;
    // the kernels count work items in 32 bits
    if ((mod || cache == Cache::kFp4) &&
        static_cast<long long>(num_seqs) * parts * num_kv_heads * col_chunks > (1LL << 30))
        return PA_ERR_INVALID_ARG;
    const size_t need = decode_ws_bytes(num_seqs, max_rows, num_q_heads, head_dim, parts);
    if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned256(workspace)) return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    const bool maps_ok =
        cache == Cache::kFp4   ? true
        : cache == Cache::kFp8 ? make_kv_map_fp8(&c.kmap, k_cache, num_blocks, num_kv_heads) &&
                                     make_kv_map_fp8(&c.vmap, v_cache, num_blocks, num_kv_heads)
                               : make_kv_map_block(&c.kmap, k_cache, num_blocks, num_kv_heads, head_dim, dtype) &&
                                     make_kv_map_block(&c.vmap, v_cache, num_blocks, num_kv_heads, head_dim, dtype);
    if (!maps_ok) return PA_ERR_CUDA;
    pa::DecodeParams& p = c.p;
    p = pa::DecodeParams{};
    p.out = out;
    p.q = q;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.err = err;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.num_blocks = num_blocks;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.group = num_q_heads / num_kv_heads;
    p.partition_tokens = part;
    p.max_parts = parts;
    p.max_q = max_q;
    p.max_rows = max_rows;
    p.num_rows = num_rows;
    p.col_chunks = col_chunks;
    p.scale_log2 = scale_log2(scale) * k_scale;
    p.v_scale = v_scale;
    p.k_pool = k_cache;
    p.v_pool = v_cache;
    if (mod) p.mod = *mod;
    carve_workspace(p, workspace);
    c.head_dim = head_dim;
    c.dtype = dtype;
    c.cache = cache;
    c.modified = mod != nullptr;
    return PA_OK;
}

static int decode_launch(const DecodeCall& c, cudaStream_t stream) {
    cudaError_t e = c.cache == Cache::kFp8   ? pa::launch_decode_fp8(c.p, c.kmap, c.vmap, c.dtype, stream)
                    : c.cache == Cache::kFp4 ? pa::launch_decode_fp4(c.p, c.head_dim, c.dtype, stream)
                    : c.modified ? pa::launch_decode_mod(c.p, c.kmap, c.vmap, c.head_dim, c.dtype, stream)
                                 : pa::launch_decode(c.p, c.kmap, c.vmap, c.head_dim, c.dtype, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

static int decode_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                       const int32_t* cu_q_lens, int num_seqs, int max_seq_len, int num_blocks, float scale,
                       int num_q_heads, int num_kv_heads, int head_dim, int partition_size, void* workspace,
                       size_t workspace_bytes, int dtype, cudaStream_t stream, int max_q, int max_rows,
                       Cache cache = Cache::k16, float k_scale = 1.f, float v_scale = 1.f,
                       const pa::ScoreMod* mod = nullptr) {
    DecodeCall c;
    const int rc = decode_prepare(c, out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                                  num_seqs, max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim,
                                  partition_size, workspace, workspace_bytes, dtype, max_q, max_rows, num_seqs, cache,
                                  k_scale, v_scale, mod);
    return rc ? rc : decode_launch(c, stream);
}

int pa_paged_attention_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                              int num_seqs, int max_seq_len, int num_blocks, float scale, int num_q_heads,
                              int num_kv_heads, int head_dim, int block_size, int partition_size,
                              void* workspace, size_t workspace_bytes, int dtype, void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || max_seq_len < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
    if (partition_size < 0 || partition_size % PA_BLOCK_SIZE) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return decode_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, nullptr, num_seqs,
                       max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim, partition_size,
                       workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), 1, num_seqs);
}

// Prefill workspace: [tile work list, 256-aligned][decode-row partials].
// prefill plan: offsets (num_seqs + 1), the cost-sorted pair list and each
// pair's sequence (pair_cap entries each, pair_cap = num_tokens / 4 +
// num_seqs).  A pair
// is two tiles of at least 2 queries (128 rows / at most PA_MAX_GROUP = 64
// heads), so a chunk of q queries has at most q / 4 + 1 pairs.
static_assert(PA_MAX_GROUP <= 64, "the plan's pair bound assumes tiles of at least 2 queries");
static size_t plan_bytes(int num_seqs, int num_tokens) {
    const size_t pairs = static_cast<size_t>(num_tokens) / 4 + static_cast<size_t>(num_seqs);
    return align256((static_cast<size_t>(num_seqs) + 1 + 2 * pairs) * sizeof(int32_t));
}

int pa_paged_kv_write_fp8(const void* key, const void* value, void* k_cache, void* v_cache,
                          const int64_t* slot_mapping, int num_tokens, int num_blocks, int num_kv_heads,
                          int head_dim, int block_size, int src_dtype, float k_scale, float v_scale, void* stream) {
    if (src_dtype != PA_F16 && src_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (block_size != PA_BLOCK_SIZE || head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0 || num_blocks > kMaxPoolBlocks)
        return PA_ERR_INVALID_ARG;
    if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    const float k_inv = 1.0f / k_scale;   // one fp32 division, as the quantiser's definition states
    const float v_inv = 1.0f / v_scale;
    cudaError_t e = pa::launch_kv_write_fp8(key, value, k_cache, v_cache, slot_mapping, num_tokens, num_blocks,
                                            num_kv_heads, src_dtype, k_inv, v_inv, err,
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_paged_attention_decode_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                  int num_seqs, int max_seq_len, int num_blocks, float scale, float k_scale,
                                  float v_scale, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                  int partition_size, void* workspace, size_t workspace_bytes, int dtype,
                                  void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_seqs > kMaxGrid || max_seq_len < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
    if (partition_size < 0 || partition_size % PA_BLOCK_SIZE) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return decode_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, nullptr, num_seqs,
                       max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim, partition_size,
                       workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), 1, num_seqs,
                       Cache::kFp8, k_scale, v_scale);
}

int pa_paged_attention_decode_fp4(void* out, const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                  int num_seqs, int max_seq_len, int num_blocks, float scale, float k_scale,
                                  float v_scale, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                  int partition_size, void* workspace, size_t workspace_bytes, int dtype,
                                  void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || max_seq_len < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
    if (partition_size < 0 || partition_size % PA_BLOCK_SIZE) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return decode_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, nullptr, num_seqs,
                       max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim, partition_size,
                       workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), 1, num_seqs,
                       Cache::kFp4, k_scale, v_scale);
}

int pa_paged_attention_decode_mod(void* out, const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                  int num_seqs, int max_seq_len, int num_blocks, float scale, float softcap,
                                  int window, const float* alibi_slopes, int num_q_heads, int num_kv_heads,
                                  int head_dim, int block_size, int partition_size, void* workspace,
                                  size_t workspace_bytes, int dtype, void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || max_seq_len < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
    if (partition_size < 0 || partition_size % PA_BLOCK_SIZE) return PA_ERR_INVALID_ARG;
    pa::ScoreMod mod;
    if (!std::isfinite(scale) || !score_mod(mod, scale, softcap, window, alibi_slopes)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return decode_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, nullptr, num_seqs,
                       max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim, partition_size,
                       workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), 1, num_seqs,
                       Cache::k16, 1.f, 1.f, &mod);
}

// Everything an append call does; `cache` says what the pools hold.
static int append_impl(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* key,
                       int64_t key_stride, const void* value, int64_t value_stride, void* k_cache, void* v_cache,
                       const int64_t* slot_mapping, const int64_t* positions, const float* cos_sin,
                       int max_positions, int num_tokens, int num_blocks, int num_q_heads, int num_kv_heads,
                       int head_dim, int rot_dim, int interleaved, int block_size, int dtype, void* stream,
                       Cache cache, float k_scale, float v_scale) {
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (block_size != PA_BLOCK_SIZE) return PA_ERR_UNSUPPORTED;
    if (head_dim != 128 && (head_dim != 64 || cache == Cache::kFp8)) return PA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_q_heads > kMaxGrid || num_kv_heads > kMaxGrid ||
        num_blocks <= 0 || num_blocks > kMaxPoolBlocks)
        return PA_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > head_dim || (interleaved != 0 && interleaved != 1)) return PA_ERR_INVALID_ARG;
    if (rot_dim % 16) return PA_ERR_UNSUPPORTED;
    if (rot_dim > 0 && max_positions <= 0) return PA_ERR_INVALID_ARG;
    if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
        return PA_ERR_INVALID_ARG;
    const float k_inv = 1.0f / k_scale, v_inv = 1.0f / v_scale;   // one fp32 division, as the definition states
    if (!std::isfinite(k_inv) || !std::isfinite(v_inv)) return PA_ERR_INVALID_ARG;
    // rows start on 16-byte boundaries and do not overlap within a token
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
    if (num_tokens > 1 && (key_stride < kv_row || value_stride < kv_row)) return PA_ERR_INVALID_ARG;
    if (num_tokens > 1 && num_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return PA_ERR_INVALID_ARG;
    if (key_stride % 8 || value_stride % 8 || (num_q_heads > 0 && (q_stride % 8 || q_out_stride % 8)))
        return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return PA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!positions || !cos_sin || !aligned16(cos_sin))) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    // in place only as a whole: a row that overlaps another row's source races
    if (num_q_heads > 0 && q == q_out && q_stride != q_out_stride && num_tokens > 1) return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    pa::AppendParams p{};
    p.q_out = q_out;
    p.q = q;
    p.key = key;
    p.value = value;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.slots = slot_mapping;
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.num_slots = static_cast<int64_t>(num_blocks) * PA_BLOCK_SIZE;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_positions = max_positions;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.k_inv = k_inv;
    p.v_inv = v_inv;
    p.err = err;
    const cudaError_t e = pa::launch_append(p, head_dim, dtype, static_cast<int>(cache),
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_paged_rope_kv_write(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* key,
                           int64_t key_stride, const void* value, int64_t value_stride, void* k_cache,
                           void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                           const float* cos_sin, int max_positions, int num_tokens, int num_blocks,
                           int num_q_heads, int num_kv_heads, int head_dim, int rot_dim, int interleaved,
                           int block_size, int dtype, void* stream) {
    if (rot_dim == 0) return PA_ERR_INVALID_ARG;
    return append_impl(q_out, q_out_stride, q, q_stride, key, key_stride, value, value_stride, k_cache, v_cache,
                       slot_mapping, positions, cos_sin, max_positions, num_tokens, num_blocks, num_q_heads,
                       num_kv_heads, head_dim, rot_dim, interleaved, block_size, dtype, stream, Cache::k16, 1.f, 1.f);
}

int pa_paged_rope_kv_write_fp8(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* key,
                               int64_t key_stride, const void* value, int64_t value_stride, void* k_cache,
                               void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                               const float* cos_sin, int max_positions, int num_tokens, int num_blocks,
                               int num_q_heads, int num_kv_heads, int head_dim, int rot_dim, int interleaved,
                               int block_size, int src_dtype, float k_scale, float v_scale, void* stream) {
    if (rot_dim == 0) return PA_ERR_INVALID_ARG;
    return append_impl(q_out, q_out_stride, q, q_stride, key, key_stride, value, value_stride, k_cache, v_cache,
                       slot_mapping, positions, cos_sin, max_positions, num_tokens, num_blocks, num_q_heads,
                       num_kv_heads, head_dim, rot_dim, interleaved, block_size, src_dtype, stream, Cache::kFp8,
                       k_scale, v_scale);
}

int pa_paged_rope_kv_write_fp4(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* key,
                               int64_t key_stride, const void* value, int64_t value_stride, void* k_cache,
                               void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                               const float* cos_sin, int max_positions, int num_tokens, int num_blocks,
                               int num_q_heads, int num_kv_heads, int head_dim, int rot_dim, int interleaved,
                               int block_size, int src_dtype, float k_scale, float v_scale, void* stream) {
    if (rot_dim == 0) return PA_ERR_INVALID_ARG;
    return append_impl(q_out, q_out_stride, q, q_stride, key, key_stride, value, value_stride, k_cache, v_cache,
                       slot_mapping, positions, cos_sin, max_positions, num_tokens, num_blocks, num_q_heads,
                       num_kv_heads, head_dim, rot_dim, interleaved, block_size, src_dtype, stream, Cache::kFp4,
                       k_scale, v_scale);
}

int pa_paged_kv_write_fp4_strided(const void* key, int64_t key_stride, const void* value, int64_t value_stride,
                                  void* k_cache, void* v_cache, const int64_t* slot_mapping, int num_tokens,
                                  int num_blocks, int num_kv_heads, int head_dim, int block_size, int src_dtype,
                                  float k_scale, float v_scale, void* stream) {
    return append_impl(nullptr, 0, nullptr, 0, key, key_stride, value, value_stride, k_cache, v_cache, slot_mapping,
                       nullptr, nullptr, 0, num_tokens, num_blocks, 0, num_kv_heads, head_dim, 0, 0, block_size,
                       src_dtype, stream, Cache::kFp4, k_scale, v_scale);
}

int pa_paged_kv_write_fp4(const void* key, const void* value, void* k_cache, void* v_cache,
                          const int64_t* slot_mapping, int num_tokens, int num_blocks, int num_kv_heads,
                          int head_dim, int block_size, int src_dtype, float k_scale, float v_scale, void* stream) {
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    return pa_paged_kv_write_fp4_strided(key, row, value, row, k_cache, v_cache, slot_mapping, num_tokens, num_blocks,
                                         num_kv_heads, head_dim, block_size, src_dtype, k_scale, v_scale, stream);
}

int pa_fp4_tile_bytes(int head_dim) { return head_dim == 64 || head_dim == 128 ? fp4_tile_bytes(head_dim) : 0; }

int pa_paged_kv_unpack_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache, int num_blocks,
                           int num_kv_heads, int head_dim, int block_size, float k_scale, float v_scale, int dtype,
                           void* stream) {
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (block_size != PA_BLOCK_SIZE || (head_dim != 64 && head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if (num_blocks < 0 || num_blocks > kMaxPoolBlocks || num_kv_heads <= 0 || num_kv_heads > kMaxGrid)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale)) return PA_ERR_INVALID_ARG;
    if (num_blocks == 0) return PA_OK;
    if (!k_out || !v_out || !k_cache || !v_cache) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    const cudaError_t e = pa::launch_unpack_fp4(k_out, v_out, k_cache, v_cache, num_blocks, num_kv_heads, head_dim,
                                                dtype, k_scale, v_scale, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Workspace of a varlen call whose decode and verify rows use partitions of
// `part` tokens.
static size_t varlen_ws_bytes(int num_seqs, int num_tokens, int num_q_heads, int head_dim, int max_seq_len, int part) {
    return plan_bytes(num_seqs, num_tokens) + decode_ws_bytes(num_seqs, verify_rows_bound(num_seqs, num_tokens), num_q_heads,
                                                  head_dim, parts_for(max_seq_len, part));
}

size_t pa_prefill_workspace_bytes(int num_seqs, int num_tokens, int num_q_heads, int head_dim, int max_seq_len) {
    if (num_seqs <= 0 || num_tokens < 0 || num_q_heads <= 0 || head_dim <= 0 || max_seq_len < 0) return 0;
    return varlen_ws_bytes(num_seqs, num_tokens, num_q_heads, head_dim, max_seq_len, effective_partition(max_seq_len, 0));
}

size_t pa_prefill_mod_workspace_bytes(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                      int max_seq_len) {
    if (num_seqs <= 0 || num_tokens < 0 || num_q_heads <= 0 || head_dim <= 0 || max_seq_len < 0) return 0;
    const int part = pa_decode_partition_for(num_seqs, num_q_heads, num_kv_heads, max_seq_len);
    return part > 0 ? varlen_ws_bytes(num_seqs, num_tokens, num_q_heads, head_dim, max_seq_len, part) : 0;
}

// FP8 varlen calls: after the 16-bit call's workspace, the chunks' 16-bit
// copy ([256 B header | chunk_seq | chunk_base | table | K copy | V copy],
// every part 256-byte aligned).  Copy blocks hold 16 rows of num_kv_heads *
// head_dim 16-bit values, for K and for V.
static size_t fp8_copy_fixed_bytes(int num_seqs, int max_blocks_per_seq) {
    return 256 + 2 * align256(static_cast<size_t>(num_seqs) * sizeof(int32_t)) +
           align256(static_cast<size_t>(num_seqs) * static_cast<size_t>(max_blocks_per_seq) * sizeof(int32_t));
}

static size_t fp8_copy_block_bytes(int num_kv_heads, int head_dim) {
    return 2 * static_cast<size_t>(PA_BLOCK_SIZE) * num_kv_heads * head_dim * 2;   // K and V
}

// The chunks' 16-bit copy of a varlen call over an FP8 or 4-bit cache.
static size_t chunk_copy_bytes(int num_seqs, int num_tokens, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                               int64_t chunk_kv_tokens) {
    // each chunk rounds its length up to whole blocks: at most one partial
    // block per chunk, and at most num_tokens / (PA_VERIFY_MAX_Q + 1) chunks
    const int64_t chunks = std::min<int64_t>(num_seqs, num_tokens / (PA_VERIFY_MAX_Q + 1));
    int64_t blocks = (chunk_kv_tokens + PA_BLOCK_SIZE - 1) / PA_BLOCK_SIZE + chunks;
    blocks = std::min<int64_t>(blocks, static_cast<int64_t>(num_seqs) * max_blocks_per_seq);
    blocks = std::min<int64_t>(blocks, kMaxPoolBlocks);
    return fp8_copy_fixed_bytes(num_seqs, max_blocks_per_seq) +
           static_cast<size_t>(blocks) * fp8_copy_block_bytes(num_kv_heads, head_dim);
}

size_t pa_prefill_fp8_workspace_bytes(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                      int head_dim, int max_seq_len, int max_blocks_per_seq,
                                      int64_t chunk_kv_tokens) {
    if (num_seqs <= 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_seq_len < 0 || max_blocks_per_seq <= 0 || chunk_kv_tokens < 0)
        return 0;
    return pa_prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, head_dim, max_seq_len) +
           chunk_copy_bytes(num_seqs, num_tokens, num_kv_heads, head_dim, max_blocks_per_seq, chunk_kv_tokens);
}

size_t pa_prefill_fp4_workspace_bytes(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                      int head_dim, int max_seq_len, int max_blocks_per_seq,
                                      int64_t chunk_kv_tokens) {
    if (num_kv_heads <= 0 || max_blocks_per_seq <= 0 || chunk_kv_tokens < 0) return 0;
    const size_t rows =
        pa_prefill_mod_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, max_seq_len);
    return rows ? rows + chunk_copy_bytes(num_seqs, num_tokens, num_kv_heads, head_dim, max_blocks_per_seq,
                                          chunk_kv_tokens)
                : 0;
}

// Everything a varlen call does, for either cache type; arguments are
// validated by the entry points.
static int prefill_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                        const int32_t* cu_q_lens, int num_seqs, int num_tokens, int max_q_len, int max_seq_len,
                        int num_blocks, float scale, int num_q_heads, int num_kv_heads, int head_dim,
                        void* workspace, size_t workspace_bytes, int dtype, cudaStream_t s, Cache cache,
                        float k_scale, float v_scale, const pa::ScoreMod* mod = nullptr) {
    // the chunks' work items are counted in 32 bits
    if ((mod || cache == Cache::kFp4) &&
        (static_cast<long long>(num_tokens) / 4 + num_seqs) * num_kv_heads > (1LL << 30))
        return PA_ERR_INVALID_ARG;
    const size_t pb = plan_bytes(num_seqs, num_tokens);
    // partitions of the decode and verify rows
    const int part = mod || cache == Cache::kFp4
                         ? pa_decode_partition_for(num_seqs, num_q_heads, num_kv_heads, max_seq_len)
                         : effective_partition(max_seq_len, 0);
    const size_t base_bytes = varlen_ws_bytes(num_seqs, num_tokens, num_q_heads, head_dim, max_seq_len, part);
    if (!workspace || workspace_bytes < base_bytes) return PA_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned256(workspace)) return PA_ERR_INVALID_ARG;
    // FP8 or 4-bit chunks: room for the 16-bit copy of at least one block
    const bool copied = cache != Cache::k16;
    pa::Fp8Copy copy{};
    if (copied && max_q_len > PA_VERIFY_MAX_Q) {
        const size_t fixed = fp8_copy_fixed_bytes(num_seqs, max_blocks_per_seq);
        const size_t per = fp8_copy_block_bytes(num_kv_heads, head_dim);
        if (workspace_bytes < base_bytes + fixed + per) return PA_ERR_WORKSPACE_TOO_SMALL;
        const size_t cap = std::min<size_t>((workspace_bytes - base_bytes - fixed) / per, kMaxPoolBlocks);
        uint8_t* c = static_cast<uint8_t*>(workspace) + base_bytes;
        copy.hdr = reinterpret_cast<int32_t*>(c);
        c += 256;
        copy.chunk_seq = reinterpret_cast<int32_t*>(c);
        c += align256(static_cast<size_t>(num_seqs) * sizeof(int32_t));
        copy.chunk_base = reinterpret_cast<int32_t*>(c);
        c += align256(static_cast<size_t>(num_seqs) * sizeof(int32_t));
        copy.table = reinterpret_cast<int32_t*>(c);
        c += align256(static_cast<size_t>(num_seqs) * static_cast<size_t>(max_blocks_per_seq) * sizeof(int32_t));
        copy.k16 = c;
        copy.v16 = c + cap * (per / 2);
        copy.cap_blocks = static_cast<int>(cap);
        copy.k_codes = k_cache;
        copy.v_codes = v_cache;
        copy.src_tables = block_tables;
        copy.src_num_blocks = num_blocks;
        copy.fp4 = cache == Cache::kFp4;
    }
    int32_t* plan = static_cast<int32_t*>(workspace);
    const int group = num_q_heads / num_kv_heads;
    // decode rows (q_len == 1) and speculative-verify rows (q_len <= PA_VERIFY_MAX_Q)
    // through the decode kernel
    const int max_q = std::max(1, std::min(max_q_len, PA_VERIFY_MAX_Q));
    DecodeCall dc;
    int rc = decode_prepare(dc, out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                            num_seqs, max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim, part,
                            static_cast<uint8_t*>(workspace) + pb, workspace_bytes - pb, dtype, max_q,
                            verify_rows_bound(num_seqs, num_tokens), num_tokens, cache, k_scale, v_scale, mod);
    if (rc) return rc;
    if (max_q_len <= PA_VERIFY_MAX_Q) return decode_launch(dc, s);
    unsigned int* err = error_word();
    pa::PrefillParams p{};
    p.out = out;
    p.q = q;
    p.block_tables = copied ? copy.table : block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.err = err;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.num_blocks = copied ? copy.cap_blocks : num_blocks;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.scale_log2 = scale_log2(scale) * k_scale;
    p.v_scale = v_scale;
    if (mod) p.mod = *mod;
    CUtensorMap kmap, vmap;
    // tiles of 128 / group queries (every supported grouping) on the tcgen05
    // tensor cores, running beside the decode rows: the decode plan and the
    // prefill kernel go first; the decode kernel then starts on the SMs the
    // prefill kernel leaves free.  K comes in one box per 64-dim half of a
    // block, V in one box per block, from the 16-bit cache or (FP8 or 4-bit
    // cache) from the chunks' 16-bit copy.
    const void* kc = copied ? copy.k16 : k_cache;
    const void* vc = copied ? copy.v16 : v_cache;
    if (!make_kv_map(&kmap, kc, p.num_blocks, num_kv_heads, head_dim, dtype) ||
        !make_kv_map_block(&vmap, vc, p.num_blocks, num_kv_heads, head_dim, dtype))
        return PA_ERR_CUDA;
    p.q_per_tile = 128 / group;
    p.pair_cap = num_tokens / 4 + num_seqs;
    CUtensorMap qmap;
    if (!make_q_map(&qmap, q, num_tokens, num_q_heads, head_dim, group, p.q_per_tile, dtype)) return PA_ERR_CUDA;
    if (pa::launch_decode_plan(dc.p, s) != cudaSuccess) return PA_ERR_CUDA;
    p.decode_units = dc.p.unit_count;
    p.overlap_ctas = std::max(1, copied ? pa::sm_count() * kOverlapPrefillNumFp8 / kOverlapPrefillDenFp8
                                     : pa::sm_count() * kOverlapPrefillNum / kOverlapPrefillDen);
    if (mod || cache == Cache::kFp4) {
        // SMs shared by work: a key tile of a pair (two 128 x 128 tiles) counts
        // as 2.0 us of one SM (capped scores 2.6 us); a key of a short row is
        // counted at an eighth of its own time (1.2 ns of 10 at 16 bits, 0.5 ns
        // of 5 at 4 bits), because the rows also run on the SMs that the chunks
        // leave at their end, and because chunks on few SMs slow down beside a
        // saturated memory.  Four chunks of 1536 beside 12, 60, 400, 2048 rows
        // (us): 4-bit 268, 291, 449, 1253; 16-bit with a distance bias 303,
        // 355, 740, 2693, with half as much weight again 308, 350, 721, 2687
        // (over other steps neither wins), with nine times as much, on earlier
        // kernels that took 323, 371, 770, 2818: 352, 469, 1593, 7403.
        // All of these are steps of 32/8 heads of 128.  col_chunks counts a verify
        // row's most columns, so a single query weighs 1, 4 and 8 at 1, 4 and 8
        // heads per kv head (4-bit) for the same bytes: with many heads the rows
        // get more of the SMs than by their own work.
        p.split = dc.p.split;
        p.decode_weight = (cache == Cache::kFp4 ? 0.5f : 1.2f) * dc.p.col_chunks / (mod && softcapped(*mod) ? 2600.f : 2000.f);
    }
    if (pa::launch_prefill_tc(p, plan, kmap, vmap, qmap, head_dim, dtype, max_q_len, num_tokens,
                              copied ? &copy : nullptr, mod != nullptr, s) !=
        cudaSuccess)
        return PA_ERR_CUDA;
    dc.p.overlap = 1;
    return decode_launch(dc, s);
}

int pa_paged_attention_prefill(void* out, const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                               const int32_t* cu_q_lens, int num_seqs, int num_tokens, int max_q_len,
                               int max_seq_len, int num_blocks, float scale, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, void* workspace, size_t workspace_bytes, int dtype,
                               void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_tokens < 0 || max_q_len < 0 || max_seq_len < 0 ||
        max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_q_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, num_seqs,
                        num_tokens, max_q_len, max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim,
                        workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), Cache::k16, 1.f, 1.f);
}

int pa_paged_attention_prefill_mod(void* out, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                   const int32_t* cu_q_lens, int num_seqs, int num_tokens, int max_q_len,
                                   int max_seq_len, int num_blocks, float scale, float softcap, int window,
                                   const float* alibi_slopes, int num_q_heads, int num_kv_heads, int head_dim,
                                   int block_size, void* workspace, size_t workspace_bytes, int dtype,
                                   void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_tokens < 0 || max_q_len < 0 || max_seq_len < 0 ||
        max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    pa::ScoreMod mod;
    if (!std::isfinite(scale) || !score_mod(mod, scale, softcap, window, alibi_slopes)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_q_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, num_seqs,
                        num_tokens, max_q_len, max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim,
                        workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), Cache::k16, 1.f, 1.f,
                        &mod);
}

int pa_paged_attention_prefill_fp4(void* out, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                   const int32_t* cu_q_lens, int num_seqs, int num_tokens, int max_q_len,
                                   int max_seq_len, int num_blocks, float scale, float k_scale, float v_scale,
                                   int num_q_heads, int num_kv_heads, int head_dim, int block_size, void* workspace,
                                   size_t workspace_bytes, int dtype, void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_tokens < 0 || max_q_len < 0 || max_seq_len < 0 ||
        max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_q_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, num_seqs,
                        num_tokens, max_q_len, max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim,
                        workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), Cache::kFp4, k_scale,
                        v_scale);
}

int pa_paged_attention_prefill_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                   const int32_t* cu_q_lens, int num_seqs, int num_tokens, int max_q_len,
                                   int max_seq_len, int num_blocks, float scale, float k_scale, float v_scale,
                                   int num_q_heads, int num_kv_heads, int head_dim, int block_size, void* workspace,
                                   size_t workspace_bytes, int dtype, void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_tokens < 0 || max_q_len < 0 || max_seq_len < 0 ||
        max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_q_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, num_seqs,
                        num_tokens, max_q_len, max_seq_len, num_blocks, scale, num_q_heads, num_kv_heads, head_dim,
                        workspace, workspace_bytes, dtype, static_cast<cudaStream_t>(stream), Cache::kFp8, k_scale,
                        v_scale);
}

// Cross attention's workspace, for chunks only: [rows of every sequence (without
// cu_q_lens) | tile plan, with the items dealt out behind its pair lists].
size_t pa_cross_workspace_bytes(int num_seqs, int num_tokens, int max_q_len) {
    if (num_seqs <= 0 || num_tokens < 0 || max_q_len <= PA_VERIFY_MAX_Q) return 0;
    return align256((static_cast<size_t>(num_seqs) + 1) * sizeof(int32_t)) + plan_bytes(num_seqs, num_tokens) +
           align256((1 + PA_DEAL_ROUNDS_ * PA_DEAL_CTAS_) * sizeof(int32_t));
}

int pa_paged_cross_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, int max_blocks_per_seq, const int32_t* enc_lens,
                             const int32_t* cu_q_lens, int num_seqs, int num_tokens, int max_q_len, int max_enc_len,
                             int num_blocks, float scale, int num_q_heads, int num_kv_heads, int head_dim,
                             int block_size, void* workspace, size_t workspace_bytes, int dtype, void* stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_blocks);
    if (rc) return rc;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_tokens < 0 || max_q_len < 0 || max_enc_len < 0 ||
        max_blocks_per_seq <= 0 || max_blocks_per_seq > kMaxPoolBlocks)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!cu_q_lens) {
        if (num_tokens % num_seqs) return PA_ERR_INVALID_ARG;
        max_q_len = num_tokens / num_seqs;
    }
    if (!out || !q || !k_cache || !v_cache || !block_tables || !enc_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    const size_t need = pa_cross_workspace_bytes(num_seqs, num_tokens, max_q_len);
    if (need) {
        if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned256(workspace)) return PA_ERR_INVALID_ARG;
    }
    const int group = num_q_heads / num_kv_heads;
    const int max_q = std::min(max_q_len, PA_VERIFY_MAX_Q);
    const int cols = std::max(1, max_q * group), chunk = cols > 8 ? 16 : 8;
    const int col_chunks = (cols + chunk - 1) / chunk;
    // CTAs (up to 8 an item) and query-tile pairs are counted in 32 bits
    if (static_cast<long long>(num_seqs) * num_kv_heads * col_chunks > (1LL << 27) ||
        (static_cast<long long>(num_tokens) / 4 + num_seqs) * num_kv_heads > (1LL << 30))
        return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap kbmap, vmap;   // one box per (block, head) tile
    if (!make_kv_map_block(&kbmap, k_cache, num_blocks, num_kv_heads, head_dim, dtype) ||
        !make_kv_map_block(&vmap, v_cache, num_blocks, num_kv_heads, head_dim, dtype))
        return PA_ERR_CUDA;
    pa::CrossParams c{};
    c.out = out;
    c.q = q;
    c.block_tables = block_tables;
    c.seq_lens = enc_lens;
    c.cu_q_lens = cu_q_lens;
    c.err = err;
    c.num_seqs = num_seqs;
    c.num_rows = num_tokens;
    c.q_per_seq = cu_q_lens ? 0 : max_q_len;
    c.max_q = max_q;
    c.max_blocks = max_blocks_per_seq;
    c.max_len = max_enc_len;
    c.num_blocks = num_blocks;
    c.num_q_heads = num_q_heads;
    c.num_kv_heads = num_kv_heads;
    c.group = group;
    c.col_chunks = col_chunks;
    c.scale_log2 = scale_log2(scale);
    if (max_q_len > PA_VERIFY_MAX_Q) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        const int32_t* cu = cu_q_lens;
        if (!cu) {
            int32_t* rows = reinterpret_cast<int32_t*>(ws);
            if (pa::launch_uniform_rows(rows, num_seqs, max_q_len, s) != cudaSuccess) return PA_ERR_CUDA;
            cu = rows;
        }
        pa::PrefillParams p{};
        p.out = out;
        p.q = q;
        p.block_tables = block_tables;
        p.seq_lens = enc_lens;
        p.cu_q_lens = cu;
        p.err = err;
        p.num_seqs = num_seqs;
        p.max_blocks = max_blocks_per_seq;
        p.max_seq_len = max_enc_len;
        p.num_blocks = num_blocks;
        p.num_q_heads = num_q_heads;
        p.num_kv_heads = num_kv_heads;
        p.group = group;
        p.scale_log2 = c.scale_log2;
        p.v_scale = 1.f;
        p.q_per_tile = 128 / group;
        p.pair_cap = num_tokens / 4 + num_seqs;
        p.cross = 1;
        CUtensorMap kmap, qmap;
        if (!make_kv_map(&kmap, k_cache, num_blocks, num_kv_heads, head_dim, dtype) ||
            !make_q_map(&qmap, q, num_tokens, num_q_heads, head_dim, group, p.q_per_tile, dtype))
            return PA_ERR_CUDA;
        int32_t* plan = reinterpret_cast<int32_t*>(ws + align256((static_cast<size_t>(num_seqs) + 1) * sizeof(int32_t)));
        if (pa::launch_prefill_tc(p, plan, kmap, vmap, qmap, head_dim, dtype, max_q_len, num_tokens, nullptr, false,
                                  s) != cudaSuccess)
            return PA_ERR_CUDA;
        if (!cu_q_lens) return PA_OK;   // every sequence is a chunk
        c.chunks_follow = 1;
        c.overlap = 1;
    }
    return pa::launch_cross(c, kbmap, vmap, head_dim, dtype, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}


size_t pa_beam_select_workspace_bytes(int num_seqs, int num_beams, int vocab, int num_out, int dtype) {
    if (num_seqs <= 0 || num_seqs > kMaxGrid || num_beams <= 0 || num_beams > PA_MAX_BEAMS || vocab <= 0 || vocab > PA_MAX_VOCAB ||
        num_out <= 0 || num_out > PA_MAX_BEAM_OUT || dtype < PA_F16 || dtype > PA_F32)
        return 0;
    if (pa::beam_cluster(num_seqs, num_beams, vocab, dtype)) return 0;
    const size_t n = static_cast<size_t>(num_seqs) * num_beams * pa::beam_pieces(vocab, dtype);
    return align256(n * sizeof(float2)) + n * 8 * sizeof(float);
}

int pa_beam_select(float* out_scores, int32_t* out_parents, int32_t* out_tokens, uint8_t* out_finished,
                   const void* logits, int64_t logits_stride, const float* scores, const uint8_t* finished,
                   int end_token, int num_seqs, int num_beams, int vocab, int num_out, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_F32) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_beams <= 0 || vocab <= 0 || num_out <= 0) return PA_ERR_INVALID_ARG;
    if (num_beams > PA_MAX_BEAMS || vocab > PA_MAX_VOCAB || num_out > PA_MAX_BEAM_OUT) return PA_ERR_UNSUPPORTED;
    if (num_out > static_cast<long long>(num_beams) * vocab) return PA_ERR_INVALID_ARG;
    if (end_token < -1 || end_token >= vocab || (finished && end_token < 0)) return PA_ERR_INVALID_ARG;
    if (logits_stride < vocab && num_seqs * num_beams > 1) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out_scores || !out_parents || !out_tokens || !logits || !scores) return PA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == PA_F32 ? 4 : 2)) return PA_ERR_INVALID_ARG;
    const size_t need = pa_beam_select_workspace_bytes(num_seqs, num_beams, vocab, num_out, dtype);
    if (need) {
        if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned256(workspace)) return PA_ERR_INVALID_ARG;
    }
    pa::BeamSelectParams p{};
    p.out_scores = out_scores;
    p.out_parents = out_parents;
    p.out_tokens = out_tokens;
    p.out_finished = out_finished;
    p.logits = logits;
    p.scores = scores;
    p.finished = finished;
    p.stride = logits_stride;
    p.num_seqs = num_seqs;
    p.beams = num_beams;
    p.vocab = vocab;
    p.k = num_out;
    p.end_token = end_token;
    p.pieces = pa::beam_pieces(vocab, dtype);
    const size_t n = static_cast<size_t>(num_seqs) * num_beams * p.pieces;
    if (n > (1u << 30)) return PA_ERR_INVALID_ARG;
    if (need) {
        p.sums = static_cast<float2*>(workspace);
        p.groups = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(n * sizeof(float2)));
    }
    return pa::launch_beam_select(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_beam_reorder(int32_t* tables_out, const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* seq_lens, const int32_t* parents, int num_seqs, int num_beams,
                    void* const* k_caches, void* const* v_caches, int num_layers, int num_blocks, int num_kv_heads,
                    int head_dim, int block_size, int cache_kind, void* stream) {
    if (block_size != PA_BLOCK_SIZE || num_beams > PA_MAX_BEAMS) return PA_ERR_UNSUPPORTED;
    if (cache_kind != PA_CACHE_16BIT && cache_kind != PA_CACHE_FP8 && cache_kind != PA_CACHE_FP4)
        return PA_ERR_UNSUPPORTED;
    if (head_dim != 128 && (head_dim != 64 || cache_kind == PA_CACHE_FP8)) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_seqs > kMaxGrid || num_beams <= 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > kMaxPoolBlocks || num_layers < 0 || num_blocks <= 0 || num_blocks > kMaxPoolBlocks ||
        num_kv_heads <= 0 || num_kv_heads > kMaxGrid)
        return PA_ERR_INVALID_ARG;
    // a request's table entries are counted in 32 bits
    if (static_cast<long long>(num_beams) * max_blocks_per_seq > (1LL << 30)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!tables_out || !block_tables || !seq_lens || !parents) return PA_ERR_INVALID_ARG;
    // in place as a whole, or apart
    const size_t bytes = static_cast<size_t>(num_seqs) * num_beams * max_blocks_per_seq * sizeof(int32_t);
    const uintptr_t a = reinterpret_cast<uintptr_t>(tables_out), b = reinterpret_cast<uintptr_t>(block_tables);
    if (a != b && a < b + bytes && b < a + bytes) return PA_ERR_INVALID_ARG;
    if (num_layers > 0 && (!k_caches || !v_caches)) return PA_ERR_INVALID_ARG;
    for (int i = 0; i < num_layers; ++i)
        if (!k_caches[i] || !v_caches[i] || !aligned16(k_caches[i]) || !aligned16(v_caches[i])) return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    pa::BeamReorderParams p{};
    p.tables = block_tables;
    p.tables_out = tables_out;
    p.seq_lens = seq_lens;
    p.parents = parents;
    p.err = err;
    p.num_seqs = num_seqs;
    p.beams = num_beams;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    if (cache_kind == PA_CACHE_FP4) {   // codes and scales of a token lie apart: whole tiles
        p.block_bytes = static_cast<int64_t>(num_kv_heads) * fp4_tile_bytes(head_dim);
    } else if (cache_kind == PA_CACHE_FP8) {
        p.block_bytes = static_cast<int64_t>(PA_BLOCK_SIZE) * num_kv_heads * head_dim;
        p.runs = num_kv_heads;
        p.run_stride = PA_BLOCK_SIZE * head_dim;
        p.token_bytes = head_dim;
    } else {
        p.block_bytes = static_cast<int64_t>(PA_BLOCK_SIZE) * num_kv_heads * head_dim * 2;
        p.runs = 1;
        p.token_bytes = num_kv_heads * head_dim * 2;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int first = 0; first == 0 || first < num_layers; first += pa::kReorderLayers) {
        p.first = first == 0;
        p.layers = std::min(num_layers - first, pa::kReorderLayers);
        for (int i = 0; i < p.layers; ++i) {
            p.k[i] = k_caches[first + i];
            p.v[i] = v_caches[first + i];
        }
        if (pa::launch_beam_copy(p, s) != cudaSuccess) return PA_ERR_CUDA;
    }
    if (tables_out == block_tables && pa::launch_beam_tables(p, s) != cudaSuccess) return PA_ERR_CUDA;
    return PA_OK;
}

int pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int num_pairs, int num_blocks,
                   int num_kv_heads, int head_dim, int elem_bytes, void* stream) {
    if (num_pairs < 0 || num_blocks <= 0 || num_blocks > kMaxPoolBlocks || num_kv_heads <= 0 || head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_ERR_UNSUPPORTED;
    const int64_t block_bytes = static_cast<int64_t>(PA_BLOCK_SIZE) * num_kv_heads * head_dim * elem_bytes;
    if (block_bytes % 16) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PA_OK;
    if (!k_cache || !v_cache || !pairs || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    cudaError_t e = pa::launch_copy_blocks(k_cache, v_cache, pairs, num_pairs, num_blocks, block_bytes, err,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_paged_kv_gather(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                       const int32_t* cu_seq_lens, int num_seqs, int max_seq_len, int num_blocks, int num_kv_heads,
                       int head_dim, int elem_bytes, void* stream) {
    if (num_seqs < 0 || num_seqs > kMaxGrid || max_seq_len < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
    if (num_blocks <= 0 || num_blocks > kMaxPoolBlocks || num_kv_heads <= 0 || head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_ERR_UNSUPPORTED;
    const int64_t row_bytes = static_cast<int64_t>(num_kv_heads) * head_dim * elem_bytes;
    if (row_bytes % 16) return PA_ERR_UNSUPPORTED;
    // FP8 pools are head-major: each head's row of head_dim codes is moved in 16-byte chunks
    const int64_t head_major_row_bytes = elem_bytes == 1 ? head_dim : 0;
    if (head_major_row_bytes % 16) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!k_out || !v_out || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_seq_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    cudaError_t e = pa::launch_kv_gather(k_out, v_out, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
                                         cu_seq_lens, num_seqs, num_blocks, row_bytes, head_major_row_bytes,
                                         max_seq_len, err,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_selftest_wait_timeout(void* stream) {
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    return pa::launch_wait_selftest(err, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_get_device_error(int* code, int clear, void* stream) {
    if (!code) return PA_ERR_INVALID_ARG;
    unsigned int* err = error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int v = 0;
    if (cudaMemcpyAsync(&v, err, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess) return PA_ERR_CUDA;
    if (clear && cudaMemsetAsync(err, 0, sizeof v, s) != cudaSuccess) return PA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return PA_ERR_CUDA;
    *code = static_cast<int>(v);
    return PA_OK;
}

}  // extern "C"
