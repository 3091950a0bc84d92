// Internal (non-ABI) declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

// Device error word bits (mirrors the PA_DEVERR_* values of the public header).
#define PA_DEVERR_BLOCK_ID_ 1u
#define PA_DEVERR_SLOT_ 2u
#define PA_DEVERR_SEQ_LEN_ 4u
#define PA_DEVERR_TIMEOUT_ 8u
#define PA_DEVERR_WORKSPACE_ 16u
#define PA_DEVERR_POSITION_ 32u
#define PA_DEVERR_BEAM_ 64u

namespace pa {

// Launch `kern` with programmatic stream serialization: it may start before
// the preceding kernel of the stream has finished; it must call pdl_wait()
// before touching anything that kernel produces.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Rows of a varlen call whose chunk has 1..PA_VERIFY_MAX_Q_ queries (decode
// rows, speculative-verify rows) run in the decode kernel; longer chunks run
// in the prefill kernels.
#define PA_VERIFY_MAX_Q_ 8
// Cross attention's chunks are dealt out to the CTAs by their work in up to so many
// rounds, to so many CTAs at the most.
#define PA_DEAL_ROUNDS_ 8
#define PA_DEAL_CTAS_ 256


// Modified scores (all zero: none).  With raw = q . k:
//   s = cap > 0 ? cap * tanh(scale * raw / cap) : scale * raw
//   s += slope[q head] * (key position - query position)
//   visible: query position - window < key position <= query position
// `cap_in` and `cap_log2` take raw to s in log2 units: tanh(x) = 1 - 2 / (1 +
// e^2x), so s log2(e) = cap_log2 - 2 cap_log2 / (1 + 2^(raw * cap_in)).
struct ScoreMod {
    float cap_in;                 // 2 log2(e) scale / cap
    float cap_log2;               // cap * log2(e); 0: no cap
    int window;                   // 0: no window
    const float* slopes;          // [Hq] or nullptr
};

struct DecodeParams {
    void* out;                    // [T, Hq, D] (T = B without cu_q_lens)
    const void* q;                // [T, Hq, D]
    const int32_t* block_tables;  // [B, max_blocks]
    const int32_t* seq_lens;      // [B]
    const int32_t* cu_q_lens;     // [B+1] or nullptr (row b = sequence b, one query each)
    float* ws_m;                  // [max_rows, Hq, max_parts] running max (log2 units)
    float* ws_l;                  // [max_rows, Hq, max_parts] running sum
    float* ws_acc;                // [max_rows, Hq, max_parts, D] unnormalised accumulator
    int32_t* units;               // [B * max_parts] (sequence << 16 | partition) work list
    int32_t* unit_count;          // number of entries in `units`
    int32_t* work_counter;        // next work item to claim (reset by the plan kernel)
    int32_t* row_base;            // [B] first partials row of a split sequence
    int32_t* rows;                // [max_rows] (sequence << 3 | query index) of every partials row
    int32_t* row_count;           // number of entries in `rows` (header of the workspace)
    int32_t* split;               // varlen calls: CTAs that take chunks (header of the workspace)
    unsigned int* err;            // device error word
    int num_seqs;
    int max_blocks;
    int max_seq_len;
    int num_blocks;
    int num_q_heads;
    int num_kv_heads;
    int head_dim;
    int group;                    // num_q_heads / num_kv_heads
    int partition_tokens;         // multiple of 16
    int max_parts;                // ceil(max_seq_len / partition_tokens)
    int max_q;                    // largest chunk handled here (1..PA_VERIFY_MAX_Q_)
    int max_rows;                 // partials rows available in the workspace
    int num_rows;                 // rows of q and out (num_seqs without cu_q_lens)
    int col_chunks;               // chunks of 8 or 16 (query, head) columns per (unit, kv head)
    float scale_log2;             // scale * log2(e) (times the K dequantisation scale for FP8)
    float v_scale;                // V dequantisation scale (1 for 16-bit caches)
    // 1: the plan kernel has already run (launched on its own) and the decode
    // kernel is launched right after a prefill kernel that allows dependent
    // launch; everything the decode kernel reads completed before that
    // prefill kernel started, so it does not wait for it
    int overlap;
    const void* k_pool;           // 4-bit pools (read without tensor maps)
    const void* v_pool;
    ScoreMod mod;
};

struct PrefillParams {
    void* out;                    // [T, Hq, D]
    const void* q;                // [T, Hq, D]
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;     // [B+1]
    unsigned int* err;
    int num_seqs;
    int max_blocks;
    int max_seq_len;
    int num_blocks;
    int num_q_heads;
    int num_kv_heads;
    int group;
    int q_per_tile;               // queries per tile: rows = q_per_tile * group <= 128
    float scale_log2;             // scale * log2(e) (times the K dequantisation scale for FP8)
    float v_scale;                // V dequantisation scale (1 for 16-bit caches)
    // when *decode_units > 0 (decode rows will run next to this kernel), only
    // the first overlap_ctas CTAs take prefill work; the others leave their SMs
    const int32_t* decode_units;
    int overlap_ctas;
    int pair_cap;                 // pair-list capacity of the plan (num_tokens / 4 + num_seqs)
    ScoreMod mod;
    // non-null: the plan shares the SMs between chunks and decode rows by their
    // work and writes the number of CTAs that take chunks here; a key of a
    // decode row costs decode_weight key tiles of a query-tile pair
    int32_t* split;
    float decode_weight;
    int cross;                    // 1: cross attention (seq_lens count the keys, which every query sees)
};

// Cross attention of short rows (at most PA_VERIFY_MAX_Q_ queries a sequence).
struct CrossParams {
    void* out;                    // [T, Hq, D]
    const void* q;
    const int32_t* block_tables;  // [B, max_blocks]
    const int32_t* seq_lens;      // [B] keys of every sequence
    const int32_t* cu_q_lens;     // [B + 1], or nullptr: q_per_seq rows each
    unsigned int* err;
    int num_seqs;
    int num_rows;                 // T
    int q_per_seq;                // without cu_q_lens
    int max_q;                    // most queries of a sequence handled here
    int chunks_follow;            // 1: sequences of more than PA_VERIFY_MAX_Q_ queries are another kernel's
    int max_blocks;
    int max_len;
    int num_blocks;
    int num_q_heads;
    int num_kv_heads;
    int group;
    int col_chunks;               // chunks of 8 or 16 (query, head) columns
    float scale_log2;
    // 1: launched right behind a prefill kernel that allows dependent launch;
    // what this one reads was complete before that one started
    int overlap;
    int longest_first;            // 1: CTAs take the sequences in order of length
};

// Selection of the best continuations (see pa_beam.cu).
constexpr int kMaxBeams = 32, kMaxBeamOut = 64;
struct BeamSelectParams {
    float* out_scores;            // [S, k]
    int32_t* out_parents;
    int32_t* out_tokens;
    uint8_t* out_finished;        // or nullptr
    const void* logits;           // [S * W, V], row stride in elements
    const float* scores;          // [S, W]
    const uint8_t* finished;      // [S, W] or nullptr
    int64_t stride;
    int num_seqs, beams, vocab, k, end_token;
    int pieces;                   // of a row (beam_pieces)
    float2* sums;                 // [S * W, pieces]: largest logit, sum of the exponentials
    float* groups;                // [S * W, pieces, 8]: largest logit of every 512 bytes
};

// Reordering of beams: kinds of pool are runs of `run_bytes` per token, `runs`
// of them `run_stride` bytes apart, or whole blocks (token_bytes 0).
constexpr int kReorderLayers = 64;   // pools of one launch
struct BeamReorderParams {
    const int32_t* tables;        // [S * W, max_blocks]
    int32_t* tables_out;          // the same, or another array
    const int32_t* seq_lens;      // [S * W]
    const int32_t* parents;       // [S, W]
    unsigned int* err;
    int num_seqs, beams, max_blocks, num_blocks;
    int64_t block_bytes;
    int runs;
    int run_stride;               // bytes between the runs of a block
    int token_bytes;              // bytes of a token in a run; 0: the whole block
    int layers;                   // of this launch
    int first;                    // the launch that reports errors (and writes tables_out, if not in place)
    void* k[kReorderLayers];
    void* v[kReorderLayers];
};

// Rotation and cache write of new tokens; strides count elements between tokens.
struct AppendParams {
    void* q_out;
    const void* q;                // [T, Hq, D]
    const void* key;              // [T, Hkv, D]
    const void* value;
    void* k_cache;
    void* v_cache;
    const int64_t* positions;     // [T]
    const float* cos_sin;         // [max_positions, rot]: cos | sin
    const int64_t* slots;         // [T]
    int64_t q_out_stride, q_stride, key_stride, value_stride;
    int64_t num_slots;
    int num_tokens;
    int num_q_heads;
    int num_kv_heads;
    int max_positions;
    int rot;                      // rotated dims of a head (a multiple of 16), 0: none
    int interleaved;
    float k_inv, v_inv;           // 1 / pool scale (quantised caches)
    unsigned int* err;
};

// FP8 (E4M3) or 4-bit cache: the prefill chunks' blocks widened to a 16-bit copy in
// the workspace, which the tensor-core kernel reads like a 16-bit cache.  The
// plan lists each chunk whose copy fits (`chunk_seq`, with its first copy
// block in `chunk_base`); sequence b's block i goes to copy block
// chunk_base[k] + i, recorded in row b of `table` (-1: not loaded).
struct Fp8Copy {
    int32_t* hdr;                 // [0] chunks listed, [1] copy blocks in use
    int32_t* chunk_seq;           // [num_seqs]
    int32_t* chunk_base;          // [num_seqs]
    int32_t* table;               // [num_seqs, max_blocks] copy block ids (rows of listed chunks)
    void* k16;                    // [cap_blocks, 16, Hkv, D] of the query type
    void* v16;
    int cap_blocks;
    const void* k_codes;          // the caller's E4M3 pools [num_blocks, Hkv, 16, D], or 4-bit pools
    const void* v_codes;
    const int32_t* src_tables;    // the caller's block table [num_seqs, max_blocks]
    int src_num_blocks;
    int fp4;                      // 1: 4-bit pools
};

// Launchers (return cudaError_t of the launch).
cudaError_t launch_slot_mapping(int64_t* slots, const int32_t* block_tables, int max_blocks,
                                const int32_t* seq_lens, const int32_t* cu_q_lens, int num_seqs,
                                int num_tokens, int num_blocks, unsigned int* err, cudaStream_t s);
cudaError_t launch_kv_write(const void* key, const void* value, void* k_cache, void* v_cache,
                            const int64_t* slots, int num_tokens, int num_blocks, int num_kv_heads,
                            int head_dim, unsigned int* err, cudaStream_t s);
cudaError_t launch_decode(const DecodeParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          int head_dim, int dtype, cudaStream_t s);
// The work-list plan alone (for p.overlap launches, which skip it; `pdl`: it
// may start before the preceding kernel of the stream has finished).
cudaError_t launch_decode_plan(const DecodeParams& p, cudaStream_t s, bool pdl = false);
// The merge of split sequences' partials (nothing when no sequence can be split).
cudaError_t launch_decode_reduce(const DecodeParams& p, int head_dim, int dtype, cudaStream_t s);
// launch_decode with p.mod applied to the scores (16-bit cache).
cudaError_t launch_decode_mod(const DecodeParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              int head_dim, int dtype, cudaStream_t s);
// 4-bit cache (p.k_pool / p.v_pool).
cudaError_t launch_decode_fp4(const DecodeParams& p, int head_dim, int dtype, cudaStream_t s);
// cu[i] = i * per, i <= num_seqs
cudaError_t launch_uniform_rows(int32_t* cu, int num_seqs, int per, cudaStream_t s);
cudaError_t launch_cross(CrossParams p, const CUtensorMap& kmap, const CUtensorMap& vmap, int head_dim, int dtype,
                         cudaStream_t s);
// dtype: 0 fp16, 1 bf16, 2 fp32
int beam_pieces(int vocab, int dtype);   // pieces of a row of logits, 4 KB each
// CTAs of the cluster that takes a request in one launch without a workspace, or 0
int beam_cluster(int num_seqs, int beams, int vocab, int dtype);
cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, cudaStream_t s);
cudaError_t launch_beam_copy(const BeamReorderParams& p, cudaStream_t s);
cudaError_t launch_beam_tables(const BeamReorderParams& p, cudaStream_t s);   // in place, behind the copies
cudaError_t launch_widen_fp4(const Fp8Copy& c, const int32_t* seq_lens, int max_blocks, int num_kv_heads,
                             int head_dim, int dtype, cudaStream_t s);
// cache: 0 the 16-bit type of the tokens, 1 FP8 (E4M3, head-major), 2 4-bit.
cudaError_t launch_append(const AppendParams& p, int head_dim, int dtype, int cache, cudaStream_t s);
cudaError_t launch_unpack_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache, int num_blocks,
                              int num_kv_heads, int head_dim, int dtype, float k_scale, float v_scale,
                              cudaStream_t s);
int sm_count();
// FP8 (E4M3) cache, head_dim 128; q/out of `dtype`.
cudaError_t launch_decode_fp8(const DecodeParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              int dtype, cudaStream_t s);
cudaError_t launch_kv_write_fp8(const void* key, const void* value, void* k_cache, void* v_cache,
                                const int64_t* slots, int num_tokens, int num_blocks, int num_kv_heads,
                                int src_dtype, float k_inv_scale, float v_inv_scale, unsigned int* err,
                                cudaStream_t s);
// pairs: device int32 [num_pairs, 2] (source block, destination block).
cudaError_t launch_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int num_pairs, int num_blocks,
                               int64_t block_bytes, unsigned int* err, cudaStream_t s);
cudaError_t launch_kv_gather(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, int max_blocks, const int32_t* seq_lens,
                             const int32_t* cu_seq_lens, int num_seqs, int num_blocks, int64_t row_bytes,
                             int64_t head_major_row_bytes, int max_seq_len, unsigned int* err, cudaStream_t s);
// One-thread kernel whose bounded mbarrier wait runs out (records a timeout).
cudaError_t launch_wait_selftest(unsigned int* err, cudaStream_t s);
// tcgen05 prefill: groups of 1 to PA_MAX_GROUP q heads per kv head; q_per_tile = 128 / group.
// `plan` is device scratch of num_seqs + 1 + 2 * pair_cap int32 (the work list
// of query-tile pairs).  With `copy` (FP8 cache, head_dim 128) the plan also
// lists the chunks' copy blocks, a kernel widens them, and K and V come from
// the copy (4-bit cache likewise, head_dim 64 or 128): p.block_tables = copy->table, p.num_blocks = copy->cap_blocks,
// kmap / vmap over copy->k16 / v16.  `modified`: apply p.mod (no copy).
cudaError_t launch_prefill_tc(const PrefillParams& p, int32_t* plan, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, const CUtensorMap& qmap, int head_dim, int dtype,
                              int max_q_len, int num_tokens, const Fp8Copy* copy, bool modified, cudaStream_t s);

}  // namespace pa
