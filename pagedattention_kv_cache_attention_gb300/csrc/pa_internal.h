// pa_internal.h -- argument blocks and launchers shared by the library's
// translation units (not part of the public ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

namespace pa {

constexpr int kMaxDevices = 64;
constexpr int kSms = 152;  // of a GB300

// What the caches hold: fp16 / bf16 elements, E4M3 codes, or FP4 tiles (pa_fp4.cuh).
enum class Kv { k16, kFp8, kFp4 };

// Raises one kernel's dynamic shared-memory limit once per device.  Safe when
// several host threads make their first call at the same time: the attribute
// is set under a lock, and later calls only read an atomic flag.  Each
// launcher keeps one function-local static instance per kernel.
class SmemLimitOnce {
 public:
  template <typename Kern>
  cudaError_t ensure(Kern kern, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lk(mu_);
    if (!done_[dev].load(std::memory_order_relaxed)) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(bytes));
      if (e != cudaSuccess) return e;
      done_[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
  }

 private:
  std::atomic<bool> done_[kMaxDevices]{};
  std::mutex mu_;
};

struct DecodeArgs {
  void *out;                    // [B, Hq, D] (used when num_parts == 1)
  const void *query;            // [B, Hq, D]
  const int32_t *block_tables;  // [B, max_blocks_per_seq]
  const int32_t *context_lens;  // [B]
  int max_blocks_per_seq;
  int num_seqs, num_q_heads, num_kv_heads, group, bs_log2;
  int64_t num_blocks;
  float scale_log2;             // scale * log2(e) (times the K dequantisation scale for FP8)
  float out_scale;              // V dequantisation scale for FP8, 1 otherwise
  int max_context_len;
  int part_tokens;              // tokens per partition (>= max_context_len when not split)
  int num_parts;
  float *ws_m, *ws_l, *ws_o;    // split partials (num_parts > 1)
  unsigned *ws_cnt;             // join counters, one per (sequence, KV head) (num_parts > 1)
  int fuse_join;                // 1: the last partition CTA of a (sequence, KV head) joins
  unsigned *err;                // device error word
  // Shared-prefix decode (nullptr / unused otherwise).  prefix_lens [B]:
  // leading tokens of each sequence held in the same physical blocks as the
  // rest of its group; group_start [num_groups + 1]: the groups are runs of
  // consecutive sequences.
  const int32_t *prefix_lens;
  const int32_t *group_start;
  int num_groups, max_group_size;
  int members_per_cta, chunks;  // sequences per shared-prefix CTA, CTAs per group
  // A chunk of few rows over FP4 caches (launch_chunk_fp4; nullptr otherwise):
  // sequence i's rows start at query_start[i], as in PrefillArgs.
  const int32_t *query_start;
  int max_q_len;
  // CTAs of a cluster that share the keys of an unsplit call over FP4 caches
  int cluster;
  int by_length;  // FP4: CTAs take the longest contexts first (seq_by_length)
  // pa_decode_sparse: block_tables [B, Hkv, max_blocks_per_seq] and context_lens [B, Hkv].
  // (Read by pa_decode_fp4.cu, whose kernel takes both kinds; pa_decode_sparse.cu takes
  // no other.)
  int per_head;
};

struct ReduceArgs {
  void *out;
  const float *ws_m, *ws_l, *ws_o;
  const int32_t *context_lens;
  int num_seqs, num_q_heads, num_parts, partition_size, max_context_len;
  // tokens the block table can address (max_blocks_per_seq * block_size); a
  // longer context is treated as invalid exactly as the decode kernel treats
  // it (INT32_MAX when the partials do not come from pa_decode)
  int64_t table_tokens;
  int warps_per_row;            // 1, 2 or 4 warps join one row
  unsigned *err;
};

struct ReshapeArgs {
  // FP8 caches: elements are stored as E4M3 codes of x / scale
  bool to_fp8;
  int src_dtype;                     // fp16 / bf16 source rows when to_fp8
  float k_scale, v_scale;
  const void *key, *value;
  int64_t key_stride, value_stride;  // elements
  void *k_cache, *v_cache;
  const int64_t *slot_mapping;
  int num_tokens, num_kv_heads, head_dim, block_size;
  int64_t num_blocks;
  unsigned *err;
};

// The FP4 cache's write (key, value are read) and read-back (they are written).
struct Fp4CacheArgs {
  void *key, *value;
  int64_t key_stride, value_stride;  // elements
  void *k_cache, *v_cache;
  const int64_t *slot_mapping;
  int num_tokens, num_kv_heads, head_dim, bs_log2;
  int64_t num_blocks;
  float k_scale, v_scale;
  unsigned *err;
};

// The rotating writes (pa_rope.cuh).
struct RopeArgs {
  void *query_out;
  const void *query, *key, *value;
  int64_t query_out_stride, query_stride, key_stride, value_stride;  // elements
  void *k_cache, *v_cache;
  const int64_t *slot_mapping, *positions;
  const float *cos_sin;              // [max_position, rotary_dim]
  int64_t max_position;
  int num_tokens, num_q_heads, num_kv_heads, rotary_dim, interleaved, bs_log2;
  int64_t num_blocks;
  float k_scale, v_scale;            // FP8 and FP4 caches
  int group_log2;                    // threads that share a token, in rope_token_heads
  unsigned *err;
};

// Threads (a power of two, at most a CTA of 256) that share a token with `items`
// items of 16 elements, so that a thread has at most three of them where it can.
inline int rope_group_log2(int items) {
  int g = 5;
  while (g < 8 && items > 3 << g) ++g;
  return g;
}

// The bounds of a block's keys (pa_sparse.cu).
struct BoundsArgs {
  int8_t *bounds;               // [num_blocks, Hkv, 2, D]: largest, smallest
  float *bound_scales;          // [num_blocks, Hkv]
  const void *k_cache;
  const int32_t *block_tables, *context_lens;
  const int32_t *query_start;   // [B + 1], or nullptr: one new token a sequence
  int max_blocks_per_seq, num_seqs, num_kv_heads, bs_log2, max_q_len;
  int64_t num_blocks;
  unsigned *err;
};

struct SelectArgs {
  int32_t *tables;              // [rows, Hkv, num_selected]
  int32_t *lens;                // [rows, Hkv]
  const void *query;            // [rows, Hq, D]
  const int8_t *bounds;
  const float *bound_scales;
  const int32_t *block_tables, *context_lens;
  const int32_t *query_start;   // [B + 1], or nullptr: row i is sequence i
  int max_blocks_per_seq, num_seqs, max_q_len, num_q_heads, num_kv_heads, group, bs_log2;
  int64_t num_blocks;
  int max_context_len, num_selected, num_sink, num_recent;
  int cluster;                  // CTAs that may share a row's blocks
  int units_per_cta;            // at least, where they are more than one
  int max_candidates;           // blocks of the longest context
  unsigned *err;
};
// Blocks of one sequence that a selection can choose from: their keys lie in shared memory.
constexpr int64_t kMaxCandidates = 49152;

struct PrefillArgs {
  void *out;                    // [total_q, Hq, D]
  const void *query;            // [total_q, Hq, D]
  const int32_t *query_start;   // [B + 1]
  const int32_t *block_tables;  // [B, max_blocks_per_seq]
  const int32_t *context_lens;  // [B], the chunk included
  int max_blocks_per_seq;
  int num_seqs, num_q_heads, num_kv_heads, group, bs_log2, max_q_len;
  int64_t num_blocks;
  float scale_log2;             // scale * log2(e) (times the K dequantisation scale for FP8)
  float out_scale;              // V dequantisation scale for FP8 caches, 1 otherwise
  unsigned *err;
  // The shared-prefix pass (the same kernel over a group's shared prefix):
  // rows are (member, query head) pairs of a group's sequences, keys the
  // partition [p part_tokens, (p + 1) part_tokens) read through the first
  // taking member's table, and each taking member's rows are written as split
  // partials (m, l, o) into the decode workspace.  Unused by pa_prefill.
  float *ws_m, *ws_l, *ws_o;
  const int32_t *prefix_lens, *group_start;
  // (chunks: in the FP4 two-tile kernel, the CTAs of a cluster)
  int num_groups, max_group_size, members_per_cta, chunks;
  int part_tokens, num_parts, max_context_len;
  int by_length;  // FP4: CTAs take the longest contexts first (seq_by_length)
};

struct BlockCopyArgs {
  const void *src[2];           // per tensor: source pool (device or mapped host memory)
  void *dst[2];                 // per tensor: destination pool
  const int64_t *mapping;       // [num_pairs, 2] (source block, destination block)
  int num_pairs;
  int64_t block_bytes;          // bytes of one block (multiple of 16)
  int64_t src_blocks, dst_blocks;
  unsigned *err;
};

// Launch `kern` on `stream` as a programmatic dependent of the work before it:
// it may start while the previous kernel finishes, and must call
// griddepcontrol.wait before reading anything that kernel writes.
// launch_clusters: the same, in clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(int cluster, void (*kern)(KArgs...), dim3 grid, dim3 block,
                            size_t smem, cudaStream_t stream, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, Args &&...args) {
  return launch_clusters(1, kern, grid, block, smem, stream, static_cast<Args &&>(args)...);
}

// Largest partition size the shared-prefix kernel takes (its shared-memory
// table holds one pool row per 16-token sub-tile of a partition).
constexpr int kMaxSharedPrefixPartition = 8192;

// The pool viewed as a 2-D tensor [num_blocks * num_kv_heads * block_size
// rows, head_dim] for TMA loads of 16-row, 128-byte boxes (128-byte swizzle).
bool encode_pool_map(CUtensorMap *map, const void *pool, int64_t rows, int head_dim, int dtype,
                     bool fp8);

// An FP4 cache of `tiles` (block, head) tiles, viewed for TMA loads of whole tiles.
bool encode_fp4_map(CUtensorMap *map, const void *pool, int64_t tiles, int block_size,
                    int head_dim, bool swizzle);

// kv_fp8: the caches hold FP8 E4M3 codes (queries and output fp16).
cudaError_t launch_decode(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                          int64_t pool_rows, int head_dim, int dtype, bool kv_fp8,
                          cudaStream_t stream, bool *map_failed);
cudaError_t launch_decode_fp4(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                              int head_dim, int dtype, cudaStream_t stream, bool *map_failed);
// pa_decode_sparse over 16-bit and FP8 caches (launch_decode_fp4 takes a.per_head itself).
cudaError_t launch_decode_sparse(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                                 int64_t pool_rows, int head_dim, int dtype, bool kv_fp8,
                                 cudaStream_t stream, bool *map_failed);
// pa_prefill_fp4 on two 128-row tiles a CTA: chunks of more than 64 rows, or of
// fewer where there are few of them (maps of whole tiles, not swizzled).
cudaError_t launch_prefill_fp4(const PrefillArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                               int head_dim, int dtype, cudaStream_t stream);
// pa_prefill_fp4 for chunks of at most kMaxChunkRows (token, head) rows a KV head.
constexpr int kMaxChunkRows = 24;
// Tokens past a sequence's end whose indexes these two kernels form: two windows
// of 32 tiles of each warp, a tile or two to a 32-token step, the warps of up to
// kFp4Cluster CTAs taking the steps in turn (65,536 tokens at block size 32, 8,192
// where the CTAs are one).  Tables end that far below 2^31 tokens.
constexpr int64_t kFp4LookAhead = int64_t(1) << 17;
constexpr int kFp4Cluster = 8;
cudaError_t launch_chunk_fp4(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                             int head_dim, int dtype, cudaStream_t stream, bool *map_failed);
cudaError_t launch_reduce(const ReduceArgs &a, int head_dim, int dtype, cudaStream_t stream);
// The shared-prefix pass of pa_decode_shared_prefix (16-bit or FP8 caches);
// the decode launch with a.prefix_lens set follows it on the same stream.
cudaError_t launch_shared_prefix(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                                 int64_t pool_rows, int head_dim, int dtype, bool kv_fp8,
                                 cudaStream_t stream, bool *map_failed);
// Sequences of one group that a shared-prefix CTA serves at query group size G.
int shared_prefix_members_per_cta(int group);
cudaError_t launch_reshape(const ReshapeArgs &a, cudaStream_t stream);
cudaError_t launch_rope(const RopeArgs &a, int head_dim, int dtype, bool to_fp8,
                        cudaStream_t stream);
cudaError_t launch_rope_fp4(const RopeArgs &a, int head_dim, int dtype, cudaStream_t stream);
cudaError_t launch_key_bounds(const BoundsArgs &a, int head_dim, int dtype, Kv kv,
                              cudaStream_t stream);
cudaError_t launch_select(const SelectArgs &a, int head_dim, int dtype, cudaStream_t stream);
cudaError_t launch_cache_fp4_write(const Fp4CacheArgs &a, int dtype, cudaStream_t stream);
cudaError_t launch_cache_fp4_read(const Fp4CacheArgs &a, int dtype, cudaStream_t stream);
cudaError_t launch_block_copy(const BlockCopyArgs &a, int num_tensors, cudaStream_t stream);
cudaError_t launch_prefill(const PrefillArgs &a, const void *k_cache, const void *v_cache,
                           int64_t pool_rows, int head_dim, int dtype, Kv kv,
                           cudaStream_t stream, bool *map_failed);

// The host-side checks of pa_decode that come before the workspace check;
// returns a pa_status value (PA_OK when pa_decode would go on to the workspace).
int32_t decode_check_args(const void *out, const void *query, const void *k_cache,
                          const void *v_cache, const int32_t *block_tables,
                          int32_t max_blocks_per_seq, const int32_t *context_lens,
                          int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, int32_t block_size, int64_t num_blocks, float scale,
                          int32_t max_context_len, int32_t partition_size, int32_t dtype);

// One CTA waiting on a barrier nothing completes (the wait-limit self-test).
cudaError_t launch_selftest_wait(unsigned *err, cudaStream_t stream);

}  // namespace pa
