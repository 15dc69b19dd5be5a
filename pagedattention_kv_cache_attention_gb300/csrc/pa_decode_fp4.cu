// pa_decode_fp4.cu -- paged decode attention over the FP4 cache (pa_decode_fp4).
//
// For each sequence i and query head h (format and exactness: pa_fp4.cuh)
//   out = sum_j softmax_j(scale q . K_j) V_j,   j < context_lens[i],
//   K_j = k_scale s e2m1(code), V_j alike, through the block table.
//
// How:
//  * One CTA per (KV head, sequence, partition) serves all G query heads of
//    the KV head, so a tile leaves HBM once per group.  Its warps take 32-token
//    steps in turn, each with its own ring of S shared-memory stages.
//  * A tile (codes and scales of one block and head, 9 or 18 lines of head_dim
//    bytes) is one 2-D TMA copy with the swizzle of its line length, so that
//    both products read shared memory without conflicts.
//  * S^T[16 tokens, 8 heads] = K Q^T on mma.sync m16n8k16.  A lane reads 16
//    (or 8) bytes of a K row, which lie within one or two scale groups:
//    cvt.f16x2.e2m1x2 makes fp16 pairs of a byte and one fp16x2 product with
//    the group's scale makes them exact values of the cache.
//  * O^T[d, 8 heads] += V^T P^T.  A lane reads the same 16 (or 8) dimensions of
//    four tokens; two tokens' nibbles are merged into bytes by three logical
//    instructions for eight codes, so that a converted pair is already (token,
//    next token) of one dimension, and its scale pair is shared by the lane's
//    dimensions.
//  * fp32 online softmax in base 2 against a reference, a score of the row, that
//    moves only when another's probability passes it by more than 2^4.  While the
//    reference's logit is small, a probability's exponent is one fma of the score;
//    a reference with a large logit is taken off the score first, since the fma
//    alone may be off by more than fp16's range (pa_fp4.cuh).  P is carried as fp16
//    (11 bits; the output has at most 11) times 2^11, so that only probabilities
//    below 2^-25 of the maximum lose bits and below 2^-35 vanish: a long context's
//    faint tail keeps its mass.
//  * Tokens that must not count get logit -inf and a V scale of zero; a code is
//    always finite, so nothing a masked slot holds (NaN scales among it)
//    reaches the output.
// What bounds it: the latency between a step's instructions, and CTAs of unequal
// length.  A warp's 32-token step is about 650 instructions in a few chains; with
// 14 warps an SM they fill 45 to 57 % of the issue slots.  Measured, 64 sequences
// of 512 to 4,096 tokens, 32 query / 8 KV heads, head_dim 128, fp16, 1,024-token
// partitions: 41 to 46 us for 161 MB by the lengths drawn (3.5 to 3.9 TB/s; bytes
// alone 24 us, instructions alone some 20); 256 sequences of up to 16,384, 64
// query heads, bf16: 109 to 117 us, 4.6 to 5.0 TB/s; 8 of 32,768 to 131,072,
// 512-token partitions: 97.5 us, 4.65 TB/s; unsplit, 256 sequences of 512 to 4,096,
// 32 / 8 heads, fp16: 126 us (floor 101); a chunk of 5 tokens x 4 heads for the
// first batch: 63 to 75 us, its three row tiles' chain of latencies at two CTAs
// an SM.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"
#include "pa_join.cuh"
#include "pa_tile.cuh"

namespace pa {

namespace {

#ifndef PA_DECODE_FP4_WARPS
#define PA_DECODE_FP4_WARPS 4
#endif
#ifndef PA_DECODE_FP4_STAGES
#define PA_DECODE_FP4_STAGES 2
#endif
#ifndef PA_DECODE_FP4_CTAS
#define PA_DECODE_FP4_CTAS 4
#endif
#ifndef PA_CHUNK_FP4_CTAS2
#define PA_CHUNK_FP4_CTAS2 3
#endif

// P is held times 2^11, against a reference that is at most 2^4 below the
// running maximum: below 2^15 then, and in fp16's normal range down to 2^-25 of
// the maximum.
constexpr float kPShift = 11.f, kGrowth = 4.f;
constexpr float kFar = kFp4FarLogit;

// Geometry of a tile in shared memory.  TMA brings it in lines of D bytes (the
// codes of two tokens; 9 lines for 16 tokens, the last of them scales) with the
// swizzle of that line length: byte address bits 4.. ^= bits 7.. (three bits at
// 128-byte lines, two at 64).  Rows 8 apart, and the two 16-token tiles of a
// 32-token unit (which start 12 lines apart), differ by half a swizzle period:
// their addresses are the same but for an offset and an XOR with kHalf.  So an
// address is one of two values of the lane (its offset, or that XOR kHalf) and
// a constant.
template <int D, int BS> struct Fp4Shape {
  static constexpr int kRow = D / 2;                     // bytes of a token's codes
  static constexpr int kScales = D / 16;                 // bytes of a token's scales
  static constexpr int kHalf = D / 2;
  static constexpr int kSlot16 = 12 * D;
  static constexpr int kUnit = 2 * kSlot16;              // 32 tokens of K or V
  static constexpr int kTiles = 32 / BS;                 // tiles of a unit
  static constexpr int kLines = BS * 9 / 16;             // lines of a tile
  static constexpr int kTileBytes = fp4_tile_bytes(BS, D);
  static constexpr int kMTiles = D / 16;
  static constexpr int kQChunks = D / 32;
};

// The lane's offset `at` (a byte of the codes of a row below 8 of a unit's
// first half), or of the unit's half h and 8 up rows on.  (at_x = at ^ kHalf)
template <int D, int BS>
__device__ __forceinline__ int code_place(int at, int at_x, int h, int up) {
  using Sh = Fp4Shape<D, BS>;
  return BS == 16 ? ((h ^ up) ? at_x : at) + h * Sh::kSlot16 + up * 8 * Sh::kRow
                  : (up ? at_x : at) + (16 * h + 8 * up) * Sh::kRow;
}
// The same for a scale byte (at: row * kScales + group, row below 8).  The
// scales of a 32-token tile's second half lie in a line of their own at 128
// bytes, whose swizzle flips unit 0.
template <int D, int BS> __device__ __forceinline__ int scale_place(int at, int h, int up) {
  using Sh = Fp4Shape<D, BS>;
  if constexpr (BS == 16)
    return at + 16 * Sh::kRow + h * Sh::kSlot16 + ((h ^ up) ? Sh::kHalf : 0);
  else
    return (D == 128 && h ? at ^ 16 : at) + (32 * Sh::kRow + (16 * h + 8 * up) * Sh::kScales);
}

// Row of a 16-token half that MMA row r stands for: a permutation that puts
// the four V rows 2c (c = 0..3) into different banks.
template <int D> __device__ __forceinline__ int token_of(int r) {
  return D == 128 ? r ^ ((r >> 1) & 1) : r ^ ((r >> 2) & 1);
}
// Byte `b` of the codes of token r in a half, in the swizzle of its lines.
template <int D> __device__ __forceinline__ int code_at(int r, int b) {
  const int at = r * (D / 2) + b;
  return at ^ (((at >> 7) & (D == 128 ? 7 : 3)) << 4);
}

// A warp's accumulators laid out in shared memory, 8 columns of kAccStride
// floats, so that the 32 lanes of each store write 32 banks (lane row g holds
// dimensions D/8 g .. D/8 g + D/8 - 1 of columns 2c and 2c + 1: in their own
// order a store would hit two banks).
template <int D> constexpr int kAccHalf = D / 2 + 8;       // from a first half-row to its second
template <int D> constexpr int kAccStride = D + 12;
template <int D> __device__ __forceinline__ int acc_place(int d) {  // of dimension d in a column
  const int g = d / (D / 8), r = d % (D / 8), mt = r % (D / 16);
  return (r >= D / 16 ? kAccHalf<D> : 0) + mt * 8 + g;
}
template <int D>
__device__ __forceinline__ void put_acc(float *dst, const float (&acc)[D / 16][4], float s0,
                                        float s1, int g, int c) {
  float *d0 = dst + 2 * c * kAccStride<D> + g, *d1 = d0 + kAccStride<D>;
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    d0[mt * 8] = acc[mt][0] * s0;
    d1[mt * 8] = acc[mt][1] * s1;
    d0[kAccHalf<D> + mt * 8] = acc[mt][2] * s0;
    d1[kAccHalf<D> + mt * 8] = acc[mt][3] * s1;
  }
}

enum class Rows { kDecode, kDecodeWarps, kWhole, kChunk };

// CTAs that share an SM: 16, 12 or 8 warps in all, by the accumulators that a
// thread holds (32, 64 or 96 registers at head_dim 128).
constexpr int ctas_per_sm(int tiles) {
  return tiles == 1 ? PA_DECODE_FP4_CTAS : tiles == 2 ? PA_CHUNK_FP4_CTAS2 : 2;
}

// T: query and output type.  NW warps, S stages each.  What the 8 NT columns of
// the products are:
//  kDecode       the heads of one query (NT = 1); the warps share a partition,
//                and the last CTA of a row joins them
//  kDecodeWarps  the same, but each warp takes a whole partition and writes its
//                partial itself (partitions joined by the reduce kernel), as in
//                the 16-bit kernel
//  kWhole        the heads of one query over its whole context, no partitions
//  kChunk        the rows of a short chunk, (token, head) pairs with token = row /
//                G, at most 8 NT of them
// In a call without partitions (kWhole, kChunk) the warps of a.cluster CTAs share
// the keys, and the CTAs join through one another's shared memory: a long context
// then takes a cluster's time and not a CTA's, and CTAs of unequal contexts fill
// the SMs more evenly.
template <typename T, int D, int BS, int NW, int S, Rows ROWS, int NT>
__global__ void __launch_bounds__(NW * 32, ctas_per_sm(NT))
    pa_decode_fp4_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const DecodeArgs a) {
  using Sh = Fp4Shape<D, BS>;
  constexpr bool WP = ROWS == Rows::kDecodeWarps, kChunk = ROWS == Rows::kChunk;
  constexpr bool kParts = ROWS == Rows::kDecode || WP;  // a context is cut into partitions
  const int cluster = kParts ? 1 : a.cluster;
  static_assert(kChunk || NT == 1, "a decode query's heads are one tile of columns");
  constexpr int kStep = 2 * Sh::kUnit;  // K then V of a 32-token step
  constexpr int kTiles = Sh::kTiles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NW * S * kStep);

  const int kvh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kParts ? 0 : static_cast<int>(blockIdx.x) % cluster;  // in the cluster
  const int part = WP ? blockIdx.x * NW + warp : kParts ? blockIdx.x : 0;
  if (WP && part >= a.num_parts) return;  // the last CTA's spare warps
  const int g = lane >> 2, c = lane & 3;
  uint8_t *my_stages = smem + warp * S * kStep;
  uint64_t *my_bars = bars + warp * S;
  // kChunk: NaNs of V at keys that not every row attends to: zeros in the
  // products, so that they do not reach the rows before them, and put back at
  // the end.  [warp][group]: the least such key, from the chunk's first token on.
  int *nan_key = reinterpret_cast<int *>(bars + NW * S);
  if (kChunk && lane < 8) nan_key[warp * 8 + lane] = 0x7fffffff;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(&my_bars[s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dependency_wait();  // the pool may come from the kernel before
  int place = blockIdx.z;
  if constexpr (!kParts) {
    if (a.by_length) {
      int *at = nan_key + NW * 8;
      if (warp == 0) {
        place = seq_by_length(a.context_lens, a.num_seqs, place, lane);
        if (lane == 0) *at = place;
      }
      __syncthreads();
      place = *at;
    }
  }
  const int seq = place;

  // Steps are 32-token windows of the sequence from the one that holds the
  // partition's first token on: a block never straddles two.  A warp's tiles
  // are numbered l in its own order; 32 lanes hold a window of 32 of them.
  const int t_begin = kParts ? part * a.part_tokens : 0;
  const int base = t_begin & ~31;
  const int64_t table = a.per_head ? static_cast<int64_t>(seq) * a.num_kv_heads + kvh : seq;
  const int32_t *bt_row = a.block_tables + table * a.max_blocks_per_seq;
  const int wid = rank * NW + warp, n_warps = NW * cluster;
  // (unsigned: max_context_len may be any int, and with it a partition past the
  // table's end may pass 2^31)
  auto step_token = [&](int k) {
    return static_cast<unsigned>(base) + (WP ? k : wid + k * n_warps) * 32;
  };
  auto block_of = [&](int l) {
    return static_cast<int>(step_token(l / kTiles) / BS) + l % kTiles;
  };
  auto table_entry = [&](int l) -> int {
    const int lb = block_of(l);
    return lb < a.max_blocks_per_seq ? bt_row[lb] : -1;
  };
  int win = table_entry(lane);  // read before the length arrives; entries past it are not used

  const int G = a.group;
  int ctx = a.context_lens[table];
  int q0 = seq, n_rows = G, base_pos = 0;  // the chunk's first token, its rows, its position
  if constexpr (kChunk) {
    q0 = a.query_start[seq];
    const int q_len = a.query_start[seq + 1] - q0;
    n_rows = q_len * G;
    base_pos = ctx - q_len;
    if (q_len < 0 || ctx < q_len || ctx > a.max_blocks_per_seq * BS || q_len > a.max_q_len) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0) atomicOr(a.err, kErrBadLen);
      return;  // (the whole cluster)
    }
    if (n_rows == 0) return;  // (n_rows <= 8 NT: the launch has NT for max_q_len)
  } else if (ctx < 0 || ctx > a.max_blocks_per_seq * BS || ctx > a.max_context_len) {
    if (threadIdx.x == 0 && part == 0 && (kvh == 0 || a.per_head)) atomicOr(a.err, kErrBadLen);
    ctx = 0;
  }
  if (part > 0 && t_begin >= ctx) return;
  const int np_seq = kParts && ctx > 0 ? (ctx - 1) / a.part_tokens + 1 : 1;
  const int t_end = kParts ? t_begin + min(ctx - t_begin, a.part_tokens) : ctx;
  const int n_step = t_end > base ? (t_end - base + 31) / 32 : 0;
  const int my_n = WP ? n_step : (n_step > wid ? (n_step - wid + n_warps - 1) / n_warps : 0);

  // First line of the warp's tile l in the pool.  Every step loads all its
  // tiles: in place of one without a token of the partition, and of an invalid
  // block id, block 0 is read and nothing of it used.
  bool bad = false;  // an invalid id was met (the same in all lanes)
  auto line_of = [&](int l, int phys) -> int {
    const int lb = block_of(l);
    const bool used = l < my_n * kTiles && lb <= (t_end - 1) / BS && lb >= t_begin / BS;
    const bool ok = phys >= 0 && static_cast<int64_t>(phys) < a.num_blocks;
    if (used && !ok) atomicOr(a.err, kErrBadBlock);
    bad = bad || __any_sync(kFull, used && !ok);
    return ((used && ok ? phys : 0) * a.num_kv_heads + kvh) * Sh::kLines;
  };
  int win_base = 0;
  win = line_of(lane, win);
  int win_next = my_n * kTiles > 32 ? line_of(32 + lane, table_entry(32 + lane)) : 0;

  const uint64_t policy = l2_policy_evict_first();
  auto fill = [&](int k, int s) {  // called for k = 0, 1, 2, ...
    if (k * kTiles >= win_base + 32) {
      win_base += 32;
      win = win_next;
      win_next = line_of(win_base + 32 + lane, table_entry(win_base + 32 + lane));
    }
    const int y0 = __shfl_sync(kFull, win, (k * kTiles) & 31);
    const int y1 = kTiles == 2 ? __shfl_sync(kFull, win, (k * kTiles + 1) & 31) : 0;
    if (lane == 0) {
      uint8_t *st = my_stages + s * kStep;
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&my_bars[s], 2 * kTiles * Sh::kTileBytes);
      tma_load_2d(st, &kmap, 0, y0, &my_bars[s], policy);
      if (kTiles == 2) tma_load_2d(st + Sh::kSlot16, &kmap, 0, y1, &my_bars[s], policy);
      tma_load_2d(st + Sh::kUnit, &vmap, 0, y0, &my_bars[s], policy);
      if (kTiles == 2)
        tma_load_2d(st + Sh::kUnit + Sh::kSlot16, &vmap, 0, y1, &my_bars[s], policy);
    }
  };
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < my_n) fill(s, s);

  // query fragments of column g of every tile, in the order of the K bytes a lane reads
  uint4 qf[NT][Sh::kQChunks];
  float sl[NT][2];  // softmax scale of the lane's columns 2c and 2c + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = 8 * nt + g;
    const T *qrow = static_cast<const T *>(a.query) +
                    (static_cast<int64_t>(q0 + (kChunk ? col / G : 0)) * a.num_q_heads + kvh * G +
                     (kChunk ? col % G : col)) * D;
#pragma unroll
    for (int i = 0; i < Sh::kQChunks; ++i)
      qf[nt][i] = col < n_rows
                      ? *reinterpret_cast<const uint4 *>(qrow + (c * Sh::kQChunks + i) * 8)
                      : make_uint4(0, 0, 0, 0);
    sl[nt][0] = sl[nt][1] = a.scale_log2;
    if constexpr (!std::is_same<T, __half>::value) {
      // bf16 queries: each row is scaled by 2^e so that its largest magnitude
      // lies in [2^14, 2^15), then rounded to fp16 (exact for every value down
      // to 2^-31 of the largest: bf16 carries 8 bits, and fp16 holds 8 bits at
      // every magnitude from 2^-17 up); 2^-e joins the row's softmax scale
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < Sh::kQChunks; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 v = Elem<T>::unpack(word_of(qf[nt][i], w));
          mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const int e = min(120, 14 + 127 - static_cast<int>((__float_as_uint(mx) >> 23) & 0xffu));
      const float f = ldexpf(1.f, e);
#pragma unroll
      for (int i = 0; i < Sh::kQChunks; ++i) {
        uint32_t w4[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 v = Elem<T>::unpack(word_of(qf[nt][i], w));
          w4[w] = Elem<__half>::pack(v.x * f, v.y * f);
        }
        qf[nt][i] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
      }
      sl[nt][0] = ldexpf(sl[nt][0], -__shfl_sync(kFull, e, 8 * c));      // a lane of column 2c
      sl[nt][1] = ldexpf(sl[nt][1], -__shfl_sync(kFull, e, 8 * c + 4));  // of column 2c + 1
    }
    sl[nt][0] = fp4_normal_scale(sl[nt][0]);
    sl[nt][1] = fp4_normal_scale(sl[nt][1]);
    if (!kChunk && a.scale_log2 < 0.f) {  // a negative scale: the query's sign (order of the scores)
#pragma unroll
      for (int i = 0; i < Sh::kQChunks; ++i) {
        qf[nt][i].x ^= 0x80008000u;
        qf[nt][i].y ^= 0x80008000u;
        qf[nt][i].z ^= 0x80008000u;
        qf[nt][i].w ^= 0x80008000u;
      }
    }
  }

  // The lane's places in a unit's first half: K row token_of(g), V rows t0 =
  // token_of(2c) and t1 = token_of(2c + 1), all below 8; the scale groups 2c
  // and 2c + 1 (or c) of K, g (or g / 2) of V.
  const int kr = token_of<D>(g), t0 = token_of<D>(2 * c), t1 = token_of<D>(2 * c + 1);
  constexpr int kBytes = D == 128 ? 16 : 8;  // of a K row; of a V row half of them
  const int k_at = code_at<D>(kr, c * kBytes), k_ax = k_at ^ Sh::kHalf;
  const int v_0 = code_at<D>(t0, g * kBytes / 2), v_0x = v_0 ^ Sh::kHalf;
  const int v_1 = code_at<D>(t1, g * kBytes / 2), v_1x = v_1 ^ Sh::kHalf;
  const int ks_at = kr * Sh::kScales + (D == 128 ? 2 * c : c);
  const int vs_0 = t0 * Sh::kScales + (D == 128 ? g : g >> 1);
  const int vs_1 = t1 * Sh::kScales + (D == 128 ? g : g >> 1);

  const float NEG_INF = -INFINITY;
  // online softmax of the lane's columns 2c and 2c + 1 in base 2: xr is the
  // reference, a score before the softmax scale (-inf before the first token), so
  // that probabilities are held as 2^((x - xr) sl + kPShift)
  float xr[NT][2], l[NT][2], acc[NT][Sh::kMTiles][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    xr[nt][0] = xr[nt][1] = NEG_INF;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < Sh::kMTiles; ++mt)
      acc[nt][mt][0] = acc[nt][mt][1] = acc[nt][mt][2] = acc[nt][mt][3] = 0.f;
  }

  // One step, its K and V at `stage`.  masked: only the tokens that `mask` has
  // count (bit i: token i of the step), and in a chunk only those up to a
  // row's own, which is token `own` + row / G; the code of whole steps is
  // apart, as the selects cost a seventh of a step's instructions.
  auto step = [&](const uint8_t *stage, bool masked, uint32_t mask, int own) {
    // ---- S^T = K Q^T
    float x[NT][2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // two chains of products, so that half of them wait for one another
      // (several tiles of columns are chains enough)
      constexpr int kChains = NT == 1 ? 2 : 1;
      float y[NT][kChains][4] = {};
      const uint8_t *ka = stage + code_place<D, BS>(k_at, k_ax, h, 0);
      const uint8_t *kb = stage + code_place<D, BS>(k_at, k_ax, h, 1);
      const uint8_t *sa = stage + scale_place<D, BS>(ks_at, h, 0);
      const uint8_t *sb = stage + scale_place<D, BS>(ks_at, h, 1);
      uint32_t pa, pb;  // the scales of rows a and b as fp16 pairs
      uint32_t wa[D / 32], wb[D / 32];
      if constexpr (D == 128) {
        const uint4 va = *reinterpret_cast<const uint4 *>(ka);
        const uint4 vb = *reinterpret_cast<const uint4 *>(kb);
        wa[0] = va.x, wa[1] = va.y, wa[2] = va.z, wa[3] = va.w;
        wb[0] = vb.x, wb[1] = vb.y, wb[2] = vb.z, wb[3] = vb.w;
        pa = e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t *>(sa));
        pb = e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t *>(sb));
      } else {
        const uint2 va = *reinterpret_cast<const uint2 *>(ka);
        const uint2 vb = *reinterpret_cast<const uint2 *>(kb);
        wa[0] = va.x, wa[1] = va.y;
        wb[0] = vb.x, wb[1] = vb.y;
        pa = e4m3x2_lo_to_f16x2(*sa * 0x101u);
        pb = e4m3x2_lo_to_f16x2(*sb * 0x101u);
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t ga = D == 64 ? pa : __byte_perm(pa, 0, w < 2 ? 0x1010 : 0x3232);
        const uint32_t gb = D == 64 ? pb : __byte_perm(pb, 0, w < 2 ? 0x1010 : 0x3232);
        uint32_t ha[4], hb[4];
        e2m1x8_to_half(wa[w], ha);
        e2m1x8_to_half(wb[w], hb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ha[i] = f16x2_mul(ha[i], ga);
          hb[i] = f16x2_mul(hb[i], gb);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Elem<__half>::mma(y[nt][0], ha[0], hb[0], ha[1], hb[1], qf[nt][w].x, qf[nt][w].y);
          Elem<__half>::mma(y[nt][kChains - 1], ha[2], hb[2], ha[3], hb[3], qf[nt][w].z,
                            qf[nt][w].w);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[nt][h][e] = kChains == 2 ? y[nt][0][e] + y[nt][kChains - 1][e] : y[nt][0][e];
    }

    uint32_t pb0[NT][2], pb1[NT][2];  // P^T as the B operand
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // a row's own token (of columns 2c and 2c + 1) within the step
      const int col = 8 * nt + 2 * c;
      const int own0 = kChunk && masked ? own + col / G : 0;
      const int own1 = kChunk && masked ? own + (col + 1) / G : 0;
      // tokens that do not count get -inf
      auto hide = [&](float (&z)[2][4]) {
        if (!masked) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ta = 16 * h + kr, tb = ta + 8;
          const bool va = (mask >> ta) & 1u, vb = (mask >> tb) & 1u;
          z[h][0] = va && (!kChunk || ta <= own0) ? z[h][0] : NEG_INF;
          z[h][1] = va && (!kChunk || ta <= own1) ? z[h][1] : NEG_INF;
          z[h][2] = vb && (!kChunk || tb <= own0) ? z[h][2] : NEG_INF;
          z[h][3] = vb && (!kChunk || tb <= own1) ? z[h][3] : NEG_INF;
        }
      };
      // 2^y are the probabilities; the reference moves only when one of them
      // passes 2^(kPShift + kGrowth), so most steps need a vote and no shuffles
      const float s0 = sl[nt][0], s1 = sl[nt][1];
      const float c0 = fmaf(-xr[nt][0], s0, kPShift), c1 = fmaf(-xr[nt][1], s1, kPShift);
      float y[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        y[h][0] = fmaf(x[nt][h][0], s0, c0);
        y[h][1] = fmaf(x[nt][h][1], s1, c1);
        y[h][2] = fmaf(x[nt][h][2], s0, c0);
        y[h][3] = fmaf(x[nt][h][3], s1, c1);
      }
      hide(y);
      float top = NEG_INF;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        top = fmaxf(top, fmaxf(fmaxf(y[h][0], y[h][1]), fmaxf(y[h][2], y[h][3])));
      // (c0, c1 are infinite before the first token)
      if (__any_sync(kFull, top > kPShift + kGrowth || fmaxf(fabsf(c0), fabsf(c1)) > kFar)) {
        hide(x[nt]);
        float mx0 = xr[nt][0], mx1 = xr[nt][1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx0 = fmaxf(mx0, fmaxf(x[nt][h][0], x[nt][h][2]));
          mx1 = fmaxf(mx1, fmaxf(x[nt][h][1], x[nt][h][3]));
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, off));
        }
        const float al0 = mx0 == xr[nt][0] ? 1.f : ex2_approx((xr[nt][0] - mx0) * s0);
        const float al1 = mx1 == xr[nt][1] ? 1.f : ex2_approx((xr[nt][1] - mx1) * s1);
        xr[nt][0] = mx0;
        xr[nt][1] = mx1;
        l[nt][0] *= al0;
        l[nt][1] *= al1;
#pragma unroll
        for (int mt = 0; mt < Sh::kMTiles; ++mt) {
          acc[nt][mt][0] *= al0;
          acc[nt][mt][1] *= al1;
          acc[nt][mt][2] *= al0;
          acc[nt][mt][3] *= al1;
        }
        const float r0 = mx0 == NEG_INF ? 0.f : mx0;  // no token yet: any finite reference
        const float r1 = mx1 == NEG_INF ? 0.f : mx1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          y[h][0] = fmaf(x[nt][h][0] - r0, s0, kPShift);
          y[h][1] = fmaf(x[nt][h][1] - r1, s1, kPShift);
          y[h][2] = fmaf(x[nt][h][2] - r0, s0, kPShift);
          y[h][3] = fmaf(x[nt][h][3] - r1, s1, kPShift);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = ex2_approx(y[h][0]), p1 = ex2_approx(y[h][1]);
        const float p2 = ex2_approx(y[h][2]), p3 = ex2_approx(y[h][3]);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        // an 8x8 transpose of the accumulator's layout
        pb0[nt][h] = movmatrix_trans(Elem<__half>::pack(p0, p1));
        pb1[nt][h] = movmatrix_trans(Elem<__half>::pack(p2, p3));
      }
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t *Vs = stage + Sh::kUnit;
      uint32_t s0 = Vs[scale_place<D, BS>(vs_0, h, 0)], s1 = Vs[scale_place<D, BS>(vs_1, h, 0)];
      uint32_t s2 = Vs[scale_place<D, BS>(vs_0, h, 1)], s3 = Vs[scale_place<D, BS>(vs_1, h, 1)];
      if (masked) {
        s0 = (mask >> (16 * h + t0)) & 1u ? s0 : 0;
        s1 = (mask >> (16 * h + t1)) & 1u ? s1 : 0;
        s2 = (mask >> (16 * h + t0 + 8)) & 1u ? s2 : 0;
        s3 = (mask >> (16 * h + t1 + 8)) & 1u ? s3 : 0;
        if constexpr (kChunk) {
          auto drop_nan = [&](uint32_t &sc, int at) {
            if ((sc & 0x7fu) == 0x7fu) {
              sc = 0;
              atomicMin(&nan_key[warp * 8 + (D == 128 ? g : g >> 1)], at - own);
            }
          };
          drop_nan(s0, 16 * h + t0);
          drop_nan(s1, 16 * h + t1);
          drop_nan(s2, 16 * h + t0 + 8);
          drop_nan(s3, 16 * h + t1 + 8);
          __syncwarp();
        }
      }
      const uint32_t g01 = e4m3x2_lo_to_f16x2(s0 | (s1 << 8));
      const uint32_t g23 = e4m3x2_lo_to_f16x2(s2 | (s3 << 8));
      // words of eight codes of tokens A and B -> (A, B) pairs of the even or the odd dimensions
      auto pairs = [](uint32_t A, uint32_t B, int odd, uint32_t s, uint32_t (&out)[4]) {
        e2m1x8_to_half(odd ? ((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u)
                           : (A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u),
                       out);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = f16x2_mul(out[i], s);
      };
      const uint8_t *p0 = Vs + code_place<D, BS>(v_0, v_0x, h, 0);
      const uint8_t *p1 = Vs + code_place<D, BS>(v_1, v_1x, h, 0);
      const uint8_t *p2 = Vs + code_place<D, BS>(v_0, v_0x, h, 1);
      const uint8_t *p3 = Vs + code_place<D, BS>(v_1, v_1x, h, 1);
      if constexpr (D == 128) {
        const uint2 w0 = *reinterpret_cast<const uint2 *>(p0);
        const uint2 w1 = *reinterpret_cast<const uint2 *>(p1);
        const uint2 w2 = *reinterpret_cast<const uint2 *>(p2);
        const uint2 w3 = *reinterpret_cast<const uint2 *>(p3);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {  // m-tiles 0, 2, 4, 6, then 1, 3, 5, 7
          uint32_t a0[4], a1[4], a2[4], a3[4];
          pairs(w0.x, w1.x, odd, g01, a0);
          pairs(w0.y, w1.y, odd, g01, a1);
          pairs(w2.x, w3.x, odd, g23, a2);
          pairs(w2.y, w3.y, odd, g23, a3);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              Elem<__half>::mma(acc[nt][2 * i + odd], a0[i], a1[i], a2[i], a3[i], pb0[nt][h],
                                pb1[nt][h]);
        }
      } else {
        const uint32_t w0 = *reinterpret_cast<const uint32_t *>(p0);
        const uint32_t w1 = *reinterpret_cast<const uint32_t *>(p1);
        const uint32_t w2 = *reinterpret_cast<const uint32_t *>(p2);
        const uint32_t w3 = *reinterpret_cast<const uint32_t *>(p3);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {  // m-tiles 0, 2, then 1, 3
          uint32_t a0[4], a2[4];
          pairs(w0, w1, odd, g01, a0);
          pairs(w2, w3, odd, g23, a2);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              Elem<__half>::mma(acc[nt][2 * i + odd], a0[i], a0[2 + i], a2[i], a2[2 + i],
                                pb0[nt][h], pb1[nt][h]);
        }
      }
    }
  };

  bool timed_out = false;
  int k = 0;
#pragma unroll 1
  for (; k < my_n; ++k) {
    const int s = k % S;
    if (!__all_sync(kFull, mbar_wait_bounded(&my_bars[s], (k / S) & 1))) {
      if (lane == 0) atomicOr(a.err, kErrTimeout);
      timed_out = true;
      break;
    }
    const uint8_t *stage = my_stages + s * kStep;
    const int step_tok = step_token(k);
    // (in a chunk every row sees the step's last token if its first row does)
    if (!bad && step_tok >= t_begin &&
        step_tok + 32 <= (kChunk ? base_pos + 1 : t_end)) {
      step(stage, false, 0xffffffffu, 0);
    } else {
      const int tok = step_tok + lane;
      bool in = tok >= t_begin && tok < t_end;
      if (bad && in) {
        const int phys = bt_row[tok / BS];
        in = phys >= 0 && static_cast<int64_t>(phys) < a.num_blocks;
      }
      step(stage, true, __ballot_sync(kFull, in), base_pos - step_tok);
    }

    // ---- refill this stage with step k + S
    __syncwarp();
    if (k + S < my_n) fill(k + S, s);
  }
  // after a wait that ran out, copies already in flight land before the CTA
  // leaves (bounded again)
  for (const int filled = min(k + S, my_n); timed_out && k < filled; ++k)
    (void)mbar_wait_bounded(&my_bars[k % S], (k / S) & 1);

  // row sums over the 8 token rows; l and acc are both held times 2^kPShift,
  // relative to xr; from here on (to is what brings them there) to m, a float
  // next to xr's logit
  float m[NT][2], to[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], off);
      m[nt][e] = fp4_reference(xr[nt][e], sl[nt][e], kPShift, to[nt][e]);
      l[nt][e] *= to[nt][e];
    }

  if constexpr (WP) {
    const int64_t first = static_cast<int64_t>(seq) * a.num_q_heads + kvh * G;
    const int h0 = 2 * c, h1 = 2 * c + 1;
    const float inv0 = l[0][0] > 0.f ? a.out_scale * to[0][0] / l[0][0] : 0.f;
    const float inv1 = l[0][1] > 0.f ? a.out_scale * to[0][1] / l[0][1] : 0.f;
    const int64_t pr0 = (first + h0) * a.num_parts + part, pr1 = (first + h1) * a.num_parts + part;
    if (g == 0) {
      if (h0 < G) {
        a.ws_m[pr0] = m[0][0];
        a.ws_l[pr0] = l[0][0];
      }
      if (h1 < G) {
        a.ws_m[pr1] = m[0][1];
        a.ws_l[pr1] = l[0][1];
      }
    }
    // out through the warp's idle stages, in whole lines
    float *mine = reinterpret_cast<float *>(my_stages);
    put_acc<D>(mine, acc[0], inv0, inv1, g, c);
    __syncwarp();
#pragma unroll 1
    for (int i = lane; i < G * (D / 4); i += 32) {
      const int h = i / (D / 4), d = i % (D / 4) * 4;
      const float *src = mine + h * kAccStride<D>;
      *reinterpret_cast<float4 *>(a.ws_o + ((first + h) * a.num_parts + part) * D + d) =
          make_float4(src[acc_place<D>(d)], src[acc_place<D>(d + 1)], src[acc_place<D>(d + 2)],
                      src[acc_place<D>(d + 3)]);
    }
    grid_launch_dependents();
    return;
  }

  // ---- merge warps through shared memory (stages are idle now), a tile of
  // columns at a time
  float *wacc = reinterpret_cast<float *>(smem);  // [NW][8][kAccStride]
  float *wml = wacc + NW * 8 * kAccStride<D>;     // [NW][8][2]
  float *cl_o = wml + NW * 8 * 2 + 4;             // [NT][8][D]: the CTA's, for its cluster
  float *cl_ml = cl_o + NT * 8 * D;               // [NT][8][2]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    __syncthreads();
    if (g == 0) {
      wml[(warp * 8 + 2 * c) * 2 + 0] = m[nt][0];
      wml[(warp * 8 + 2 * c) * 2 + 1] = l[nt][0];
      wml[(warp * 8 + 2 * c + 1) * 2 + 0] = m[nt][1];
      wml[(warp * 8 + 2 * c + 1) * 2 + 1] = l[nt][1];
    }
    put_acc<D>(wacc + warp * 8 * kAccStride<D>, acc[nt], to[nt][0], to[nt][1], g, c);
    __syncthreads();
    constexpr int kChunks = D / 8;
    const int cols = min(8, n_rows - 8 * nt);
    for (int item = threadIdx.x; item < cols * kChunks; item += NW * 32) {
      const int h = item / kChunks, ch = item % kChunks;
      float M = NEG_INF;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, wml[(w * 8 + h) * 2]);
      float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = exp2f(wml[(w * 8 + h) * 2] - M);
        L += wml[(w * 8 + h) * 2 + 1] * f;
        const float *src = wacc + (w * 8 + h) * kAccStride<D>;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += src[acc_place<D>(ch * 8 + e)] * f;
      }
      if constexpr (kChunk) {
        int first_nan = nan_key[ch / 2];
#pragma unroll
        for (int w = 1; w < NW; ++w) first_nan = min(first_nan, nan_key[w * 8 + ch / 2]);
        if (first_nan <= (8 * nt + h) / G) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __int_as_float(0x7fffffff);
        }
      }
      if (!kParts && cluster > 1) {
        float4 *dst = reinterpret_cast<float4 *>(cl_o + (nt * 8 + h) * D + ch * 8);
        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        if (ch == 0) {
          cl_ml[(nt * 8 + h) * 2] = M;
          cl_ml[(nt * 8 + h) * 2 + 1] = L;
        }
        continue;
      }
      const int col = 8 * nt + h;
      const int64_t row = static_cast<int64_t>(q0 + (kChunk ? col / G : 0)) * a.num_q_heads +
                          kvh * G + (kChunk ? col % G : col);
      const float inv = L > 0.f ? a.out_scale / L : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= inv;
      if (!kParts || (a.fuse_join && np_seq == 1)) {
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D + ch * 8) =
            make_uint4(Elem<T>::pack(o[0], o[1]), Elem<T>::pack(o[2], o[3]),
                       Elem<T>::pack(o[4], o[5]), Elem<T>::pack(o[6], o[7]));
      } else {
        const int64_t pr = row * a.num_parts + part;
        float4 *dst = reinterpret_cast<float4 *>(a.ws_o + pr * D + ch * 8);
        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        if (ch == 0) {
          a.ws_m[pr] = M;
          a.ws_l[pr] = L;
        }
      }
    }
  }
  if (!kParts && cluster > 1) {
    // the cluster's CTAs share the rows of the join out
    cluster_sync();
    constexpr int kChunks = D / 8;
    const int cols = min(8 * NT, n_rows);
    for (int item = threadIdx.x + rank * NW * 32; item < cols * kChunks;
         item += NW * 32 * cluster) {
      const int col = item / kChunks, ch = item % kChunks;
      float M = NEG_INF;
      for (int r = 0; r < cluster; ++r)
        M = fmaxf(M, ld_cluster_f2(cluster_addr(cl_ml + col * 2, r)).x);
      float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int r = 0; r < cluster; ++r) {
        const float2 ml = ld_cluster_f2(cluster_addr(cl_ml + col * 2, r));
        const uint32_t src = cluster_addr(cl_o + col * D + ch * 8, r);
        const float4 x = ld_cluster_f4(src), y = ld_cluster_f4(src + 16);
        const float f = exp2f(ml.x - M);
        L += ml.y * f;
        o[0] += x.x * f;
        o[1] += x.y * f;
        o[2] += x.z * f;
        o[3] += x.w * f;
        o[4] += y.x * f;
        o[5] += y.y * f;
        o[6] += y.z * f;
        o[7] += y.w * f;
      }
      const int64_t row = static_cast<int64_t>(q0 + (kChunk ? col / G : 0)) * a.num_q_heads +
                          kvh * G + (kChunk ? col % G : col);
      const float inv = L > 0.f ? a.out_scale / L : 0.f;
      *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D + ch * 8) = make_uint4(
          Elem<T>::pack(o[0] * inv, o[1] * inv), Elem<T>::pack(o[2] * inv, o[3] * inv),
          Elem<T>::pack(o[4] * inv, o[5] * inv), Elem<T>::pack(o[6] * inv, o[7] * inv));
    }
    cluster_sync();  // nobody leaves while its memory is read
  }
  if (kParts && a.fuse_join && np_seq > 1) {
    if (last_to_arrive(a, seq, kvh, np_seq, reinterpret_cast<uint32_t *>(wml + NW * 8 * 2)))
      join_partitions<T, D, NW>(a, seq, kvh, np_seq);
  }
  grid_launch_dependents();
}

template <typename T, int D, int BS, int NW, int S, Rows ROWS, int NT>
cudaError_t launch_rows(DecodeArgs a, const CUtensorMap &km, const CUtensorMap &vm,
                        unsigned grid_x, cudaStream_t stream) {
  constexpr size_t stages = static_cast<size_t>(NW) * S * 2 * Fp4Shape<D, BS>::kUnit;
  constexpr bool kParts = ROWS == Rows::kDecode || ROWS == Rows::kDecodeWarps;
  constexpr size_t smem = 1024 + stages + NW * S * 8 + (kParts ? 0 : NW * 8 * 4 + 4);
  static_assert((static_cast<size_t>(NW) * (kAccStride<D> + 2) + NT * (D + 2)) * 32 + 16 <= stages,
                "merge buffers and the join flag must fit in the stage area");
  static_assert(smem <= 227 * 1024, "shared memory");
  static_assert((64 / Fp4Shape<D, BS>::kTiles * NW * (kParts ? 1 : kFp4Cluster) + 1) * 32 <=
                    kFp4LookAhead,
                "token indexes past the end of the longest table");
  auto kern = pa_decode_fp4_kernel<T, D, BS, NW, S, ROWS, NT>;
  static SmemLimitOnce smem_limit;
  const cudaError_t e = smem_limit.ensure(kern, smem);
  if (e != cudaSuccess) return e;
  // Longest contexts first where the CTAs are more than run at once and the
  // table leaves room for unequal contexts.  Contexts of 512 to 4,096, 32 / 8 heads:
  // 64 sequences of 20 rows 68 us against 82, of 16 rows 57 against 63; 128 unsplit
  // sequences 74 against 87, 256 126 against 140.  (256 of up to 300 tokens, 8 rows,
  // under a table of 32,768: 27 against 26.)  Calls with partitions lose: 256
  // sequences of up to 16,384 128 us against 117, since every empty partition's CTA
  // asks for its sequence too.
  const int64_t ctas = static_cast<int64_t>(grid_x) * a.num_kv_heads * a.num_seqs;
  a.by_length = !kParts && a.cluster == 1 && !a.per_head &&
                a.num_seqs > 1 && a.num_seqs <= kMaxByLength && ctas > kSms * ctas_per_sm(NT) &&
                (static_cast<int64_t>(a.max_blocks_per_seq) << a.bs_log2) >= kMinByLength &&
                (ROWS == Rows::kChunk || a.max_context_len >= kMinByLength);
  return launch_clusters(a.cluster, kern, dim3(grid_x, a.num_kv_heads, a.num_seqs),
                         dim3(NW * 32), smem, stream, km, vm, a);
}

// How many CTAs share the keys of a sequence and KV head in a call without
// partitions: as many as the SMs still have room for, while a warp keeps two steps of the longest
// context that the table can hold.  Few sequences gain (one of 8,000 tokens and
// one KV head 20 us, with one CTA 93; eight KV heads of 4,096 tokens 11 against
// 33), and beyond that room a CTA's 4 to 6 us of start and join cost more than
// the evener load gives (64 sequences of 512 to 4,096 tokens, 20 rows, taken
// as they come: 82 us alone, 88 in pairs, 115 in fours).  Tables per head, 32 / 8
// heads x 128: 8 rows of 2,048 tokens 11.3 us, 16.5 without clusters; 64 of 512 12.5
// (two warps a CTA 11.0 and 12.3, but 256 rows of up to 1,024, 64 / 8 heads, 62 us
// against 53.7 with four).
int cluster_of(const DecodeArgs &a, int64_t ctas, int warps, int per_sm) {
  const int64_t steps = (static_cast<int64_t>(a.max_blocks_per_seq) << a.bs_log2) / 32;
  int n = 1;
  while (n < kFp4Cluster && 2 * n * ctas <= kSms * per_sm && steps >= 4 * n * warps) n *= 2;
  return n;
}

template <typename T, int D, int BS>
cudaError_t launch_decode_t(DecodeArgs a, const CUtensorMap &km, const CUtensorMap &vm,
                            cudaStream_t stream) {
  a.cluster = 1;
  constexpr int NW = PA_DECODE_FP4_WARPS, S = PA_DECODE_FP4_STAGES;
  if (a.num_parts > 1 && !a.fuse_join)
    return launch_rows<T, D, BS, NW, S, Rows::kDecodeWarps, 1>(a, km, vm,
                                                               (a.num_parts + NW - 1) / NW, stream);
  if (a.num_parts > 1)
    return launch_rows<T, D, BS, NW, S, Rows::kDecode, 1>(a, km, vm, a.num_parts, stream);
  a.cluster = cluster_of(a, static_cast<int64_t>(a.num_seqs) * a.num_kv_heads, NW, ctas_per_sm(1));
  return launch_rows<T, D, BS, NW, S, Rows::kWhole, 1>(a, km, vm, a.cluster, stream);
}

template <typename T, int D, int BS>
cudaError_t launch_chunk_t(DecodeArgs a, const CUtensorMap &km, const CUtensorMap &vm,
                           cudaStream_t stream) {
  const int rows = a.max_q_len * a.group;
  auto launch = [&](auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    a.cluster = cluster_of(a, static_cast<int64_t>(a.num_seqs) * a.num_kv_heads, 4,
                           ctas_per_sm(NT));
    return launch_rows<T, D, BS, 4, 2, Rows::kChunk, NT>(a, km, vm, a.cluster, stream);
  };
  if (rows <= 8) return launch(std::integral_constant<int, 1>{});
  if (rows <= 16) return launch(std::integral_constant<int, 2>{});
  return launch(std::integral_constant<int, 3>{});
}

// f(head_dim, block_size) with both as compile-time constants
template <typename F> cudaError_t by_shape(int head_dim, int bs_log2, F &&f) {
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  using B16 = std::integral_constant<int, 16>;
  using B32 = std::integral_constant<int, 32>;
  if (head_dim == 128) return bs_log2 == 4 ? f(D128{}, B16{}) : f(D128{}, B32{});
  return bs_log2 == 4 ? f(D64{}, B16{}) : f(D64{}, B32{});
}

bool encode_maps(CUtensorMap *km, CUtensorMap *vm, const DecodeArgs &a, const void *k_cache,
                 const void *v_cache, int head_dim) {
  const int64_t tiles = a.num_blocks * a.num_kv_heads;
  return encode_fp4_map(km, k_cache, tiles, 1 << a.bs_log2, head_dim, true) &&
         encode_fp4_map(vm, v_cache, tiles, 1 << a.bs_log2, head_dim, true);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                              int head_dim, int dtype, cudaStream_t stream, bool *map_failed) {
  CUtensorMap km, vm;
  *map_failed = !encode_maps(&km, &vm, a, k_cache, v_cache, head_dim);
  if (*map_failed) return cudaErrorInvalidValue;
  return by_shape(head_dim, a.bs_log2, [&](auto d, auto bs) {
    return dtype == 0 ? launch_decode_t<__half, d(), bs()>(a, km, vm, stream)
                      : launch_decode_t<__nv_bfloat16, d(), bs()>(a, km, vm, stream);
  });
}

cudaError_t launch_chunk_fp4(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                             int head_dim, int dtype, cudaStream_t stream, bool *map_failed) {
  CUtensorMap km, vm;
  *map_failed = !encode_maps(&km, &vm, a, k_cache, v_cache, head_dim);
  if (*map_failed) return cudaErrorInvalidValue;
  return by_shape(head_dim, a.bs_log2, [&](auto d, auto bs) {
    return dtype == 0 ? launch_chunk_t<__half, d(), bs()>(a, km, vm, stream)
                      : launch_chunk_t<__nv_bfloat16, d(), bs()>(a, km, vm, stream);
  });
}

}  // namespace pa
