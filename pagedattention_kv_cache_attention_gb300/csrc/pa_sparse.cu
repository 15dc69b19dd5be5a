// pa_sparse.cu -- the cheap score of sparse attention: bounds of a block's keys
// (pa_update_key_bounds and its FP8 and FP4 forms), and the choice of blocks
// by them (pa_select_blocks).
//
// Bounds of a (block, KV head), over its tokens: with a the largest magnitude
// and 2^e the least power of two with a <= 127 2^e (e >= -126), every channel's
// largest and smallest key over 2^e, rounded up and down to an integer.  Then
//   q . k <= sum_d max(q_d hi_d, q_d lo_d) 2^e  for every key k of the block.
//
// Score of a block for a KV head's group of queries.  The queries become
// integers c = rint(q / 2^f), 2^f the least power of two with the group's
// largest magnitude <= 4095 2^f.  The bounds of c 2^f, all heads, add up to
//   2^f 2^e I,   I = sum_d P_d hi_d + N_d lo_d,
//   P_d, N_d = the sums of the group's positive, of its negative c_d,
// one integer product of 2 D terms for the whole group: |P_d| + |N_d| <= 8 * 4095,
// so that P and N fit 16 bits and |I| <= 127 * 32760 * 128 fits 32.  I does not
// depend on the order of its sum, so neither does the choice; 2^f is common to
// the blocks and left out.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The least e >= -126 with a <= (2^n - 1) 2^e; a finite, > 0.
__device__ __forceinline__ int exponent_for(float a, int n) {
  // a = m 2^x, 0.5 <= m < 1 (a below the normal numbers: e is -126 at once)
  const uint32_t bits = __float_as_uint(a);
  const int x = static_cast<int>(bits >> 23) - 126;
  const float m = __uint_as_float((bits & 0x7fffffu) | 0x3f000000u);
  const float most = 1.f - pow2(-n);
  return max(x - n + (m > most ? 1 : 0), -126);
}

// ---------------------------------------------------------------- key bounds

// Larger and smaller of two fp16 or bf16 pairs, NaN if either is.
template <typename T> __device__ __forceinline__ void extremes2(uint32_t x, uint32_t &hi, uint32_t &lo) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = *reinterpret_cast<const __half2 *>(&x);
    const __half2 h = __hmax2_nan(*reinterpret_cast<const __half2 *>(&hi), v);
    const __half2 l = __hmin2_nan(*reinterpret_cast<const __half2 *>(&lo), v);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
  } else {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&x);
    const __nv_bfloat162 h = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&hi), v);
    const __nv_bfloat162 l = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&lo), v);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
  }
}

// A lane's share of a token's row: 8 elements of a 16-bit cache, 16 of an FP8 or
// FP4 one (as fp16, exact), in W words of pairs; kLanes lanes hold a row.
template <int D, Kv KV> struct KeyShare {
  static constexpr int kElems = KV == Kv::k16 ? 8 : 16;
  static constexpr int kWords = kElems / 2;
  static constexpr int kLanes = D / kElems;
  static constexpr int kRows = 32 / kLanes;  // rows that a warp reads at once
  // raw bytes of the share of row r of a block whose bytes begin at `block`
  struct Raw {
    uint4 x;
    uint32_t scale;
  };
  static __device__ __forceinline__ Raw load(const uint8_t *block, int bs, int r, int share) {
    Raw raw;
    raw.scale = 0;
    if constexpr (KV == Kv::kFp4) {
      const uint2 c = *reinterpret_cast<const uint2 *>(block + r * (D / 2) + share * 8);
      raw.x = make_uint4(c.x, c.y, 0, 0);
      raw.scale = block[fp4_code_bytes(bs, D) + r * (D / 16) + share];
    } else {
      raw.x = *reinterpret_cast<const uint4 *>(block + r * (D * (KV == Kv::k16 ? 2 : 1)) + share * 16);
    }
    return raw;
  }
  static __device__ __forceinline__ void widen(const Raw &raw, uint32_t (&w)[kWords]) {
    if constexpr (KV == Kv::k16) {
      w[0] = raw.x.x, w[1] = raw.x.y, w[2] = raw.x.z, w[3] = raw.x.w;
    } else if constexpr (KV == Kv::kFp8) {
      e4m3x16_to_half(raw.x, w);
    } else {
      uint32_t a[4], b[4];
      e2m1x8_to_half(raw.x.x, a);
      e2m1x8_to_half(raw.x.y, b);
      const uint32_t s = e4m3x2_lo_to_f16x2(raw.scale | (raw.scale << 8));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = f16x2_mul(a[i], s);
        w[4 + i] = f16x2_mul(b[i], s);
      }
    }
  }
};

// Elementwise larger of two pairs, NaN if either is.
template <typename T> __device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  uint32_t unused = y;
  extremes2<T>(x, y, unused);
  return y;
}

// A CTA for a block, a warp for a KV head of it (more heads in turn): every lane
// keeps the extremes of its channels over the rows that it reads.  The lanes that
// hold the same channels then share these out in a butterfly, largest ones to the
// lower half of the warp and the negated smallest to the upper one, so that all
// that is left is a maximum.
// Latency bounds it (length, table entry, keys: three loads one after another): a
// step's 256 sequences x 8 heads x 32 tokens x 128, bf16, 2.9 us for 9 MB; 16 chunks
// of 1,031 tokens, 8 heads x 128, fp16 7.5 us for 36 MB, FP8 5.5, FP4 5.8 (with all
// lanes of a channel taking all of its maxima 3.7, 9.8, 7.1 and 7.3: instructions).
constexpr int kBoundsWarps = 8;

template <typename T, int D, Kv KV>
__global__ void __launch_bounds__(kBoundsWarps * 32) key_bounds_kernel(const BoundsArgs a) {
  using Share = KeyShare<D, KV>;
  using MT = typename std::conditional<KV == Kv::k16, T, __half>::type;
  constexpr int W = Share::kWords, kLanes = Share::kLanes, kRows = Share::kRows;
  constexpr int kTake = KV == Kv::k16 ? 8 : 4;  // rows that a lane has in flight
  constexpr int kKeep = 2 * W * kLanes / 32;    // words that a lane ends with
  grid_dependency_wait();  // the keys may come from the kernel before
  const int seq = blockIdx.y, lane = threadIdx.x & 31;
  const int bs = 1 << a.bs_log2;
  const int ctx = a.context_lens[seq];
  int new_tokens = min(ctx, 1);
  if (a.query_start) new_tokens = a.query_start[seq + 1] - a.query_start[seq];
  if (new_tokens < 0 || ctx < new_tokens || new_tokens > a.max_q_len ||
      ctx > static_cast<int64_t>(a.max_blocks_per_seq) << a.bs_log2) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.err, kErrBadLen);
    return;
  }
  if (new_tokens == 0) return;
  const int64_t j = ((ctx - new_tokens) >> a.bs_log2) + static_cast<int64_t>(blockIdx.x);
  if (j > (ctx - 1) >> a.bs_log2) return;
  const int phys = a.block_tables[static_cast<int64_t>(seq) * a.max_blocks_per_seq + j];
  if (phys < 0 || phys >= a.num_blocks) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrBadBlock);
    return;
  }
  const int rows = min(bs, static_cast<int>(ctx - (j << a.bs_log2)));
  const int block_bytes = KV == Kv::kFp4 ? fp4_tile_bytes(bs, D) : bs * D * (KV == Kv::k16 ? 2 : 1);
  const int share = lane % kLanes, r0 = lane / kLanes;
  for (int h = threadIdx.x >> 5; h < a.num_kv_heads; h += blockDim.x >> 5) {
    const int64_t cell = static_cast<int64_t>(phys) * a.num_kv_heads + h;
    const uint8_t *block = static_cast<const uint8_t *>(a.k_cache) + cell * block_bytes;
    // (row 0 counts always: rows past the end are read as that one)
    uint32_t v[2 * W];  // the largest, then the smallest
    for (int r = r0; r < bs; r += kRows * kTake) {
      typename Share::Raw raw[kTake];
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        const int at = r + i * kRows;
        raw[i] = Share::load(block, bs, at < rows ? at : 0, share);
      }
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        uint32_t x[W];
        Share::widen(raw[i], x);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (i == 0 && r == r0) v[w] = v[W + w] = x[w];
          extremes2<MT>(x[w], v[w], v[W + w]);
        }
      }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) v[W + w] ^= 0x80008000u;
#pragma unroll
    for (int off = 16, n = W; off >= kLanes; off >>= 1, n >>= 1) {
      const bool up = lane & off;
#pragma unroll
      for (int w = 0; w < n; ++w) {
        const uint32_t keep = up ? v[n + w] : v[w], give = up ? v[w] : v[n + w];
        v[w] = max2<MT>(__shfl_xor_sync(kAll, give, off), keep);
      }
    }
    // the largest magnitude is the largest of all that is left; an infinity or a NaN
    // is one of those, too
    float x[2 * kKeep], top = 0.f;
#pragma unroll
    for (int w = 0; w < kKeep; ++w) {
      const float2 p = Elem<MT>::unpack(v[w]);
      x[2 * w] = p.x, x[2 * w + 1] = p.y;
      top = p.x < INFINITY ? fmaxf(top, p.x) : INFINITY;
      top = p.y < INFINITY ? fmaxf(top, p.y) : INFINITY;
    }
    top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(top)));
    const bool odd = top == INFINITY, none = odd || top == 0.f;
    const int e = none ? 0 : exponent_for(top, 7);
    const float inv = none ? 0.f : pow2(-e);
    const bool smallest = lane & 16;
    uint32_t out[kKeep / 2];
#pragma unroll
    for (int q = 0; q < kKeep / 2; ++q) {
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // (2^-e is exact, and so is the product but for one below 2^-126, which, rounded
        // up, stays above 0 if it is above 0)
        const int c = none ? 0 : __float2int_ru(__fmul_ru(x[4 * q + b], inv));
        word |= static_cast<uint32_t>((smallest ? -c : c) & 0xff) << (8 * b);
      }
      out[q] = word;
    }
    // the lane's words: the part of its share that its place among the lanes of
    // equal channels in its half of the warp stands for
    int first = 0;
#pragma unroll
    for (int off = 8, n = W / 2; off >= kLanes; off >>= 1, n >>= 1) first += lane & off ? n : 0;
    int8_t *dst = a.bounds + (cell * 2 + (smallest ? 1 : 0)) * D + share * Share::kElems + 2 * first;
    if constexpr (kKeep == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
    else
      *reinterpret_cast<uint32_t *>(dst) = out[0];
    if (lane == 0) a.bound_scales[cell] = odd ? INFINITY : none ? 0.f : pow2(e);
  }
}

template <typename T, int D, Kv KV>
cudaError_t launch_bounds(const BoundsArgs &a, cudaStream_t stream) {
  // blocks that max_q_len new tokens can reach into
  int64_t blocks = ((static_cast<int64_t>(a.max_q_len) - 1) >> a.bs_log2) + 2;
  blocks = blocks < a.max_blocks_per_seq ? blocks : a.max_blocks_per_seq;
  if (a.max_q_len == 1) blocks = 1;
  const int warps = a.num_kv_heads < kBoundsWarps ? a.num_kv_heads : kBoundsWarps;
  return launch_dependent(key_bounds_kernel<T, D, KV>, dim3(static_cast<unsigned>(blocks), a.num_seqs),
                          dim3(warps * 32), 0, stream, a);
}

template <typename T, int D>
cudaError_t launch_bounds_kv(const BoundsArgs &a, Kv kv, cudaStream_t stream) {
  if (kv == Kv::kFp8) return launch_bounds<__half, D, Kv::kFp8>(a, stream);
  if (kv == Kv::kFp4) return launch_bounds<__half, D, Kv::kFp4>(a, stream);
  return launch_bounds<T, D, Kv::k16>(a, stream);
}

// ---------------------------------------------------------------- selection

constexpr uint32_t kForced = 0xffffffffu;  // above the key of every score

// An unsigned key in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A sequence's rows and the tokens that they see.
struct SelectRows {
  int64_t row0;  // its first row
  int rows;      // how many
  int base;      // tokens that row t sees, less t
  // false if there is nothing to do for the sequence (a bad length is flagged by
  // one thread of the grid)
  __device__ __forceinline__ bool load(const SelectArgs &a, int seq, bool tell) {
    const int ctx = a.context_lens[seq];
    const bool fine = ctx >= 0 && ctx <= a.max_context_len &&
                      ctx <= static_cast<int64_t>(a.max_blocks_per_seq) << a.bs_log2;
    if (!a.query_start) {
      if (!fine && tell) atomicOr(a.err, kErrBadLen);
      row0 = seq;
      rows = 1;
      base = fine ? ctx : 0;
      return true;
    }
    const int q0 = a.query_start[seq], q_len = a.query_start[seq + 1] - q0;
    row0 = q0;
    rows = q_len;
    base = ctx - q_len + 1;
    if (fine && q_len >= 0 && q_len <= ctx && q_len <= a.max_q_len) return true;
    if (tell) atomicOr(a.err, kErrBadLen);
    return false;
  }
};

// A row's group of queries, in one warp: lane l holds channels D / 32 l .. of all heads.
template <typename T, int D> struct Queries {
  static constexpr int kPer = D / 32;
  uint32_t w[8][kPer / 2];
  __device__ __forceinline__ void load(const SelectArgs &a, int64_t row, int kvh, int lane) {
    const T *q = static_cast<const T *>(a.query) + (row * a.num_q_heads + kvh * a.group) * D + lane * kPer;
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i)
        w[h][i] = h < a.group ? reinterpret_cast<const uint32_t *>(q + h * D)[i] : 0;
  }
};

// I of 16 blocks and up to 4 rows is a product on the tensor cores: the blocks'
// codes as fp16 integers times 2^-24 (a byte in the low bits of a half is that
// subnormal number; with 128 added codes are unsigned), the weights P and N of a
// row as two columns, their low bytes (0 to 255) and high ones (-128 to 127).  A
// column's sum is below 255 * 255 * 256 < 2^24 units of 2^-24, so fp32 holds every
// partial sum exactly.  I = low + 256 high - 128 (sum of the weights).
// (By integer dot products a row takes 64 of them for 16 blocks, at half rate, and
// sums over lanes; the codes' three instructions for 4 of them here are shared by
// the rows.  5 drafted tokens of 64 sequences, contexts of 512 to 4,096, 32 / 8
// heads: 12.4 us, by dot products 16.8, at the time.)
//
// The order of the 2 D codes in the product is one that lets a lane take 16
// consecutive codes of a block: code 64 i + 16 c + 4 w + e is column c's e-th of
// step 4 i + w.
template <int D> struct Weights {
  static constexpr int kSteps = 2 * D / 16;
  uint2 frag[kSteps][32];  // the B operand of a step in each lane: columns 2 r, 2 r + 1 are row r's
  int bias[4];             // 128 times the sum of a row's weights

  // Row r of the tile, from its group of queries (nullptr: zeros).  For a whole warp.
  template <typename T>
  __device__ __forceinline__ void put(const Queries<T, D> *q, int r, int lane) {
    constexpr int kPer = D / 32;
    int p[kPer], m[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = m[i] = 0;
    if (q) {
      uint32_t top = 0;  // magnitudes are ordered like their bits; a NaN is above infinity
#pragma unroll
      for (int h = 0; h < 8; ++h)
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) {
          const float2 v = Elem<T>::unpack(q->w[h][i]);
          top = max(top, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))));
        }
      top = __reduce_max_sync(kAll, top);
      if (top > 0 && top < 0x7f800000u) {
        const float inv = pow2(-exponent_for(__uint_as_float(top), 12));
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const float2 v = Elem<T>::unpack(q->w[h][i / 2]);
            const int c = __float2int_rn((i & 1 ? v.y : v.x) * inv);
            p[i] += max(c, 0);
            m[i] += min(c, 0);
            sum += c;
          }
      }
    }
    sum = __reduce_add_sync(kAll, sum);
    if (lane == 0) bias[r] = 128 * sum;
    // kPer consecutive codes are part of one lane's four of a step
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int code = n * D + lane * kPer;
      const int step = code / 64 * 4 + code % 16 / 4, c = code % 64 / 16;
#pragma unroll
      for (int high = 0; high < 2; ++high) {
        uint32_t h[kPer / 2];
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
          const int a = n ? m[i] : p[i], b = n ? m[i + 1] : p[i + 1];
          h[i / 2] = high ? Elem<__half>::pack(static_cast<float>(a >> 8), static_cast<float>(b >> 8))
                          : Elem<__half>::pack(static_cast<float>(a & 255), static_cast<float>(b & 255));
        }
        uint32_t *dst = reinterpret_cast<uint32_t *>(&frag[step][(2 * r + high) * 4 + c]) +
                        code % 4 / 2;
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) dst[i] = h[i];
      }
    }
  }
};

// 16 blocks of a row's table, in one warp: lane (g, c) holds codes 64 i + 16 c ..
// of blocks g and g + 8, and their scales.
template <int D> struct Unit {
  static constexpr int kBlocks = 16;
  static constexpr int kLoads = 2 * D / 64;
  uint4 x[2][kLoads];
  float scale[2];
  bool ok[2];

  // phys: blocks g and g + 8, -1 for none
  __device__ __forceinline__ void load(const SelectArgs &a, int kvh, const int (&phys)[2], int c) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      ok[b] = phys[b] >= 0;
      const int64_t cell = static_cast<int64_t>(phys[b]) * a.num_kv_heads + kvh;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        x[b][i] = make_uint4(0, 0, 0, 0);
        if (ok[b])
          x[b][i] = *reinterpret_cast<const uint4 *>(a.bounds + cell * (2 * D) + 64 * i + 16 * c);
      }
      scale[b] = ok[b] ? a.bound_scales[cell] : 0.f;
    }
  }
  // The keys of blocks g and g + 8 for rows c of kTiles tiles.
  template <int kTiles>
  __device__ __forceinline__ void keys(const Weights<D> *w, int lane, uint32_t (&key)[kTiles][2]) const {
    float acc[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int s = 0; s < Weights<D>::kSteps; ++s) {
      const uint32_t u0 = word_of(x[0][s / 4], s % 4) ^ 0x80808080u;
      const uint32_t u1 = word_of(x[1][s / 4], s % 4) ^ 0x80808080u;
      const uint32_t a0 = __byte_perm(u0, 0, 0x4140), a2 = __byte_perm(u0, 0, 0x4342);
      const uint32_t a1 = __byte_perm(u1, 0, 0x4140), a3 = __byte_perm(u1, 0, 0x4342);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const uint2 f = w[n].frag[s][lane];
        Elem<__half>::mma(acc[n], a0, a1, a2, a3, f.x, f.y);
      }
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int bias = w[n].bias[lane & 3];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int total = __float2int_rn(acc[n][2 * b] * 0x1p24f) +
                          256 * __float2int_rn(acc[n][2 * b + 1] * 0x1p24f) - bias;
        key[n][b] = 0;
        if (ok[b])
          // (+ 0: a scale of 0 gives 0, not -0, whose key is another)
          key[n][b] = key_of(
              scale[b] < INFINITY ? __fmul_rn(__int2float_rn(total), scale[b]) + 0.f : INFINITY);
      }
    }
  }
};

// A sequence's table, 16 blocks (g and g + 8 of a lane) at a time: entries may be
// read before the length is known, blocks are what is left of them then.
struct Table {
  const int32_t *row;
  int width;
  __device__ __forceinline__ Table(const SelectArgs &a, int seq)
      : row(a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq),
        width(a.max_blocks_per_seq) {}
  __device__ __forceinline__ void entries(int j, int (&e)[2]) const {
    e[0] = j < width ? row[j] : -1;
    e[1] = j + 8 < width ? row[j + 8] : -1;
  }
  // -1 for entry e of block j >= n, or (flagged) for one that is no block
  static __device__ __forceinline__ int block(const SelectArgs &a, int e, int j, int n) {
    if (j >= n) return -1;
    if (e >= 0 && e < a.num_blocks) return e;
    atomicOr(a.err, kErrBadBlock);
    return -1;
  }
};

// The largest t in [lo, hi] with at_least(t) >= want, or one with at_least(t) <=
// enough (>= want) too.  at_least(c) counts the keys >= c, at_least(lo) = count >=
// want, and no key that can be told from others is above hi; count becomes
// at_least(t).  Every second guess is where t would lie if the keys were spread
// evenly, the others halve the range (some five to nine guesses for exactly `want`
// of 256 keys, in place of twenty bits one by one).
template <typename F>
__device__ __forceinline__ uint32_t threshold(uint32_t lo, uint32_t hi, int &count, int want,
                                              int enough, F &&at_least) {
  int above = 0;  // keys > hi
  bool even = true;
  while (lo != hi && count > enough) {
    const uint32_t room = hi - lo;  // c - lo is 1 .. room
    uint32_t off = room / 2;
    if (even)
      off = static_cast<uint32_t>(static_cast<float>(room) *
                                  __fdividef(static_cast<float>(count - want),
                                             static_cast<float>(count - above)));
    even = !even;
    const uint32_t c = lo + 1 + min(off, room - 1);
    const int here = at_least(c);
    if (here >= want) {
      lo = c;
      count = here;
    } else {
      hi = c - 1;
      above = here;
    }
  }
  return lo;
}

// The keys of a row (key i * 32 + lane of n in k[i]; 0 past n): calls take(i, place)
// in the lanes of the `want` largest, ties to the first; want < n, and more than
// the forced ones or as many.
template <int KPL, typename F>
__device__ __forceinline__ void pick(const uint32_t (&k)[KPL], int n, int forced, int want, int lane,
                                     F &&take) {
  uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    if (i * 32 + lane < n && k[i] != kForced) {
      lo = min(lo, k[i]);
      hi = max(hi, k[i]);
    }
  }
  lo = __reduce_min_sync(kAll, lo);
  hi = __reduce_max_sync(kAll, hi);
  int count = n;
  uint32_t t = kForced;
  if (want == forced)
    count = want;
  else
    t = threshold(lo, hi, count, want, want, [&](uint32_t c) {
      int here = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) here += k[i] >= c ? 1 : 0;
      return static_cast<int>(__reduce_add_sync(kAll, here));
    });
  // keys above t are taken, and of those equal to it (the count has count - want
  // too many) the first
  int equal = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) equal += i * 32 + lane < n && k[i] == t ? 1 : 0;
  equal = __reduce_add_sync(kAll, equal);
  int left = equal - (count - want), place = 0;
  const uint32_t below = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    if (i * 32 >= n) break;
    const bool in = i * 32 + lane < n;
    const uint32_t eqs = __ballot_sync(kAll, in && k[i] == t);
    const bool mine = in && (k[i] > t || (k[i] == t && __popc(eqs & below) < left));
    const uint32_t all = __ballot_sync(kAll, mine);
    if (mine) take(i, place + __popc(all & below));
    place += __popc(all);
    left -= __popc(eqs);
  }
}

// Short contexts: at most 32 KPL blocks.  A CTA takes up to 4 TILES rows of a
// sequence and one KV head: its warps score 16 blocks at a time for all rows, so
// that bounds are read once for them; then a warp a row picks, with the row's keys
// in registers and no barrier.
// (Neither selection kernel lets the next one start early: its CTAs would wait on
// the SMs that this one's are on; drafted rows back to back 12.6 us, 11.5 without.)
template <typename T, int D, int KPL, int TILES, int NW>
__global__ void __launch_bounds__(NW * 32, KPL == 8 ? 4 : 1) select_short_kernel(const SelectArgs a) {
  using U = Unit<D>;
  constexpr int kRows = 4 * TILES;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Weights<D> *weights = reinterpret_cast<Weights<D> *>(smem_raw);
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem_raw + TILES * sizeof(Weights<D>));  // [rows][stride]
  const int stride = a.max_candidates;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.y, seq = blockIdx.z;
  const int bs = 1 << a.bs_log2, K = a.num_selected;
  grid_dependency_wait();  // queries, bounds and lengths may come from the kernel before
  const Table table(a, seq);
  const int32_t *bt_row = table.row;
  int j0 = warp * U::kBlocks, e[2];
  table.entries(j0 + g, e);
  Queries<T, D> q;  // (a row of its own needs no length to be found)
  if (!a.query_start && warp == 0) q.load(a, seq, kvh, lane);
  SelectRows rows;
  if (!rows.load(a, seq, tid == 0 && blockIdx.x == 0 && kvh == 0)) return;
  const int t0 = blockIdx.x * kRows, count = min(kRows, rows.rows - t0);
  if (count <= 0) return;
  const int most = (rows.base + t0 + count - 1 + bs - 1) >> a.bs_log2;  // blocks of the last row
  if (most > K) {
    static_assert(kRows <= NW, "a warp a row");
    if (warp < kRows) {
      if (a.query_start && warp < count) q.load(a, rows.row0 + t0 + warp, kvh, lane);
      weights[warp / 4].put(warp < count ? &q : nullptr, warp % 4, lane);
    }
    __syncthreads();
    for (; j0 < most; j0 += NW * U::kBlocks) {
      const int phys[2] = {Table::block(a, e[0], j0 + g, most), Table::block(a, e[1], j0 + 8 + g, most)};
      U unit;
      unit.load(a, kvh, phys, c);
      if (j0 + NW * U::kBlocks < most) table.entries(j0 + NW * U::kBlocks + g, e);
      uint32_t key[TILES][2];
      unit.template keys<TILES>(weights, lane, key);
#pragma unroll
      for (int n = 0; n < TILES; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          if (4 * n + c < count && j0 + 8 * b + g < most)
            keys[(4 * n + c) * stride + j0 + 8 * b + g] = key[n][b];
    }
    __syncthreads();
  }
  for (int r = warp; r < count; r += NW) {
    const int seen = rows.base + t0 + r, n = (seen + bs - 1) >> a.bs_log2;
    const int64_t at = (rows.row0 + t0 + r) * a.num_kv_heads + kvh;
    int32_t *out = a.tables + at * K;
    if (n <= K) {  // all of them
      for (int i = lane; i < K; i += 32) out[i] = i < n ? bt_row[i] : -1;
      if (lane == 0) a.lens[at] = seen;
      continue;
    }
    uint32_t k[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = i * 32 + lane;
      k[i] = j < n ? keys[r * stride + j] : 0;
      if (j < n && (j < a.num_sink || j >= n - a.num_recent)) k[i] = kForced;
    }
    bool last = false;
    pick<KPL>(k, n, a.num_sink + a.num_recent, K, lane, [&](int i, int place) {
      out[place] = bt_row[i * 32 + lane];
      last = last || i * 32 + lane == n - 1;
    });
    const bool any = __any_sync(kAll, last);
    if (lane == 0) a.lens[at] = K * bs - (any ? n * bs - seen : 0);
  }
}

// Long contexts: the CTAs of a cluster score a share of a row's blocks each, into
// the keys of the first one, which then picks.  What bounds it: HBM while blocks are
// scored (8 contexts of 32,768 to 131,072 tokens, 32 / 8 heads x 128: 51 MB, 9 to 10
// of 20.7 us), and the chain of latencies around that: the length, the queries'
// weights and the cluster's start 2.5 us, the pick 4 us in some 15 barriers.
constexpr int kBins = 2048, kBinBits = 11;
constexpr int kMaxSelCluster = 8;
constexpr int kRunKeys = 16;  // keys that a thread holds in registers at most

// Shared memory of a CTA, before the keys.
template <int D, int NT> struct SelectShared {
  Weights<D> weights;
  uint32_t bins[kBins];
  uint32_t part[NT / 32];
  uint32_t lo, hi;  // of the keys that are not forced
  uint32_t chosen_bin, chosen_above, chosen_count;
  uint32_t few[32], few_count;
  uint32_t few_keys[NT], few_at[NT];  // keys that may be taken, and where they are
};

// Sum over the CTA's threads before this one; `all`: over all of them.
template <int NT>
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t *part, uint32_t &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(kAll, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const uint32_t x = part[w];
    before += w < warp ? x : 0;
    all += x;
  }
  return before + incl - v;
}

// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void red_cluster_min(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_max(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The K largest of n > K keys, ties to the first; the keys' indexes take their
// places in order from keys[0] on.  For a whole CTA.  In a turn thread i takes
// keys L i .. L i + L - 1, from one of its own on around (different lanes,
// different banks).  ONE: one turn does (n <= NT L), the keys stay in registers.
template <int NT, int L, bool ONE, typename Shared>
__device__ __forceinline__ void pick_long(const SelectArgs &a, Shared &sh, uint32_t *keys, int n) {
  const int tid = threadIdx.x, lane = tid & 31;
  constexpr int kTurn = NT * L;
  const int first = lane * L / 32;
  uint32_t k[L];  // k[i] is key (first + i) % L of the run; 0 past n
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int j = j0 + tid * L + ((first + i) & (L - 1));
      k[i] = j < n ? keys[j] : 0;
    }
  };
  if (ONE) load(0);
  // f() with every turn's keys in k
  auto turns = [&](auto &&f) {
    if (ONE) {
      f();
    } else {
      for (int j0 = 0; j0 < n; j0 += kTurn) {
        load(j0);
        f();
      }
    }
  };
  uint32_t lo = sh.lo, hi = sh.hi;
  const int forced = a.num_sink + a.num_recent;
  int need = a.num_selected - forced;  // fewer than the keys not forced
  if (ONE && need > 0 && need <= n / L) {
    // As many whole runs as are wanted: what `need` of the runs' largest keys reach,
    // the need-th largest key does, too.  With a bound that half as many more of
    // them reach some 240 keys of 8,192 in 512 runs are left for the 128 largest;
    // among these a thread a key picks.  (Cutting the whole range instead, as below:
    // 4.8 us for 8,192 keys in 256 runs, against 4.)
    uint32_t top = lo;
#pragma unroll
    for (int i = 0; i < L; ++i) top = max(top, k[i] == kForced ? 0 : k[i]);
    int count = n / L;
    const uint32_t least = threshold(lo, hi, count, need, need + need / 2, [&](uint32_t c) {
      return __syncthreads_count(tid < n / L && top >= c);
    });
    uint32_t mine = 0, all;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int at = (first + i) & (L - 1);
      mine |= (tid * L + at < n && k[i] >= least ? 1u : 0u) << at;
    }
    int place = sum_before<NT>(__popc(mine), sh.part, all);
    if (all <= NT) {
      while (mine) {
        const int i = __ffs(mine) - 1;
        mine &= mine - 1;
        sh.few_keys[place] = keys[tid * L + i];
        sh.few_at[place++] = tid * L + i;
      }
      __syncthreads();
      const bool real = tid < static_cast<int>(all);
      const uint32_t x = real ? sh.few_keys[tid] : 0;
      count = all;
      const uint32_t t = threshold(least, hi, count, a.num_selected, a.num_selected, [&](uint32_t c) {
        return __syncthreads_count(real && x >= c);
      });
      // keys above t are taken, and of those equal to it the first
      const bool eq = real && x == t;
      const int left = a.num_selected - __syncthreads_count(real && x > t);
      const uint32_t before = sum_before<NT>((real && x > t ? 1u : 0u) | (eq ? 0x10000u : 0u), sh.part, all);
      const int ties = before >> 16;
      if ((real && x > t) || (eq && ties < left))
        keys[(before & 0xffff) + min(ties, left)] = sh.few_at[tid];
      __syncthreads();
      return;
    }
    lo = least;  // the general way
    __syncthreads();
  }
  bool whole = need == 0;  // every key of [lo, hi] is taken
  if (whole) lo = hi = kForced;
  // The need-th largest key: the range [lo, hi] that holds it is cut into kBins
  // equal parts, their keys counted, and the part that holds it taken, until
  // what is left of the range is taken whole, is one value or holds few keys.
  while (!whole && lo != hi) {
    const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
#pragma unroll
    for (int i = 0; i < kBins; i += NT) sh.bins[i + tid] = 0;
    if (tid == 0) sh.few_count = 0;
    __syncthreads();
    turns([&] {
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (k[i] >= lo && k[i] <= hi) atomicAdd(&sh.bins[(k[i] - lo) >> shift], 1u);
    });
    __syncthreads();
    // the part with the need-th largest key: sums over the parts from the top;
    // thread i holds some parts, from part kBins - 1 - kPer i down
    constexpr int kPer = kBins / NT;
    uint32_t mine[kPer], sum = 0, all;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      mine[b] = sh.bins[kBins - 1 - tid * kPer - b];
      sum += mine[b];
    }
    uint32_t before = sum_before<NT>(sum, sh.part, all);
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      if (before < static_cast<uint32_t>(need) && before + mine[b] >= static_cast<uint32_t>(need)) {
        sh.chosen_bin = kBins - 1 - tid * kPer - b;
        sh.chosen_above = before;
        sh.chosen_count = mine[b];
      }
      before += mine[b];
    }
    __syncthreads();
    const int count = sh.chosen_count;
    need -= sh.chosen_above;
    whole = count == need;
    lo += sh.chosen_bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1));
    if (!whole && lo != hi && count <= 32) {
      // the need-th largest of them: its rank is the number of larger ones, and of
      // equal ones before it
      turns([&] {
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (k[i] >= lo && k[i] <= hi) sh.few[atomicAdd(&sh.few_count, 1u)] = k[i];
      });
      __syncthreads();
      const uint32_t x = lane < count ? sh.few[lane] : 0;
      int rank = 0, above = 0;
      for (int i = 0; i < count; ++i) {
        const uint32_t other = __shfl_sync(kAll, x, i);
        rank += other > x || (other == x && i < lane) ? 1 : 0;
        above += other > x ? 1 : 0;
      }
      const int who = __ffs(__ballot_sync(kAll, lane < count && rank == need - 1)) - 1;
      lo = hi = __shfl_sync(kAll, x, who);
      need -= __shfl_sync(kAll, above, who);
    }
  }
  // Keys above hi are taken, those of [lo, hi] too if `whole`; otherwise they are
  // one value, and the first `need` of them are.  (A key's index is at least its
  // place: written over the keys, it meets none that is still to be read.)
  int place0 = 0, j0 = 0;  // taken before this turn's keys, which begin at j0
  turns([&] {
    uint32_t above = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int at = (first + i) & (L - 1);
      const bool in = j0 + tid * L + at < n;
      above |= (in && (whole ? k[i] >= lo : k[i] > lo) ? 1u : 0u) << at;
      equal |= (in && !whole && k[i] == lo ? 1u : 0u) << at;
    }
    uint32_t all;
    __syncthreads();  // sh.part is free
    const uint32_t before = sum_before<NT>(__popc(above) | (__popc(equal) << 16), sh.part, all);
    const int ties = before >> 16;
    int place = place0 + static_cast<int>(before & 0xffff) + min(ties, need);
    int left = max(0, need - ties);
    uint32_t todo = above | equal;
    while (todo) {
      const int i = __ffs(todo) - 1;
      todo &= todo - 1;
      if ((equal >> i) & 1u) {
        if (left == 0) continue;
        --left;
      }
      keys[place++] = j0 + tid * L + i;
    }
    place0 += static_cast<int>(all & 0xffff) + min(static_cast<int>(all >> 16), need);
    need -= min(static_cast<int>(all >> 16), need);
    j0 += kTurn;
  });
  __syncthreads();
}

// ROWS: rows of a sequence that a cluster scores at once, 1 or 4 (four rows are one
// product); row r's keys gather in CTA r, which picks for it.  (4 rows of 4 contexts
// of 32,768 to 131,072 tokens 20.0 us, 5 rows 33, where a cluster for each row took
// 42.6 and 49.  Eight rows in two products: 25 us for the 5 rows, but as slow or up to
// 12 % slower where more clusters are to be served than run at once.)
template <typename T, int D, int NT, int ROWS>
__global__ void __launch_bounds__(NT, 1024 / NT) select_long_kernel(const SelectArgs a) {
  using U = Unit<D>;
  static_assert(ROWS == 1 || ROWS == 4, "of one product");
  using Shared = SelectShared<D, NT>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem_raw + sizeof(Shared));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % a.cluster;
  const int t0 = static_cast<int>(blockIdx.x) / a.cluster * ROWS;  // first row of the sequence's
  // (heads last: neighbouring clusters are of different sequences, so that the
  // long ones do not meet on the same SMs)
  const int seq = blockIdx.y, kvh = blockIdx.z;
  const int bs = 1 << a.bs_log2, K = a.num_selected;
  if (tid == 0) sh.lo = 0xffffffffu, sh.hi = 0;
  grid_dependency_wait();  // queries, bounds and lengths may come from the kernel before

  const Table table(a, seq);
  const int32_t *bt_row = table.row;
  Queries<T, D> q;  // (a row of its own needs no length to be found)
  if (!a.query_start && warp == 0) q.load(a, seq, kvh, lane);
  SelectRows rows;
  if (!rows.load(a, seq, tid == 0 && blockIdx.x == 0 && kvh == 0) || t0 >= rows.rows)
    return;  // (the whole cluster)
  const int count = ROWS == 1 ? 1 : min(ROWS, rows.rows - t0);
  // of row r < count: the tokens and blocks that it sees, more than the row before
  auto seen_by = [&](int r) { return rows.base + t0 + r; };
  auto blocks_of = [&](int r) { return (seen_by(r) + bs - 1) >> a.bs_log2; };
  auto cell_of = [&](int r) { return (rows.row0 + t0 + r) * a.num_kv_heads + kvh; };
  auto take_all = [&](int r) {
    const int n = blocks_of(r);
    for (int i = tid; i < K; i += NT) a.tables[cell_of(r) * K + i] = i < n ? bt_row[i] : -1;
    if (tid == 0) a.lens[cell_of(r)] = seen_by(r);
  };
  const int most = blocks_of(count - 1);
  if (most <= K) {
    for (int r = rank; r < count; r += a.cluster) take_all(r);
    return;  // (the whole cluster)
  }
  // CTAs that have work; the others make room (a CTA that has left counts as
  // arrived at the cluster's barriers)
  const int units = (most + U::kBlocks - 1) / U::kBlocks;
  const int ctas = max(count, min(a.cluster, (units + a.units_per_cta - 1) / a.units_per_cta));
  if (rank >= ctas) return;
  if (ctas > 1) cluster_arrive();
  // the warp's units, `step` blocks apart; the next one's entries are read while one
  // is worked on
  const int step = ctas * (NT / 32) * U::kBlocks;
  int j0 = (rank * (NT / 32) + warp) * U::kBlocks, e[2];
  table.entries(j0 + g, e);
  U unit;
  auto fetch = [&] {
    const int phys[2] = {Table::block(a, e[0], j0 + g, most), Table::block(a, e[1], j0 + 8 + g, most)};
    unit.load(a, kvh, phys, c);
    if (j0 + step < most) table.entries(j0 + step + g, e);
  };
  // (four warps make the weights, the others' first loads are under way meanwhile)
  if (warp < 4) {
    if (a.query_start && warp < count) q.load(a, rows.row0 + t0 + warp, kvh, lane);
    sh.weights.put(warp < count ? &q : nullptr, warp, lane);
  } else if (j0 < most) {
    fetch();
  }
  __syncthreads();
  if (ctas > 1) cluster_wait();  // the CTAs that pick have started: their shared memory is there
  // the lane's row c: its blocks (none if there is no such row), where its keys go
  const int n_of = c < count ? blocks_of(c) : 0;
  const uint32_t keys_at = ctas > 1 ? cluster_addr(keys, c < count ? c : 0) : 0;
  uint32_t lo = 0xffffffffu, hi = 0;  // of the keys that are not forced
  for (bool there = warp >= 4; j0 < most; j0 += step, there = false) {
    if (!there) fetch();
    uint32_t key[1][2];
    unit.template keys<1>(&sh.weights, lane, key);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = j0 + 8 * b + g;
      if (j < n_of) {
        uint32_t k = key[0][b];
        if (j < a.num_sink || j >= n_of - a.num_recent) {
          k = kForced;
        } else {
          lo = min(lo, k);
          hi = max(hi, k);
        }
        if (ctas > 1)
          st_cluster_u32(keys_at + j * 4, k);
        else
          keys[j] = k;
      }
    }
  }
  if constexpr (ROWS == 1) {
    lo = __reduce_min_sync(kAll, lo);
    hi = __reduce_max_sync(kAll, hi);
  } else {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      lo = min(lo, __shfl_xor_sync(kAll, lo, off));
      hi = max(hi, __shfl_xor_sync(kAll, hi, off));
    }
  }
  if (lane < count) {
    if (ctas > 1) {
      red_cluster_min(cluster_addr(&sh.lo, lane), lo);
      red_cluster_max(cluster_addr(&sh.hi, lane), hi);
    } else {
      atomicMin(&sh.lo, lo);
      atomicMax(&sh.hi, hi);
    }
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();
  if (rank >= count) return;
  const int r = ROWS == 1 ? 0 : rank, n = blocks_of(r);
  if (ROWS > 1 && n <= K) {
    take_all(r);
    return;
  }
  if (n <= NT * 4)
    pick_long<NT, 4, true>(a, sh, keys, n);
  else if (n <= NT * kRunKeys)
    pick_long<NT, kRunKeys, true>(a, sh, keys, n);
  else
    pick_long<NT, kRunKeys, false>(a, sh, keys, n);
  int32_t *out = a.tables + cell_of(r) * K;
  for (int i = tid; i < K; i += NT) out[i] = bt_row[keys[i]];
  if (tid == 0)
    a.lens[cell_of(r)] =
        K * bs - (keys[K - 1] == static_cast<uint32_t>(n - 1) ? n * bs - seen_by(r) : 0);
}

template <typename T, int D, int NT, int ROWS> cudaError_t launch_long(SelectArgs a, cudaStream_t stream) {
  const size_t smem = sizeof(SelectShared<D, NT>) + static_cast<size_t>(a.max_candidates) * 4;
  constexpr size_t most = sizeof(SelectShared<D, NT>) + kMaxCandidates * 4;
  static_assert(most <= 227 * 1024, "shared memory");
  auto kern = select_long_kernel<T, D, NT, ROWS>;
  static SmemLimitOnce smem_limit;
  const cudaError_t e = smem_limit.ensure(kern, most);
  if (e != cudaSuccess) return e;
  const int tiles = (a.max_q_len - 1) / ROWS + 1;
  const int64_t clusters = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * tiles;
  // CTAs that may share a row: as many as run at once (2 kSms), each with 128 blocks
  // at least; twice as many where each has 512, since those of the shorter
  // contexts then leave at once.  (32 / 8 heads x 128, one row a sequence, with this
  // rule and with one CTA: 16,000 tokens 6.2 and 11.5 us, 131,072 tokens 12.2 and 44,
  // 16 x 1,000 to 16,000 10.3 and 12.0, 16 x 16,000 to 65,000 25.4 and 43.6; with twice
  // as many from 128 blocks on 8 x 16,000 take 16.3 us in place of 8.5, with only as
  // many as run at once 16 x 16,000 to 65,000 29.8 in place of 25.4.)
  a.cluster = ROWS;  // a CTA for each row that a cluster picks for
  for (int c = a.cluster; c < kMaxSelCluster; c *= 2) {
    const int64_t ctas = 2 * c * clusters;
    if (!(ctas <= 2 * kSms && a.max_candidates >= 128 * c) &&
        !(ctas <= 4 * kSms && a.max_candidates >= 512 * c))
      break;
    a.cluster = 2 * c;
  }
  // where they are more than run at once, four units a warp
  a.units_per_cta = NT / 32 * (a.cluster * clusters <= 2 * kSms ? 1 : 4);
  return launch_clusters(a.cluster, kern,
                         dim3(static_cast<unsigned>(a.cluster * tiles), a.num_seqs, a.num_kv_heads),
                         dim3(NT), smem, stream, a);
}

template <typename T, int D, int KPL, int TILES, int NW>
cudaError_t launch_short(const SelectArgs &a, cudaStream_t stream) {
  constexpr int kRows = 4 * TILES;
  const int rows = a.max_q_len < kRows ? a.max_q_len : kRows;
  constexpr size_t fixed = TILES * sizeof(Weights<D>);
  const size_t smem = fixed + static_cast<size_t>(rows) * a.max_candidates * 4;
  static_assert(fixed + static_cast<size_t>(kRows) * 32 * KPL * 4 <= 48 * 1024,
                "shared memory that needs no leave");
  const unsigned tiles = (static_cast<unsigned>(a.max_q_len) + kRows - 1) / kRows;
  return launch_dependent(select_short_kernel<T, D, KPL, TILES, NW>,
                          dim3(tiles, a.num_kv_heads, a.num_seqs), dim3(NW * 32), smem, stream, a);
}

// Which kernel (32 / 8 heads x 128, GPU time of a call).
// Single rows: up to 256 candidates the short one, 64 x 512 to 4,096 tokens 9.5 us
// (long, 256 threads: 10.2); above, the long one, 64 x 2,000 to 8,000 tokens 15.3 us
// (20.6), 256 of them 44 (56), one of 16,000 6.2 (20.9).
// The long one has 256 threads, four CTAs an SM, while their registers hold the keys
// of the longest context, and else 512: 64 x 2,000 to 8,000 tokens 15.3 us (512:
// 20.6), 200 x 8,000 to 30,000 95 (106); 131,072 tokens 12.2 us with 512 and 15.0
// with 256.
// Several rows a sequence: up to 256 candidates the short one, 5 rows of 64 x 512 to
// 4,096 tokens 11.5 us (34.5 with a cluster for each row); up to 1,024 too, where
// there are so many tiles of four rows that the long one's clusters would wait for
// one another: 64 x 2,000 to 8,000 tokens, 4 rows 22.4 us (long 34), 5 rows 27.3 (55);
// 200 x 4,000 to 9,000, 4 rows 69 (100); 16 x 4,000 to 16,000, 5 rows 18.2 (22.4).
// The long one for fewer: 8 x 2,000 to 8,000, 2 rows 7.8 us (short 12.9); 8 x 4,000
// to 16,000, 8 rows 13.1 (18.4); 32 x 8,000 to 16,000, 4 rows 25.3 (38.3).
template <typename T, int D> cudaError_t launch_select_t(const SelectArgs &a, cudaStream_t stream) {
  if (a.max_q_len == 1) {
    if (a.max_candidates > 256 * kRunKeys) return launch_long<T, D, 512, 1>(a, stream);
    if (a.max_candidates > 256) return launch_long<T, D, 256, 1>(a, stream);
    return launch_short<T, D, 8, 1, 4>(a, stream);
  }
  if (a.max_candidates > 256 * kRunKeys) return launch_long<T, D, 512, 4>(a, stream);
  const int64_t tiles = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * ((a.max_q_len - 1) / 4 + 1);
  const int few = a.max_candidates <= 512 ? kSms / 2 : a.max_q_len > 4 ? kSms : 2 * kSms;
  if (a.max_candidates > 1024 || (a.max_candidates > 256 && tiles <= few))
    return launch_long<T, D, 256, 4>(a, stream);
  if (a.max_q_len > 4) {
    if (a.max_candidates > 512) return launch_short<T, D, 32, 2, 8>(a, stream);
    if (a.max_candidates > 256) return launch_short<T, D, 16, 2, 8>(a, stream);
    return launch_short<T, D, 8, 2, 8>(a, stream);
  }
  if (a.max_candidates > 512) return launch_short<T, D, 32, 1, 4>(a, stream);
  if (a.max_candidates > 256) return launch_short<T, D, 16, 1, 4>(a, stream);
  return launch_short<T, D, 8, 1, 4>(a, stream);
}

}  // namespace

cudaError_t launch_key_bounds(const BoundsArgs &a, int head_dim, int dtype, Kv kv,
                              cudaStream_t stream) {
  if (dtype == 0)
    return head_dim == 128 ? launch_bounds_kv<__half, 128>(a, kv, stream)
                           : launch_bounds_kv<__half, 64>(a, kv, stream);
  return head_dim == 128 ? launch_bounds_kv<__nv_bfloat16, 128>(a, kv, stream)
                         : launch_bounds_kv<__nv_bfloat16, 64>(a, kv, stream);
}

cudaError_t launch_select(const SelectArgs &a, int head_dim, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return head_dim == 128 ? launch_select_t<__half, 128>(a, stream)
                           : launch_select_t<__half, 64>(a, stream);
  return head_dim == 128 ? launch_select_t<__nv_bfloat16, 128>(a, stream)
                         : launch_select_t<__nv_bfloat16, 64>(a, stream);
}

}  // namespace pa
