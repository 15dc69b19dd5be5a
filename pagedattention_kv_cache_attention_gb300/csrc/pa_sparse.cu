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
// largest magnitude <= 4095 2^f.  The bounds of the group's heads add up to
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

constexpr int kBoundsWarps = 4;

// A warp for a (block, KV head): every lane keeps the extremes of its channels
// over the rows that it reads, lanes of the same channels are joined by shuffles.
template <typename T, int D, Kv KV>
__global__ void __launch_bounds__(kBoundsWarps * 32) key_bounds_kernel(const BoundsArgs a) {
  using Share = KeyShare<D, KV>;
  using MT = typename std::conditional<KV == Kv::k16, T, __half>::type;
  constexpr int W = Share::kWords, kLanes = Share::kLanes, kRows = Share::kRows;
  constexpr int kTake = KV == Kv::k16 ? 8 : 4;  // rows that a lane has in flight
  grid_dependency_wait();  // the keys may come from the kernel before
  grid_launch_dependents();
  const int seq = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kBoundsWarps + (threadIdx.x >> 5);
  const int h = static_cast<int>(item % a.num_kv_heads);
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
  const int64_t j = ((ctx - new_tokens) >> a.bs_log2) + item / a.num_kv_heads;
  if (j > (ctx - 1) >> a.bs_log2) return;
  const int phys = a.block_tables[static_cast<int64_t>(seq) * a.max_blocks_per_seq + j];
  if (phys < 0 || phys >= a.num_blocks) {
    if (lane == 0) atomicOr(a.err, kErrBadBlock);
    return;
  }
  const int rows = min(bs, static_cast<int>(ctx - (j << a.bs_log2)));
  const int64_t cell = static_cast<int64_t>(phys) * a.num_kv_heads + h;
  const int block_bytes = KV == Kv::kFp4 ? fp4_tile_bytes(bs, D) : bs * D * (KV == Kv::k16 ? 2 : 1);
  const uint8_t *block = static_cast<const uint8_t *>(a.k_cache) + cell * block_bytes;

  const int share = lane % kLanes, r0 = lane / kLanes;
  // (row 0 counts always: rows past the end are read as that one)
  uint32_t hi[W], lo[W];
  Share::widen(Share::load(block, bs, 0, share), hi);
#pragma unroll
  for (int w = 0; w < W; ++w) lo[w] = hi[w];
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
      for (int w = 0; w < W; ++w) extremes2<MT>(x[w], hi[w], lo[w]);
    }
  }
  float top = 0.f;
  bool odd = false;  // an infinity or a NaN
  float up[2 * W], down[2 * W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
#pragma unroll
    for (int off = kLanes; off < 32; off <<= 1) {
      const uint32_t oh = __shfl_xor_sync(kAll, hi[w], off), ol = __shfl_xor_sync(kAll, lo[w], off);
      uint32_t unused = ol;
      extremes2<MT>(oh, hi[w], unused);
      unused = oh;
      extremes2<MT>(ol, unused, lo[w]);
    }
    const float2 x = Elem<MT>::unpack(hi[w]), y = Elem<MT>::unpack(lo[w]);
    up[2 * w] = x.x, up[2 * w + 1] = x.y, down[2 * w] = y.x, down[2 * w + 1] = y.y;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float m = fmaxf(fabsf(up[2 * w + e]), fabsf(down[2 * w + e]));
      odd = odd || !(fabsf(up[2 * w + e]) < INFINITY) || !(fabsf(down[2 * w + e]) < INFINITY);
      top = fmaxf(top, m);
    }
  }
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
  odd = __any_sync(kAll, odd);
  const bool none = odd || top == 0.f;
  const int e = none ? 0 : exponent_for(top, 7);
  const float inv = none ? 0.f : pow2(-e);
  // group 0 of the lanes writes the largest, group 1 the smallest
  if (r0 < 2) {
    uint32_t out[Share::kElems / 4];
#pragma unroll
    for (int q = 0; q < Share::kElems / 4; ++q) {
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = 4 * q + b;
        // (2^-e is exact, and so is the product but for results below 2^-149)
        const int code = none ? 0 : r0 == 0 ? __float2int_ru(up[i] * inv) : __float2int_rd(down[i] * inv);
        word |= static_cast<uint32_t>(code & 0xff) << (8 * b);
      }
      out[q] = word;
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.bounds + (cell * 2 + r0) * D + share * Share::kElems);
#pragma unroll
    for (int q = 0; q < Share::kElems / 4; q += 2)
      *reinterpret_cast<uint2 *>(dst + q) = make_uint2(out[q], out[q + 1]);
    if (lane == 0) a.bound_scales[cell] = odd ? INFINITY : none ? 0.f : pow2(e);
  }
}

template <typename T, int D, Kv KV>
cudaError_t launch_bounds(const BoundsArgs &a, cudaStream_t stream) {
  // blocks that max_q_len new tokens can reach into
  int64_t blocks = ((static_cast<int64_t>(a.max_q_len) - 1) >> a.bs_log2) + 2;
  blocks = blocks < a.max_blocks_per_seq ? blocks : a.max_blocks_per_seq;
  if (a.max_q_len == 1) blocks = 1;
  const int64_t ctas = (blocks * a.num_kv_heads + kBoundsWarps - 1) / kBoundsWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_dependent(key_bounds_kernel<T, D, KV>, dim3(static_cast<unsigned>(ctas), a.num_seqs),
                          dim3(kBoundsWarps * 32), 0, stream, a);
}

template <typename T, int D>
cudaError_t launch_bounds_kv(const BoundsArgs &a, Kv kv, cudaStream_t stream) {
  if (kv == Kv::kFp8) return launch_bounds<__half, D, Kv::kFp8>(a, stream);
  if (kv == Kv::kFp4) return launch_bounds<__half, D, Kv::kFp4>(a, stream);
  return launch_bounds<T, D, Kv::k16>(a, stream);
}

// ---------------------------------------------------------------- selection

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048, kBinBits = 11;
constexpr uint32_t kForced = 0xffffffffu;  // above the key of every score

// An unsigned key in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ int dp2a_lo(uint32_t a, uint32_t b, int c) {
  return __dp2a_lo(static_cast<int>(a), static_cast<int>(b), c);
}
__device__ __forceinline__ int dp2a_hi(uint32_t a, uint32_t b, int c) {
  return __dp2a_hi(static_cast<int>(a), static_cast<int>(b), c);
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Shared memory of a CTA, after the keys [max_candidates].
template <int D> struct SelectShared {
  uint32_t bins[kBins];
  int16_t w[2][D];              // P, N
  uint16_t q[8][D];             // the group's queries
  uint32_t part[3][kSelWarps];
  uint32_t chosen_bin, chosen_above, chosen_count;
};

// Sum over lanes of a warp of R values held by R lanes each ... in a butterfly
// that halves the values as it goes: lane r of a group of R ends with the sum of
// v[r] over its group.
template <int R> __device__ __forceinline__ int transpose_sum(int (&v)[R], int lane) {
#pragma unroll
  for (int half = R / 2; half > 0; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const int keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(kAll, give, half);
    }
  }
  return v[0];
}

// The cluster's CTAs score a share of the row's blocks each, into the keys of the
// first one, which then picks and writes.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  constexpr int kLanes = 2 * D / 16;      // lanes that hold a block's bounds, 16 codes each
  constexpr int kSteps = kLanes;          // blocks of a warp's window of 32 that a lane sees
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem_raw);
  SelectShared<D> &sh = *reinterpret_cast<SelectShared<D> *>(
      smem_raw + ((static_cast<size_t>(a.max_candidates) * 4 + 15) & ~static_cast<size_t>(15)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = a.cluster, rank = static_cast<int>(blockIdx.x) % cluster;
  const int t = static_cast<int>(blockIdx.x) / cluster;  // row of the sequence's chunk
  const int kvh = blockIdx.y, seq = blockIdx.z;
  const int bs = 1 << a.bs_log2, K = a.num_selected;
  grid_dependency_wait();  // queries, bounds and lengths may come from the kernel before
  grid_launch_dependents();

  // the row, and the tokens that it sees
  const int ctx = a.context_lens[seq];
  int64_t row = seq;
  int seen = ctx;
  bool fine = ctx >= 0 && ctx <= a.max_context_len &&
              ctx <= static_cast<int64_t>(a.max_blocks_per_seq) << a.bs_log2;
  if (a.query_start) {
    const int q0 = a.query_start[seq], q_len = a.query_start[seq + 1] - q0;
    fine = fine && q_len >= 0 && q_len <= ctx && q_len <= a.max_q_len;
    if (!fine && tid == 0 && blockIdx.x == 0 && kvh == 0) atomicOr(a.err, kErrBadLen);
    if (!fine || t >= q_len) return;  // (the whole cluster)
    row = q0 + t;
    seen = ctx - q_len + t + 1;
  } else if (!fine) {
    if (tid == 0 && blockIdx.x == 0 && kvh == 0) atomicOr(a.err, kErrBadLen);
    seen = 0;
  }
  const int n = (seen + bs - 1) >> a.bs_log2;
  const int32_t *bt_row = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
  int32_t *out = a.tables + (row * a.num_kv_heads + kvh) * K;
  int32_t *out_len = a.lens + row * a.num_kv_heads + kvh;
  if (n <= K) {  // all of them
    if (rank == 0) {
      for (int i = tid; i < K; i += kSelThreads) out[i] = i < n ? bt_row[i] : -1;
      if (tid == 0) *out_len = seen;
    }
    return;  // (the whole cluster)
  }

  // the group's queries as integers, and their sums by sign
  const int G = a.group;
  const T *q = static_cast<const T *>(a.query) + (row * a.num_q_heads + kvh * G) * D;
  {
    float top = 0.f;
    for (int i = tid; i < G * (D / 8); i += kSelThreads) {
      const uint4 x = reinterpret_cast<const uint4 *>(q)[i];
      *reinterpret_cast<uint4 *>(&sh.q[0][0] + i * 8) = x;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 v = Elem<T>::unpack(word_of(x, w));
        // (a NaN becomes an infinity: both are left out)
        const float m0 = fabsf(v.x), m1 = fabsf(v.y);
        top = fmaxf(top, fmaxf(m0 == m0 ? m0 : INFINITY, m1 == m1 ? m1 : INFINITY));
      }
    }
    // (magnitudes are ordered like their bits)
    const uint32_t most = __reduce_max_sync(kAll, __float_as_uint(top));
    if (lane == 0) sh.part[0][warp] = most;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) all = max(all, sh.part[0][w]);
    top = __uint_as_float(all);
    if (tid < D) {
      int p = 0, m = 0;
      if (top > 0.f && top < INFINITY) {
        const float inv = pow2(-exponent_for(top, 12));
        for (int h = 0; h < G; ++h) {
          const uint16_t b = sh.q[h][tid];
          const float x = Elem<T>::unpack(b).x;
          const int c = __float2int_rn(x * inv);
          p += max(c, 0);
          m += min(c, 0);
        }
      }
      sh.w[0][tid] = static_cast<int16_t>(p);
      sh.w[1][tid] = static_cast<int16_t>(m);
    }
    __syncthreads();
  }
  uint32_t w[8];  // the 16 sums that the lane's codes meet
  {
    const uint4 *src = reinterpret_cast<const uint4 *>(&sh.w[0][0] + (lane % kLanes) * 16);
    const uint4 x = src[0], y = src[1];
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }

  if (cluster > 1) cluster_sync();  // the first CTA has started: its shared memory is there
  const uint32_t keys_at = cluster > 1 ? cluster_addr(keys, 0) : 0;
  // windows of 32 blocks, one warp's each: lane l ends with the score of block l
  for (int j0 = (rank * kSelWarps + warp) * 32; j0 < n; j0 += cluster * kSelWarps * 32) {
    const int j = j0 + lane;
    int phys = j < n ? bt_row[j] : -1;
    if (phys >= a.num_blocks || phys < 0) {
      if (j < n) atomicOr(a.err, kErrBadBlock);
      phys = -1;
    }
    const int64_t mine = static_cast<int64_t>(phys) * a.num_kv_heads + kvh;
    const float scale = phys >= 0 ? a.bound_scales[mine] : 0.f;
    uint4 x[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int p = __shfl_sync(kAll, phys, (lane / kLanes) * kSteps + i);
      x[i] = make_uint4(0, 0, 0, 0);
      if (p >= 0)
        x[i] = *reinterpret_cast<const uint4 *>(
            a.bounds + (static_cast<int64_t>(p) * a.num_kv_heads + kvh) * (2 * D) + (lane % kLanes) * 16);
    }
    int v[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      int s = dp2a_lo(w[0], x[i].x, 0);
      s = dp2a_hi(w[1], x[i].x, s);
      s = dp2a_lo(w[2], x[i].y, s);
      s = dp2a_hi(w[3], x[i].y, s);
      s = dp2a_lo(w[4], x[i].z, s);
      s = dp2a_hi(w[5], x[i].z, s);
      s = dp2a_lo(w[6], x[i].w, s);
      v[i] = dp2a_hi(w[7], x[i].w, s);
    }
    const int total = transpose_sum<kSteps>(v, lane % kLanes);
    uint32_t key = 0;
    if (phys >= 0)
      key = key_of(scale < INFINITY ? __fmul_rn(__int2float_rn(total), scale) : INFINITY);
    if (j < a.num_sink || j >= n - a.num_recent) key = kForced;
    if (j < n) {
      if (cluster > 1)
        st_cluster_u32(keys_at + j * 4, key);
      else
        keys[j] = key;
    }
  }
  if (cluster > 1) cluster_sync(); else __syncthreads();
  if (rank != 0) return;

  // The K-th largest key: the range [lo, hi] that holds it is cut into kBins
  // equal parts, their keys counted, and the part that holds it taken, until
  // what is left of the range is taken whole or is one value.
  uint32_t lo = 0xffffffffu, hi = 0;
  int forced = 0;
  for (int i = tid; i < n; i += kSelThreads) {
    const uint32_t k = keys[i];
    if (k == kForced) {
      ++forced;
    } else {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
  lo = __reduce_min_sync(kAll, lo);
  hi = __reduce_max_sync(kAll, hi);
  forced = __reduce_add_sync(kAll, forced);
  if (lane == 0) sh.part[0][warp] = lo, sh.part[1][warp] = hi, sh.part[2][warp] = forced;
  __syncthreads();
  forced = 0;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    lo = min(lo, sh.part[0][i]);
    hi = max(hi, sh.part[1][i]);
    forced += sh.part[2][i];
  }
  int need = K - forced;  // >= 0: the call's checks; fewer than n - forced
  bool whole = need == 0;  // every key of [lo, hi] is taken
  if (whole) lo = kForced, hi = kForced;
  while (!whole && lo != hi) {
    const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
    __syncthreads();
    for (int i = tid; i < kBins; i += kSelThreads) sh.bins[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&sh.bins[(k - lo) >> shift], 1u);
    }
    __syncthreads();
    // the part with the need-th largest key: sums over the parts from the top;
    // thread i holds 8 parts, from part kBins - 1 - 8 i down
    constexpr int kPer = kBins / kSelThreads;
    uint32_t mine[kPer], sum = 0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      mine[b] = sh.bins[kBins - 1 - tid * kPer - b];
      sum += mine[b];
    }
    uint32_t before = sum;  // inclusive over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(kAll, before, off);
      if (lane >= off) before += x;
    }
    if (lane == 31) sh.part[0][warp] = before;
    __syncthreads();
    before -= sum;
    for (int i = 0; i < warp; ++i) before += sh.part[0][i];
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
    need -= sh.chosen_above;
    whole = sh.chosen_count == static_cast<uint32_t>(need);
    lo += sh.chosen_bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1));
  }
  // keys above hi are taken, those of [lo, hi] too if `whole`; otherwise they
  // are one value, and the first `need` of them are.  A warp takes a run of
  // the blocks, so that places and ties follow the blocks' order.
  const int per = ((n + kSelThreads - 1) / kSelThreads) * 32;  // blocks of a warp
  const int begin = min(warp * per, n), end = min(begin + per, n);
  int above = 0, equal = 0;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const uint32_t k = i0 + lane < end ? keys[i0 + lane] : 0;
    const bool in = i0 + lane < end;
    above += __popc(__ballot_sync(kAll, in && (whole ? k >= lo : k > lo)));
    equal += __popc(__ballot_sync(kAll, in && !whole && k == lo));
  }
  __syncthreads();
  if (lane == 0) sh.part[0][warp] = above, sh.part[1][warp] = equal;
  __syncthreads();
  int place = 0, ties = 0;  // taken, and equal ones, before this warp's blocks
  for (int i = 0; i < warp; ++i) {
    place += sh.part[0][i] + min(static_cast<int>(sh.part[1][i]), max(0, need - ties));
    ties += sh.part[1][i];
  }
  bool last = false;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int j = i0 + lane;
    const bool in = j < end;
    const uint32_t k = in ? keys[j] : 0;
    const bool eq = in && !whole && k == lo;
    const uint32_t eqs = __ballot_sync(kAll, eq);
    const int tie = ties + __popc(eqs & ((1u << lane) - 1));
    const bool take = in && ((whole ? k >= lo : k > lo) || (eq && tie < need));
    const uint32_t takes = __ballot_sync(kAll, take);
    if (take) {
      out[place + __popc(takes & ((1u << lane) - 1))] = bt_row[j];
      last = last || j == n - 1;
    }
    place += __popc(takes);
    ties += __popc(eqs);
  }
  const int any = __syncthreads_or(last ? 1 : 0);
  if (tid == 0) *out_len = K * bs - (any ? n * bs - seen : 0);
}

template <typename T, int D> cudaError_t launch_select_t(SelectArgs a, cudaStream_t stream) {
  const size_t smem = ((static_cast<size_t>(a.max_candidates) * 4 + 15) & ~static_cast<size_t>(15)) +
                      sizeof(SelectShared<D>);
  constexpr size_t most = kMaxCandidates * 4 + sizeof(SelectShared<D>);
  static_assert(most <= 227 * 1024, "shared memory");
  auto kern = select_kernel<T, D>;
  static SmemLimitOnce smem_limit;
  const cudaError_t e = smem_limit.ensure(kern, most);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * a.max_q_len;
  a.cluster = 1;
  while (a.cluster < 8 && 2 * a.cluster * rows <= 4 * kSms && a.max_candidates >= 512 * a.cluster)
    a.cluster *= 2;
  return launch_clusters(a.cluster, kern,
                         dim3(static_cast<unsigned>(a.cluster * a.max_q_len), a.num_kv_heads, a.num_seqs),
                         dim3(kSelThreads), smem, stream, a);
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
