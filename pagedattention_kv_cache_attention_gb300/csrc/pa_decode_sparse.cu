// pa_decode_sparse.cu -- decode attention over a block table and a length for
// each (row, KV head), 16-bit and FP8 caches (pa_decode_sparse,
// pa_decode_sparse_fp8):
//   out = sum_j softmax_j(scale q . K_j) V_j,   j < lens[row, KV head].
//
// How:
//  * The warps of a cluster of 1 to 8 CTAs share the tokens of one (row, KV
//    head) and serve its G query heads.  A warp takes steps of NSUB 16-token
//    sub-tiles in turn, brought in by TMA into its own ring of S stages, and
//    computes on them as the dense decode kernel does (pa_tile.cuh): S^T = K Q^T
//    and O^T += V^T P^T on mma.sync, fp32 online softmax, P in two parts.
//  * The warps' (m, l, o) are merged through shared memory, the CTAs' through one
//    another's: no workspace, no second kernel.
// What bounds it: HBM, and of small calls the chain of latencies from the table
// over the first tiles to the join.  Measured (32 / 8 heads x 128, fp16 or bf16):
// 64 rows of 512 tokens 23.1 us for 135 MB, 5.9 TB/s; 8 rows of 2,048 tokens 15.0 us
// for 67 MB, 4.5 TB/s; FP8, 256 rows of up to 1,024 tokens, 64 / 8 heads: 67 us for
// 420 MB, 6.2 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tile.cuh"

namespace pa {

namespace {

constexpr int kMaxCluster = 8;

template <typename T, int D, int NW, int S, bool F8, int NSUB>
__global__ void __launch_bounds__(NW * 32)
    sparse_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const DecodeArgs a) {
  using Sh = Shape<D, F8>;
  using MT = typename std::conditional<F8, __half, T>::type;  // E4M3 is exact in fp16
  static_assert(NSUB == 1 || NSUB == 2 || NSUB == 4, "a step's sub-tiles lie in one window");
  static_assert(S * NSUB <= 32, "stage bits; the first window holds every stage's sub-tiles");
  constexpr int kStepBytes = 2 * NSUB * Sh::kTileBytes;  // K and V of one step
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NW * S * kStepBytes);

  const int cluster = a.cluster, rank = static_cast<int>(blockIdx.x);
  const int kvh = blockIdx.y, row = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int wid = rank * NW + warp, n_warps = NW * cluster;

  uint8_t *my_stages = smem + warp * S * kStepBytes;
  uint64_t *my_bars = bars + warp * S;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(&my_bars[s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dependency_wait();  // tables, queries and the pool may come from the kernel before

  // Step k of the warp covers sub-tiles (wid + k n_warps) NSUB + h.  "Local"
  // sub-tile l = k NSUB + h; the lanes hold the block ids of a window of 32.
  const int64_t table = static_cast<int64_t>(row) * a.num_kv_heads + kvh;
  const int32_t *bt_row = a.block_tables + table * a.max_blocks_per_seq;
  const int bs_mask = (1 << a.bs_log2) - 1;
  auto sub_of = [&](int l) -> int64_t {
    return (wid + static_cast<int64_t>(l / NSUB) * n_warps) * NSUB + l % NSUB;
  };
  auto table_entry = [&](int l) -> int {
    const int64_t lb = sub_of(l) * kTile >> a.bs_log2;
    return lb < a.max_blocks_per_seq ? bt_row[lb] : -1;
  };
  int win = table_entry(lane);  // read before the length arrives; entries past it are not used
  int len = a.context_lens[table];
  if (len < 0 || len > a.max_context_len) {
    if (threadIdx.x == 0 && rank == 0) atomicOr(a.err, kErrBadLen);
    len = 0;
  }
  const int n_sub = (len + kTile - 1) / kTile, n_step = (n_sub + NSUB - 1) / NSUB;
  const int my_n = n_step > wid ? (n_step - wid + n_warps - 1) / n_warps : 0;

  // physical block of local sub-tile l, -1 if past the end or invalid (flagged; its
  // tokens are masked)
  auto checked = [&](int l, int phys) -> int {
    if (l >= my_n * NSUB || sub_of(l) >= n_sub) return -1;
    if (phys < 0 || static_cast<int64_t>(phys) >= a.num_blocks) {
      atomicOr(a.err, kErrBadBlock);
      return -1;
    }
    return phys;
  };
  const uint64_t policy = l2_policy_evict_first();
  auto issue = [&](int k, const int (&phys)[NSUB], int s) {  // lane 0
    uint64_t *bar = &my_bars[s];
    uint32_t bytes = 0;
#pragma unroll
    for (int h = 0; h < NSUB; ++h) bytes += phys[h] >= 0 ? 2 * Sh::kTileBytes : 0;
    if (bytes == 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, bytes);
    uint8_t *st = my_stages + s * kStepBytes;
#pragma unroll
    for (int h = 0; h < NSUB; ++h) {
      if (phys[h] < 0) continue;
      const int tok = static_cast<int>(sub_of(k * NSUB + h)) * kTile;
      const int y = ((phys[h] * a.num_kv_heads + kvh) << a.bs_log2) + (tok & bs_mask);
#pragma unroll
      for (int b = 0; b < Sh::kBoxes; ++b) {
        tma_load_2d(st + h * Sh::kTileBytes + b * Sh::kBoxBytes, &kmap, b * Sh::kBoxElems, y, bar,
                    policy);
        tma_load_2d(st + (NSUB + h) * Sh::kTileBytes + b * Sh::kBoxBytes, &vmap,
                    b * Sh::kBoxElems, y, bar, policy);
      }
    }
  };

  int win_base = 0;
  win = checked(lane, win);
  int win_next = my_n * NSUB > 32 ? checked(32 + lane, table_entry(32 + lane)) : -1;
  uint32_t stage_ok = 0;  // bit s NSUB + h: sub-tile h of the step in stage s is valid
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (s < my_n) {
      int phys[NSUB];
#pragma unroll
      for (int h = 0; h < NSUB; ++h) {
        phys[h] = __shfl_sync(kFull, win, s * NSUB + h);
        stage_ok |= (phys[h] >= 0 ? 1u : 0u) << (s * NSUB + h);
      }
      if (lane == 0) issue(s, phys, s);
    }
  }

  // query fragments of head g, in the order in which the keys are read
  const int G = a.group;
  uint4 qf[Sh::kQChunks];
  float scale0 = a.scale_log2, scale1 = a.scale_log2;  // of heads 2c, 2c + 1
  {
    const T *q = static_cast<const T *>(a.query) +
                 (static_cast<int64_t>(row) * a.num_q_heads + kvh * G + g) * D;
#pragma unroll
    for (int i = 0; i < Sh::kQChunks; ++i) {
      const int ch = F8 ? 2 * (c * (D / 64) + (i >> 1)) + (i & 1) : q_chunk(i, c);
      qf[i] = g < G ? *reinterpret_cast<const uint4 *>(q + ch * 8) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (F8 && !std::is_same<T, __half>::value)
      column_scales(a.scale_log2 * queries_to_half(qf), c, scale0, scale1);
  }

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1
  float acc[Sh::kMTiles][4];
#pragma unroll
  for (int mt = 0; mt < Sh::kMTiles; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;

  int k = 0;
  bool timed_out = false;
#pragma unroll 1
  for (; k < my_n; ++k) {
    const int s = k % S;
    if (!__all_sync(kFull, mbar_wait_bounded(&my_bars[s], (k / S) & 1))) {
      if (lane == 0) atomicOr(a.err, kErrTimeout);
      timed_out = true;
      break;
    }
    const uint8_t *stage = my_stages + s * kStepBytes;
    int nvalid[NSUB];
    float sc[NSUB][4], p[NSUB][4];
#pragma unroll
    for (int h = 0; h < NSUB; ++h) {
      const bool ok = (stage_ok >> (s * NSUB + h)) & 1u;
      const int tok = static_cast<int>(sub_of(k * NSUB + h)) * kTile;
      nvalid[h] = ok ? max(0, min(kTile, len - tok)) : 0;
      if constexpr (F8)
        qk_subtile_8<D>(stage + h * Sh::kTileBytes, qf, g, c, sc[h]);
      else
        qk_subtile_16<MT, D>(stage + h * Sh::kTileBytes, qf, g, c, sc[h]);
    }
    softmax_step<NSUB, Sh::kMTiles>(sc, nvalid, g, scale0, scale1, m0, m1, l0, l1, acc, p);
#pragma unroll
    for (int h = 0; h < NSUB; ++h) {
      uint32_t pb0, pb1, pr0, pr1;
      p_operands<MT>(p[h], pb0, pb1, pr0, pr1);
      const uint8_t *Vs = stage + (NSUB + h) * Sh::kTileBytes;
      if constexpr (F8)
        pv_subtile_8<D>(Vs, nvalid[h], g, c, pb0, pb1, pr0, pr1, acc);
      else
        pv_subtile_16<MT, D>(Vs, nvalid[h], g, c, pb0, pb1, pr0, pr1, acc);
    }
    // refill this stage with step k + S
    __syncwarp();
    const int nk = k + S;
    if (nk < my_n) {
      if (nk * NSUB >= win_base + 32) {
        win_base += 32;
        win = win_next;
        win_next = checked(win_base + 32 + lane, table_entry(win_base + 32 + lane));
      }
      int phys[NSUB];
#pragma unroll
      for (int h = 0; h < NSUB; ++h) {
        phys[h] = __shfl_sync(kFull, win, nk * NSUB + h - win_base);
        stage_ok = (stage_ok & ~(1u << (s * NSUB + h))) |
                   ((phys[h] >= 0 ? 1u : 0u) << (s * NSUB + h));
      }
      if (lane == 0) {
        fence_proxy_async_smem();
        issue(nk, phys, s);
      }
    }
  }
  // after a wait that ran out, copies already in flight land before the CTA
  // leaves (bounded again)
  for (const int filled = min(k + S, my_n); timed_out && k < filled; ++k)
    (void)mbar_wait_bounded(&my_bars[k % S], (k / S) & 1);

  // row sums over the 8 token rows (lanes differing in g)
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(kFull, l0, off);
    l1 += __shfl_xor_sync(kFull, l1, off);
  }
  // ---- merge the warps through shared memory (stages are idle now)
  __syncthreads();
  float *wacc = reinterpret_cast<float *>(smem);  // [NW][8][D]
  float *wml = wacc + NW * 8 * D;                 // [NW][8][2]
  float *cl_o = wml + NW * 8 * 2;                 // [8][D]: the CTA's, for its cluster
  float *cl_ml = cl_o + 8 * D;                    // [8][2]
  if (g == 0) {
    wml[(warp * 8 + 2 * c) * 2 + 0] = m0;
    wml[(warp * 8 + 2 * c) * 2 + 1] = l0;
    wml[(warp * 8 + 2 * c + 1) * 2 + 0] = m1;
    wml[(warp * 8 + 2 * c + 1) * 2 + 1] = l1;
  }
  store_partial_o<D, F8>(wacc + (warp * 8 + 2 * c) * D, wacc + (warp * 8 + 2 * c + 1) * D, true,
                         true, acc, 1.f, 1.f, g);
  __syncthreads();
  constexpr int kChunks = D / 8;
  T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(row) * a.num_q_heads + kvh * G) * D;
  auto put = [&](int h, int ch, float L, float (&o)[8]) {
    const float inv = L > 0.f ? a.out_scale / L : 0.f;
    *reinterpret_cast<uint4 *>(out + h * D + ch * 8) = make_uint4(
        Elem<T>::pack(o[0] * inv, o[1] * inv), Elem<T>::pack(o[2] * inv, o[3] * inv),
        Elem<T>::pack(o[4] * inv, o[5] * inv), Elem<T>::pack(o[6] * inv, o[7] * inv));
  };
  for (int item = threadIdx.x; item < G * kChunks; item += NW * 32) {
    const int h = item / kChunks, ch = item % kChunks;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wml[(w * 8 + h) * 2]);
    float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = wml[(w * 8 + h) * 2];
      const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      L += wml[(w * 8 + h) * 2 + 1] * f;
      const float *src = wacc + (w * 8 + h) * D + ch * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += src[e] * f;
    }
    if (cluster == 1) {
      put(h, ch, L, o);
      continue;
    }
    float4 *dst = reinterpret_cast<float4 *>(cl_o + h * D + ch * 8);
    dst[0] = make_float4(o[0], o[1], o[2], o[3]);
    dst[1] = make_float4(o[4], o[5], o[6], o[7]);
    if (ch == 0) {
      cl_ml[h * 2] = M;
      cl_ml[h * 2 + 1] = L;
    }
  }
  if (cluster > 1) {
    // the cluster's CTAs share the heads' chunks of the join out
    cluster_sync();
    for (int item = threadIdx.x + rank * NW * 32; item < G * kChunks; item += NW * 32 * cluster) {
      const int h = item / kChunks, ch = item % kChunks;
      float M = -INFINITY;
      for (int r = 0; r < cluster; ++r)
        M = fmaxf(M, ld_cluster_f2(cluster_addr(cl_ml + h * 2, r)).x);
      float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int r = 0; r < cluster; ++r) {
        const float2 ml = ld_cluster_f2(cluster_addr(cl_ml + h * 2, r));
        const uint32_t src = cluster_addr(cl_o + h * D + ch * 8, r);
        const float4 x = ld_cluster_f4(src), y = ld_cluster_f4(src + 16);
        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
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
      put(h, ch, L, o);
    }
    cluster_sync();  // nobody leaves while its memory is read
  }
  grid_launch_dependents();
}

// One instance of the kernel: its shared memory, and how many CTAs of it an SM
// takes at least (by shared memory, and at most 136 registers a thread).
template <typename T, int D, int NW, int S, bool F8, int NSUB> struct Instance {
  static constexpr int kStepTokens = NSUB * kTile;
  static constexpr size_t kStages = static_cast<size_t>(NW) * S * 2 * NSUB * Shape<D, F8>::kTileBytes;
  static constexpr size_t kSmem = 1024 + kStages + NW * S * 8;
  static constexpr int kPerSm = static_cast<int>(227 * 1024 / (kSmem + 1024));
  static_assert((static_cast<size_t>(NW) + 1) * 8 * (D + 2) * 4 <= kStages,
                "merge buffers must fit in the stage area");

  // CTAs that share a row's tokens: as many as the SMs have room for, while a warp
  // keeps four steps of the longest table.
  static int cluster_of(const DecodeArgs &a) {
    const int64_t ctas = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
    const int64_t steps = a.max_context_len / kStepTokens;
    int n = 1;
    while (n < kMaxCluster && 2 * n * ctas <= kSms * kPerSm && steps >= 4 * n * NW) n *= 2;
    return n;
  }
  static cudaError_t launch(DecodeArgs a, const CUtensorMap &km, const CUtensorMap &vm,
                            cudaStream_t stream) {
    auto kern = sparse_decode_kernel<T, D, NW, S, F8, NSUB>;
    static SmemLimitOnce smem_limit;
    const cudaError_t e = smem_limit.ensure(kern, kSmem);
    if (e != cudaSuccess) return e;
    a.cluster = cluster_of(a);
    return launch_clusters(a.cluster, kern, dim3(a.cluster, a.num_kv_heads, a.num_seqs),
                           dim3(NW * 32), kSmem, stream, km, vm, a);
  }
};

// Warps of a CTA.  16-bit caches: four where they share a row in clusters (8 rows of
// 2,048 tokens, 32 / 8 heads x 128: 15.0 us; 16.0 with two), else two, of whose CTAs
// an SM takes six (64 rows of 512 tokens: 23.1 us; 27.9 with four, whose 512 CTAs
// are more than the 456 that run at once; 23.6 with three, 24.3 with one).  FP8
// caches: four (256 rows of up to 1,024 tokens, 64 / 8 heads x 128: 67 us; 71 with
// two, 72 with three, 79 with one, 98 with eight; 8 rows of 2,048 tokens, 32 / 8 heads
// 11.1 us, 12.1 with two).  For 64 rows of 512 tokens two would be better, for the
// reason above: 14.1 us, 17.6 with four.  Three stages in place of two: 23.5 and 77 us
// with two warps, 24.8 and 76 with four.
template <typename T, int D>
cudaError_t launch_d(const DecodeArgs &a, bool kv_fp8, const CUtensorMap &km,
                     const CUtensorMap &vm, cudaStream_t stream) {
  using Wide = Instance<T, D, 4, 2, false, D == 64 ? 2 : 1>;
  using Narrow = Instance<T, D, 2, 2, false, D == 64 ? 2 : 1>;
  using Fp8 = Instance<T, D, 4, D == 64 ? 4 : 2, true, 2>;
  if (kv_fp8) return Fp8::launch(a, km, vm, stream);
  return Wide::cluster_of(a) > 1 ? Wide::launch(a, km, vm, stream)
                                 : Narrow::launch(a, km, vm, stream);
}

}  // namespace

cudaError_t launch_decode_sparse(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                                 int64_t pool_rows, int head_dim, int dtype, bool kv_fp8,
                                 cudaStream_t stream, bool *map_failed) {
  CUtensorMap km, vm;
  *map_failed = !encode_pool_map(&km, k_cache, pool_rows, head_dim, dtype, kv_fp8) ||
                !encode_pool_map(&vm, v_cache, pool_rows, head_dim, dtype, kv_fp8);
  if (*map_failed) return cudaErrorInvalidValue;
  if (dtype == 0)
    return head_dim == 128 ? launch_d<__half, 128>(a, kv_fp8, km, vm, stream)
                           : launch_d<__half, 64>(a, kv_fp8, km, vm, stream);
  return head_dim == 128 ? launch_d<__nv_bfloat16, 128>(a, kv_fp8, km, vm, stream)
                         : launch_d<__nv_bfloat16, 64>(a, kv_fp8, km, vm, stream);
}

}  // namespace pa
