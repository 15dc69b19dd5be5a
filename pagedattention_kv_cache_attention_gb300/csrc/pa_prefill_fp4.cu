// pa_prefill_fp4.cu -- chunked-prefill attention over the FP4 cache on the
// fifth-generation tensor core, for chunks of more than 64 (token, head) rows a KV
// head, and for shorter ones down to 25 rows where the (sequence, KV head) pairs
// are fewer than two for each SM (pa_prefill_fp4; the others run in
// pa_prefill_tc.cu, those of at most 24 rows in pa_decode_fp4.cu).
//
// The arithmetic is pa_prefill_tc.cu's: two 128-row query tiles of one
// (sequence, KV head) per CTA, rows (token, head), 64-key steps; S = Q K^T and
// O += P V by tcgen05 with the accumulators in tensor memory, an online softmax
// in base 2 with thread r of a tile owning row r.  Differences:
//  * K and V arrive as FP4 tiles (codes and scales in one TMA copy) in a ring
//    of raw steps; four warps widen them to the exact fp16 stages that the
//    products read, each 32 rows of every 64-key step of K or of V.
//  * P takes the place of the scores it comes from: of a tile's 256 columns of
//    tensor memory, 128 are two score buffers (step n in buffer n % 2) and the
//    rest O; the softmax writes P, as fp16, over the first half of the buffer it
//    has just read.  Q K^T of step n + 1 so waits only for P V of step n - 1 and
//    runs beside the softmax of step n.
//  * The issuing warps run their loops whole and elect a lane for the tcgen05
//    instructions: operands then stay in uniform registers (a product's issue
//    took 113 cycles in a single-lane branch, 65 like this).
// What bounds it: a step takes 1,730 cycles; the shared memory is busy for 1,430
// of them (Q's 64 KB, K's and V's 32 KB each, read by the products, 32 KB
// written by the widening), a tile's softmax for 1,300.  Measured: 8,111-token
// prompt, 64 query / 8 KV heads, head_dim 128, bf16: 841 us, 1.28 PFLOP/s (0.67
// of cuBLAS bf16).  In an earlier state of this kernel (975 us) separate columns
// for P took 1,022; products of 128 keys (a third less of Q's traffic) with the
// scores' buffer whole 1,144, since a tile's next scores then wait for its last
// P V; two threads a row 1,207.
//
// Where the call has too few CTAs to fill the SMs, a cluster of up to eight
// shares a tile pair's keys: each CTA takes a run of the steps, leaves its O,
// maximum and sum in shared memory, and the CTAs share the rows of the join.
//
// Warp roles: warps 0 and 2 widen K, 1 and 3 V; 4-7 softmax of tile 0, 8-11 of
// tile 1; 12-15 issue (Q K^T and P V of tile 0, of tile 1).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"
#include "pa_tc.cuh"

namespace pa {

namespace {

constexpr int kThreads = 512;
// P is held times 2^11 with the running maximum at most 2^4 behind, so that it
// stays below 2^15 and keeps fp16's precision down to 2^-25 of the maximum: a
// long context's faint tail keeps its mass.
constexpr float kPShift = 11.f, kGrowth = 4.f;
constexpr float kFar = kFp4FarLogit;

#ifndef PA_PREFILL_FP4_KSTAGES
#define PA_PREFILL_FP4_KSTAGES 3
#endif
#ifndef PA_PREFILL_FP4_VSTAGES
#define PA_PREFILL_FP4_VSTAGES 3
#endif
#ifndef PA_PREFILL_FP4_RAW
#define PA_PREFILL_FP4_RAW 3
#endif

// First warps of the roles (the widening first, which the schedulers then
// favour: 975 us against 983 with it last, then).
constexpr int kLoad0 = 0, kSoft0 = 4, kIssue0 = 12;

// Shared memory.  An atom is 64 dimensions of 128-byte rows.
template <int D> struct Layout {
  static constexpr int kAtoms = D / 64;
  static constexpr int kSK = PA_PREFILL_FP4_KSTAGES;  // widened stages of K, 64 keys each
  static constexpr int kSV = PA_PREFILL_FP4_VSTAGES;  // and of V
  static constexpr int kRaw = PA_PREFILL_FP4_RAW;     // raw steps of 64 keys
  static constexpr int kQAtom = kTcRows * 128;
  static constexpr int kKAtom = kPairKeys * 128;
  static constexpr int kVAtom = kPairKeys * 128;
  static_assert(kKAtom == kVAtom, "one widening code for both");
  static constexpr int kRawStep = kPairKeys / 16 * kRawSlot16<D>;
  static constexpr int kKOff = 2 * kAtoms * kQAtom;
  static constexpr int kVOff = kKOff + kSK * kAtoms * kKAtom;
  static constexpr int kRawOff = kVOff + kSV * kAtoms * kVAtom;
  static constexpr int kBarOff = kRawOff + 2 * kRaw * kRawStep;
  static constexpr int kBars = 2 * kSK + 2 * kSV + 4 + 4 + 4 + 1 + 4 * kRaw;
  static constexpr size_t kSmem = 1024 + kBarOff + kBars * 8 + 16 + (D / 16 + 1) * 4;
  // join in a cluster: O [tile][row][D] fp32 over the idle Q and stages, 16-byte
  // unit u of row r at u ^ (r & 7); then (maximum, sum) [tile][row]
  static constexpr int kMlOff = 2 * kTcRows * D * 4;
  static_assert(kMlOff + 2 * kTcRows * 8 <= kRawOff, "the join fits in Q and the stages");
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    pa_prefill_fp4_kernel(const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const PrefillArgs a) {
  using L = Layout<D>;
  constexpr int kAtoms = L::kAtoms, kSK = L::kSK, kSV = L::kSV, kRaw = L::kRaw;
  constexpr int kSub = kPairKeys / 16;  // 16-key sub-tiles of a step
  constexpr uint32_t kAllSub = (1u << kSub) - 1;
  constexpr bool kBf16 = !std::is_same<T, __half>::value;
  constexpr int kOCol = 128;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
  uint64_t *k_empty = k_full + kSK;
  uint64_t *v_full = k_empty + kSK;
  uint64_t *v_empty = v_full + kSV;
  uint64_t *s_full = v_empty + kSV;   // [tile][buffer]: a step's scores computed
  uint64_t *p_full = s_full + 4;      // [tile][buffer]: its P in their place
  uint64_t *pv_done = p_full + 4;     // [tile][buffer]: its P V done
  uint64_t *q_ready = pv_done + 4;
  uint64_t *raw_land = q_ready + 1;   // [4 warps][kRaw]: a warp's raw tiles of a step are in
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(raw_land + 4 * kRaw);
  // NaNs of V at keys that not every row attends to: zeros in the products, so
  // that they do not reach the rows before them, and put back at the end
  int *nan_key = reinterpret_cast<int *>(tmem_slot + 4);

  const int cluster = a.chunks, cluster_log2 = 31 - __clz(cluster);  // a power of two
  const int kvh = blockIdx.x >> cluster_log2, seq = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group;
  const int tpc = 2 * kTcRows / G;  // tokens per CTA

  if (tid == 0) {
    for (int s = 0; s < kSK; ++s) {
      mbar_init(&k_full[s], 2);  // filled by two widening warps
      mbar_init(&k_empty[s], 2);  // released by both tiles' issuers
    }
    for (int s = 0; s < kSV; ++s) {
      mbar_init(&v_full[s], 2);
      mbar_init(&v_empty[s], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kTcRows);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_ready, 2 * kTcRows);
    for (int s = 0; s < 4 * kRaw; ++s) mbar_init(&raw_land[s], 1);
    fence_barrier_init();
    for (int i = 0; i <= D / 16; ++i) nan_key[i] = 0x7fffffff;
  }
  if (warp == kIssue0) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the chunk's K/V may come from the kernel before

  const int q0 = a.query_start[seq];
  const int q_len = a.query_start[seq + 1] - q0;
  const int ctx = a.context_lens[seq];
  bool active = true;
  if (q_len < 0 || ctx < q_len || ctx > (a.max_blocks_per_seq << a.bs_log2) ||
      q_len > a.max_q_len) {
    if (tid == 0) atomicOr(a.err, kErrBadLen);
    active = false;  // (in the whole cluster, here and below)
  }
  const int rank = blockIdx.x & (cluster - 1);
  // a sequence's tiles start together, those with the most keys first, so that
  // its K and V come from L2
  const int t_first = (gridDim.y - 1 - blockIdx.y) * tpc;
  if (t_first >= q_len) active = false;
  const int t_last = min(q_len, t_first + tpc) - 1;
  const int base_pos = ctx - q_len;
  const int n_keys = base_pos + t_last + 1;
  const int32_t *bt_row = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
  // Steps of 64 keys that each tile needs (tile 1 holds the later tokens, so it
  // reads every step tile 0 reads).  Tile 0's rows
  // reach token (kTcRows - 1) / G; tile 1's begin at token kTcRows / G.
  const int last0 = min(t_last, t_first + (kTcRows - 1) / G);
  const int last1 = t_first + kTcRows / G <= t_last ? t_last : -1;
  // In a cluster, from step_base on the CTA's share of them.
  const int all0 = active ? (base_pos + last0 + kPairKeys) / kPairKeys : 0;
  const int all1 = active && last1 >= 0 ? (n_keys + kPairKeys - 1) / kPairKeys : 0;
  const int all = max(all0, all1);
  const int step_base = (all * rank) >> cluster_log2;  // (all < 2^26, rank < 8)
  const int n_steps = ((all * (rank + 1)) >> cluster_log2) - step_base;
  const int steps0 = max(0, min(n_steps, all0 - step_base));
  const int steps1 = all1 > 0 ? n_steps : 0;
  const int n_sub = (n_keys + 15) / 16;

  // the softmax threads' row, for the join in a cluster: its reference, a score
  // before the softmax scale, and the scale
  float x_ref = -INFINITY, l = 0.f, sl2 = a.scale_log2;
  bool row_done = false;  // the row's O is in tensor memory
  if (active && warp >= kSoft0 && warp < kSoft0 + 8) {
    // ------------------------------------------------------------ softmax warps
    const int t = (warp - kSoft0) >> 2;
    const int r = tid & (kTcRows - 1);  // row within the tile = TMEM lane
    const int rc = t * kTcRows + r;     // row within the CTA
    const int tok = t_first + rc / G;
    const bool row_ok = tok <= t_last;
    const int pos = base_pos + tok;     // keys up to pos are attended to
    const int my_steps = t == 0 ? steps0 : steps1;
    // Q and the output move in whole rows: lane ch of a group of kLanes holds
    // unit ch of the row, kRowsAt rows at a time; the rows' offsets from the
    // tile pair's first (in rows of D; -1: past the chunk) are asked of their
    // threads.  A thread that walks its own row touches a line with every lane
    // of every access instead: 3 us more a CTA (of 13 for one step of keys).
    constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;
    const int sub = lane / kLanes, ch = lane % kLanes;
    const int row_off = row_ok ? (rc / G) * a.num_q_heads + rc % G : -1;
    const int64_t tile_at =
        (static_cast<int64_t>(q0 + t_first) * a.num_q_heads + kvh * G) * D;
    // 16-byte unit c of row i of this warp in the swizzled Q tile
    auto q_unit = [&](int i, int c) {
      return reinterpret_cast<uint4 *>(smem + (t * kAtoms + (c >> 3)) * L::kQAtom +
                                       ((warp & 3) * 32 + i) * 128 + (((c & 7) ^ (i & 7)) << 4));
    };
    {
      const T *qbase = static_cast<const T *>(a.query) + tile_at + ch * 8;
#pragma unroll
      for (int i = 0; i < 32 / kRowsAt; ++i) {
        const int off = __shfl_sync(kFullMask, row_off, i * kRowsAt + sub);
        // rows past the chunk: zeros (nothing read)
        cp_async16(q_unit(i * kRowsAt + sub, ch),
                   qbase + static_cast<int64_t>(max(off, 0)) * D, off >= 0);
      }
      cp_async_wait_all();
      // bf16 queries: the row is scaled by 2^e so that its largest magnitude
      // lies in [2^14, 2^15), then rounded to fp16 (exact for every value down
      // to 2^-31 of the largest: bf16 carries 8 significant bits, and fp16
      // holds 8 bits at every magnitude from 2^-17 up), and 2^-e joins the
      // row's softmax scale.  Each thread rewrites its own row: a third of the
      // instructions of rewriting what it fetched, which needs a maximum over
      // lanes for every unit (4,500 cycles a CTA more).
      if constexpr (kBf16) {
        __syncwarp();
        uint4 v[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) v[c] = *q_unit(lane, c);
        uint32_t mx = 0;  // the largest exponent: of the magnitudes' bits, two at a time
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu),
                                     __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
        const int e = min(120, 14 + 127 - static_cast<int>(max(mx >> 23, (mx >> 7) & 0xffu)));
        const float qf = ldexpf(1.f, e);
        sl2 = ldexpf(sl2, -e);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t w4[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 f = Elem<T>::unpack(word_of(v[c], w));
            w4[w] = Elem<__half>::pack(f.x * qf, f.y * qf);
          }
          *q_unit(lane, c) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      }
      sl2 = fp4_normal_scale(sl2);
      fence_proxy_async_smem();
      mbar_arrive(q_ready);
    }
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 256;
    // table entry of sub-tile `lane` of step n; whether the loaders took it
    auto entry = [&](int n) -> int {
      const int u = (step_base + n) * kSub + lane;
      return lane < kSub && u < n_sub ? bt_row[(u * 16) >> a.bs_log2] : -1;
    };
    auto valid = [&](int phys) -> uint32_t {
      return __ballot_sync(kFullMask, phys >= 0 && static_cast<int64_t>(phys) < a.num_blocks) &
             kAllSub;
    };
    bool ok_run = true;
    uint32_t vmask_next = my_steps > 0 ? valid(entry(0)) : 0;
    for (int n = 0; n < my_steps; ++n) {
      const int h = n & 1;
      const uint32_t vmask = vmask_next;
      if (!__all_sync(kFullMask, mbar_wait_bounded(&s_full[2 * t + h], (n >> 1) & 1))) {
        ok_run = false;
        break;
      }
      tc_fence_after();
      float sv[kPairKeys];
      {
        // both loads in flight before the one wait
        float t0[32], t1[32];
        tmem_ld32(lane_addr + 64 * h, t0);
        tmem_ld32(lane_addr + 64 * h + 32, t1);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          sv[i] = t0[i];
          sv[32 + i] = t1[i];
        }
      }
      // loaded now, used at the end of the step: its latency hides behind the softmax
      const int bt_next = n + 1 < my_steps ? entry(n + 1) : -1;
      const int key0 = (step_base + n) * kPairKeys;
      // rows past the chunk (zeros, never stored) attend like the last one, so that
      // they do not send their warp through the masking at every step (255 of 256
      // rows in use: 143 us became 118)
      if (!(key0 + kPairKeys - 1 <= pos && vmask == kAllSub)) {
#pragma unroll
        for (int c = 0; c < kPairKeys; ++c) {
          const bool ok = key0 + c <= pos && ((vmask >> (c >> 4)) & 1u);
          sv[c] = ok ? sv[c] : -INFINITY;
        }
      }
      // row max: three-input max, 64 -> 22 -> 8 -> 3 -> 1
      float t22[22], t8[8];
#pragma unroll
      for (int j = 0; j < 21; ++j) t22[j] = fmax3(sv[3 * j], sv[3 * j + 1], sv[3 * j + 2]);
      t22[21] = sv[63];
#pragma unroll
      for (int j = 0; j < 7; ++j) t8[j] = fmax3(t22[3 * j], t22[3 * j + 1], t22[3 * j + 2]);
      t8[7] = t22[21];
      const float xmax = fmax3(fmax3(t8[0], t8[1], t8[2]), fmax3(t8[3], t8[4], t8[5]),
                               fmaxf(t8[6], t8[7]));  // the scale is positive: same order
      const float grow = (xmax - x_ref) * sl2;
      const bool move = grow > kGrowth;  // includes the first finite max
      const float alpha = move ? ex2_approx(-grow) : 1.f;
      if (move) {
        l *= alpha;
        x_ref = xmax;
      }
      const float ref = x_ref == -INFINITY ? 0.f : x_ref;
      float neg_m = fmaf(-ref, sl2, kPShift);
      if (__any_sync(kFullMask, fabsf(neg_m) > kFar)) {  // a large logit: see kFp4FarLogit
#pragma unroll
        for (int c = 0; c < kPairKeys; ++c) sv[c] -= ref;
        neg_m = kPShift;
      }
      const uint64_t scale2 = f2_pack(sl2, sl2), negm2 = f2_pack(neg_m, neg_m);
      uint64_t ls2[4] = {0, 0, 0, 0};  // +0.0f pairs
      uint32_t ph[kPairKeys / 2];
#pragma unroll
      for (int e = 0; e < kPairKeys / 2; ++e) {
        const float2 x = f2_unpack(f2_fma(f2_pack(sv[2 * e], sv[2 * e + 1]), scale2, negm2));
        const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
        ls2[e & 3] = f2_add(ls2[e & 3], f2_pack(p0, p1));
        ph[e] = Elem<__half>::pack(p0, p1);
      }
      const float2 sm = f2_unpack(f2_add(f2_add(ls2[0], ls2[1]), f2_add(ls2[2], ls2[3])));
      l += sm.x + sm.y;
      // P of this half into the score columns that this thread has read
      tmem_st16(lane_addr + 64 * h, ph);
      tmem_st16(lane_addr + 64 * h + 16, ph + 16);
      // O must hold P V of every earlier step before it is rescaled
      if (n > 0 && __any_sync(kFullMask, move)) {  // whole warp: rows that did not move use 1
        if (!__all_sync(kFullMask, mbar_wait_bounded(&pv_done[2 * t + (1 - h)],
                                                     ((n - 1) >> 1) & 1))) {
          ok_run = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          float o[32];
          tmem_ld32(lane_addr + kOCol + cb * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(lane_addr + kOCol + cb * 32, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[2 * t + h]);
      vmask_next = valid(bt_next);
    }
    // ---- epilogue: O / l for this row
    if (ok_run && my_steps > 0) {
      const int last = my_steps - 1;
      ok_run = __all_sync(kFullMask,
                          mbar_wait_bounded(&pv_done[2 * t + (last & 1)], (last >> 1) & 1));
      row_done = ok_run;
      if (ok_run && cluster == 1) {
        tc_fence_after();
        const float inv = l > 0.f ? a.out_scale / l : 0.f;  // times the V scale
        // through the Q tile, whose readers are done
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          float o[32];
          tmem_ld32(lane_addr + kOCol + cb * 32, o);
          tmem_wait_ld();
          if (nan_key[D / 16] <= pos) put_nans(o, nan_key, cb, pos);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *q_unit(lane, cb * 4 + q) =
                make_uint4(Elem<T>::pack(o[q * 8 + 0] * inv, o[q * 8 + 1] * inv),
                           Elem<T>::pack(o[q * 8 + 2] * inv, o[q * 8 + 3] * inv),
                           Elem<T>::pack(o[q * 8 + 4] * inv, o[q * 8 + 5] * inv),
                           Elem<T>::pack(o[q * 8 + 6] * inv, o[q * 8 + 7] * inv));
        }
        __syncwarp();
        T *obase = static_cast<T *>(a.out) + tile_at + ch * 8;
#pragma unroll
        for (int b = 0; b < 32; b += 8 * kRowsAt) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = *q_unit(b + i * kRowsAt + sub, ch);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int off = __shfl_sync(kFullMask, row_off, b + i * kRowsAt + sub);
            if (off >= 0) *reinterpret_cast<uint4 *>(obase + static_cast<int64_t>(off) * D) = v[i];
          }
        }
      }
    }
    if (!ok_run && lane == 0) atomicOr(a.err, kErrTimeout);
  } else if (active && warp >= kIssue0) {
    // ------------------------------------------------------------ MMA issuers
    // Q K^T of a step once K is in and the P that took the buffer's place two
    // steps ago has been used; P V of a step once P and V are in place.  Each
    // issuer releases every K (or V) stage once; for those its tile does not
    // read it waits for the stage to fill first, so its release lands in that
    // phase.
    // The whole warp runs the loops and one elected lane issues, so that the
    // operands stay in uniform registers.
    const bool leader = elect_one();
    auto arrived = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(kFullMask, mbar_wait_bounded(bar, parity)) != 0;
    };
    bool ok_run = true;
    auto issue_qk = [&](int t, int steps) {
      const uint32_t tt = tmem + t * 256;
      const uint32_t id_qk = umma_idesc_f16(0, false, kTcRows, kPairKeys);
      // every operand is one of two descriptors plus a byte offset / 16 in the
      // address field (shared memory lies below 2^18 bytes, so the 14-bit field
      // never carries)
      const uint64_t dq = umma_desc_sw128(smem_addr(smem) + t * kAtoms * L::kQAtom, 16, 1024);
      const uint64_t dk0 = umma_desc_sw128(smem_addr(smem + L::kKOff), 16, 1024);
      ok_run = arrived(q_ready, 0);
      for (int n = 0; n < steps && ok_run; ++n) {
        const int s = n % kSK, h = n & 1;
        if (!arrived(&k_full[s], (n / kSK) & 1) ||
            (n > 1 && !arrived(&pv_done[2 * t + h], ((n - 2) >> 1) & 1))) {
          ok_run = false;
          break;
        }
        tc_fence_after();
        const uint64_t dk = dk0 + static_cast<uint64_t>((s * kAtoms * L::kKAtom) >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_f16(tt + 64 * h,
                     dq + static_cast<uint64_t>(((k >> 2) * L::kQAtom + (k & 3) * 32) >> 4),
                     dk + static_cast<uint64_t>(((k >> 2) * L::kKAtom + (k & 3) * 32) >> 4), id_qk,
                     k > 0);
          umma_commit(&s_full[2 * t + h]);
          umma_commit(&k_empty[s]);
        }
        __syncwarp();
      }
      for (int n = steps; n < n_steps && ok_run; ++n) {
        ok_run = arrived(&k_full[n % kSK], (n / kSK) & 1);
        if (ok_run && leader) mbar_arrive(&k_empty[n % kSK]);
      }
    };
    auto issue_pv = [&](int t, int steps) {
      const uint32_t tt = tmem + t * 256;
      const uint32_t id_pv = umma_idesc_f16(0, true, kTcRows, D);
      const uint64_t dv0 = umma_desc_sw128(smem_addr(smem + L::kVOff), L::kVAtom, 1024);
      for (int n = 0; n < steps && ok_run; ++n) {
        const int s = n % kSV, h = n & 1;
        if (!arrived(&v_full[s], (n / kSV) & 1) || !arrived(&p_full[2 * t + h], (n >> 1) & 1)) {
          ok_run = false;
          break;
        }
        tc_fence_after();
        const uint64_t dv = dv0 + static_cast<uint64_t>((s * kAtoms * L::kVAtom) >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kPairKeys / 16; ++kk)
            umma_f16_ts(tt + kOCol, tt + 64 * h + 8 * kk,
                        dv + static_cast<uint64_t>((kk * 2048) >> 4), id_pv, n > 0 || kk > 0);
          umma_commit(&pv_done[2 * t + h]);
          umma_commit(&v_empty[s]);
        }
        __syncwarp();
      }
      for (int n = steps; n < n_steps && ok_run; ++n) {
        ok_run = arrived(&v_full[n % kSV], (n / kSV) & 1);
        if (ok_run && leader) mbar_arrive(&v_empty[n % kSV]);
      }
    };
    if (warp == kIssue0)
      issue_qk(0, steps0);
    else if (warp == kIssue0 + 1)
      issue_pv(0, steps0);
    else if (warp == kIssue0 + 2)
      issue_qk(1, steps1);
    else
      issue_pv(1, steps1);
    if (!ok_run && lane == 0) atomicOr(a.err, kErrTimeout);
  } else if (active) {
    // ------------------------------------------------------------ widening warps
    const bool k_role = (warp & 1) == 0;
    uint64_t *full = k_role ? k_full : v_full, *empty = k_role ? k_empty : v_empty;
    const uint64_t policy = l2_policy_evict_normal();  // the chunk's other tiles read it too
    const bool ok_run = f4_widen_share<D, kSK, kSV, kRaw, L::kRawStep, L::kKAtom>(
        a, k_role ? &kmap : &vmap, bt_row, kvh, lane, k_role,
        warp - kLoad0 >= 2 ? kF4Share : 0, step_base, n_steps, n_keys, base_pos + t_first + 1, full,
        empty, raw_land + (warp - kLoad0) * kRaw, smem + (k_role ? L::kKOff : L::kVOff),
        smem + L::kRawOff + (k_role ? 0 : kRaw * L::kRawStep), nan_key, policy);
    if (!ok_run && lane == 0) atomicOr(a.err, kErrTimeout);
  }

  // ---- teardown: every tcgen05 operation is complete once each tile's last
  // P V has been observed by its softmax warps (its Q K^T products came
  // before it), or the tile had no work
  tc_fence_before();
  __syncthreads();
  if (cluster > 1 && active) {
    float2 *ml = reinterpret_cast<float2 *>(smem + L::kMlOff);
    if (warp >= kSoft0 && warp < kSoft0 + 8) {
      const int t = (warp - kSoft0) >> 2, r = tid & (kTcRows - 1);
      const uint32_t addr =
          tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 256 + kOCol;
      float4 *row = reinterpret_cast<float4 *>(smem + (t * kTcRows + r) * D * 4);
      const int pos = base_pos + t_first + (t * kTcRows + r) / G;
      float to;  // O and l relative to m, and no longer times 2^kPShift
      const float m = fp4_reference(x_ref, sl2, kPShift, to);
      tc_fence_after();
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        float o[32];
        tmem_ld32(addr + cb * 32, o);
        tmem_wait_ld();
        if (nan_key[D / 16] <= pos) put_nans(o, nan_key, cb, pos);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          row[(cb * 8 + q) ^ (r & 7)] =
              row_done ? make_float4(o[4 * q] * to, o[4 * q + 1] * to, o[4 * q + 2] * to,
                                     o[4 * q + 3] * to)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      ml[t * kTcRows + r] = row_done ? make_float2(m, l * to) : make_float2(-INFINITY, 0.f);
      tc_fence_before();
    }
    cluster_sync();
    // the pair's 256 rows, an equal share of them for each CTA, 8 columns at a time
    const int rows = 2 * kTcRows / cluster;
    for (int i = tid; i < rows * (D / 8); i += kThreads) {
      const int rc = rank * rows + i / (D / 8), ch = i % (D / 8);
      const int tok = t_first + rc / G;
      if (tok > t_last) continue;
      float M = -INFINITY, sum = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < cluster; ++k) M = fmaxf(M, ld_cluster_f2(cluster_addr(ml + rc, k)).x);
      const float ref = M == -INFINITY ? 0.f : M;
      for (int k = 0; k < cluster; ++k) {
        const float2 part = ld_cluster_f2(cluster_addr(ml + rc, k));
        const uint32_t row = cluster_addr(smem + rc * D * 4, k);
        const float4 x = ld_cluster_f4(row + (((2 * ch) ^ (rc & 7)) << 4));
        const float4 y = ld_cluster_f4(row + (((2 * ch + 1) ^ (rc & 7)) << 4));
        const float f = exp2f(part.x - ref);
        sum += part.y * f;
        o[0] += x.x * f;
        o[1] += x.y * f;
        o[2] += x.z * f;
        o[3] += x.w * f;
        o[4] += y.x * f;
        o[5] += y.y * f;
        o[6] += y.z * f;
        o[7] += y.w * f;
      }
      const float inv = sum > 0.f ? a.out_scale / sum : 0.f;
      T *orow = static_cast<T *>(a.out) +
                (static_cast<int64_t>(q0 + tok) * a.num_q_heads + kvh * G + rc % G) * D;
      *reinterpret_cast<uint4 *>(orow + ch * 8) = make_uint4(
          Elem<T>::pack(o[0] * inv, o[1] * inv), Elem<T>::pack(o[2] * inv, o[3] * inv),
          Elem<T>::pack(o[4] * inv, o[5] * inv), Elem<T>::pack(o[6] * inv, o[7] * inv));
    }
    cluster_sync();  // nobody leaves while its memory is read
  }
  if (warp == kIssue0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  grid_launch_dependents();
}

template <typename T, int D>
cudaError_t launch_t(const PrefillArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                     cudaStream_t stream) {
  constexpr size_t smem = Layout<D>::kSmem;
  static_assert(smem <= 227 * 1024, "shared memory");
  auto kern = pa_prefill_fp4_kernel<T, D>;
  static SmemLimitOnce smem_limit;
  const cudaError_t e = smem_limit.ensure(kern, smem);
  if (e != cudaSuccess) return e;
  // as many CTAs on a tile pair's keys as the SMs have room for, while each
  // keeps four steps of the longest context that the table can hold
  PrefillArgs b = a;
  const int tpc = 2 * kTcRows / a.group;
  // (no chunk is longer than what the table can hold)
  const int64_t room = static_cast<int64_t>(a.max_blocks_per_seq) << a.bs_log2;
  b.max_q_len = static_cast<int>(std::min<int64_t>(a.max_q_len, std::max<int64_t>(room, 1)));
  const int64_t tiles = (b.max_q_len - 1) / tpc + 1;
  const int64_t ctas = tiles * a.num_kv_heads * a.num_seqs, steps = room / kPairKeys;
  b.chunks = 1;
  while (b.chunks < 8 && 2 * b.chunks * ctas <= kSms && steps >= 8 * b.chunks) b.chunks *= 2;
  return launch_clusters(b.chunks, kern,
                         dim3(a.num_kv_heads * b.chunks, static_cast<unsigned>(tiles), a.num_seqs),
                         dim3(kThreads), smem, stream, km, vm, b);
}

}  // namespace

cudaError_t launch_prefill_fp4(const PrefillArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                               int head_dim, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return head_dim == 128 ? launch_t<__half, 128>(a, km, vm, stream)
                           : launch_t<__half, 64>(a, km, vm, stream);
  return head_dim == 128 ? launch_t<__nv_bfloat16, 128>(a, km, vm, stream)
                         : launch_t<__nv_bfloat16, 64>(a, km, vm, stream);
}

}  // namespace pa
