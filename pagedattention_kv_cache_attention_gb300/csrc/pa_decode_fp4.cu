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
//  * A tile (codes and scales of one block and head, 18 or 36 rows of
//    head_dim / 2 bytes) is one 2-D TMA copy with the swizzle of its row
//    length, so that both products read shared memory without conflicts.
//  * S^T[16 tokens, 8 heads] = K Q^T on mma.sync m16n8k16.  A lane reads 16
//    (or 8) bytes of a K row, which lie within one or two scale groups:
//    cvt.f16x2.e2m1x2 makes fp16 pairs of a byte and one fp16x2 product with
//    the group's scale makes them exact values of the cache.
//  * O^T[d, 8 heads] += V^T P^T.  A lane reads the same 16 (or 8) dimensions of
//    four tokens; two tokens' nibbles are merged into bytes by three logical
//    instructions for eight codes, so that a converted pair is already (token,
//    next token) of one dimension, and its scale pair is shared by the lane's
//    dimensions.
//  * fp32 online softmax in base 2.  P is carried as fp16 (11 bits; the output
//    has at most 11) scaled by 2^15, so that only probabilities below 2^-29 of
//    the running maximum lose bits and below 2^-39 vanish: a long context's
//    faint tail keeps its mass.
//  * Tokens that must not count get logit -inf and a V scale of zero; a code is
//    always finite, so nothing a masked slot holds (NaN scales among it)
//    reaches the output.
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

constexpr float kPShift = 15.f;  // P is held times 2^15

// Geometry of a tile in shared memory: rows of D / 2 bytes in the swizzle of
// that row length (64 bytes: 16-byte unit u of row r at u ^ ((r >> 1) & 3);
// 32 bytes: u ^ ((r >> 2) & 1)), the scales in the rows after the codes.
template <int D> struct Fp4Shape {
  static constexpr int kRow = D / 2;                   // bytes of a token's codes
  static constexpr int kScales = D / 16;               // bytes of a token's scales
  static constexpr int kSwizzle = D == 128 ? 3 : 1;    // units that a row's XOR reaches
  static constexpr int kSlot16 = D == 128 ? 1536 : 768;  // a 16-token tile, on a swizzle period
  static constexpr int kUnit = 2 * kSlot16;            // 32 tokens of K or V (one or two tiles)
  static constexpr int kMTiles = D / 16;
  static constexpr int kQChunks = D / 32;
};

// Row of a 16-token sub-tile that MMA row r stands for: a permutation that
// puts the four V rows 2c (c = 0..3) into different banks.
template <int D> __device__ __forceinline__ int token_of(int r) {
  return D == 128 ? r ^ ((r >> 1) & 1) : r ^ ((r >> 2) & 1);
}

// T: query and output type.  NW warps, S stages each, U 32-token units per
// step.  WP: each warp takes a whole partition and writes its partial itself
// (partitions joined by the reduce kernel), as in the 16-bit kernel.
template <typename T, int D, int NW, int S, int U, bool WP>
__global__ void __launch_bounds__(NW * 32)
    pa_decode_fp4_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const DecodeArgs a) {
  using Sh = Fp4Shape<D>;
  constexpr int kStep = 2 * U * Sh::kUnit;  // K then V of a step
  constexpr int kSubs = 2 * U;              // 16-token sub-tiles of a step
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NW * S * kStep);

  const int kvh = blockIdx.y, seq = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = WP ? blockIdx.x * NW + warp : blockIdx.x;
  if (WP && part >= a.num_parts) return;  // the last CTA's spare warps
  const int g = lane >> 2, c = lane & 3;
  uint8_t *my_stages = smem + warp * S * kStep;
  uint64_t *my_bars = bars + warp * S;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(&my_bars[s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dependency_wait();  // the pool may come from the kernel before

  // Units are 32-token windows of the sequence from the one that holds the
  // partition's first token on: a block never straddles two.  A warp's tiles
  // (tpu = 32 / block_size of them a unit) are numbered l in its own order; 32
  // lanes hold the block ids of a window of them.
  const int t_begin = part * a.part_tokens;
  const int base = t_begin & ~31;
  const int tsh = 5 - a.bs_log2, tpu = 1 << tsh;  // 1 or 2 tiles a unit
  const int32_t *bt_row = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
  auto unit_of = [&](int lu) {  // the warp's local unit -> the partition's
    return WP ? lu : (warp + (lu / U) * NW) * U + lu % U;
  };
  auto block_of = [&](int l) { return (base >> a.bs_log2) + (unit_of(l >> tsh) << tsh) + (l & (tpu - 1)); };
  auto table_entry = [&](int l) -> int {
    const int lb = block_of(l);
    return lb < a.max_blocks_per_seq ? bt_row[lb] : -1;
  };
  int win = table_entry(lane);  // read before the length arrives; entries past it are not used

  int ctx = a.context_lens[seq];
  if (ctx < 0 || ctx > (a.max_blocks_per_seq << a.bs_log2) || ctx > a.max_context_len) {
    if (threadIdx.x == 0 && part == 0 && kvh == 0) atomicOr(a.err, kErrBadLen);
    ctx = 0;
  }
  if (part > 0 && t_begin >= ctx) return;
  const int np_seq = ctx > 0 ? (ctx + a.part_tokens - 1) / a.part_tokens : 1;
  const int t_end = min(ctx, t_begin + a.part_tokens);
  const int n_unit = t_end > base ? (t_end - base + 31) / 32 : 0;
  const int n_grp = (n_unit + U - 1) / U;
  const int my_n = WP ? n_grp : (n_grp > warp ? (n_grp - warp + NW - 1) / NW : 0);

  // block id of the warp's tile l; -1 if it holds no token of the partition or is invalid
  auto checked = [&](int l, int phys) -> int {
    const int lb = block_of(l);
    if (l >= ((my_n * U) << tsh) || lb > ((t_end - 1) >> a.bs_log2) || lb < (t_begin >> a.bs_log2))
      return -1;
    if (phys < 0 || static_cast<int64_t>(phys) >= a.num_blocks) {
      atomicOr(a.err, kErrBadBlock);
      return -1;
    }
    return phys;
  };

  const uint64_t policy = l2_policy_evict_first();
  const uint32_t tile_bytes = fp4_tile_bytes(1 << a.bs_log2, D);
  const int tile_rows = 18 << (a.bs_log2 - 4);
  // lane 0: load the tiles of a step (phys of tile i in unit-tile order) into stage s
  auto issue = [&](const int (&phys)[kSubs], int s) {
    uint64_t *bar = &my_bars[s];
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < kSubs; ++i) bytes += i < (U << tsh) && phys[i] >= 0 ? 2 * tile_bytes : 0;
    if (bytes == 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, bytes);
    uint8_t *st = my_stages + s * kStep;
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
      if (i >= (U << tsh) || phys[i] < 0) continue;
      const int y = (phys[i] * a.num_kv_heads + kvh) * tile_rows;
      uint8_t *dst = st + (i >> tsh) * Sh::kUnit + (i & (tpu - 1)) * Sh::kSlot16;
      tma_load_2d(dst, &kmap, 0, y, bar, policy);
      tma_load_2d(dst + U * Sh::kUnit, &vmap, 0, y, bar, policy);
    }
  };

  int win_base = 0;
  win = checked(lane, win);
  const int my_tiles = (my_n * U) << tsh;
  int win_next = my_tiles > 32 ? checked(32 + lane, table_entry(32 + lane)) : -1;
  uint32_t stage_ok = 0;  // bit s kSubs + i: tile i of stage s is loaded
  auto tiles_of = [&](int k, int s, int (&phys)[kSubs]) {
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
      phys[i] = __shfl_sync(kFull, win, (((k * U) << tsh) + i - win_base) & 31);
      const uint32_t bit = 1u << (s * kSubs + i);
      stage_ok = phys[i] >= 0 && i < (U << tsh) ? stage_ok | bit : stage_ok & ~bit;
    }
  };
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (s < my_n) {
      int phys[kSubs];
      tiles_of(s, s, phys);
      if (lane == 0) issue(phys, s);
    }
  }

  // query fragments of head g, in the order of the K bytes a lane reads
  const int G = a.group;
  uint4 qf[Sh::kQChunks];
  float sl0 = a.scale_log2, sl1 = a.scale_log2;  // of the lane's columns 2c and 2c + 1
  {
    const T *qrow = static_cast<const T *>(a.query) +
                    (static_cast<int64_t>(seq) * a.num_q_heads + kvh * G + g) * D;
#pragma unroll
    for (int i = 0; i < Sh::kQChunks; ++i)
      qf[i] = g < G ? *reinterpret_cast<const uint4 *>(qrow + (c * Sh::kQChunks + i) * 8)
                    : make_uint4(0, 0, 0, 0);
    if constexpr (!std::is_same<T, __half>::value) {
      // bf16 queries: each head is scaled by 2^e so that its largest magnitude
      // lies in [2^14, 2^15), then rounded to fp16 (exact for every value down
      // to 2^-31 of the largest: bf16 carries 8 bits, and fp16 holds 8 bits at
      // every magnitude from 2^-17 up); 2^-e joins the head's softmax scale
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < Sh::kQChunks; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 v = Elem<T>::unpack(word_of(qf[i], w));
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
          const float2 v = Elem<T>::unpack(word_of(qf[i], w));
          w4[w] = Elem<__half>::pack(v.x * f, v.y * f);
        }
        qf[i] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
      }
      sl0 = ldexpf(sl0, -__shfl_sync(kFull, e, 8 * c));      // a lane of head 2c
      sl1 = ldexpf(sl1, -__shfl_sync(kFull, e, 8 * c + 4));  // of head 2c + 1
    }
  }

  // The lane's places in a sub-tile: K rows token_of(g) and + 8, V rows
  // t0 = token_of(2c), t1 = token_of(2c + 1) and + 8 (rows 8 apart share their
  // swizzle and lie 8 kRow bytes apart).
  const int kr = token_of<D>(g), t0 = token_of<D>(2 * c), t1 = token_of<D>(2 * c + 1);
  int k_at, v_at0, v_at1;
  if constexpr (D == 128) {
    k_at = kr * 64 + ((c ^ ((kr >> 1) & 3)) << 4);
    const int in_row = (((g >> 1) ^ c) << 4) + (g & 1) * 8;  // (t0 >> 1) & 3 = (t1 >> 1) & 3 = c
    v_at0 = t0 * 64 + in_row;
    v_at1 = t1 * 64 + in_row;
  } else {
    k_at = kr * 32 + (((c >> 1) ^ ((kr >> 2) & 1)) << 4) + (c & 1) * 8;
    const int in_row = (((g >> 2) ^ (c >> 1)) << 4) + (g & 3) * 4;  // (t0 >> 2) & 1 = c >> 1
    v_at0 = t0 * 32 + in_row;
    v_at1 = t1 * 32 + in_row;
  }
  const int kb = D == 128 ? 2 * c : c, vb = D == 128 ? g : g >> 1;  // scale groups of the lane
  // a 16-token sub-tile h of a unit: its codes and its scales.  The scales of
  // the upper half of a 32-token tile lie in rows whose swizzle flips unit 0.
  const bool bs16 = a.bs_log2 == 4;
  const int sub_step = bs16 ? Sh::kSlot16 : 16 * Sh::kRow;
  const int sc_base = bs16 ? 16 * Sh::kRow : 32 * Sh::kRow;
  const int sc_step = bs16 ? Sh::kSlot16 : 16 * Sh::kScales;
  const int sc_flip = D == 128 && !bs16 ? 16 : 0;

  const float NEG_INF = -INFINITY;
  float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1
  float acc[Sh::kMTiles][4];
#pragma unroll
  for (int mt = 0; mt < Sh::kMTiles; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;

  bool timed_out = false;
  int k_stop = my_n;
#pragma unroll 1
  for (int k = 0; k < my_n; ++k) {
    const int s = k % S;
    if (!__all_sync(kFull, mbar_wait_bounded(&my_bars[s], (k / S) & 1))) {
      if (lane == 0) atomicOr(a.err, kErrTimeout);
      timed_out = true;
      k_stop = k;
      break;
    }
    const uint8_t *stage = my_stages + s * kStep;
    // valid tokens [lo, hi) of each sub-tile
    int lo[kSubs], hi[kSubs];
    bool whole = true;
#pragma unroll
    for (int h = 0; h < kSubs; ++h) {
      const int tile = bs16 ? h : h >> 1;
      const int tok = base + unit_of(k * U + (h >> 1)) * 32 + (h & 1) * 16;
      const bool ok = (stage_ok >> (s * kSubs + tile)) & 1u;
      lo[h] = max(0, t_begin - tok);
      hi[h] = ok ? max(0, min(16, t_end - tok)) : 0;
      whole = whole && lo[h] == 0 && hi[h] == 16;
    }

    // ---- S^T = K Q^T
    float x[kSubs][4];
#pragma unroll
    for (int h = 0; h < kSubs; ++h) {
      const uint8_t *unit = stage + (h >> 1) * Sh::kUnit;
      const uint8_t *Ks = unit + (h & 1) * sub_step + k_at;
      const uint8_t *sc = unit + sc_base + (h & 1) * sc_step;
      const int flip = (h & 1) * sc_flip;
      const int sa = ((kr * Sh::kScales) ^ flip) + kb, sb = (((kr + 8) * Sh::kScales) ^ flip) + kb;
      x[h][0] = x[h][1] = x[h][2] = x[h][3] = 0.f;
      if constexpr (D == 128) {
        const uint4 wa = *reinterpret_cast<const uint4 *>(Ks);
        const uint4 wb = *reinterpret_cast<const uint4 *>(Ks + 8 * Sh::kRow);
        const uint32_t pa = e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + sa));
        const uint32_t pb = e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + sb));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t ga = __byte_perm(pa, 0, w < 2 ? 0x1010 : 0x3232);
          const uint32_t gb = __byte_perm(pb, 0, w < 2 ? 0x1010 : 0x3232);
          uint32_t ha[4], hb[4];
          e2m1x8_to_half(word_of(wa, w), ha);
          e2m1x8_to_half(word_of(wb, w), hb);
          Elem<__half>::mma(x[h], f16x2_mul(ha[0], ga), f16x2_mul(hb[0], gb), f16x2_mul(ha[1], ga),
                            f16x2_mul(hb[1], gb), qf[w].x, qf[w].y);
          Elem<__half>::mma(x[h], f16x2_mul(ha[2], ga), f16x2_mul(hb[2], gb), f16x2_mul(ha[3], ga),
                            f16x2_mul(hb[3], gb), qf[w].z, qf[w].w);
        }
      } else {
        const uint2 wa = *reinterpret_cast<const uint2 *>(Ks);
        const uint2 wb = *reinterpret_cast<const uint2 *>(Ks + 8 * Sh::kRow);
        const uint32_t p = e4m3x2_lo_to_f16x2(sc[sa] | (static_cast<uint32_t>(sc[sb]) << 8));
        const uint32_t ga = __byte_perm(p, 0, 0x1010), gb = __byte_perm(p, 0, 0x3232);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t ha[4], hb[4];
          e2m1x8_to_half(w == 0 ? wa.x : wa.y, ha);
          e2m1x8_to_half(w == 0 ? wb.x : wb.y, hb);
          Elem<__half>::mma(x[h], f16x2_mul(ha[0], ga), f16x2_mul(hb[0], gb), f16x2_mul(ha[1], ga),
                            f16x2_mul(hb[1], gb), qf[w].x, qf[w].y);
          Elem<__half>::mma(x[h], f16x2_mul(ha[2], ga), f16x2_mul(hb[2], gb), f16x2_mul(ha[3], ga),
                            f16x2_mul(hb[3], gb), qf[w].z, qf[w].w);
        }
      }
    }

    // ---- online softmax in base 2, one reduction for the step's tokens
#pragma unroll
    for (int h = 0; h < kSubs; ++h) {
      x[h][0] *= sl0;
      x[h][1] *= sl1;
      x[h][2] *= sl0;
      x[h][3] *= sl1;
    }
    if (!whole) {
#pragma unroll
      for (int h = 0; h < kSubs; ++h) {
        const bool va = kr >= lo[h] && kr < hi[h], vz = kr + 8 >= lo[h] && kr + 8 < hi[h];
        x[h][0] = va ? x[h][0] : NEG_INF;
        x[h][1] = va ? x[h][1] : NEG_INF;
        x[h][2] = vz ? x[h][2] : NEG_INF;
        x[h][3] = vz ? x[h][3] : NEG_INF;
      }
    }
    float mx0 = m0, mx1 = m1;
#pragma unroll
    for (int h = 0; h < kSubs; ++h) {
      mx0 = fmaxf(mx0, fmaxf(x[h][0], x[h][2]));
      mx1 = fmaxf(mx1, fmaxf(x[h][1], x[h][3]));
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, off));
    }
    const float r0 = mx0 == NEG_INF ? 0.f : mx0 - kPShift;  // no valid token yet: any reference
    const float r1 = mx1 == NEG_INF ? 0.f : mx1 - kPShift;
    if (__any_sync(kFull, mx0 != m0 || mx1 != m1)) {
      const float al0 = ex2_approx(m0 - kPShift - r0), al1 = ex2_approx(m1 - kPShift - r1);
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int mt = 0; mt < Sh::kMTiles; ++mt) {
        acc[mt][0] *= al0;
        acc[mt][1] *= al1;
        acc[mt][2] *= al0;
        acc[mt][3] *= al1;
      }
      m0 = mx0;
      m1 = mx1;
    }
    uint32_t pb0[kSubs], pb1[kSubs];
#pragma unroll
    for (int h = 0; h < kSubs; ++h) {
      const float p0 = ex2_approx(x[h][0] - r0), p1 = ex2_approx(x[h][1] - r1);
      const float p2 = ex2_approx(x[h][2] - r0), p3 = ex2_approx(x[h][3] - r1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      // P^T as the B operand: an 8x8 transpose of the accumulator's layout
      pb0[h] = movmatrix_trans(Elem<__half>::pack(p0, p1));
      pb1[h] = movmatrix_trans(Elem<__half>::pack(p2, p3));
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int h = 0; h < kSubs; ++h) {
      const uint8_t *unit = stage + (U + (h >> 1)) * Sh::kUnit;
      const uint8_t *Vs = unit + (h & 1) * sub_step;
      const uint8_t *sc = unit + sc_base + (h & 1) * sc_step + vb;
      const int flip = (h & 1) * sc_flip;
      uint32_t s0 = sc[(t0 * Sh::kScales) ^ flip], s1 = sc[(t1 * Sh::kScales) ^ flip];
      uint32_t s2 = sc[((t0 + 8) * Sh::kScales) ^ flip], s3 = sc[((t1 + 8) * Sh::kScales) ^ flip];
      if (!whole) {
        s0 = t0 >= lo[h] && t0 < hi[h] ? s0 : 0;
        s1 = t1 >= lo[h] && t1 < hi[h] ? s1 : 0;
        s2 = t0 + 8 >= lo[h] && t0 + 8 < hi[h] ? s2 : 0;
        s3 = t1 + 8 >= lo[h] && t1 + 8 < hi[h] ? s3 : 0;
      }
      const uint32_t g01 = e4m3x2_lo_to_f16x2(s0 | (s1 << 8));
      const uint32_t g23 = e4m3x2_lo_to_f16x2(s2 | (s3 << 8));
      // words of eight codes of tokens (A, B) -> even dimensions' pairs, odd dimensions' pairs
      auto pairs = [](uint32_t A, uint32_t B, uint32_t (&even)[4], uint32_t (&odd)[4]) {
        e2m1x8_to_half((A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u), even);
        e2m1x8_to_half(((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u), odd);
      };
      if constexpr (D == 128) {
        const uint2 v0 = *reinterpret_cast<const uint2 *>(Vs + v_at0);
        const uint2 v1 = *reinterpret_cast<const uint2 *>(Vs + v_at1);
        const uint2 v2 = *reinterpret_cast<const uint2 *>(Vs + v_at0 + 8 * Sh::kRow);
        const uint2 v3 = *reinterpret_cast<const uint2 *>(Vs + v_at1 + 8 * Sh::kRow);
        uint32_t a0[2][4], a1[2][4], a2[2][4], a3[2][4];
        pairs(v0.x, v1.x, a0[0], a0[1]);
        pairs(v0.y, v1.y, a1[0], a1[1]);
        pairs(v2.x, v3.x, a2[0], a2[1]);
        pairs(v2.y, v3.y, a3[0], a3[1]);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
          Elem<__half>::mma(acc[mt], f16x2_mul(a0[mt & 1][mt >> 1], g01),
                            f16x2_mul(a1[mt & 1][mt >> 1], g01), f16x2_mul(a2[mt & 1][mt >> 1], g23),
                            f16x2_mul(a3[mt & 1][mt >> 1], g23), pb0[h], pb1[h]);
      } else {
        uint32_t a0[2][4], a2[2][4];
        pairs(*reinterpret_cast<const uint32_t *>(Vs + v_at0),
              *reinterpret_cast<const uint32_t *>(Vs + v_at1), a0[0], a0[1]);
        pairs(*reinterpret_cast<const uint32_t *>(Vs + v_at0 + 8 * Sh::kRow),
              *reinterpret_cast<const uint32_t *>(Vs + v_at1 + 8 * Sh::kRow), a2[0], a2[1]);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
          Elem<__half>::mma(acc[mt], f16x2_mul(a0[mt & 1][mt >> 1], g01),
                            f16x2_mul(a0[mt & 1][2 + (mt >> 1)], g01), f16x2_mul(a2[mt & 1][mt >> 1], g23),
                            f16x2_mul(a2[mt & 1][2 + (mt >> 1)], g23), pb0[h], pb1[h]);
      }
    }

    // ---- refill this stage with step k + S
    __syncwarp();
    const int nk = k + S;
    if (nk < my_n) {
      if (((nk * U) << tsh) >= win_base + 32) {
        win_base += 32;
        win = win_next;
        win_next = checked(win_base + 32 + lane, table_entry(win_base + 32 + lane));
      }
      int phys[kSubs];
      tiles_of(nk, s, phys);
      if (lane == 0) {
        fence_proxy_async_smem();
        issue(phys, s);
      }
    }
  }

  if (timed_out) {
    // let copies already in flight land before the CTA leaves (bounded again)
    for (int kk = k_stop; kk < min(k_stop + S, my_n); ++kk)
      (void)mbar_wait_bounded(&my_bars[kk % S], (kk / S) & 1);
  }

  // row sums over the 8 token rows; l and acc are both held times 2^kPShift
  const float unshift = exp2f(-kPShift);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(kFull, l0, off);
    l1 += __shfl_xor_sync(kFull, l1, off);
  }
  l0 *= unshift;
  l1 *= unshift;

  if constexpr (WP) {
    const int64_t row0 = static_cast<int64_t>(seq) * a.num_q_heads + kvh * G;
    const int h0 = 2 * c, h1 = 2 * c + 1;
    const float inv0 = l0 > 0.f ? a.out_scale * unshift / l0 : 0.f;
    const float inv1 = l1 > 0.f ? a.out_scale * unshift / l1 : 0.f;
    const int64_t pr0 = (row0 + h0) * a.num_parts + part, pr1 = (row0 + h1) * a.num_parts + part;
    if (g == 0) {
      if (h0 < G) {
        a.ws_m[pr0] = m0;
        a.ws_l[pr0] = l0;
      }
      if (h1 < G) {
        a.ws_m[pr1] = m1;
        a.ws_l[pr1] = l1;
      }
    }
    store_partial_o<D, true>(a.ws_o + pr0 * D, a.ws_o + pr1 * D, h0 < G, h1 < G, acc, inv0, inv1,
                             g);
    grid_launch_dependents();
    return;
  }

  // ---- merge warps through shared memory (stages are idle now)
  __syncthreads();
  float *wacc = reinterpret_cast<float *>(smem);  // [NW][8][D]
  float *wml = wacc + NW * 8 * D;                 // [NW][8][2]
  if (g == 0) {
    wml[(warp * 8 + 2 * c) * 2 + 0] = m0;
    wml[(warp * 8 + 2 * c) * 2 + 1] = l0;
    wml[(warp * 8 + 2 * c + 1) * 2 + 0] = m1;
    wml[(warp * 8 + 2 * c + 1) * 2 + 1] = l1;
  }
  {
    float *h0 = wacc + (warp * 8 + 2 * c) * D;
    store_partial_o<D, true>(h0, h0 + D, true, true, acc, unshift, unshift, g);
  }
  __syncthreads();
  constexpr int kChunks = D / 8;
  for (int item = threadIdx.x; item < G * kChunks; item += NW * 32) {
    const int h = item / kChunks, ch = item % kChunks;
    float M = NEG_INF;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wml[(w * 8 + h) * 2]);
    float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = wml[(w * 8 + h) * 2];
      const float f = mw == NEG_INF ? 0.f : exp2f(mw - M);
      L += wml[(w * 8 + h) * 2 + 1] * f;
      const float *src = wacc + (w * 8 + h) * D + ch * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += src[e] * f;
    }
    const int64_t row = static_cast<int64_t>(seq) * a.num_q_heads + kvh * G + h;
    const float inv = L > 0.f ? a.out_scale / L : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    if (a.num_parts == 1 || (a.fuse_join && np_seq == 1)) {
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
  if (a.fuse_join && np_seq > 1) {
    if (last_to_arrive(a, seq, kvh, np_seq, reinterpret_cast<uint32_t *>(wml + NW * 8 * 2)))
      join_partitions<T, D, NW>(a, seq, kvh, np_seq);
  }
  grid_launch_dependents();
}

#ifndef PA_DECODE_FP4_WARPS
#define PA_DECODE_FP4_WARPS 4
#endif
#ifndef PA_DECODE_FP4_STAGES
#define PA_DECODE_FP4_STAGES 2
#endif
#ifndef PA_DECODE_FP4_UNITS
#define PA_DECODE_FP4_UNITS 1
#endif

template <typename T, int D, bool WP>
cudaError_t launch_w(const DecodeArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                     cudaStream_t stream) {
  constexpr int NW = PA_DECODE_FP4_WARPS, S = PA_DECODE_FP4_STAGES, U = PA_DECODE_FP4_UNITS;
  constexpr size_t stages = static_cast<size_t>(NW) * S * 2 * U * Fp4Shape<D>::kUnit;
  constexpr size_t smem = 1024 + stages + NW * S * 8;
  static_assert(static_cast<size_t>(NW) * 8 * D * 4 + NW * 8 * 2 * 4 + 16 <= stages,
                "merge buffers and the join flag must fit in the stage area");
  static_assert(S * 2 * U <= 32, "stage bits");
  auto kern = pa_decode_fp4_kernel<T, D, NW, S, U, WP>;
  static SmemLimitOnce smem_limit;
  const cudaError_t e = smem_limit.ensure(kern, smem);
  if (e != cudaSuccess) return e;
  const unsigned gx = WP ? static_cast<unsigned>((a.num_parts + NW - 1) / NW)
                         : static_cast<unsigned>(a.num_parts);
  return launch_dependent(kern, dim3(gx, a.num_kv_heads, a.num_seqs), dim3(NW * 32), smem, stream,
                          km, vm, a);
}

template <typename T, int D>
cudaError_t launch_t(const DecodeArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                     cudaStream_t stream) {
  return a.num_parts > 1 && !a.fuse_join ? launch_w<T, D, true>(a, km, vm, stream)
                                         : launch_w<T, D, false>(a, km, vm, stream);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeArgs &a, const void *k_cache, const void *v_cache,
                              int head_dim, int dtype, cudaStream_t stream, bool *map_failed) {
  CUtensorMap km, vm;
  const int64_t tiles = a.num_blocks * a.num_kv_heads;
  *map_failed = !encode_fp4_map(&km, k_cache, tiles, 1 << a.bs_log2, head_dim, true) ||
                !encode_fp4_map(&vm, v_cache, tiles, 1 << a.bs_log2, head_dim, true);
  if (*map_failed) return cudaErrorInvalidValue;
  if (dtype == 0)
    return head_dim == 128 ? launch_t<__half, 128>(a, km, vm, stream)
                           : launch_t<__half, 64>(a, km, vm, stream);
  return head_dim == 128 ? launch_t<__nv_bfloat16, 128>(a, km, vm, stream)
                         : launch_t<__nv_bfloat16, 64>(a, km, vm, stream);
}

}  // namespace pa
