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
//  * fp32 online softmax in base 2 against a reference that moves only when a
//    score passes it by more than 4.  P is carried as fp16 (11 bits; the output
//    has at most 11) times 2^11, so that only probabilities below 2^-25 of the
//    maximum lose bits and below 2^-35 vanish: a long context's faint tail
//    keeps its mass.
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

#ifndef PA_DECODE_FP4_WARPS
#define PA_DECODE_FP4_WARPS 4
#endif
#ifndef PA_DECODE_FP4_STAGES
#define PA_DECODE_FP4_STAGES 2
#endif
#ifndef PA_DECODE_FP4_CTAS
#define PA_DECODE_FP4_CTAS 4
#endif

// P is held times 2^11, against a reference that is at most 2^4 below the
// running maximum: below 2^15 then, and in fp16's normal range down to 2^-25 of
// the maximum.
constexpr float kPShift = 11.f, kGrowth = 4.f;

// Geometry of a tile in shared memory.  TMA brings it in lines of D bytes (the
// codes of two tokens; 9 lines for 16 tokens, the last of them scales) with the
// swizzle of that line length: byte address bits 4.. ^= bits 7.. (three bits at
// 128-byte lines, two at 64).  A 16-token tile takes a place of 12 lines, so
// that the second tile of a 32-token unit (and of no other pair of places)
// starts half a swizzle period off: all its addresses are XORed with kOdd.
template <int D, int BS> struct Fp4Shape {
  static constexpr int kRow = D / 2;                     // bytes of a token's codes
  static constexpr int kScales = D / 16;                 // bytes of a token's scales
  static constexpr int kSlot16 = 12 * D;
  static constexpr int kUnit = 2 * kSlot16;              // 32 tokens of K or V
  static constexpr int kTiles = 32 / BS;                 // tiles of a unit
  static constexpr int kLines = BS * 9 / 16;             // lines of a tile
  static constexpr int kTileBytes = fp4_tile_bytes(BS, D);
  static constexpr int kOdd = BS == 16 ? D / 2 : 0;
  // codes and scales of the unit's 16-token half h
  __host__ __device__ static constexpr int codes(int h) { return h * (BS == 16 ? kSlot16 : 16 * kRow); }
  __host__ __device__ static constexpr int scales(int h) {
    return BS == 16 ? h * kSlot16 + 16 * kRow : 32 * kRow + h * 16 * kScales;
  }
  __host__ __device__ static constexpr int flip_codes(int h) { return h * kOdd; }
  // (the second half's scales of a 32-token tile lie in the line that the
  // 128-byte swizzle XORs with one 16-byte unit)
  __host__ __device__ static constexpr int flip_scales(int h) { return h * (BS == 16 ? kOdd : (D == 128 ? 16 : 0)); }
  static constexpr int kMTiles = D / 16;
  static constexpr int kQChunks = D / 32;
};

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

// T: query and output type.  NW warps, S stages each.  WP: each warp takes a
// whole partition and writes its partial itself (partitions joined by the
// reduce kernel), as in the 16-bit kernel.
template <typename T, int D, int BS, int NW, int S, bool WP>
__global__ void __launch_bounds__(NW * 32, PA_DECODE_FP4_CTAS)
    pa_decode_fp4_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const DecodeArgs a) {
  using Sh = Fp4Shape<D, BS>;
  constexpr int kStep = 2 * Sh::kUnit;  // K then V of a 32-token step
  constexpr int kTiles = Sh::kTiles;
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

  // Steps are 32-token windows of the sequence from the one that holds the
  // partition's first token on: a block never straddles two.  A warp's tiles
  // are numbered l in its own order; 32 lanes hold a window of 32 of them.
  const int t_begin = part * a.part_tokens;
  const int base = t_begin & ~31;
  const int32_t *bt_row = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
  auto step_token = [&](int k) { return base + (WP ? k : warp + k * NW) * 32; };
  auto block_of = [&](int l) { return step_token(l / kTiles) / BS + l % kTiles; };
  auto table_entry = [&](int l) -> int {
    const int lb = block_of(l);
    return lb < a.max_blocks_per_seq ? bt_row[lb] : -1;
  };
  int win = table_entry(lane);  // read before the length arrives; entries past it are not used

  int ctx = a.context_lens[seq];
  if (ctx < 0 || ctx > a.max_blocks_per_seq * BS || ctx > a.max_context_len) {
    if (threadIdx.x == 0 && part == 0 && kvh == 0) atomicOr(a.err, kErrBadLen);
    ctx = 0;
  }
  if (part > 0 && t_begin >= ctx) return;
  const int np_seq = ctx > 0 ? (ctx + a.part_tokens - 1) / a.part_tokens : 1;
  const int t_end = min(ctx, t_begin + a.part_tokens);
  const int n_step = t_end > base ? (t_end - base + 31) / 32 : 0;
  const int my_n = WP ? n_step : (n_step > warp ? (n_step - warp + NW - 1) / NW : 0);

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

  // The lane's places in a half: K rows token_of(g) and + 8, V rows t0 =
  // token_of(2c), t1 = token_of(2c + 1) and + 8.  Row r + 8 lies 8 kRow bytes
  // on, in lines whose 128-byte swizzle differs in unit bit 2 (a 64-byte line's
  // in none).
  const int kr = token_of<D>(g), t0 = token_of<D>(2 * c), t1 = token_of<D>(2 * c + 1);
  constexpr int kBytes = D == 128 ? 16 : 8;  // of a K row; of a V row half of them
  const int k_a = code_at<D>(kr, c * kBytes), k_b = code_at<D>(kr + 8, c * kBytes);
  const int v_0 = code_at<D>(t0, g * kBytes / 2), v_1 = code_at<D>(t1, g * kBytes / 2);
  const int v_2 = code_at<D>(t0 + 8, g * kBytes / 2), v_3 = code_at<D>(t1 + 8, g * kBytes / 2);
  // scale groups of the lane: 2c and 2c + 1 (or c) of K, g (or g / 2) of V
  const int ks_a = kr * Sh::kScales + (D == 128 ? 2 * c : c), ks_b = ks_a + 8 * Sh::kScales;
  const int vs_0 = t0 * Sh::kScales + (D == 128 ? g : g >> 1);
  const int vs_1 = t1 * Sh::kScales + (D == 128 ? g : g >> 1);

  const float NEG_INF = -INFINITY;
  // online softmax of the lane's heads 2c and 2c + 1 in base 2: c0 = kPShift -
  // the reference of head 2c, so that probabilities are held as 2^(x + c0);
  // before the first token the reference is far below any score
  float c0 = 1e30f, c1 = 1e30f, l0 = 0.f, l1 = 0.f;
  float acc[Sh::kMTiles][4];
#pragma unroll
  for (int mt = 0; mt < Sh::kMTiles; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;

  // One step, its K and V at `stage`.  masked: only the tokens that `mask` has
  // count (bit i: token i of the step); the code of whole steps is apart, as
  // the selects cost a seventh of a step's instructions.
  auto step = [&](const uint8_t *stage, bool masked, uint32_t mask) {
    // ---- S^T = K Q^T
    float x[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t *Ks = stage + Sh::codes(h);
      const uint8_t *sc = stage + Sh::scales(h);
      // two chains of products, so that half of them wait for one another
      float y[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int ca = k_a ^ Sh::flip_codes(h), cb = k_b ^ Sh::flip_codes(h);
      const int sa = ks_a ^ Sh::flip_scales(h), sb = ks_b ^ Sh::flip_scales(h);
      uint32_t pa, pb;  // the scales of rows a and b as fp16 pairs
      uint32_t wa[D / 32], wb[D / 32];
      if constexpr (D == 128) {
        const uint4 va = *reinterpret_cast<const uint4 *>(Ks + ca);
        const uint4 vb = *reinterpret_cast<const uint4 *>(Ks + cb);
        wa[0] = va.x, wa[1] = va.y, wa[2] = va.z, wa[3] = va.w;
        wb[0] = vb.x, wb[1] = vb.y, wb[2] = vb.z, wb[3] = vb.w;
        pa = e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + sa));
        pb = e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + sb));
      } else {
        const uint2 va = *reinterpret_cast<const uint2 *>(Ks + ca);
        const uint2 vb = *reinterpret_cast<const uint2 *>(Ks + cb);
        wa[0] = va.x, wa[1] = va.y;
        wb[0] = vb.x, wb[1] = vb.y;
        pa = e4m3x2_lo_to_f16x2(sc[sa] * 0x101u);
        pb = e4m3x2_lo_to_f16x2(sc[sb] * 0x101u);
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t ga = D == 64 ? pa : __byte_perm(pa, 0, w < 2 ? 0x1010 : 0x3232);
        const uint32_t gb = D == 64 ? pb : __byte_perm(pb, 0, w < 2 ? 0x1010 : 0x3232);
        uint32_t ha[4], hb[4];
        e2m1x8_to_half(wa[w], ha);
        e2m1x8_to_half(wb[w], hb);
        Elem<__half>::mma(y[0], f16x2_mul(ha[0], ga), f16x2_mul(hb[0], gb), f16x2_mul(ha[1], ga),
                          f16x2_mul(hb[1], gb), qf[w].x, qf[w].y);
        Elem<__half>::mma(y[1], f16x2_mul(ha[2], ga), f16x2_mul(hb[2], gb), f16x2_mul(ha[3], ga),
                          f16x2_mul(hb[3], gb), qf[w].z, qf[w].w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = y[0][e] + y[1][e];
    }

    // z = scores + (b0, b1); tokens that do not count get -inf
    auto logits = [&](float (&z)[2][4], float b0, float b1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        z[h][0] = fmaf(x[h][0], sl0, b0);
        z[h][1] = fmaf(x[h][1], sl1, b1);
        z[h][2] = fmaf(x[h][2], sl0, b0);
        z[h][3] = fmaf(x[h][3], sl1, b1);
        if (masked) {
          const bool va = (mask >> (16 * h + kr)) & 1u, vz = (mask >> (16 * h + kr + 8)) & 1u;
          z[h][0] = va ? z[h][0] : NEG_INF;
          z[h][1] = va ? z[h][1] : NEG_INF;
          z[h][2] = vz ? z[h][2] : NEG_INF;
          z[h][3] = vz ? z[h][3] : NEG_INF;
        }
      }
    };
    // 2^y are the probabilities; the reference moves only when one of them
    // passes 2^(kPShift + kGrowth), so most steps need a vote and no shuffles
    float y[2][4];
    logits(y, c0, c1);
    float top = NEG_INF;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      top = fmaxf(top, fmaxf(fmaxf(y[h][0], y[h][1]), fmaxf(y[h][2], y[h][3])));
    if (__any_sync(kFull, top > kPShift + kGrowth)) {
      logits(y, 0.f, 0.f);
      float mx0 = kPShift - c0, mx1 = kPShift - c1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx0 = fmaxf(mx0, fmaxf(y[h][0], y[h][2]));
        mx1 = fmaxf(mx1, fmaxf(y[h][1], y[h][3]));
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, off));
        mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, off));
      }
      const float n0 = kPShift - mx0, n1 = kPShift - mx1;
      const float al0 = ex2_approx(n0 - c0), al1 = ex2_approx(n1 - c1);
      c0 = n0;
      c1 = n1;
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int mt = 0; mt < Sh::kMTiles; ++mt) {
        acc[mt][0] *= al0;
        acc[mt][1] *= al1;
        acc[mt][2] *= al0;
        acc[mt][3] *= al1;
      }
      logits(y, c0, c1);
    }
    uint32_t pb0[2], pb1[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float p0 = ex2_approx(y[h][0]), p1 = ex2_approx(y[h][1]);
      const float p2 = ex2_approx(y[h][2]), p3 = ex2_approx(y[h][3]);
      l0 += p0 + p2;
      l1 += p1 + p3;
      // P^T as the B operand: an 8x8 transpose of the accumulator's layout
      pb0[h] = movmatrix_trans(Elem<__half>::pack(p0, p1));
      pb1[h] = movmatrix_trans(Elem<__half>::pack(p2, p3));
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t *Vs = stage + Sh::kUnit + Sh::codes(h);
      const uint8_t *sc = stage + Sh::kUnit + Sh::scales(h);
      uint32_t s0 = sc[vs_0 ^ Sh::flip_scales(h)], s1 = sc[vs_1 ^ Sh::flip_scales(h)];
      uint32_t s2 = sc[(vs_0 + 8 * Sh::kScales) ^ Sh::flip_scales(h)];
      uint32_t s3 = sc[(vs_1 + 8 * Sh::kScales) ^ Sh::flip_scales(h)];
      if (masked) {
        s0 = (mask >> (16 * h + t0)) & 1u ? s0 : 0;
        s1 = (mask >> (16 * h + t1)) & 1u ? s1 : 0;
        s2 = (mask >> (16 * h + t0 + 8)) & 1u ? s2 : 0;
        s3 = (mask >> (16 * h + t1 + 8)) & 1u ? s3 : 0;
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
      const int c_0 = v_0 ^ Sh::flip_codes(h), c_1 = v_1 ^ Sh::flip_codes(h);
      const int c_2 = v_2 ^ Sh::flip_codes(h), c_3 = v_3 ^ Sh::flip_codes(h);
      if constexpr (D == 128) {
        const uint2 w0 = *reinterpret_cast<const uint2 *>(Vs + c_0);
        const uint2 w1 = *reinterpret_cast<const uint2 *>(Vs + c_1);
        const uint2 w2 = *reinterpret_cast<const uint2 *>(Vs + c_2);
        const uint2 w3 = *reinterpret_cast<const uint2 *>(Vs + c_3);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {  // m-tiles 0, 2, 4, 6, then 1, 3, 5, 7
          uint32_t a0[4], a1[4], a2[4], a3[4];
          pairs(w0.x, w1.x, odd, g01, a0);
          pairs(w0.y, w1.y, odd, g01, a1);
          pairs(w2.x, w3.x, odd, g23, a2);
          pairs(w2.y, w3.y, odd, g23, a3);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            Elem<__half>::mma(acc[2 * i + odd], a0[i], a1[i], a2[i], a3[i], pb0[h], pb1[h]);
        }
      } else {
        const uint32_t w0 = *reinterpret_cast<const uint32_t *>(Vs + c_0);
        const uint32_t w1 = *reinterpret_cast<const uint32_t *>(Vs + c_1);
        const uint32_t w2 = *reinterpret_cast<const uint32_t *>(Vs + c_2);
        const uint32_t w3 = *reinterpret_cast<const uint32_t *>(Vs + c_3);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {  // m-tiles 0, 2, then 1, 3
          uint32_t a0[4], a2[4];
          pairs(w0, w1, odd, g01, a0);
          pairs(w2, w3, odd, g23, a2);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            Elem<__half>::mma(acc[2 * i + odd], a0[i], a0[2 + i], a2[i], a2[2 + i], pb0[h],
                              pb1[h]);
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
    if (!bad && step_tok >= t_begin && step_tok + 32 <= t_end) {
      step(stage, false, 0xffffffffu);
    } else {
      const int tok = step_tok + lane;
      bool in = tok >= t_begin && tok < t_end;
      if (bad && in) {
        const int phys = bt_row[tok / BS];
        in = phys >= 0 && static_cast<int64_t>(phys) < a.num_blocks;
      }
      step(stage, true, __ballot_sync(kFull, in));
    }

    // ---- refill this stage with step k + S
    __syncwarp();
    if (k + S < my_n) fill(k + S, s);
  }
  // after a wait that ran out, copies already in flight land before the CTA
  // leaves (bounded again)
  for (const int filled = min(k + S, my_n); timed_out && k < filled; ++k)
    (void)mbar_wait_bounded(&my_bars[k % S], (k / S) & 1);

  // row sums over the 8 token rows; l and acc are both held times 2^kPShift
  const float unshift = exp2f(-kPShift);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(kFull, l0, off);
    l1 += __shfl_xor_sync(kFull, l1, off);
  }
  l0 *= unshift;
  l1 *= unshift;
  const float m0 = kPShift - c0, m1 = kPShift - c1;  // the references

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

template <typename T, int D, int BS, bool WP>
cudaError_t launch_w(const DecodeArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                     cudaStream_t stream) {
  constexpr int NW = PA_DECODE_FP4_WARPS, S = PA_DECODE_FP4_STAGES;
  constexpr size_t stages = static_cast<size_t>(NW) * S * 2 * Fp4Shape<D, BS>::kUnit;
  constexpr size_t smem = 1024 + stages + NW * S * 8;
  static_assert(static_cast<size_t>(NW) * 8 * D * 4 + NW * 8 * 2 * 4 + 16 <= stages,
                "merge buffers and the join flag must fit in the stage area");
  auto kern = pa_decode_fp4_kernel<T, D, BS, NW, S, WP>;
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
  const bool wp = a.num_parts > 1 && !a.fuse_join;
  if (a.bs_log2 == 4)
    return wp ? launch_w<T, D, 16, true>(a, km, vm, stream)
              : launch_w<T, D, 16, false>(a, km, vm, stream);
  return wp ? launch_w<T, D, 32, true>(a, km, vm, stream)
            : launch_w<T, D, 32, false>(a, km, vm, stream);
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
