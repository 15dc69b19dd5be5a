// pa_tc.cuh -- what the tcgen05 prefill kernels share: wrappers of the
// instructions that they use beyond pa_device.cuh's, packed fp32 arithmetic, and
// the widening of FP4 tiles to the fp16 stages of the matrix products.
#pragma once

#include <stdint.h>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kTcRows = 128;     // query rows per tile = TMEM lanes
constexpr int kPairKeys = 64;                  // keys per step
constexpr unsigned kFullMask = 0xffffffffu;

// D (TMEM) [+]= A (TMEM, K-major: lane = row, column c = elements 2c, 2c+1) * B (smem)
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// 16 consecutive 32-bit columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Non-blocking look at an mbarrier phase (acquire, CTA scope): true once the
// phase with the given parity has completed.
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Packed fp32 pairs (sm_100 and later): two IEEE fp32 operations per instruction,
// each rounded exactly as the scalar one.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Place of a raw 16-token FP4 tile (TMA copies start on 128 bytes); a 32-token
// tile takes two.
template <int D> constexpr int kRawSlot16 = D == 128 ? 1152 : 640;

// FP4 caches: 32 rows of raw tiles (unswizzled) at a time become rows of the
// fp16 tile that the MMA reads, every value s * e2m1(code) exact there.  A lane
// takes 32 dimensions of a row, four words of eight codes, each one 16-byte
// store.  Its words are taken in an order i = t ^ f that differs between lanes:
// with it the 32 word loads of a step t hit 32 banks, and the eight stores of
// a phase (two rows of four lanes, or four rows of two) eight different
// 16-byte bank groups of the swizzled rows.  f and every offset depend on the
// lane alone and are worked out once: worked out for each row, the widening took
// as long as the whole step (2,030 of 2,100 cycles, measured), and with them it
// takes 1,400.
template <int D> struct F4Widen {
  static constexpr int kPerRow = D / 32;          // lanes per row
  static constexpr int kRows = 32 / kPerRow;      // rows per pass: 8 or 16
  static constexpr int kPasses = 16 / kRows;      // passes of a 16-row group
  int row, read[4], write[4], scale;
  uint32_t sel_lo, sel_hi;  // the scale pair's halves for words t < 2 and t >= 2
  int group1, scale0, scale1;  // second 16-row group, scales of the first and of the second

  // atom_bytes: from one 64-dimension atom of the fp16 stage to the next
  __device__ __forceinline__ F4Widen(int lane, int bs_log2, int atom_bytes) {
    const int u = lane % kPerRow;
    row = lane / kPerRow;
    const int f = D == 128 ? ((row >> 1) & 3) ^ (u >> 1) ^ ((row & 1) << 1) : (row >> 2) & 3;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int i = t ^ f;
      read[t] = row * (D / 2) + u * 16 + (i << 2);
      write[t] = (u >> 1) * atom_bytes + row * 128 + ((((u & 1) * 4 + i) ^ (row & 7)) << 4);
    }
    scale = row * (D / 16) + 2 * u;
    sel_lo = f & 2 ? 0x3232 : 0x1010;
    sel_hi = f & 2 ? 0x1010 : 0x3232;
    const bool bs16 = bs_log2 == 4;
    group1 = bs16 ? kRawSlot16<D> : 16 * (D / 2);
    scale0 = (bs16 ? 16 : 32) * (D / 2);
    scale1 = bs16 ? kRawSlot16<D> + 16 * (D / 2) : 32 * (D / 2) + D;
  }

  // The lane's pair of scales (of groups 2 u and 2 u + 1, u = lane % kPerRow)
  // without NaNs, which are noted: nan[group] becomes the least key with a NaN
  // scale in the group, nan[D / 16] that of all groups.
  static __device__ __forceinline__ uint32_t drop_nans(uint32_t sc, int lane, int key, int *nan) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (((sc >> (8 * i)) & 0x7fu) == 0x7fu) {
        sc &= ~(0xffu << (8 * i));
        atomicMin(&nan[2 * (lane % kPerRow) + i], key);
        atomicMin(&nan[D / 16], key);
      }
    return sc;
  }

  // rows 0..31 of raw to rows 0..31 at st, with the scales fix(row, pair); a
  // scale of zero makes zeros: a code is always finite
  template <typename Fix>
  __device__ __forceinline__ void operator()(const uint8_t *raw, uint8_t *st, Fix fix) const {
    uint32_t w[2][kPasses][4], sc[2][kPasses];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const uint8_t *codes = raw + (q ? group1 : 0) + p * kRows * (D / 2);
#pragma unroll
        for (int t = 0; t < 4; ++t) w[q][p][t] = *reinterpret_cast<const uint32_t *>(codes + read[t]);
        sc[q][p] = *reinterpret_cast<const uint16_t *>(raw + (q ? scale1 : scale0) +
                                                       p * kRows * (D / 16) + scale);
      }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r0 = 16 * q + p * kRows;
        const uint32_t s2 = e4m3x2_lo_to_f16x2(fix(r0 + row, sc[q][p]));
        const uint32_t lo = __byte_perm(s2, 0, sel_lo), hi = __byte_perm(s2, 0, sel_hi);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t g = t < 2 ? lo : hi;
          uint32_t h[4];
          e2m1x8_to_half(w[q][p][t], h);
          *reinterpret_cast<uint4 *>(st + r0 * 128 + write[t]) =
              make_uint4(f16x2_mul(h[0], g), f16x2_mul(h[1], g), f16x2_mul(h[2], g),
                         f16x2_mul(h[3], g));
        }
      }
  }
};

// One widening warp's work: its share, kF4Share rows from share0 on of every 64-key
// step of K or of V.  Its own copies bring the share's tiles into its part of the
// raw ring, RAW steps ahead; it widens them into the fp16 stage, hands its part
// over (full) and refills the raw place that it has just read.  Steps are counted
// from step_base on.  Of V, rows that must not contribute become zeros (K's are
// masked by the softmax), and NaNs at keys from all_rows on, which not every row
// attends to, are noted in nan_key.  False where a wait ran out; copies in flight
// have then landed or been waited for.
constexpr int kF4Share = 32;
template <int D, int SK, int SV, int RAW, int RAW_STEP, int ATOM>
__device__ __forceinline__ bool f4_widen_share(
    const PrefillArgs &a, const CUtensorMap *map, const int32_t *bt_row, int kvh, int lane,
    bool k_role, int share0, int step_base, int n_steps, int n_keys, int all_rows, uint64_t *full,
    uint64_t *empty, uint64_t *land, uint8_t *ring, uint8_t *raw, int *nan_key, uint64_t policy) {
  const int tsh = a.bs_log2 == 4 ? 1 : 0;  // 1 << tsh tiles of a share
  const uint32_t tile_bytes = fp4_tile_bytes(1 << a.bs_log2, D);
  const int tile_lines = 9 << (a.bs_log2 - 4);
  const F4Widen<D> widen(lane, a.bs_log2, ATOM);
  raw += share0 / 16 * kRawSlot16<D>;
  // block of the warp's tile l (its tiles are numbered over all steps)
  auto tile_block = [&](int l) -> int {
    const int key = (step_base + (l >> tsh)) * kPairKeys + share0 + (tsh ? (l & 1) * 16 : 0);
    if (key >= n_keys) return -1;
    const int phys = bt_row[key >> a.bs_log2];
    if (phys < 0 || static_cast<int64_t>(phys) >= a.num_blocks) {
      atomicOr(a.err, kErrBadBlock);
      return -1;
    }
    return phys;
  };
  int win_base = 0, win = tile_block(lane);
  uint32_t loaded = 0;  // bits 2 rs and up: tiles of the share in raw place rs
  auto fetch = [&](int m) {
    const int rs = m % RAW;
    if ((m << tsh) >= win_base + 32) {
      win_base += 32;
      win = tile_block(win_base + lane);
    }
    const int phys = __shfl_sync(kFullMask, win, (m << tsh) + (tsh & lane) - win_base);
    const uint32_t mask = __ballot_sync(kFullMask, lane < 1 << tsh && phys >= 0);
    loaded = (loaded & ~(3u << (2 * rs))) | (mask << (2 * rs));
    if (lane == 0) {
      if (mask == 0)
        mbar_arrive(&land[rs]);
      else
        mbar_arrive_expect_tx(&land[rs], __popc(mask) * tile_bytes);
    }
    __syncwarp();
    if (lane < 1 << tsh && phys >= 0)
      tma_load_2d(raw + rs * RAW_STEP + lane * kRawSlot16<D>, map, 0,
                  (phys * a.num_kv_heads + kvh) * tile_lines, &land[rs], policy);
  };
  for (int m = 0; m < min(RAW, n_steps); ++m) fetch(m);
  bool ok_run = true;
  int m = 0;
  for (; m < n_steps; ++m) {
    const int rs = m % RAW;
    const int S = k_role ? SK : SV, s = m % S;
    if (!__all_sync(kFullMask, mbar_wait_bounded(&land[rs], (m / RAW) & 1) &&
                                   (m < S || mbar_wait_bounded(&empty[s], ((m / S) - 1) & 1)))) {
      ok_run = false;
      break;
    }
    const uint32_t ok = (loaded >> (2 * rs)) & 3u;
    const int key0 = (step_base + m) * kPairKeys;
    const int past = n_keys - key0 - share0;  // the share's first row past the keys
    uint8_t *st = ring + s * (D / 64) * ATOM + share0 * 128;
    const uint8_t *from = raw + rs * RAW_STEP;
    if (k_role || (ok == (1u << (1 << tsh)) - 1 && key0 + kPairKeys <= all_rows))
      widen(from, st, [](int, uint32_t sc) { return sc; });
    else
      widen(from, st, [&](int r, uint32_t sc) {
        return r < past && ((ok >> (r >> a.bs_log2)) & 1u)
                   ? F4Widen<D>::drop_nans(sc, lane, key0 + share0 + r, nan_key)
                   : 0u;
      });
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[s]);
    if (m + RAW < n_steps) fetch(m + RAW);
  }
  // after a wait that ran out, copies already in flight land before the CTA
  // leaves (bounded again)
  for (int k = m; !ok_run && k < min(m + RAW, n_steps); ++k)
    (void)mbar_wait_bounded(&land[k % RAW], (k / RAW) & 1);
  return ok_run;
}

// 32 output values of a row, from dimension 32 cb on: NaN where the row attends
// to a key whose V has a NaN scale there (what drop_nans noted; pos: the row's
// last key).
__device__ __forceinline__ void put_nans(float (&o)[32], const int *nan, int cb, int pos) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (nan[2 * cb + i] <= pos) {
#pragma unroll
      for (int e = 0; e < 16; ++e) o[16 * i + e] = __int_as_float(0x7fffffff);
    }
}

}  // namespace pa
