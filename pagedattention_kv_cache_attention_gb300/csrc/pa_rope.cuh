// pa_rope.cuh -- the rotation of queries and keys by their positions, on the
// way into the cache (pa_rope_and_cache and its FP8 and FP4 forms).
//
// Of the first r = rotary_dim elements of a head, pairs (x, y) become
//   x' = x cos - y sin,   y' = y cos + x sin,
// cosines and sines read from the caller's table (fp32, one row a position:
// r / 2 cosines, then r / 2 sines), x and y being elements i and i + r / 2, or
// 2 i and 2 i + 1.  Products and sums are IEEE fp32 operations of their own,
// not an fma: the result, rounded to the row's type, is then the same wherever
// it is computed, and with it the codes of an FP8 or FP4 cache.
//
// A thread's item is two 8-element chunks of one head that hold whole pairs:
// chunks u and u + r / 16 (or 2 u and 2 u + 1), so that 16-byte loads and
// stores do for both orders, and a thread's cosines and sines, pairs 8 u ..
// 8 u + 7, are the same for all the heads that it takes of its token.
#pragma once

#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

constexpr unsigned kErrBadPos = 64u;  // of the device error word (mirrors include/pa.h)

// x cos - y sin and y cos + x sin of the pair (x, y).
__device__ __forceinline__ void rope_pair(float x, float y, float c, float s, float &xr, float &yr) {
  xr = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  yr = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// A token's slot and position: false if it is to be left out (no slot, or one
// of the two outside its range, which `tell` says to flag).
__device__ __forceinline__ bool rope_token(const RopeArgs &a, int64_t slot, int64_t pos, bool tell) {
  if (slot < 0) return false;
  const bool bad_slot = slot >= (a.num_blocks << a.bs_log2);
  const bool bad_pos = pos < 0 || pos >= a.max_position;
  if ((bad_slot || bad_pos) && tell)
    atomicOr(a.err, (bad_slot ? kErrBadSlot : 0u) | (bad_pos ? kErrBadPos : 0u));
  return !bad_slot && !bad_pos;
}

// The two chunks of item u of a head, and its cosines and sines: c[i], s[i]
// belong to pair 8 u + i.  Items from r / 16 on are copied.
template <int D> struct RopeItem {
  int a, b;  // chunks
  bool turn;
  float c[8], s[8];
  __device__ __forceinline__ RopeItem(int u, int rotary, int interleaved) {
    const int turned = rotary / 16;
    turn = u < turned;
    a = interleaved || !turn ? 2 * u : u;
    b = interleaved || !turn ? 2 * u + 1 : u + turned;
  }
  __device__ __forceinline__ void load(const float *row, int u, int rotary) {
    if (!turn) return;
    const float4 *cos = reinterpret_cast<const float4 *>(row + 8 * u);
    const float4 *sin = reinterpret_cast<const float4 *>(row + rotary / 2 + 8 * u);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = cos[i], y = sin[i];
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
  }
  // Rotates the 16 elements of both chunks in place.
  template <typename T>
  __device__ __forceinline__ void apply(uint4 &va, uint4 &vb, int interleaved) const {
    if (!turn) return;
    uint32_t wa[4], wb[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 x = Elem<T>::unpack(word_of(va, w)), y = Elem<T>::unpack(word_of(vb, w));
      float p0, p1, q0, q1;
      if (interleaved) {  // pairs within a word: 8 u + w of chunk a, 8 u + 4 + w of chunk b
        rope_pair(x.x, x.y, c[w], s[w], p0, p1);
        rope_pair(y.x, y.y, c[4 + w], s[4 + w], q0, q1);
      } else {
        rope_pair(x.x, y.x, c[2 * w], s[2 * w], p0, q0);
        rope_pair(x.y, y.y, c[2 * w + 1], s[2 * w + 1], p1, q1);
      }
      wa[w] = Elem<T>::pack(p0, p1);
      wb[w] = Elem<T>::pack(q0, q1);
    }
    va = make_uint4(wa[0], wa[1], wa[2], wa[3]);
    vb = make_uint4(wb[0], wb[1], wb[2], wb[3]);
  }
};

// 8 consecutive 16-bit elements -> 8 E4M3 codes of x / scale (IEEE division,
// nearest even, magnitudes beyond 448 clamped).
template <typename T> __device__ __forceinline__ uint2 quantise8_e4m3(const uint4 &x, float scale) {
  uint32_t q[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 v = Elem<T>::unpack(word_of(x, w));
    q[w] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v.x, scale), __fdiv_rn(v.y, scale)),
                                    __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// The first `heads` of a token's query, key and value heads (in that order),
// by 1 << a.group_log2 threads, of which this is number `me`.
template <typename T, int D, bool F8>
__device__ __forceinline__ void rope_token_heads(const RopeArgs &a, int64_t token, int me,
                                                 int heads) {
  constexpr int kItems = D / 16, kBatch = 3;
  const int64_t slot = a.slot_mapping[token], pos = a.positions[token];
  const int u = me % kItems, step = (1 << a.group_log2) / kItems;
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  RopeItem<D> item(u, a.rotary_dim, a.interleaved);
  const T *query = static_cast<const T *>(a.query) + token * a.query_stride;
  const T *key = static_cast<const T *>(a.key) + token * a.key_stride;
  const T *value = static_cast<const T *>(a.value) + token * a.value_stride;
  bool first = true;
  int64_t cell = 0;  // head 0 of the token's slot, in rows of the cache
  for (int h0 = me / kItems; h0 < heads; h0 += step * kBatch) {
    uint4 va[kBatch], vb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step;
      const T *row = h < hq ? query + h * D
                            : h < hq + hkv ? key + (h - hq) * D : value + (h - hq - hkv) * D;
      va[i] = vb[i] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        va[i] = *reinterpret_cast<const uint4 *>(row + item.a * 8);
        vb[i] = *reinterpret_cast<const uint4 *>(row + item.b * 8);
      }
    }
    if (first) {  // (after the rows' loads: slot and position are two more of a chain)
      if (!rope_token(a, slot, pos, me == 0)) return;
      item.load(a.cos_sin + pos * a.rotary_dim, u, a.rotary_dim);
      const int64_t blk = slot >> a.bs_log2;
      cell = ((blk * hkv) << a.bs_log2) + (slot & ((1 << a.bs_log2) - 1));
      first = false;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step;
      if (h >= heads) break;
      const bool is_value = h >= hq + hkv;
      if (!is_value) item.template apply<T>(va[i], vb[i], a.interleaved);
      if (h < hq) {
        T *out = static_cast<T *>(a.query_out) + token * a.query_out_stride + h * D;
        *reinterpret_cast<uint4 *>(out + item.a * 8) = va[i];
        *reinterpret_cast<uint4 *>(out + item.b * 8) = vb[i];
        continue;
      }
      const int64_t row = cell + (static_cast<int64_t>(h - hq - (is_value ? hkv : 0)) << a.bs_log2);
      if constexpr (F8) {
        const float g = is_value ? a.v_scale : a.k_scale;
        uint8_t *dst = static_cast<uint8_t *>(is_value ? a.v_cache : a.k_cache) + row * D;
        *reinterpret_cast<uint2 *>(dst + item.a * 8) = quantise8_e4m3<T>(va[i], g);
        *reinterpret_cast<uint2 *>(dst + item.b * 8) = quantise8_e4m3<T>(vb[i], g);
      } else {
        T *dst = static_cast<T *>(is_value ? a.v_cache : a.k_cache) + row * D;
        *reinterpret_cast<uint4 *>(dst + item.a * 8) = va[i];
        *reinterpret_cast<uint4 *>(dst + item.b * 8) = vb[i];
      }
    }
  }
}

}  // namespace pa
