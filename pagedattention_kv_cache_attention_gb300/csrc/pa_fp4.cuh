// pa_fp4.cuh -- the FP4 KV cache's number format and tile layout.
//
// A cached element is an E2M1 code (1 sign, 2 exponent bits with bias 1, 1
// fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives); 16
// consecutive elements of a head_dim row share one E4M3 scale, and a cache has
// one fp32 scale g: code c under scale s stands for g * s * e2m1(c).
//
// The tile of one (physical block, KV head) is block_size * head_dim * 9 / 16
// consecutive bytes: the codes of its tokens row by row (head_dim / 2 bytes a
// token, the even element of a byte in its low nibble), then their scales row
// by row (head_dim / 16 bytes a token).  Codes and scales of a tile are so
// fetched in one copy.
//
// e2m1 * E4M3 has at most 2 + 4 significant bits and is 0 or lies between
// 2^-10 and 2688 in magnitude, so s * e2m1(c) is exact in fp16: the attention
// kernels form it there (one fp16x2 product for two elements) and fold g into
// the softmax scale or the output.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

constexpr uint32_t kFp4NanScale = 0x7f;  // E4M3 NaN: the scale of a group with a NaN in it

// Bytes of one (block, KV head) tile, and of its codes.
__host__ __device__ constexpr int fp4_tile_bytes(int bs, int d) { return bs * d * 9 / 16; }
__host__ __device__ constexpr int fp4_code_bytes(int bs, int d) { return bs * d / 2; }

// Eight E2M1 codes (element 0 in the lowest nibble) to four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight fp32 values to E2M1 codes (nearest, ties to the even code, magnitudes
// beyond 6 to 6), value 0 in the lowest nibble.
__device__ __forceinline__ uint32_t float8_to_e2m1x8(const float (&y)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

// Product of two fp16 pairs.
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  const __half2 p = __hmul2(*reinterpret_cast<const __half2 *>(&a),
                            *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&p);
}

// E4M3 code (low byte of b) to fp32, exact.
__device__ __forceinline__ float e4m3_to_float(uint32_t b) {
  const uint32_t h = e4m3x2_lo_to_f16x2(b & 0xffu);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

// Logits of any size.  A probability is 2^((x - xr) sl + shift): x a score, xr
// the row's reference (a score, too), sl > 0 the softmax scale in base 2.  As one
// fma of x, with shift - xr sl rounded to c, its exponent is off by what c lost,
// the same for all of the row: up to half a unit of xr sl in its last place, 2^-16
// at 2^8, but more than fp16's range from 2^27 on.  From kFp4FarLogit on xr is
// therefore taken off x first (exact, or off by 2^-24 of the difference).
constexpr float kFp4FarLogit = 256.f;

// The softmax scale of a row as a normal number: small cache scales times small
// powers of two of a bf16 row may fall below, and 0 x -inf would be NaN.  (What
// the row's logits then lose is below 2^-90: scores are below 2^35.)  Of a
// negative scale, the magnitude.
__device__ __forceinline__ float fp4_normal_scale(float sl) {
  return fminf(fmaxf(fabsf(sl), 0x1p-126f), 0x1.fffffep127f);
}

// Sums held relative to the score xr, and times 2^shift, are to be joined with
// others by logits: returns the float next to xr sl, and in `to` what makes them
// relative to it.  (Bounded: where the rounding of xr sl is larger than 16, logits
// of other parts cannot be told apart any more finely, and sums and their
// reciprocals times a cache scale of 2^100 stay within fp32.)
__device__ __forceinline__ float fp4_reference(float xr, float sl, float shift, float &to) {
  const float m = fminf(fmaxf(xr * sl, -0x1.fffffep127f), 0x1.fffffep127f);
  to = exp2f(fminf(fmaxf(fmaf(xr, sl, -m), -16.f), 16.f) - shift);
  return m;
}

// fp32 to the nearest E4M3 code (ties to even, at most 448; NaN stays NaN).
__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
  return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// The most sequences that are put in order: a lane holds eight lengths in registers.
// What the order gives falls with their number, as the last CTAs are a smaller part
// of the call: of 5-token chunks 17 % at 64 sequences, 4 % at 256.
constexpr int kMaxByLength = 256;
constexpr int kMinByLength = 1024;  // tokens of the longest context

// The sequence of place z when n <= kMaxByLength sequences are put in order of
// their context lengths, longest first, in 16 to 32 classes of equal width (in a
// class by index).  For a whole warp.  A grid of more CTAs than run at once ends
// with its last CTAs: with the short contexts there it ends earlier.  Where no
// context reaches kMinByLength the places stay as they are.  (Functions of their
// own: inlined, their registers cost the kernels up to 10 %.)
template <int kWords>  // a lane holds the lengths of kWords sequences
static __device__ __noinline__ int place_by_length(const int32_t *lens, int n, int z, int lane) {
  int c[kWords], top = 0;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    c[i] = i * 32 + lane < n ? max(lens[i * 32 + lane], 0) : -1;
    top = max(top, c[i]);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (top < kMinByLength) return z;
  const int shift = 27 - __clz(top);  // top >> shift is at most 31
#pragma unroll
  for (int i = 0; i < kWords; ++i) c[i] >>= shift;  // (-1 stays)
  int cls = 0, rem = z;  // the class, a bit at a time; the place among what is left
#pragma unroll
  for (int bit = 4; bit >= 0; --bit) {
    const int want = (cls >> bit) | 1;
    int count = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      count += __popc(__ballot_sync(0xffffffffu, c[i] >> bit == want));
    if (rem < count)
      cls |= 1 << bit;
    else
      rem -= count;
  }
  uint32_t in = 0;  // the word of the class that holds place rem
  int word = 0, first = 0;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const uint32_t these = __ballot_sync(0xffffffffu, c[i] == cls);
    if (first <= rem) {
      in = these;
      word = i;
      z = rem - first;  // among the word's
    }
    first += __popc(these);
  }
  const bool here = ((in >> lane) & 1u) && __popc(in & ((1u << lane) - 1)) == z;
  return word * 32 + __ffs(__ballot_sync(0xffffffffu, here)) - 1;
}
__device__ __forceinline__ int seq_by_length(const int32_t *lens, int n, int z, int lane) {
  return n <= 64 ? place_by_length<2>(lens, n, z, lane)
                 : place_by_length<kMaxByLength / 32>(lens, n, z, lane);
}

}  // namespace pa
