// pa_join.cuh -- the log-sum-exp join of split-context partitions inside a
// decode kernel: counting the partitions of a (sequence, KV head) in, and the
// join by the CTA that completes the count.
#pragma once

#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Atomic add with acquire-release semantics at GPU scope; returns the old value.
__device__ __forceinline__ unsigned atom_add_acq_rel_gpu(unsigned *p, unsigned v) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v)
               : "memory");
  return old;
}

// Each partition CTA adds kJoinArrive to its (sequence, KV head) counter: after
// k arrivals both 16-bit halves hold k, so a counter that did not start at zero
// (a workspace whose counter words were not cleared) is recognised.
constexpr unsigned kJoinArrive = 0x00010001u;

// Log-sum-exp join of the np partitions of one (sequence, KV head), run by the
// CTA that finished last: out = sum_p w_p o_p / sum_p w_p, w_p = l_p 2^(m_p - M),
// M = max_p m_p, for the G query heads of the KV head.  Thread items are
// 4-element chunks of one head's output; partitions are taken 8 at a time with
// a running maximum, so every group costs one round trip to L2.  The partials
// were written by other CTAs of this grid: they are read through L2 (ld.cg).
template <typename T, int D, int NW>
__device__ __forceinline__ void join_partitions(const DecodeArgs &a, int seq, int kvh, int np) {
  constexpr int kQuads = D / 4;
  constexpr int kGroup = 8;
  const int G = a.group;
  for (int item = threadIdx.x; item < G * kQuads; item += NW * 32) {
    const int h = item / kQuads, c4 = item % kQuads;
    const int64_t row = static_cast<int64_t>(seq) * a.num_q_heads + kvh * G + h;
    const float *mrow = a.ws_m + row * a.num_parts;
    const float *lrow = a.ws_l + row * a.num_parts;
    const float *orow = a.ws_o + row * a.num_parts * D + c4 * 4;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < np; p0 += kGroup) {
      float mp[kGroup], lp[kGroup];
      float4 op[kGroup];
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        if (p0 + u < np) {
          mp[u] = __ldcg(mrow + p0 + u);
          lp[u] = __ldcg(lrow + p0 + u);
          op[u] = __ldcg(reinterpret_cast<const float4 *>(orow + static_cast<int64_t>(p0 + u) * D));
        } else {
          mp[u] = -INFINITY;
          lp[u] = 0.f;
          op[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      float Mn = M;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) Mn = fmaxf(Mn, mp[u]);
      const float ref = Mn == -INFINITY ? 0.f : Mn;  // no token yet: any finite reference
      const float al = exp2f(M - ref);
      L *= al;
      acc.x *= al;
      acc.y *= al;
      acc.z *= al;
      acc.w *= al;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const float wgt = lp[u] * exp2f(mp[u] - ref);
        L += wgt;
        acc.x += wgt * op[u].x;
        acc.y += wgt * op[u].y;
        acc.z += wgt * op[u].z;
        acc.w += wgt * op[u].w;
      }
      M = Mn;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const uint2 pk = make_uint2(Elem<T>::pack(acc.x * inv, acc.y * inv),
                                Elem<T>::pack(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * D + c4 * 4) = pk;
  }
}

// Count this CTA's partition of (sequence, KV head) in; true for the whole CTA
// if it is the last of `arrivals`, so that every partial is visible to it.
// The first barrier orders every thread's partial stores before thread 0's
// acquire-release add, which publishes them (release, cumulative) and, for the
// last CTA, makes every other CTA's partials visible (acquire).
__device__ __forceinline__ bool last_to_arrive(const DecodeArgs &a, int seq, int kvh,
                                               int arrivals_wanted, uint32_t *last_flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned *cnt = a.ws_cnt + static_cast<int64_t>(seq) * a.num_kv_heads + kvh;
    const unsigned prev = atom_add_acq_rel_gpu(cnt, kJoinArrive);
    const unsigned k = prev & 0xffffu;
    const unsigned arrivals = static_cast<unsigned>(arrivals_wanted);  // CTAs that count in
    uint32_t last = 0;
    if ((prev >> 16) != k || k >= arrivals) {
      atomicOr(a.err, kErrWorkspace);  // the counter did not start at zero
    } else if (k == arrivals - 1) {
      last = 1;
      atomicExch(cnt, 0u);  // every partition has arrived: ready for the next call
    }
    *last_flag = last;
  }
  __syncthreads();
  return *last_flag != 0;
}

}  // namespace pa
