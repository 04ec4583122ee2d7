// mala_decode_mass.cuh -- the second kernel of a decode that also collects
// each key's attention weight.
//
// The split kernel (mala_decode.cuh, kScores) has written every live key's
// scores and the splits' (O_s, LSE_s). What is left is, per (b, query head),
//   LSE = log sum_s exp(LSE_s),   O = sum_s exp(LSE_s - LSE) O_s,
// and per (b, KV head, key j), over the group's query heads h,
//   mass_j = decay * mass_j' + sum_h exp(s_hj - LSE_h),
// the newest key (the query's own) starting from 0. MALA scores every tile,
// kept or skipped, so the weights cost no second pass over K: G scores (4 G
// bytes) are written and read per key and KV head, against 4 d bytes of K and V.
//
// One launch does both: the first blocks merge the splits, a warp per (b,
// query head); the others take 1024 keys of one (b, KV head) each and form the
// LSEs of its G heads from the partials again (G x n_splits values, from L2),
// so they wait for nothing.
#pragma once

#include "mala_ptx.cuh"

namespace mala {

struct DecMassParams {
  const float* o_part;    // [B, Hq, S, d]
  const float* lse_part;  // [B, Hq, S]
  uint16_t* o;            // [B, Hq, d]
  float* lse;             // [B, Hq]
  const float* scores;    // [B, Hkv, ld_scores, G], log2 units
  const int32_t* seqlens;
  const float* mass_in;   // [B, Hkv, ld], nullable
  float* mass_out;
  int B, Hq, Hkv, G, n_splits, ld, ld_scores, max_len;
  int merge_blocks, key_blocks;  // blocks of the merge; blocks per (b, KV head)
  float decay;
};

constexpr int kDecMassThreads = 256;
constexpr int kDecMassKeys = 1024;  // keys per block

// log sum exp over the splits of one row, by a warp (every lane returns it)
__device__ __forceinline__ float merged_lse(const float* lp, int n_splits, int lane) {
  float mx = -INFINITY;
  for (int s = lane; s < n_splits; s += 32) mx = fmaxf(mx, __ldg(lp + s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float z = 0.f;
  for (int s = lane; s < n_splits; s += 32) {
    const float x = __ldg(lp + s);
    z += x == -INFINITY ? 0.f : __expf(x - mx);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return mx == -INFINITY ? -INFINITY : mx + __logf(z);
}

template <int D>
__global__ void __launch_bounds__(kDecMassThreads) mala_decode_mass_kernel(const DecMassParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < p.merge_blocks) {
    const int row = blockIdx.x * (kDecMassThreads / 32) + warp;
    if (row >= p.B * p.Hq) return;
    const float* lp = p.lse_part + static_cast<size_t>(row) * p.n_splits;
    const float L = merged_lse(lp, p.n_splits, lane);
    constexpr int PER = D / 32;
    float out[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) out[e] = 0.f;
    for (int s = 0; s < p.n_splits; ++s) {
      const float ls = __ldg(lp + s);
      if (ls == -INFINITY) continue;
      const float w = __expf(ls - L);
      const float* src = p.o_part + (static_cast<size_t>(row) * p.n_splits + s) * D + lane * PER;
#pragma unroll
      for (int e = 0; e < PER; ++e) out[e] = fmaf(w, src[e], out[e]);
    }
#pragma unroll
    for (int e = 0; e < PER; e += 2)
      *reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(row) * D + lane * PER + e) =
          pack_bf16x2(out[e], out[e + 1]);
    if (lane == 0) p.lse[row] = L;
    return;
  }

  const int blk = blockIdx.x - p.merge_blocks;
  const int bk = blk / p.key_blocks, j0 = (blk % p.key_blocks) * kDecMassKeys;
  const int b = bk / p.Hkv, hkv = bk % p.Hkv;
  int L = __ldg(p.seqlens + b);
  if (L < 0 || L > p.max_len) L = 0;  // reported by the split kernel; the sequence has no weights
  const float* min = p.mass_in ? p.mass_in + static_cast<size_t>(bk) * p.ld : nullptr;
  float* mout = p.mass_out + static_cast<size_t>(bk) * p.ld;
  const int j1 = ::min(j0 + kDecMassKeys, p.ld);
  __shared__ float lse2[8];
  if (j0 < L && warp < p.G) {
    const float x = merged_lse(p.lse_part + (static_cast<size_t>(b) * p.Hq + hkv * p.G + warp) * p.n_splits,
                               p.n_splits, lane);
    if (lane == 0) lse2[warp] = x * 1.4426950408889634f;
  }
  __syncthreads();
  const float* sc = p.scores + static_cast<size_t>(bk) * p.ld_scores * p.G;
  for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += kDecMassThreads) {
    float m = 0.f;
    if (j < L) {
      const float* s = sc + static_cast<size_t>(j) * p.G;
      if (p.G == 4) {  // one 16-byte load
        const float4 x = *reinterpret_cast<const float4*>(s);
        m = (ex2_approx(x.x - lse2[0]) + ex2_approx(x.y - lse2[1])) +
            (ex2_approx(x.z - lse2[2]) + ex2_approx(x.w - lse2[3]));
      } else {
        for (int g = 0; g < p.G; ++g) m += ex2_approx(s[g] - lse2[g]);
      }
      if (min != nullptr && p.decay != 0.f && j < L - 1) m = fmaf(p.decay, min[j], m);
    }
    mout[j] = m;  // past the sequence's keys: 0
  }
}

}  // namespace mala
