// mala_decode_mass.cuh -- the second kernel of a decode that also collects
// each key's attention weight.
//
// The first kernel (mala_decode.cuh with kScores behind a gate, else
// mala_decode_flat.cuh) has written every live key's scores and partial results
// (O_s, LSE_s). What is left is, per (b, query head),
//   LSE = log sum_s exp(LSE_s),   O = sum_s exp(LSE_s - LSE) O_s,
// and per (b, KV head, key j), over the group's query heads h,
//   mass_j = decay * mass_j' + sum_h exp(s_hj - LSE_h),
// the newest key (the query's own) starting from 0. MALA scores every tile,
// kept or skipped, so the weights cost no second pass over K: G scores (4 G
// bytes) are written and read per key and KV head, against 4 d bytes of K and V.
//
// One launch does both: the first blocks merge the partials, a warp per (b,
// query head); the others take 1024 keys of one (b, KV head) each and form the
// LSEs of its G heads from the partials again (a few dozen values a head, from
// L2), so they wait for nothing but the first kernel.
#pragma once

#include "mala_decode_flat.cuh"

namespace mala {

struct DecMassParams {
  const float* o_part;    // [B, Hq, slots, d]
  const float* lse_part;  // [B, Hq, slots]
  uint16_t* o;            // [B, Hq, d]
  float* lse;             // [B, Hq]
  const float* scores;    // [B, Hkv, G, max_len], log2 units
  const int32_t* seqlens;
  const float* mass_in;   // [B, Hkv, ld], nullable
  float* mass_out;
  const int* plan;        // mala_decode_flat_kernel's (null: every unit has `slots` partials)
  int32_t* kept_tiles;    // with a plan: written here (every tile is kept)
  uint8_t* keep_map;
  int B, Hq, Hkv, G, slots, ld, max_len, max_pages, page;
  int merge_blocks, key_blocks;  // blocks of the merge; blocks per (b, KV head)
  float decay;
};

constexpr int kDecMassThreads = 256;
constexpr int kDecMassKeys = 1024;  // keys per block, four consecutive ones to a thread

// length of sequence b (0: idle, or invalid and reported by the first kernel)
__device__ __forceinline__ int mass_len(const DecMassParams& p, int b) {
  const int L = __ldg(p.seqlens + b);
  return L < 0 || L > p.max_len ? 0 : L;
}

// partial results of (b, KV head)
__device__ __forceinline__ int mass_parts(const DecMassParams& p, int b, int hkv, int len) {
  if (p.plan == nullptr) return p.slots;
  const int nt = (len + kFlatTile - 1) / kFlatTile, run = p.plan[p.B];
  if (nt == 0) return 0;
  const int at = p.plan[b] + hkv * nt;
  return (at + nt - 1) / run - at / run + 1;
}

// log sum exp of n values, by a warp (every lane returns it); the lane's own first value in x0
__device__ __forceinline__ float merged_lse(const float* lp, int n, int lane, float& x0) {
  x0 = lane < n ? lp[lane] : -INFINITY;
  float mx = x0;
  for (int s = lane + 32; s < n; s += 32) mx = fmaxf(mx, lp[s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (mx == -INFINITY) return -INFINITY;
  float z = __expf(x0 - mx);
  for (int s = lane + 32; s < n; s += 32) z += __expf(lp[s] - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return mx + __logf(z);
}

// GP: the group's heads rounded up to 1, 2, 4 or 8 (scores a thread holds at once).
template <int D, int GP>
__global__ void __launch_bounds__(kDecMassThreads) mala_decode_mass_kernel(const DecMassParams p) {
  cudaGridDependencySynchronize();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < p.merge_blocks) {
    const int row = blockIdx.x * (kDecMassThreads / 32) + warp;
    if (row >= p.B * p.Hq) return;
    const int b = row / p.Hq, len = mass_len(p, b);
    const int n = mass_parts(p, b, row % p.Hq / p.G, len);
    const float* lp = p.lse_part + static_cast<size_t>(row) * p.slots;
    float x0;
    const float L = merged_lse(lp, n, lane, x0);
    // the partials' weights a lane each, 32 partials at a time
    constexpr int PER = D / 32;
    float out[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) out[e] = 0.f;
    const float* src = p.o_part + static_cast<size_t>(row) * p.slots * D + lane * PER;
    for (int s0 = 0; s0 < n; s0 += 32) {
      const float x = s0 == 0 ? x0 : s0 + lane < n ? lp[s0 + lane] : -INFINITY;
      const float wl = x == -INFINITY ? 0.f : __expf(x - L);
      const int cnt = min(32, n - s0);
#pragma unroll 8
      for (int s = 0; s < cnt; ++s) {
        const float w = __shfl_sync(0xffffffffu, wl, s);
        float v[PER];
        if constexpr (PER == 4) {
          const float4 t = *reinterpret_cast<const float4*>(src + static_cast<size_t>(s0 + s) * D);
          v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
        } else {
          const float2 t = *reinterpret_cast<const float2*>(src + static_cast<size_t>(s0 + s) * D);
          v[0] = t.x; v[1] = t.y;
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) out[e] = fmaf(w, v[e], out[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < PER; e += 2)
      *reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(row) * D + lane * PER + e) =
          pack_bf16x2(out[e], out[e + 1]);
    if (lane == 0) p.lse[row] = L;
    if (p.plan != nullptr) {
      const int pages = (len + p.page - 1) / p.page;
      if (lane == 0) p.kept_tiles[row] = pages;
      if (p.keep_map != nullptr)
        for (int i = lane; i < pages; i += 32) p.keep_map[static_cast<size_t>(row) * p.max_pages + i] = 1;
    }
    return;
  }

  const int blk = blockIdx.x - p.merge_blocks;
  const int bk = blk / p.key_blocks;
  const int b = bk / p.Hkv, hkv = bk % p.Hkv;
  const int L = mass_len(p, b);
  const int j0 = (blk % p.key_blocks) * kDecMassKeys;
  __shared__ float lse2[8];
  const int j = j0 + 4 * static_cast<int>(threadIdx.x);
  // the keys' scores and earlier masses, on their way while the LSEs are formed
  float4 x[GP];
  const float* sc = p.scores + static_cast<size_t>(bk) * p.G * p.max_len + j;
#pragma unroll
  for (int g = 0; g < GP; ++g)
    x[g] = j < L && g < p.G ? *reinterpret_cast<const float4*>(sc + static_cast<size_t>(g) * p.max_len)
                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  const size_t at = static_cast<size_t>(bk) * p.ld + j;
  const bool old = p.mass_in != nullptr && p.decay != 0.f && j < L - 1;
  const bool words = (p.ld & 3) == 0;  // whole 16-byte words
  float before[4] = {0.f, 0.f, 0.f, 0.f};
  if (old && words) {
    const float4 v = *reinterpret_cast<const float4*>(p.mass_in + at);
    before[0] = v.x; before[1] = v.y; before[2] = v.z; before[3] = v.w;
  } else if (old) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < L - 1) before[e] = p.mass_in[at + e];
  }
  if (j0 < L && warp < p.G) {
    float x0;
    const float l = merged_lse(p.lse_part + (static_cast<size_t>(b) * p.Hq + hkv * p.G + warp) * p.slots,
                               mass_parts(p, b, hkv, L), lane, x0);
    if (lane == 0) lse2[warp] = l * 1.4426950408889634f;
  }
  __syncthreads();
  if (j >= p.ld) return;
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    const float l2 = j < L && g < p.G ? lse2[g] : 0.f;  // what is not there adds exp2(-inf) = 0
    m[0] += ex2_approx(x[g].x - l2);
    m[1] += ex2_approx(x[g].y - l2);
    m[2] += ex2_approx(x[g].z - l2);
    m[3] += ex2_approx(x[g].w - l2);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (j + e >= L) m[e] = 0.f;  // past the sequence's keys
    if (old && j + e < L - 1) m[e] = fmaf(p.decay, before[e], m[e]);
  }
  if (words) {
    *reinterpret_cast<float4*>(p.mass_out + at) = make_float4(m[0], m[1], m[2], m[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < p.ld) p.mass_out[at + e] = m[e];
  }
}

}  // namespace mala
