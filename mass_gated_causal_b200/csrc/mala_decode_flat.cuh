// mala_decode_flat.cuh -- ungated (tau = 0) paged decode that keeps its scores, for
// mala_decode_paged_mass.
//
// Without a gate no tile waits for a decision, so the schedule is free: the key
// tiles of all (sequence, KV head) units are laid end to end and cut into equal
// runs, one per CTA, two CTAs to an SM, whatever the sequences' lengths. (Splitting
// every sequence into the same number of ranges left SMs idle behind the longest:
// 8 sequences of 64K to 128K keys took 797 us.) A run that ends inside a unit
// leaves a partial (O, LSE); the second kernel merges a unit's partials, whose
// number follows from the lengths.
//
//   warps 0-3  compute: warp w owns keys 16 w .. 16 w + 15 of every 64-key tile,
//              with an online softmax of its own; nothing is exchanged between
//              warps until the unit ends
//   warp  4    producer: K and V tiles by TMA through one ring, across units
//
// The products are small (at most eight query rows) and the kernel is bound by
// HBM, so they run on warp-level MMAs (m16n8k16), whose operands come straight
// from the swizzled tiles by ldmatrix: S (heads x keys) = Q K^T with the group's
// heads as rows 0-7, O (heads x d) += P V with P in two bf16 parts, p = hi + lo,
// as rows 0-7 and 8-15 of one operand, so that P loses nothing at bf16 size (hi and
// lo hold 16 bits) and the second half of the rows is not wasted. On the FMA pipes
// the same products took 3,500 cycles a tile pair, more than HBM needs.
#pragma once

#include "mala_ptx.cuh"

namespace mala {

struct FlatParams {
  int B, Hq, Hkv, G;
  const int* seqlens;
  const int* block_table;
  int max_pages, num_pages, page_shift, max_len;
  const uint16_t* q;  // [B, Hq, d]
  float scale_log2;
  float* o_part;      // [B, Hq, slots, d]
  float* lse_part;    // [B, Hq, slots] natural log
  float* scores;      // [B, Hkv, G, max_len] log2 units
  int* plan;          // [B + 1]: first tile of each sequence (times Hkv heads), then the run length
  int slots;
  unsigned* status;
  uint64_t wait_ns;
  int stall_tile;
};

constexpr int kFlatTile = 64;      // keys per tile
constexpr int kFlatLeastRun = 2;   // tiles: a run is not cut shorter
constexpr int kFlatThreads = 160;

template <int D>
struct FlatLayout {
  static constexpr int T_BYTES = kFlatTile * D * 2;  // a K or V tile
  static constexpr int NS = D == 128 ? 3 : 6;        // ring stages (K and V)
  static constexpr int OFF_RED = 2 * NS * T_BYTES;   // fp32 [2][8][D]: the warps' partials
  static constexpr int OFF_ML = OFF_RED + 2 * 8 * D * 4;  // m, l: [4 warps][8 heads] each
  static constexpr int OFF_BAR = OFF_ML + 2 * 4 * 8 * 4;
  static constexpr int OFF_MISC = OFF_BAR + 3 * NS * 8;  // k_full, v_full, empty
  static constexpr int BYTES = OFF_MISC + 48;
  static constexpr int ALLOC_BYTES = BYTES + 1024;
  static_assert(ALLOC_BYTES <= 113 * 1024, "two CTAs to an SM");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Key tiles of sequence b (0 for an idle slot or an invalid length).
__device__ __forceinline__ int flat_tiles(const FlatParams& p, int b) {
  const int len = __ldg(p.seqlens + b);
  return len < 0 || len > p.max_len ? 0 : (len + kFlatTile - 1) / kFlatTile;
}

template <int D>
__global__ void __launch_bounds__(kFlatThreads, 2)
    mala_decode_flat_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const FlatParams p) {
  using Lay = FlatLayout<D>;
  constexpr int NS = Lay::NS, TB = Lay::T_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;  // stage s: K at 2 s TB, V at (2 s + 1) TB
  float* sRed = reinterpret_cast<float*>(smem + Lay::OFF_RED);
  float* sM = reinterpret_cast<float*>(smem + Lay::OFF_ML);
  float* sL = sM + 32;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* v_full = k_full + NS;
  uint64_t* empty = v_full + NS;
  int* misc = reinterpret_cast<int*>(smem + Lay::OFF_MISC);
  int* abort_flag = misc;  // then: first sequence, its first tile, the run's length, tiles in all
  int* gave_up = misc + 8;  // [4] per compute warp, of the unit at hand

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    // tiles in all, the run length, and the sequence in which this CTA's run begins
    long long all = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int n = b0 + lane < p.B ? flat_tiles(p, b0 + lane) : 0;
      all += __reduce_add_sync(0xffffffffu, n);
    }
    all *= p.Hkv;  // below 2^31 (checked on the host for the longest lengths)
    const int run = max(static_cast<int>((all + gridDim.x - 1) / gridDim.x), kFlatLeastRun);
    const long long pos = static_cast<long long>(blockIdx.x) * run;
    long long at = 0;
    int first = p.B, first_at = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int n = b0 + lane < p.B ? flat_tiles(p, b0 + lane) * p.Hkv : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const long long lo = at + incl - n;
      if (blockIdx.x == 0 && b0 + lane < p.B) {
        p.plan[b0 + lane] = static_cast<int>(lo);
        const int len = __ldg(p.seqlens + b0 + lane);
        if (len < 0 || len > p.max_len) atomicOr(p.status, kStatusSeqTable);
      }
      const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && pos >= lo && pos < lo + n);
      if (hit) {
        const int src = __ffs(hit) - 1;
        first = b0 + src;
        first_at = static_cast<int>(__shfl_sync(0xffffffffu, lo, src));
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      if (blockIdx.x == 0) p.plan[p.B] = run;
      misc[1] = first;
      misc[2] = first_at;
      misc[3] = run;
      misc[4] = static_cast<int>(all);
    }
  }
  __syncthreads();
  const int run = misc[3], all = misc[4];
  const long long begin = static_cast<long long>(blockIdx.x) * run;
  if (begin >= all) return;
  const int pos0 = static_cast<int>(begin), pos1 = min(all, pos0 + run);
  const FailState fs{abort_flag, p.status, p.wait_ns};

  // A walk over the run: unit (b, hkv) and its tiles [t, t1) in the run.
  struct Walk {
    int b, hkv, nt, t, t1, at;  // at: the unit's first tile among all
  };
  auto start = [&]() {
    Walk w;
    w.b = misc[1];
    w.nt = flat_tiles(p, w.b);
    w.hkv = (pos0 - misc[2]) / w.nt;
    w.at = misc[2] + w.hkv * w.nt;
    w.t = pos0 - w.at;
    w.t1 = min(w.nt, pos1 - w.at);
    return w;
  };
  auto next = [&](Walk& w) {  // false: the run ends with this unit
    w.at += w.nt;
    if (w.at >= pos1) return false;
    if (++w.hkv == p.Hkv) {
      w.hkv = 0;
      do w.nt = flat_tiles(p, ++w.b); while (w.nt == 0);
    }
    w.t = 0;
    w.t1 = min(w.nt, pos1 - w.at);
    return true;
  };

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const int shift = p.page_shift - 6, sub = (1 << shift) - 1;  // tiles of a page
      // the page of a tile, checked: an id outside the pool is reported and read as
      // zeros (a TMA load outside the tensor fills)
      auto page_of = [&](const Walk& w, int t) {
        const int pg = __ldg(p.block_table + static_cast<size_t>(w.b) * p.max_pages + (t >> shift));
        if (pg >= 0 && pg < p.num_pages) return pg;
        atomicOr(p.status, kStatusSeqTable);
        return p.num_pages;
      };
      Walk w = start();
      int n = 0, st = 0;
      uint32_t par = 1;
      bool ok = true;
      do {
        int pg_next = page_of(w, w.t);  // page ids are read a tile ahead
        for (int t = w.t; ok && t < w.t1; ++t, ++n) {
          const int pg = pg_next;
          if (t + 1 < w.t1) pg_next = page_of(w, t + 1);
          if (n >= NS && !mbar_wait(&empty[st], par, fs)) {
            ok = false;
            break;
          }
          // test hook: a phase that cannot complete before this tile is loaded
          if (n == p.stall_tile && !mbar_wait(&k_full[st], (n / NS) & 1, fs)) {
            ok = false;
            break;
          }
          const int row = (t & sub) * kFlatTile;
          uint8_t* dst = sKV + 2 * st * TB;
          mbar_arrive_expect_tx(&k_full[st], TB);
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(&tm_k, &k_full[st], dst + h * (kFlatTile * 128), h * 64, w.hkv, row, pg);
          mbar_arrive_expect_tx(&v_full[st], TB);
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(&tm_v, &v_full[st], dst + TB + h * (kFlatTile * 128), h * 64, w.hkv, row, pg);
          if (++st == NS) {
            st = 0;
            par ^= 1u;  // the first wait for a stage is for its first release (phase 0)
          }
        }
      } while (ok && next(w));
      for (int i = max(0, n - NS); i < n; ++i) {
        mbar_wait_drain(&k_full[i % NS], (i / NS) & 1);
        mbar_wait_drain(&v_full[i % NS], (i / NS) & 1);
      }
    }
    return;  // the other warps synchronise with named barrier 1
  }

  // ---------------------------------------------------------- compute warps
  const int g = lane >> 2, c = lane & 3;  // this lane's head (row of S and O) and column pair
  const int mat = lane >> 3, r8 = lane & 7;
  // ldmatrix rows: K: matrices (keys 0-7, 8 values), (keys 0-7, next 8), (keys 8-15, ..), ..;
  // V, transposed: (keys 0-7, 8 values), (keys 8-15, same), (keys 0-7, next 8), ..
  const int k_row = warp * 16 + (mat >> 1) * 8 + r8, k_half = mat & 1;
  const int v_row = warp * 16 + (mat & 1) * 8 + r8, v_half = mat >> 1;
  const uint32_t kv = smem_u32(sKV);
  int st = 0;
  uint32_t par = 0;
  bool aborted = false;
  Walk w = start();
  do {
    const int len = __ldg(p.seqlens + w.b);
    const int unit = w.b * p.Hkv + w.hkv;
    uint32_t qa[D / 16][2];  // rows 0-7 of Q; rows 8-15 are zero
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][0] = qa[kk][1] = 0u;
      if (g < p.G) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<size_t>(w.b) * p.Hq + w.hkv * p.G + g) * D + kk * 16 + 2 * c);
        qa[kk][0] = __ldg(src);
        qa[kk][1] = __ldg(src + 4);
      }
    }
    float o[D / 8][4];  // rows g (P's high part) and g + 8 (its low part)
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m = -INFINITY, l = 0.f;
    float* score = p.scores + (static_cast<size_t>(unit) * p.G + g) * p.max_len + warp * 16 + 2 * c;

    for (int t = w.t; t < w.t1; ++t) {
      const uint32_t kt = kv + 2 * st * TB, vt = kt + TB;
      if (!aborted) aborted = !mbar_wait_warp(&k_full[st], par, fs);
      if (aborted) break;
      float s[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int ch = kk * 2 + k_half;
        uint32_t b[4];
        ldsm_x4(kt + (ch >> 3) * (kFlatTile * 128) + sw128_offset(k_row, ch & 7), b);
        mma_bf16(s[0], qa[kk][0], 0u, qa[kk][1], 0u, b[0], b[1]);
        mma_bf16(s[1], qa[kk][0], 0u, qa[kk][1], 0u, b[2], b[3]);
      }
      // scores of head g and keys 2c, 2c + 1, 2c + 8, 2c + 9 of the warp's 16
      float x[4] = {s[0][0] * p.scale_log2, s[0][1] * p.scale_log2, s[1][0] * p.scale_log2, s[1][1] * p.scale_log2};
      const int key0 = t * kFlatTile + warp * 16;
      if (g < p.G) {
        *reinterpret_cast<float2*>(score + t * kFlatTile) = make_float2(x[0], x[1]);
        *reinterpret_cast<float2*>(score + t * kFlatTile + 8) = make_float2(x[2], x[3]);
      }
      const bool tail = key0 + 16 > len;  // uniform over the warp: some of its keys are past the last
      if (tail) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 2 * c + (e & 1) + (e >> 1) * 8 >= len) x[e] = -INFINITY;
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool grows = top > m + 8.f;  // lazy rescale: the offset moves only when the maximum grew by > 2^8
      if (__any_sync(0xffffffffu, grows)) {
        const float a = grows ? ex2_approx(m - top) : 1.f;
        if (grows) m = top;
        l *= a;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= a;
      }
      const float off = m == -INFINITY ? 0.f : m;  // no key yet: every probability is exp2(-inf - 0) = 0
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(x[e] - off);
      l += (pr[0] + pr[1]) + (pr[2] + pr[3]);
      const uint32_t h0 = pack_bf16x2(pr[0], pr[1]), h1 = pack_bf16x2(pr[2], pr[3]);
      const uint32_t l0 = pack_bf16x2(pr[0] - bf16lo_to_f32(h0), pr[1] - bf16hi_to_f32(h0));
      const uint32_t l1 = pack_bf16x2(pr[2] - bf16lo_to_f32(h1), pr[3] - bf16hi_to_f32(h1));

      aborted = !mbar_wait_warp(&v_full[st], par, fs);
      if (aborted) break;
      if (tail) {
        // V rows past the last key are whatever the page held, perhaps not finite, and 0 times that
        // is not 0: the warp clears its own
        for (int i = lane; i < 16 * (D / 8); i += 32) {
          const int row = i / (D / 8), ch = i % (D / 8);
          if (key0 + row >= len)
            st_shared_v4(vt + (ch >> 3) * (kFlatTile * 128) + sw128_offset(warp * 16 + row, ch & 7), 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // before the stage is refilled
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const int ch = j * 2 + v_half;
        uint32_t b[4];
        ldsm_x4_trans(vt + (ch >> 3) * (kFlatTile * 128) + sw128_offset(v_row, ch & 7), b);
        mma_bf16(o[2 * j], h0, l0, h1, l1, b[0], b[1]);
        mma_bf16(o[2 * j + 1], h0, l0, h1, l1, b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);  // this warp has read K and V
      if (++st == NS) {
        st = 0;
        par ^= 1u;
      }
    }

    // the unit's part of this run: the warps' results into one
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c == 0) {
      sM[warp * 8 + g] = m;
      sL[warp * 8 + g] = l;
    }
    if (lane == 0) gave_up[warp] = aborted ? 1 : 0;
    named_bar_sync(1, 128);
    // one warp that gave up ends the run for all: the next unit's barriers need every warp
    aborted = (gave_up[0] | gave_up[1] | gave_up[2] | gave_up[3]) != 0;
    const float top = fmaxf(fmaxf(sM[g], sM[8 + g]), fmaxf(sM[16 + g], sM[24 + g]));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) z += sM[i * 8 + g] == -INFINITY ? 0.f : sL[i * 8 + g] * ex2_approx(sM[i * 8 + g] - top);
    const float a = m == -INFINITY ? 0.f : ex2_approx(m - top);
    // warps 2 and 3 hand theirs to 0 and 1, then 1 to 0
    if (warp >= 2) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(sRed + (warp - 2) * 8 * D + g * D + j * 8 + 2 * c) =
            make_float2((o[j][0] + o[j][2]) * a, (o[j][1] + o[j][3]) * a);
    }
    named_bar_sync(1, 128);
    if (warp < 2) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const float2 v = *reinterpret_cast<const float2*>(sRed + warp * 8 * D + g * D + j * 8 + 2 * c);
        o[j][0] = fmaf(o[j][0] + o[j][2], a, v.x);
        o[j][1] = fmaf(o[j][1] + o[j][3], a, v.y);
        if (warp == 1) *reinterpret_cast<float2*>(sRed + 8 * D + g * D + j * 8 + 2 * c) = make_float2(o[j][0], o[j][1]);
      }
    }
    named_bar_sync(1, 128);
    if (warp == 0 && g < p.G && !aborted) {
      const int slot = static_cast<int>(blockIdx.x) - w.at / run;
      const size_t at = (static_cast<size_t>(w.b) * p.Hq + w.hkv * p.G + g) * p.slots + slot;
      const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const float2 v = *reinterpret_cast<const float2*>(sRed + 8 * D + g * D + j * 8 + 2 * c);
        *reinterpret_cast<float2*>(p.o_part + at * D + j * 8 + 2 * c) =
            make_float2((o[j][0] + v.x) * inv, (o[j][1] + v.y) * inv);
      }
      if (c == 0) p.lse_part[at] = z > 0.f ? (top + lg2_approx(z)) * 0.69314718055994531f : -INFINITY;
    }
    // (the next unit's first barrier comes after its tiles: sM, sL and sRed are read by then)
  } while (!aborted && next(w));
}

}  // namespace mala
