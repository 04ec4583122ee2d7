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
//
// Short caches (kShort): a cluster of CTAs takes one (sequence, KV head), its
// tiles dealt in turn, and everything ends there: the scores stay in shared
// memory, the CTAs read each other's maxima, sums and O through distributed shared
// memory, and each writes a slice of O and the masses of its own keys. One launch,
// no workspace: 2 sequences of up to 2K keys, 2 KV heads, 7.5 us in a graph against
// 12.5 for the two kernels.
#pragma once

#include "mala_ptx.cuh"
#include "mala_short_cluster.h"

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
  // kShort only (the others' are written by the second kernel)
  uint16_t* o;           // [B, Hq, d]
  float* lse;            // [B, Hq]
  const float* mass_in;  // [B, Hkv, ld], nullable
  float* mass_out;
  int32_t* kept_tiles;
  uint8_t* keep_map;
  float decay;
  int ld;
  int cluster;  // CTAs per (sequence, KV head)
  int pitch;    // floats between the heads' scores in shared memory
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
  static constexpr int PAIR_BYTES = 113 * 1024;  // two CTAs to an SM
  static_assert(ALLOC_BYTES <= PAIR_BYTES);

  // kShort: the warps' partials take the first stage once its tiles are read, and
  // the scores, [G][pitch] fp32, lie behind the rest. Eight floats more than the
  // tiles fill put the heads of a warp's stores into different banks.
  static constexpr int SHORT_NS = D == 128 ? 3 : 4;
  static constexpr int SHORT_ML = 2 * SHORT_NS * T_BYTES;
  static constexpr int SHORT_BAR = SHORT_ML + 2 * 4 * 8 * 4;
  static constexpr int SHORT_MISC = SHORT_BAR + 3 * SHORT_NS * 8;
  static constexpr int SHORT_SCORES = SHORT_MISC + 48;
  static constexpr int short_pitch(int tiles) { return tiles * kFlatTile + 8; }
  static constexpr int short_bytes(int G, int tiles) { return SHORT_SCORES + G * short_pitch(tiles) * 4 + 1024; }
  static_assert(2 * 8 * D * 4 <= 2 * T_BYTES && SHORT_SCORES % 8 == 0);
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

template <int D, bool kShort>
__global__ void __launch_bounds__(kFlatThreads, 2)
    mala_decode_flat_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const FlatParams p) {
  using Lay = FlatLayout<D>;
  constexpr int NS = kShort ? Lay::SHORT_NS : Lay::NS, TB = Lay::T_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;  // stage s: K at 2 s TB, V at (2 s + 1) TB
  float* sRed = reinterpret_cast<float*>(smem + (kShort ? 0 : Lay::OFF_RED));
  float* sM = reinterpret_cast<float*>(smem + (kShort ? Lay::SHORT_ML : Lay::OFF_ML));
  float* sL = sM + 32;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + (kShort ? Lay::SHORT_BAR : Lay::OFF_BAR));
  uint64_t* v_full = k_full + NS;
  uint64_t* empty = v_full + NS;
  int* misc = reinterpret_cast<int*>(smem + (kShort ? Lay::SHORT_MISC : Lay::OFF_MISC));
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
  if (!kShort && warp == 0) {
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
  const int run = kShort ? 1 : misc[3], all = kShort ? 0 : misc[4];
  const long long begin = kShort ? 0 : static_cast<long long>(blockIdx.x) * run;
  if (!kShort && begin >= all) return;
  const int pos0 = static_cast<int>(begin), pos1 = min(all, pos0 + run);
  const FailState fs{abort_flag, p.status, p.wait_ns};
  const int rank = kShort ? static_cast<int>(blockIdx.x) % p.cluster : 0;
  const int step = kShort ? p.cluster : 1;  // between the tiles of a walk

  // A walk over the run: unit (b, hkv) and its tiles [t, t1) in the run.
  struct Walk {
    int b, hkv, nt, t, t1, at;  // at: the unit's first tile among all
  };
  auto start = [&]() {
    Walk w;
    if constexpr (kShort) {
      const int unit = static_cast<int>(blockIdx.x) / p.cluster;
      w.b = unit / p.Hkv;
      w.hkv = unit % p.Hkv;
      w.nt = w.t1 = flat_tiles(p, w.b);
      w.t = rank;
      w.at = 0;
      return w;
    }
    w.b = misc[1];
    w.nt = flat_tiles(p, w.b);
    w.hkv = (pos0 - misc[2]) / w.nt;
    w.at = misc[2] + w.hkv * w.nt;
    w.t = pos0 - w.at;
    w.t1 = min(w.nt, pos1 - w.at);
    return w;
  };
  auto next = [&](Walk& w) {  // false: the run ends with this unit
    if constexpr (kShort) return false;
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
      auto page_at = [&](int b, int t) { return __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + (t >> shift)); };
      // an id outside the pool is reported and read as zeros (a TMA load outside the tensor fills)
      auto checked = [&](int pg) {
        if (pg >= 0 && pg < p.num_pages) return pg;
        atomicOr(p.status, kStatusSeqTable);
        return p.num_pages;
      };
      // kShort: the first page id is on its way while the length is (perhaps one past the last page: not used then)
      const int pg_first = kShort ? page_at(static_cast<int>(blockIdx.x) / p.cluster / p.Hkv,
                                            min(rank, ((p.max_pages - 1) << shift)))
                                  : 0;
      Walk w = start();
      int n = 0, st = 0;
      uint32_t par = 1;
      bool ok = true;
      do {
        int pg_next = kShort ? pg_first : page_at(w.b, w.t);  // page ids are read a tile ahead
        for (int t = w.t; ok && t < w.t1; t += step, ++n) {
          const int pg = checked(pg_next);
          if (t + step < w.t1) pg_next = page_at(w.b, t + step);
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
    if constexpr (kShort) {  // the cluster's two barriers count every thread
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
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
    const int len = kShort && w.nt == 0 ? 0 : __ldg(p.seqlens + w.b);
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
    float* score;  // of head g and this lane's keys in a tile
    if constexpr (kShort) {
      score = reinterpret_cast<float*>(smem + Lay::SHORT_SCORES) + g * p.pitch + warp * 16 + 2 * c;
      const size_t row = static_cast<size_t>(unit) * p.ld;
      for (int j = w.nt * kFlatTile + rank * 128 + static_cast<int>(threadIdx.x); j < p.ld; j += step * 128)
        p.mass_out[row + j] = 0.f;
      if (rank == 0) {
        const int pages = (len + (1 << p.page_shift) - 1) >> p.page_shift;
        const size_t first = static_cast<size_t>(w.b) * p.Hq + w.hkv * p.G;
        if (static_cast<int>(threadIdx.x) < p.G) p.kept_tiles[first + threadIdx.x] = pages;
        if (p.keep_map != nullptr)
          for (int h = 0; h < p.G; ++h)
            for (int i = threadIdx.x; i < pages; i += 128) p.keep_map[(first + h) * p.max_pages + i] = 1;
        const int given = __ldg(p.seqlens + w.b);
        if (w.hkv == 0 && threadIdx.x == 0 && (given < 0 || given > p.max_len)) atomicOr(p.status, kStatusSeqTable);
      }
    } else {
      score = p.scores + (static_cast<size_t>(unit) * p.G + g) * p.max_len + warp * 16 + 2 * c;
    }

    for (int t = w.t; t < w.t1; t += step) {
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
        float* to = kShort ? score : score + t * kFlatTile;
        *reinterpret_cast<float2*>(to) = make_float2(x[0], x[1]);
        *reinterpret_cast<float2*>(to + 8) = make_float2(x[2], x[3]);
        if constexpr (kShort) score += kFlatTile;
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

    float before[kShortTiles / 2];  // kShort: earlier masses of this thread's keys, on their way while the cluster meets
    if constexpr (kShort) {
#pragma unroll
      for (int u = 0; u < kShortTiles / 2; ++u) {
        const int i = static_cast<int>(threadIdx.x) + 128 * u;
        const int j = (rank + (i >> 6) * step) * kFlatTile + (i & 63);
        before[u] = p.mass_in != nullptr && p.decay != 0.f && j < len - 1
                        ? p.mass_in[static_cast<size_t>(unit) * p.ld + j]
                        : 0.f;
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
    if constexpr (kShort) {
      const int tid = threadIdx.x, n_cta = p.cluster;
      // this CTA's O (relative to its maxima), maxima and sums, for the cluster to read
      if (warp == 0) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float2 v = *reinterpret_cast<const float2*>(sRed + 8 * D + g * D + j * 8 + 2 * c);
          *reinterpret_cast<float2*>(sRed + g * D + j * 8 + 2 * c) = make_float2(o[j][0] + v.x, o[j][1] + v.y);
        }
        if (c == 0) {
          sM[g] = top;
          sL[g] = z;
        }
      }
      cluster_arrive();
      cluster_wait();
      // weight of CTA r in head h, and the heads' LSEs (log2 units): 16 threads a head
      float* weight = sRed + 8 * D;  // [8][kShortCluster]
      float* lse2 = weight + 8 * kShortCluster;
      {
        const int h = tid / kShortCluster, r = tid % kShortCluster;
        float mt = -INFINITY, zt = 0.f;
        if (r < n_cta) {
          mt = ld_cluster_f32(sM + h, r);
          zt = ld_cluster_f32(sL + h, r);
        }
        float mx = mt;
#pragma unroll
        for (int i = kShortCluster / 2; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        const float e = mt == -INFINITY ? 0.f : ex2_approx(mt - mx);
        float sum = zt * e;
#pragma unroll
        for (int i = kShortCluster / 2; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        weight[tid] = sum > 0.f ? e / sum : 0.f;
        const float l2 = sum > 0.f ? mx + lg2_approx(sum) : -INFINITY;
        if (r == 0) lse2[h] = l2;
        if (r == 0 && rank == 0 && h < p.G)
          p.lse[static_cast<size_t>(w.b) * p.Hq + w.hkv * p.G + h] = l2 * 0.69314718055994531f;
      }
      named_bar_sync(1, 128);
      // a slice of O: pairs of values rank, rank + cluster, ..
      for (int i = rank + n_cta * tid; i < p.G * (D / 2); i += n_cta * 128) {
        const int h = i / (D / 2), e = i % (D / 2) * 2;
        float x = 0.f, y = 0.f;
#pragma unroll 8
        for (int r = 0; r < n_cta; ++r) {
          const float2 v = ld_cluster_2f32(sRed + h * D + e, r);
          const float f = weight[h * kShortCluster + r];
          x = fmaf(f, v.x, x);
          y = fmaf(f, v.y, y);
        }
        *reinterpret_cast<uint32_t*>(p.o + (static_cast<size_t>(w.b) * p.Hq + w.hkv * p.G + h) * D + e) =
            pack_bf16x2(x, y);
      }
      cluster_arrive();  // the others' shared memory is read
      const float* sc = reinterpret_cast<const float*>(smem + Lay::SHORT_SCORES);
#pragma unroll
      for (int u = 0; u < kShortTiles / 2; ++u) {
        const int i = tid + 128 * u, t = rank + (i >> 6) * step;
        if (t >= w.nt) break;
        const int j = t * kFlatTile + (i & 63);
        float mass = 0.f;
        for (int h = 0; h < p.G; ++h) mass += ex2_approx(sc[h * p.pitch + i] - lse2[h]);
        p.mass_out[static_cast<size_t>(unit) * p.ld + j] = j < len ? fmaf(p.decay, before[u], mass) : 0.f;
      }
      cluster_wait();  // no CTA leaves while another may read its shared memory
      return;
    }
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
