// mala_key_mass_window.cuh -- key mass of a few query rows against a long cache
// (the last rows of a prompt, a short chunk).
//
// Mathematics as in mala_key_mass.cuh. With G x W rows in all (W rows that
// count, G heads of the group) small enough for shared memory, the roles turn:
// Q stays, K streams. One CTA takes one (b, KV head) and a run of its key tiles;
// Q of all G heads is one operand of up to 512 columns, loaded once, so a key
// tile costs its K and one MMA of N = kCols columns per half-row step, and no
// start-up per key block (walks as in mala_key_mass_kernel took 174 us for the
// case below, most of it the walks' starts).
//   warps 0-15  compute, two teams of eight that do not wait for each other's tiles, so
//               that one's waits are filled by the other's exponentials: up to 256
//               columns (one block) they take the tiles in turn, else a block each of
//               every tile. A warp has 32 keys and half of the block's columns; the
//               parts' sums meet in shared memory, and the first part's warps write
//               the result. At the start they lay out the LSEs, while Q and K are on their way
//   warp  16    producer: Q once, K tiles through a ring
//   warp  17    MMA issuer (one thread): S^T = K Q^T, two TMEM buffers in turn
// Columns past a head's rows hold zeros in Q and -infinity in place of -LSE, so
// they add nothing. Bound: G x W exponentials per key on the
// special-function unit (at 256 columns 2,048 cycles a tile against 760 for reading
// K at the HBM rate), a quarter of them moved to the FMA pipes (exp2_poly2). 64 rows
// of 32 heads over 8 KV heads against 2 x 32,000 keys: 41 us over two sets of inputs in
// turn (43 with an eighth on the FMA pipes, 44.7 with three eighths; all sixteen warps on
// one tile took 15% longer), 49 where every pass has inputs that no cache holds; one row,
// which only reads K, 27.5 us, of which 21 are K's bytes.
#pragma once

#include "mala_key_mass.cuh"

namespace mala {

constexpr int kWinMaxCols = 512;  // query rows of all heads that a CTA holds
constexpr int kWinPoly = 2;       // of every eight packed pairs, how many go through exp2_poly2

struct WinParams {
  KeyMassParams m;  // n_blocks, n_chunks, chunk_q and part are not used
  int rows_pad;     // W rounded up to 8: a head's columns
  int parts;        // CTAs per (b, KV head)
  int k_stages;     // K ring
};

template <int D, int kCols, int kBlocks>
struct WinLayout {
  static constexpr int THREADS = 18 * 32;
  static constexpr int K_BYTES = 128 * D * 2;
  static constexpr int MAX_STAGES = 4;
  static constexpr int STEP = kBlocks == 1 ? 2 : 1;  // between a team's tiles
  static constexpr int AHEAD = 6 / STEP;  // a team's tiles that the earlier masses are fetched ahead (a tile may take 0.3 us)
  // pos [512], sums [2][4][128], earlier masses [STEP][AHEAD + 1][128], then barriers
  static constexpr int OFF_POS = 0;
  static constexpr int OFF_RED = OFF_POS + kWinMaxCols * 4;
  static constexpr int OFF_OLD = OFF_RED + 2 * 4 * 128 * 4;
  static constexpr int OFF_BAR = OFF_OLD + STEP * (AHEAD + 1) * 128 * 4;
  // k_full[4], k_empty[4], s_full[2], s_empty[2], q_full, q_ready, mma_final
  static constexpr int N_BARS = 2 * MAX_STAGES + 4 + 3;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int OFF_Q = (OFF_MISC + 16 + 1023) & ~1023;
  // behind Q the LSEs' channels of its columns and those of the keys (16 each, lse_offset), then the K ring
  static constexpr int OFF_LSE = OFF_Q + kBlocks * kCols * D * 2;
  static constexpr int OFF_ONE = OFF_LSE + kBlocks * kCols * 32;
  static constexpr int OFF_K = OFF_ONE + 128 * 32;
  static_assert(OFF_K % 1024 == 0, "swizzled tiles");
  static constexpr int bytes(int stages) { return OFF_K + stages * K_BYTES + 1024; }
};

template <int D, int kCols, int kBlocks>
__global__ void __launch_bounds__(WinLayout<D, kCols, kBlocks>::THREADS, 1)
    mala_key_mass_window_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                                const WinParams wp) {
  using Lay = WinLayout<D, kCols, kBlocks>;
  const KeyMassParams& p = wp.m;
  constexpr uint32_t IDESC = idesc_bf16(128, kCols, false, false);
  constexpr int STEP = Lay::STEP;
  constexpr int CG = kCols / 2;  // columns per compute warp
  static_assert(CG % 32 == 0, "a warp reads its columns 32 at a time");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sLse = smem_u32(smem + Lay::OFF_LSE), sOne = smem_u32(smem + Lay::OFF_ONE);
  int* sPos = reinterpret_cast<int*>(smem + Lay::OFF_POS);
  float* sRed = reinterpret_cast<float*>(smem + Lay::OFF_RED);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* k_empty = k_full + Lay::MAX_STAGES;
  uint64_t* s_full = k_empty + Lay::MAX_STAGES;
  uint64_t* s_empty = s_full + 2;
  uint64_t* q_full = s_empty + 2;
  uint64_t* q_ready = q_full + 1;
  uint64_t* mma_final = q_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  uint8_t* sQ = smem + Lay::OFF_Q;
  constexpr int cols = kBlocks * kCols;  // columns in all
  uint8_t* sK = smem + Lay::OFF_K;
  const int NK = wp.k_stages;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bk = static_cast<int>(blockIdx.x) % (p.B * p.Hkv), part = static_cast<int>(blockIdx.x) / (p.B * p.Hkv);
  const int b = bk / p.Hkv, hkv = bk % p.Hkv;
  const KeyMassSeq sq = key_mass_seq(p, b);
  if (!sq.ok) {  // nothing of this sequence is touched
    if (threadIdx.x == 0 && part == 0) atomicOr(p.status, kStatusSeqTable);
    return;
  }
  const int rows = sq.Lq - sq.first;  // rows of a head that count (<= rows_pad)
  const int n_tiles = (sq.Lk + 127) / 128;
  const int per = (n_tiles + wp.parts - 1) / wp.parts;
  const int t0 = min(part * per, n_tiles), T = min(per, n_tiles - t0);
  const size_t row_at = static_cast<size_t>(bk) * p.ld;
  // the entries past the keys, by the last part
  if (part == wp.parts - 1)
    for (int j = sq.Lk + static_cast<int>(threadIdx.x); j < p.ld; j += Lay::THREADS) p.mass_out[row_at + j] = 0.f;
  if (T <= 0) return;
  if (rows <= 0) {  // a sequence without queries: its keys keep what they have
    for (int j = t0 * 128 + static_cast<int>(threadIdx.x); j < min((t0 + T) * 128, sq.Lk); j += Lay::THREADS)
      p.mass_out[row_at + j] =
          p.mass_in != nullptr && p.decay != 0.f && j < sq.P0 ? p.decay * p.mass_in[row_at + j] : 0.f;
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::MAX_STAGES; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    mbar_init(q_full, 1);
    mbar_init(q_ready, 16);
    mbar_init(mma_final, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const FailState fs{abort_flag, p.status, p.wait_ns};

  if (warp == 16) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const int bt = p.cu_q != nullptr ? 0 : b;
      mbar_arrive_expect_tx(q_full, p.G * wp.rows_pad * D * 2);
      for (int g = 0; g < p.G; ++g)
        for (int h = 0; h < D / 64; ++h)
          tma_load_4d(&tm_q, q_full, sQ + h * (cols * 128) + g * wp.rows_pad * 128, h * 64, hkv * p.G + g,
                      sq.q_off + sq.first, bt);
      int st = 0, issued = 0;
      uint32_t par = 1;
      for (int t = 0; t < T; ++t) {
        if (t >= NK && !mbar_wait(&k_empty[st], par, fs)) break;
        mbar_arrive_expect_tx(&k_full[st], Lay::K_BYTES);
        for (int h = 0; h < D / 64; ++h)
          tma_load_4d(&tm_k, &k_full[st], sK + st * Lay::K_BYTES + h * 16384, h * 64, hkv,
                      sq.k_off + (t0 + t) * 128, bt);
        issued = t + 1;
        if (++st == NK) {
          st = 0;
          par ^= 1u;  // the first wait for a slot is for its first release (phase 0)
        }
      }
      mbar_wait_drain(q_full, 0);
      for (int t = max(0, issued - NK); t < issued; ++t) mbar_wait_drain(&k_full[t % NK], (t / NK) & 1);
    }
    __syncwarp();
  } else if (warp == 17) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dK = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dLse = lse_desc(sLse), dOne = lse_desc(sOne);
      bool ok = mbar_wait(q_ready, 0, fs);
      int st = 0, n = 0;
      uint32_t par = 0;
      for (int t = 0; ok && t < T; ++t) {
        // test hook: wait on a barrier only this thread completes (after the
        // loop), so the bounded wait expires and the CTA takes its abort path
        if (t == p.stall_tile && !mbar_wait(mma_final, 0, fs)) break;
        if (!mbar_wait(&k_full[st], par, fs)) break;
        for (int y = 0; y < kBlocks; ++y, ++n) {
          if (n >= 2 && !mbar_wait(&s_empty[n & 1], ((n >> 1) - 1) & 1, fs)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            umma_bf16_ss(tmem + (n & 1) * 256, sdesc_add(dK, st * Lay::K_BYTES + (kk >> 2) * 16384 + (kk & 3) * 32),
                         sdesc_add(dQ, (kk >> 2) * (cols * 128) + y * (kCols * 128) + (kk & 3) * 32), IDESC,
                         kk > 0 ? 1u : 0u);
            if (kk + 1 == lse_step(D))
              umma_bf16_ss(tmem + (n & 1) * 256, dOne, sdesc_add(dLse, y * (kCols * 32)), IDESC, 1u);
          }
          umma_commit(&s_full[n & 1]);
        }
        if (ok) umma_commit(&k_empty[st]);
        if (++st == NK) {
          st = 0;
          par ^= 1u;
        }
      }
      umma_commit(mma_final);  // completes once every MMA above has finished
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute warps
    const int wq = warp & 3, cg = (warp >> 2) & 1, team = warp >> 3;
    const int y = kBlocks == 1 ? 0 : team;  // this warp's block
    const int tid = wq * 32 + lane;  // key within the tile
    // the columns' LSEs and positions, and 1 in the LSEs' channels for every key, while Q and K are on their way
    for (int c = threadIdx.x; c < cols; c += 16 * 32) {
      const int g = c / wp.rows_pad, r = c % wp.rows_pad, i = sq.first + r;
      uint2 w = make_uint2(0xff80u, 0u);  // -infinity: a column of no row
      if (g < p.G && r < rows) {
        const int hq = hkv * p.G + g;
        w = lse_operand(p, __ldg(p.cu_q != nullptr ? p.lse + static_cast<size_t>(hq) * p.total_q + sq.q_off + i
                                                   : p.lse + (static_cast<size_t>(b) * p.Hq + hq) * sq.Lq + i));
      }
      st_shared_v4(sLse + lse_offset(c, 0), w.x, w.y, 0u, 0u);
      st_shared_v4(sLse + lse_offset(c, 1), 0u, 0u, 0u, 0u);
      sPos[c] = sq.P0 + i;
    }
    if (threadIdx.x < 128) {
      st_shared_v4(sOne + lse_offset(threadIdx.x, 0), 0x3f803f80u, 0x3f803f80u, 0u, 0u);
      st_shared_v4(sOne + lse_offset(threadIdx.x, 1), 0u, 0u, 0u, 0u);
    }
    bool aborted = !mbar_wait_warp(q_full, 0, fs);
    // rows that do not count: of a head past its rows (another sequence's, perhaps), and past the last head
    for (int i = warp * 32 + lane; i < cols * (D / 8); i += 16 * 32) {
      const int c = i / (D / 8), ch = i % (D / 8);
      if (c / wp.rows_pad >= p.G || c % wp.rows_pad >= rows)
        st_shared_v4(smem_u32(sQ) + (ch >> 3) * (cols * 128) + sw128_offset(c, ch & 7), 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_ready);
    if (!aborted) aborted = !mbar_wait_warp(q_ready, 0, fs);  // every warp's positions are in place

    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2);
    const uint32_t tS = tmem + team * 256 + cg * CG + lane_base;  // each team has its own buffer of scores
    const int* pos_a = sPos + y * kCols + cg * CG;
    const int p_min = sq.P0 + sq.first;  // position of the first row that counts
    // The warps of the first columns add the earlier masses: each thread copies its key's into its own
    // slot of a ring in shared memory, AHEAD tiles before it reads it. A sequence's own tokens start from 0.
    constexpr int AHEAD = Lay::AHEAD;
    const bool first = cg == 0 && y == 0;
    const bool has_old = first && p.mass_in != nullptr && p.decay != 0.f;
    float* sOld = reinterpret_cast<float*>(smem + Lay::OFF_OLD) + (STEP == 2 ? team * (AHEAD + 1) * 128 : 0) + tid;
    auto fetch_old = [&](int t, int slot) {
      const int key = (t0 + t) * 128 + tid;
      if (has_old && t < T && key < sq.P0) cp_async_4(smem_u32(sOld + slot * 128), p.mass_in + row_at + key);
      cp_async_commit();  // one group a tile, empty or not, so that the counting holds
    };
    const int t_first = STEP == 2 ? team : 0;  // the team's first tile
    for (int i = 0; i < AHEAD; ++i) fetch_old(t_first + i * STEP, i);
    int slot = 0;
    // this key's weights summed over the warp's columns; kPlain: every row sees every key of the tile
    auto strip = [&](auto plain_c, int key) -> float {
      constexpr bool kPlain = decltype(plain_c)::value;
      uint64_t acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = 0ull;  // (+0, +0)
#pragma unroll 2  // (all four at once spill)
      for (int c0 = 0; c0 < CG; c0 += 32) {
        uint32_t sv[32];
        tmem_ld32(tS + c0, sv);
        tmem_ld_wait();
        if (c0 == CG - 32) {  // the block is out of TMEM: its columns go back to the MMA issuer
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[team]);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          uint64_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = f2_mul(f2_pack(__uint_as_float(sv[j + 2 * e]), __uint_as_float(sv[j + 2 * e + 1])), sl2);
          const int* pos = pos_a + c0 + j;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (kPlain && e % 2 == 1 && e < 2 * kWinPoly) {
              v[e] = exp2_poly2(v[e]);
            } else {
              float lo, hi;
              f2_unpack(v[e], lo, hi);
              if (!kPlain) {
                lo = key <= pos[2 * e] ? lo : -INFINITY;
                hi = key <= pos[2 * e + 1] ? hi : -INFINITY;
              }
              v[e] = f2_pack(ex2_approx(lo), ex2_approx(hi));
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e & 3] = f2_add(acc[e & 3], v[e]);
        }
      }
      float lo, hi;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
      return lo + hi;
    };
    int use = 0;  // of the team's buffer
    for (int t = t_first; t < T; t += STEP, ++use) {
      const int k0 = (t0 + t) * 128, key = k0 + tid;
      fetch_old(t + AHEAD * STEP, slot == 0 ? AHEAD : slot - 1);
      float sum = 0.f;
      if (!aborted) aborted = !mbar_wait_warp(&s_full[team], use & 1, fs);
      if (!aborted) {  // (the barriers below are met in any case)
        tc_fence_after();
        sum = k0 + 127 <= p_min ? strip(std::true_type(), key) : strip(std::false_type(), key);
      }
      // Where the parts' sums meet: one block, both halves of the team's tile; two, those of the second
      // team too, which runs up to two tiles ahead of the first.
      float* red = sRed + (kBlocks == 1 ? team * 2 + (use & 1) : 2 * (use & 1)) * 256 + tid;
      if (kBlocks == 1) {
        red[cg * 128] = sum;
        named_bar_sync(1 + team, 256);  // the team's next tile writes the other half of red
      } else {
        if (team == 1 && use >= 2) named_bar_sync(3 + (use & 1), 512);  // the first team has read
        red[(2 * y + cg) * 128] = sum;
        if (team == 1) named_bar_arrive(1 + (use & 1), 512);
        else named_bar_sync(1 + (use & 1), 512);
      }
      if (first && key < sq.Lk && !aborted && !abort_raised(fs)) {
        float m = red[0] + red[128];
        if constexpr (kBlocks == 2) m += red[256] + red[384];
        cp_async_wait<AHEAD>();
        if (has_old && key < sq.P0) m = fmaf(p.decay, sOld[slot * 128], m);
        p.mass_out[row_at + key] = m;
      }
      if (kBlocks == 2 && team == 0 && t + 2 < T) named_bar_arrive(3 + (use & 1), 512);
      slot = slot == AHEAD ? 0 : slot + 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    if (lane == 0) mbar_wait_drain(mma_final, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace mala
