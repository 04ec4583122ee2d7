// mala_key_mass.cuh -- the attention weight every key of a prompt has collected.
//
// Mathematics: with s_ij = scale <q_i, k_j> and LSE_i the log-normaliser that
// the attention call left for row i, key j of KV head hkv collects
//   mass_j = decay * mass_j' + sum_{i in rows, j <= P0 + i} sum_{h in group} exp(s_ij - LSE_i)
// (column sums of the softmax matrix). The matrix is never formed: the scores
// are recomputed tile by tile, as in the backward, and only their exponentials'
// sums are kept.
//
// mala_key_mass_kernel: one CTA owns two tiles of 128 keys of one (b, KV head) and
// walks the query tiles that see them, each for all heads of the GQA group. The
// scores are computed transposed, S^T = K Q^T: the keys are the M rows, so a
// thread owns one key (one TMEM lane) and its sum over the queries needs no
// exchange with other threads. K is copied into tensor memory once and is the A
// operand of every MMA; only Q passes through shared memory, which halves the
// operand traffic of an MMA whose both operands lie there (at N = 128 that
// traffic is as long as the MMA itself).
// The LSEs go through the tensor cores too: -LSE / scale in four bf16 parts (exact to
// 2^-33) are four more channels of a row of Q, against ones on the keys' side, so that
// what comes out is s - LSE and a thread only scales it. That is for the bits that the
// accumulator drops (toward zero, about half a step of every partial sum but the last):
// taken off at the end, the partial sums run up to s and every weight is too small, by
// 1.2e-6 on average over an 8K prompt and 1.9e-6 with scores of 40; taken off in the
// first place, they run from -LSE and it is too large. After five eighths of the
// channels (lse_step) the sums before and after partly cancel, for concentrated rows
// (s near LSE) and diffuse ones (s small against it): 1.8e-7 to 6.9e-7 in relative L2
// for prompts, random keys and large scores, and sums without dropped bits stay exact.
// It also spares a thread the loads of the LSEs, which pays for the step.
//   warps 0-15  compute: warps 8 x .. 8 x + 7 work on tile x, four on the first 64
//               queries of a query tile and four on the others; a thread reads its
//               key's 64 scores out of TMEM, hands the columns back, and sums the
//               exponentials
//   warp  16    producer: Q tiles by TMA and the rows' LSEs, a ring
//   warp  17    MMA issuer (one thread), the tiles in turn
// TMEM: S (2 x 128 columns) | K (2 x D / 2 columns) | ones (8 columns).
//
// Bound: with d = 128 a 128 x 128 tile takes 576 cycles of MMA (64 of them for the
// LSEs) and 16,384 exponentials, 1,024 cycles at the special-function unit's 16 a
// cycle; one of every eight pairs goes through packed FMAs instead (exp2_poly2). At
// 32K keys, 32 heads over 8 KV heads, 4.5 to 4.6 ms (repeats on the same inputs; 4.7
// with inputs that change), where the products alone would take 2.7 ms at the measured
// burst rate and the special-function unit 3.3 ms; the GPU runs at its power limit by
// then (1,000 W at 1.8 GHz), so that more pairs on the FMA pipes are slower although
// they relieve the unit (none 4.69 ms, one 4.53, two 4.80, three 5.02).
//
// Splits: when the key tiles alone do not fill the GPU, each CTA takes
// chunk_q query tiles and writes partial sums; mala_key_mass_join_kernel adds
// them in a fixed order, so results do not depend on the schedule.
#pragma once

#include <type_traits>

#include "mala_ptx.cuh"

namespace mala {

struct KeyMassParams {
  int B, Hq, Hkv, G;
  int Lq, Lk;           // packed batches: the longest sequence's
  int window;           // rows that count: the last `window` (0: all)
  int chunk_q;          // query tiles a CTA takes
  int n_chunks;         // grid: chunks per (b, KV head, key block)
  int n_blocks;         // key blocks that the grid covers (256 keys each)
  const uint16_t* k;    // [B, Lk, Hkv, d]
  const float* lse;     // [B, Hq, Lq]; packed batches: [Hq, total_q]
  const int* cu_q;      // packed batch (else null)
  const int* cu_k;
  int total_q, total_k;
  float scale_log2, decay;
  float inv_hi, inv_lo;  // 1 / scale, in two parts (lse_operand)
  const float* mass_in;  // [B, Hkv, ld], nullable
  float* mass_out;
  int ld;
  float* part;  // n_chunks > 1: [B * Hkv, n_chunks, part_ld] partial sums
  int part_ld;  // keys of a row of partials
  unsigned* status;
  uint64_t wait_ns;
  int stall_tile;  // test hook (-1: off): the MMA thread stalls before this item
};

constexpr int kMassTiles = 2;                   // key tiles of a CTA
constexpr int kMassKeys = kMassTiles * 128;     // its keys

template <int D>
struct KeyMassLayout {
  static constexpr int NT = kMassTiles;
  static constexpr int NQ = 4;       // Q ring
  static constexpr int CW = 8 * NT;  // compute warps
  static constexpr int THREADS = (CW + 2) * 32;
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int LSE_BYTES = 128 * 32;  // [NQ][128 rows][16 bf16]: the LSEs' channels (lse_offset)
  static constexpr int OFF_LSE = OFF_Q + NQ * Q_BYTES;
  static constexpr int OFF_RED = OFF_LSE + NQ * LSE_BYTES;  // fp32 [NT][128]: the second half's sums
  static constexpr int OFF_BAR = OFF_RED + NT * 512;
  // q_full[NQ], q_empty[NQ], s_full[NT], s_empty[NT], k_ready, mma_final
  static constexpr int N_BARS = 2 * NQ + 2 * NT + 2;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  // at least half of an SM's shared memory: a second CTA on the SM would wait for tensor memory
  static constexpr int LEAST = 118 * 1024;
  static constexpr int ALLOC_BYTES = (BYTES > LEAST ? BYTES : LEAST) + 1024;
  static constexpr int COL_S = 0, COL_K = NT * 128, COL_ONE = COL_K + NT * (D / 2);
  static constexpr int TMEM_COLS = 512;
  static_assert(ALLOC_BYTES <= 232448, "shared memory exceeds the per-CTA limit");
};

// One sequence's walk over the query tiles; the same in the join.
struct KeyMassSeq {
  int Lq, Lk, P0, first, q_off, k_off, n_qt;  // first: first row that counts; n_qt: query tiles from it
  bool ok;
};
__device__ __forceinline__ KeyMassSeq key_mass_seq(const KeyMassParams& p, int b) {
  KeyMassSeq s;
  s.Lq = p.Lq;
  s.Lk = p.Lk;
  s.q_off = s.k_off = 0;
  s.ok = true;
  if (p.cu_q != nullptr) {
    s.q_off = __ldg(p.cu_q + b);
    s.Lq = __ldg(p.cu_q + b + 1) - s.q_off;
    s.k_off = __ldg(p.cu_k + b);
    s.Lk = __ldg(p.cu_k + b + 1) - s.k_off;
    s.ok = !(s.q_off < 0 || s.Lq < 0 || s.Lq > p.Lq || s.q_off + s.Lq > p.total_q || s.k_off < 0 || s.Lk < s.Lq ||
             s.Lk > p.Lk || s.k_off + s.Lk > p.total_k);
  }
  s.P0 = s.Lk - s.Lq;
  s.first = p.window > 0 && p.window < s.Lq ? s.Lq - p.window : 0;
  s.n_qt = (s.Lq - s.first + 127) / 128;
  return s;
}
// the first query tile with a row that sees key k0
__device__ __forceinline__ int key_mass_qt0(const KeyMassSeq& s, int k0) {
  return max(0, k0 - s.P0 - s.first) / 128;
}

// -LSE in the units of the products q k, as four bf16 values whose sum is exact to 2^-33:
// the four channels that the MMA issuer adds to a row of Q.
__device__ __forceinline__ uint2 lse_operand(const KeyMassParams& p, float lse) {
  const float a = lse * p.inv_hi;
  const bool fin = fabsf(a) < INFINITY;
  const float e = fin ? fmaf(lse, p.inv_hi, -a) + lse * p.inv_lo : 0.f;
  const float hi = bf16lo_to_f32(pack_bf16x2(-a, 0.f));
  const float r = fin ? -a - hi : 0.f;  // (an infinity or NaN stands alone)
  const uint32_t w0 = pack_bf16x2(hi, r);
  return make_uint2(w0, pack_bf16x2(r - bf16hi_to_f32(w0), -e));
}

// Where chunk `chunk` (of two) of row `row` of that operand lies: 8-row blocks of each chunk.
__device__ __forceinline__ uint32_t lse_offset(int row, int chunk) {
  return (row >> 3) * 256 + chunk * 128 + (row & 7) * 16;
}
__device__ __forceinline__ uint64_t lse_desc(uint32_t saddr) { return sdesc_plain(saddr, 128, 256); }

// After how many of the D / 16 steps over the channels the LSEs' step comes (see above).
constexpr int lse_step(int d) { return (5 * (d / 16) + 7) / 8; }

// 2^x of a packed pair on the FMA pipes: x = n + f with n the nearest integer,
// |f| <= 1/2; 2^f by a polynomial of degree 5 (minimax in the relative error, by
// the Remez exchange: 7.5e-8, with fp32 rounding 2.1e-7, about ex2.approx's own
// error), times 2^n, whose exponent field n + 127 is the low byte of x + kShift.
// Outside fp32's range as ex2.approx, up to where it ends: 0 below -126.5 (n = -127
// has the field of zero, so a masked or empty row adds exactly nothing), infinity
// from 127.5, and NaN stays NaN (the clamps keep it, and so does the product).
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x) {
  constexpr float kShift = 12582912.f + 127.f;  // 1.5 * 2^23: adding it rounds to an integer in the low bits
  float lo, hi;
  f2_unpack(x, lo, hi);
  x = f2_pack(clamp_nan(lo, -127.f, 128.f), clamp_nan(hi, -127.f, 128.f));
  const uint64_t m = f2_add(x, f2_pack(kShift, kShift));
  const uint64_t n = f2_add(m, f2_pack(-kShift, -kShift));
  const uint64_t f = f2_fma(n, f2_pack(-1.f, -1.f), x);
  uint64_t r = f2_pack(0.0013276472454890609f, 0.0013276472454890609f);
  r = f2_fma(r, f, f2_pack(0.009675540961325169f, 0.009675540961325169f));
  r = f2_fma(r, f, f2_pack(0.05550713092088699f, 0.05550713092088699f));
  r = f2_fma(r, f, f2_pack(0.24022120237350464f, 0.24022120237350464f));
  r = f2_fma(r, f, f2_pack(0.6931469440460205f, 0.6931469440460205f));
  r = f2_fma(r, f, f2_pack(1.0000001192092896f, 1.0000001192092896f));
  float mlo, mhi;
  f2_unpack(m, mlo, mhi);
  return f2_mul(r, f2_pack(__uint_as_float(__float_as_uint(mlo) << 23), __uint_as_float(__float_as_uint(mhi) << 23)));
}

constexpr int kMassPoly = 1;  // of every eight packed pairs, how many go through exp2_poly2 (see above)

template <int D>
__global__ void __launch_bounds__(KeyMassLayout<D>::THREADS, 1)
    mala_key_mass_kernel(const __grid_constant__ CUtensorMap tm_q, const KeyMassParams p) {
  using Lay = KeyMassLayout<D>;
  constexpr int NT = Lay::NT, NQ = Lay::NQ, CW = Lay::CW;
  constexpr uint32_t IDESC = idesc_bf16(128, 128, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + Lay::OFF_Q;
  const uint32_t sLse = smem_u32(smem + Lay::OFF_LSE);
  float* sRed = reinterpret_cast<float*>(smem + Lay::OFF_RED);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* q_empty = q_full + NQ;
  uint64_t* s_full = q_empty + NQ;
  uint64_t* s_empty = s_full + NT;
  uint64_t* k_ready = s_empty + NT;
  uint64_t* mma_final = k_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA order: key blocks ascending, so the longest walks (the earliest keys) start first
  const int chunk = static_cast<int>(blockIdx.x) % p.n_chunks;
  const int bk = (static_cast<int>(blockIdx.x) / p.n_chunks) % (p.B * p.Hkv);
  const int blk = static_cast<int>(blockIdx.x) / (p.n_chunks * p.B * p.Hkv);
  const int b = bk / p.Hkv, hkv = bk % p.Hkv;
  const int k0 = blk * kMassKeys;
  const KeyMassSeq sq = key_mass_seq(p, b);
  if (!sq.ok) {  // nothing of this sequence is touched
    if (threadIdx.x == 0) atomicOr(p.status, kStatusSeqTable);
    return;
  }
  const int qt_a = key_mass_qt0(sq, k0) + chunk * p.chunk_q;
  const int qt_b = k0 < sq.Lk ? min(sq.n_qt, qt_a + p.chunk_q) : 0;
  const int N = max(0, qt_b - qt_a) * p.G;  // items: (query tile, head of the group), heads fastest
  const bool direct = p.n_chunks == 1;
  // compute warps: this thread's tile, half of the queries and key
  const int x = warp >> 3, half = (warp >> 2) & 1, wq = warp & 3;
  const int tid = wq * 32 + lane;
  const int key = k0 + x * 128 + tid;

  auto finish = [&](float sum) {  // one key's result
    if (!direct) {
      p.part[(static_cast<size_t>(bk) * p.n_chunks + chunk) * p.part_ld + key] = sum;
    } else if (key < p.ld) {
      const size_t at = static_cast<size_t>(bk) * p.ld + key;
      if (p.mass_in != nullptr && p.decay != 0.f && key < sq.P0) sum = fmaf(p.decay, p.mass_in[at], sum);
      p.mass_out[at] = key < sq.Lk ? sum : 0.f;
    }
  };
  if (N == 0) {  // no query sees these keys (the join reads no chunk that is empty)
    if (direct && warp < CW && half == 0) finish(0.f);
    return;
  }

  constexpr int W = D / 4;  // 32-bit words of half a row of K
  uint32_t w[32];           // compute warps: half of this key's row, on its way while the CTA sets up
  if (warp < CW && key < sq.Lk) {
    const size_t row = p.cu_q != nullptr ? static_cast<size_t>(sq.k_off) + key : static_cast<size_t>(b) * sq.Lk + key;
    const uint4* src = reinterpret_cast<const uint4*>(p.k + (row * p.Hkv + hkv) * D + half * (D / 2));
#pragma unroll
    for (int e = 0; e < W / 4; ++e) {
      const uint4 v = __ldg(src + e);
      w[4 * e] = v.x;
      w[4 * e + 1] = v.y;
      w[4 * e + 2] = v.z;
      w[4 * e + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) w[e] = 0u;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 2);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    mbar_init(k_ready, CW);
    mbar_init(mma_final, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == CW) {
    tmem_alloc(tmem_slot, Lay::TMEM_COLS);
    tmem_relinquish();
    if (lane == 0) prefetch_tensormap(&tm_q);
  }
  for (int i = threadIdx.x; i < NQ * Lay::LSE_BYTES / 16; i += Lay::THREADS)  // channels 4 .. 15 stay 0
    st_shared_v4(sLse + i * 16, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const FailState fs{abort_flag, p.status, p.wait_ns};

  if (warp == CW) {
    // ------------------------------------------------------------ producer
    const int bt = p.cu_q != nullptr ? 0 : b;
    // lane's four rows of an item's -LSE, read a whole item ahead of their use
    auto load_lse = [&](int i0, int g, float (&v)[4]) {
      const int hq = hkv * p.G + g;
      const float* src = p.cu_q != nullptr ? p.lse + static_cast<size_t>(hq) * p.total_q + sq.q_off
                                           : p.lse + (static_cast<size_t>(b) * p.Hq + hq) * sq.Lq;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * 32 + lane;
        v[e] = i < sq.Lq ? __ldg(src + i) : 0.f;
      }
    };
    float cur[4], nxt[4];
    int i0 = sq.first + qt_a * 128, g = 0, st = 0, issued = 0;
    uint32_t par = 1;
    load_lse(i0, 0, cur);
    for (int n = 0; n < N; ++n) {
      const int g_n = g + 1 == p.G ? 0 : g + 1, i0_n = g_n == 0 ? i0 + 128 : i0;
      if (n + 1 < N) load_lse(i0_n, g_n, nxt);
      if (n >= NQ && !mbar_wait_warp(&q_empty[st], par, fs)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[st], Lay::Q_BYTES);
        for (int h = 0; h < D / 64; ++h)
          tma_load_4d(&tm_q, &q_full[st], sQ + st * Lay::Q_BYTES + h * 16384, h * 64, hkv * p.G + g, sq.q_off + i0,
                      bt);
      }
      issued = n + 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint2 w = lse_operand(p, cur[e]);
        st_shared_v2(sLse + st * Lay::LSE_BYTES + lse_offset(e * 32 + lane, 0), w.x, w.y);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[st]);
#pragma unroll
      for (int e = 0; e < 4; ++e) cur[e] = nxt[e];
      g = g_n;
      i0 = i0_n;
      if (++st == NQ) {
        st = 0;
        par ^= 1u;  // the first wait for a slot is for its first release (phase 0)
      }
    }
    if (lane == 0)
      for (int n = max(0, issued - NQ); n < issued; ++n) mbar_wait_drain(&q_full[n % NQ], (n / NQ) & 1);
    __syncwarp();
  } else if (warp == CW + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dLse = lse_desc(sLse);
      bool ok = mbar_wait(k_ready, 0, fs);
      tc_fence_after();
      for (int n = 0; ok && n < N; ++n) {
        const int st = n % NQ;
        // test hook: wait on a barrier only this thread completes (after the
        // loop), so the bounded wait expires and the CTA takes its abort path
        if (n == p.stall_tile && !mbar_wait(mma_final, 0, fs)) break;
        if (!mbar_wait(&q_full[st], (n / NQ) & 1, fs)) break;
        for (int y = 0; y < NT; ++y) {
          if (n > 0 && !mbar_wait(&s_empty[y], (n - 1) & 1, fs)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            umma_f16_ts(tmem + Lay::COL_S + y * 128, tmem + Lay::COL_K + y * (D / 2) + kk * 8,
                        sdesc_add(dQ, st * Lay::Q_BYTES + (kk >> 2) * 16384 + (kk & 3) * 32), IDESC,
                        kk > 0 ? 1u : 0u);
            if (kk + 1 == lse_step(D))
              umma_f16_ts(tmem + Lay::COL_S + y * 128, tmem + Lay::COL_ONE, sdesc_add(dLse, st * Lay::LSE_BYTES),
                          IDESC, 1u);
          }
          umma_commit(&s_full[y]);
        }
        if (ok) umma_commit(&q_empty[st]);
      }
      umma_commit(mma_final);  // completes once every MMA above has finished
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute warps
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    {  // half of this key's row into tensor memory (A operand: two values to a column)
      const uint32_t tK = tmem + Lay::COL_K + x * (D / 2) + half * W + lane_base;
      __syncwarp();
      if constexpr (W == 32) tmem_st32(tK, w);
      else tmem_st16(tK, *reinterpret_cast<uint32_t(*)[16]>(w));
      if (x == 0 && half == 0) {  // channels 0 .. 3 of the LSEs' step: 1 for every key
        uint32_t one[16] = {0x3f803f80u, 0x3f803f80u};
        tmem_st16(tmem + Lay::COL_ONE + lane_base, one);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_ready);
    }
    const uint32_t tS = tmem + Lay::COL_S + x * 128 + half * 64 + lane_base;
    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2);
    const int kw0 = k0 + x * 128 + wq * 32;  // the warp's first key
    float sum = 0.f, comp = 0.f;  // compensated over the tiles: a key may be seen by 10^5 queries
    bool aborted = false;
    // one 64 x 1 strip of an item: the sum of this key's weights over the strip's queries.
    // kPlain: every row of the strip counts and sees every key of the warp.
    auto strip = [&](auto plain_c, int c_lo, int c_hi) -> float {
      constexpr bool kPlain = decltype(plain_c)::value;
      uint64_t acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = 0ull;  // (+0, +0)
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t sv[32];
        tmem_ld32(tS + c0, sv);
        tmem_ld_wait();
        if (c0 == 32) {  // the scores are out of TMEM: its columns go back to the MMA issuer
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[x]);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          uint64_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = f2_mul(f2_pack(__uint_as_float(sv[j + 2 * e]), __uint_as_float(sv[j + 2 * e + 1])), sl2);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (kPlain && e % 2 == 1 && e < 2 * kMassPoly) {
              v[e] = exp2_poly2(v[e]);
            } else {
              float lo, hi;
              f2_unpack(v[e], lo, hi);
              if (!kPlain) {  // columns c with key <= position of row c, rows below Lq. What is masked may be
                              // anything (the next sequence's rows), so it is replaced, not multiplied
                const int c = c0 + j + 2 * e;
                lo = c >= c_lo && c < c_hi ? lo : -INFINITY;
                hi = c + 1 >= c_lo && c + 1 < c_hi ? hi : -INFINITY;
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
    int g = 0;
    uint32_t s_par = 0;
    int r0 = sq.first + qt_a * 128 + half * 64;  // this warp's first row of the item
    for (int n = 0; n < N; ++n) {
      if (!mbar_wait_warp(&s_full[x], s_par, fs)) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const int pos0 = sq.P0 + r0;  // position of the first row
      float tile = 0.f;
      if (kw0 + 31 <= pos0 && r0 + 64 <= sq.Lq) {
        tile = strip(std::true_type(), 0, 0);
      } else if (kw0 <= pos0 + 63 && r0 < sq.Lq && kw0 < sq.Lk) {
        tile = strip(std::false_type(), key - pos0, sq.Lq - r0);
      } else {  // no row sees a key of the warp
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[x]);
      }
      const float y = tile - comp, t = sum + y;
      comp = (t - sum) - y;
      sum = t;
      s_par ^= 1u;
      if (++g == p.G) {
        g = 0;
        r0 += 128;
      }
    }
    if (half == 1) sRed[x * 128 + tid] = sum;
    named_bar_sync(1, CW * 32);
    if (half == 0 && !aborted && !abort_raised(fs)) finish(sum + sRed[x * 128 + tid]);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == CW) {
    if (lane == 0) mbar_wait_drain(mma_final, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Lay::TMEM_COLS);
  }
}

// Adds the chunks' partial sums of each key, in order, and the earlier mass.
// (A template so that more than one translation unit may include this file.)
template <int kThreads>
__global__ void __launch_bounds__(kThreads) mala_key_mass_join_kernel(const KeyMassParams p) {
  cudaGridDependencySynchronize();
  const int bk = blockIdx.y, b = bk / p.Hkv;
  const int key = blockIdx.x * kThreads + threadIdx.x;
  const KeyMassSeq sq = key_mass_seq(p, b);
  if (!sq.ok || key >= p.ld) return;
  float sum = 0.f;
  if (key < sq.Lk) {
    const int tiles = sq.n_qt - key_mass_qt0(sq, key & ~(kMassKeys - 1));
    const int n = tiles > 0 ? (tiles + p.chunk_q - 1) / p.chunk_q : 0;
    const float* src = p.part + static_cast<size_t>(bk) * p.n_chunks * p.part_ld + key;
#pragma unroll 4
    for (int c = 0; c < n; ++c) sum += src[static_cast<size_t>(c) * p.part_ld];
    if (p.mass_in != nullptr && p.decay != 0.f && key < sq.P0)
      sum = fmaf(p.decay, p.mass_in[static_cast<size_t>(bk) * p.ld + key], sum);
  }
  p.mass_out[static_cast<size_t>(bk) * p.ld + key] = sum;
}

}  // namespace mala
