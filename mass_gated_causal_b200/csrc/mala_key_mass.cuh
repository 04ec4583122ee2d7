// mala_key_mass.cuh -- the attention weight every key of a prompt has collected.
//
// Mathematics: with s_ij = scale <q_i, k_j> and LSE_i the log-normaliser that
// the attention call left for row i, key j of KV head hkv collects
//   mass_j = decay * mass_j' + sum_{i in rows, j <= P0 + i} sum_{h in group} exp(s_ij - LSE_i)
// (column sums of the softmax matrix). The matrix is never formed: the scores
// are recomputed tile by tile, as in the backward, and only their exponentials'
// sums are kept.
//
// mala_key_mass_kernel: one CTA owns 256 keys (two tiles A, B of 128) of one (b,
// KV head) and walks the query tiles that see them, each for all heads of the
// GQA group. The scores are computed transposed, S^T = K Q^T: the keys are the
// M rows, so a thread owns one key (one TMEM lane) and its sum over the queries
// needs no exchange with other threads. K is copied into tensor memory once and
// is the A operand of every MMA; only Q passes through shared memory, which
// halves the operand traffic of an MMA whose both operands lie there (at N = 128
// that traffic is as long as the MMA itself).
//   warps 0-3  tile A: thread t = key row t; load K, then per query tile read
//   warps 4-7  tile B  128 scores out of TMEM, hand the columns back, sum exps
//   warp  8    producer: Q tiles by TMA and the rows' -LSE log2(e) through a ring
//   warp  9    MMA issuer (one thread), alternating between the tiles
// TMEM: S_A | S_B | K_A | K_B (128 + 128 + D / 2 + D / 2 columns).
//
// Bound: with d = 128 a 128 x 128 tile takes 512 cycles of MMA and 16,384
// exponentials, 1,024 cycles at the special-function unit's 16 a cycle. So a
// share of the exponentials is computed with packed FMAs instead (exp2_poly2).
//
// Splits: when the key tiles alone do not fill the GPU, each CTA takes
// chunk_q query tiles and writes partial sums; mala_key_mass_join_kernel adds
// them in a fixed order, so results do not depend on the schedule.
#pragma once

#include "mala_ptx.cuh"

namespace mala {

struct KeyMassParams {
  int B, Hq, Hkv, G;
  int Lq, Lk;           // packed batches: the longest sequence's
  int window;           // rows that count: the last `window` (0: all)
  int chunk_q;          // query tiles a CTA takes
  int n_chunks;         // grid: chunks per (b, KV head, key pair)
  int n_pairs;          // key pairs that the grid covers (256 keys each)
  const uint16_t* k;    // [B, Lk, Hkv, d]
  const float* lse;     // [B, Hq, Lq]; packed batches: [Hq, total_q]
  const int* cu_q;      // packed batch (else null)
  const int* cu_k;
  int total_q, total_k;
  float scale_log2, decay;
  const float* mass_in;  // [B, Hkv, ld], nullable
  float* mass_out;
  int ld;
  float* part;  // n_chunks > 1: [B * Hkv, n_chunks, n_pairs * 256] partial sums
  unsigned* status;
  uint64_t wait_ns;
  int stall_tile;  // test hook (-1: off): the MMA thread stalls before this item
};

template <int D>
struct KeyMassLayout {
  static constexpr int NQ = 4;  // Q ring
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_LSE = OFF_Q + NQ * Q_BYTES;  // fp32 [NQ][128]
  static constexpr int OFF_BAR = OFF_LSE + NQ * 512;
  // q_full[NQ], q_empty[NQ], s_full[2], s_empty[2], k_ready, mma_final
  static constexpr int N_BARS = 2 * NQ + 6;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  // at least half of an SM's shared memory: a second CTA on the SM would wait for tensor memory
  static constexpr int ALLOC_BYTES = (BYTES > 118 * 1024 ? BYTES : 118 * 1024) + 1024;
  static constexpr int COL_S = 0, COL_K = 256;
  static constexpr int TMEM_COLS = 512;
  static_assert(ALLOC_BYTES <= 232448, "shared memory exceeds the per-CTA limit");
};

// What a (b, KV head, key pair) has to do; the same on the device and in the join.
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

// 2^x of a packed pair on the FMA pipes: x = n + f with n the nearest integer,
// |f| <= 1/2; 2^f by a polynomial of degree 5 (minimax in the relative error, by
// the Remez exchange: 7.5e-8, with fp32 rounding 2.1e-7, about ex2.approx's own
// error), n added to the exponent. x is held above -126 (2^-126 counts as
// nothing); it must stay below 127.
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x) {
  constexpr float kShift = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer in the low bits
  float lo, hi;
  f2_unpack(x, lo, hi);
  x = f2_pack(fmaxf(lo, -126.f), fmaxf(hi, -126.f));
  const uint64_t m = f2_add(x, f2_pack(kShift, kShift));
  const uint64_t n = f2_add(m, f2_pack(-kShift, -kShift));
  const uint64_t f = f2_fma(n, f2_pack(-1.f, -1.f), x);
  uint64_t r = f2_pack(0.0013276472454890609f, 0.0013276472454890609f);
  r = f2_fma(r, f, f2_pack(0.009675540961325169f, 0.009675540961325169f));
  r = f2_fma(r, f, f2_pack(0.05550713092088699f, 0.05550713092088699f));
  r = f2_fma(r, f, f2_pack(0.24022120237350464f, 0.24022120237350464f));
  r = f2_fma(r, f, f2_pack(0.6931469440460205f, 0.6931469440460205f));
  r = f2_fma(r, f, f2_pack(1.0000001192092896f, 1.0000001192092896f));
  float mlo, mhi, rlo, rhi;
  f2_unpack(m, mlo, mhi);
  f2_unpack(r, rlo, rhi);
  return f2_pack(__uint_as_float(__float_as_uint(rlo) + (__float_as_uint(mlo) << 23)),
                 __uint_as_float(__float_as_uint(rhi) + (__float_as_uint(mhi) << 23)));
}

constexpr int kMassPoly = 3;  // of every eight packed pairs, how many go through exp2_poly2

template <int D>
__global__ void __launch_bounds__(320, 1)
    mala_key_mass_kernel(const __grid_constant__ CUtensorMap tm_q, const KeyMassParams p) {
  using Lay = KeyMassLayout<D>;
  constexpr int NQ = Lay::NQ;
  constexpr uint32_t IDESC = idesc_bf16(128, 128, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + Lay::OFF_Q;
  float* sLse = reinterpret_cast<float*>(smem + Lay::OFF_LSE);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* q_empty = q_full + NQ;
  uint64_t* s_full = q_empty + NQ;
  uint64_t* s_empty = s_full + 2;
  uint64_t* k_ready = s_empty + 2;
  uint64_t* mma_final = k_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA order: key pairs ascending, so the longest walks (the earliest keys) start first
  const int chunk = static_cast<int>(blockIdx.x) % p.n_chunks;
  const int bk = (static_cast<int>(blockIdx.x) / p.n_chunks) % (p.B * p.Hkv);
  const int pair = static_cast<int>(blockIdx.x) / (p.n_chunks * p.B * p.Hkv);
  const int b = bk / p.Hkv, hkv = bk % p.Hkv;
  const int k0 = pair * 256;
  const KeyMassSeq sq = key_mass_seq(p, b);
  if (!sq.ok) {  // nothing of this sequence is touched
    if (threadIdx.x == 0) atomicOr(p.status, kStatusSeqTable);
    return;
  }
  const int qt_a = key_mass_qt0(sq, k0) + chunk * p.chunk_q;
  const int qt_b = k0 < sq.Lk ? min(sq.n_qt, qt_a + p.chunk_q) : 0;
  const int N = max(0, qt_b - qt_a) * p.G;  // items: (query tile, head of the group), heads fastest
  const bool direct = p.n_chunks == 1;
  const int tid = threadIdx.x & 127, x = (warp >> 2) & 1;
  const int key = k0 + x * 128 + tid;  // compute warps: this thread's key
  const size_t row_at = static_cast<size_t>(bk) * p.ld;

  auto finish = [&](float sum) {  // one key's result
    if (!direct) {
      p.part[(static_cast<size_t>(bk) * p.n_chunks + chunk) * (p.n_pairs * 256) + key] = sum;
    } else if (key < p.ld) {
      if (p.mass_in != nullptr && p.decay != 0.f && key < sq.P0)
        sum = fmaf(p.decay, p.mass_in[row_at + key], sum);
      p.mass_out[row_at + key] = key < sq.Lk ? sum : 0.f;
    }
  };
  if (N == 0) {  // no query sees these keys (the join reads no chunk that is empty)
    if (direct && warp < 8) finish(0.f);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 2);
      mbar_init(&q_empty[i], 1 + 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 128);
    }
    mbar_init(k_ready, 256);
    mbar_init(mma_final, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, Lay::TMEM_COLS);
    tmem_relinquish();
    if (lane == 0) prefetch_tensormap(&tm_q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const FailState fs{abort_flag, p.status, p.wait_ns};

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    const int bt = p.cu_q != nullptr ? 0 : b;
    // lane's four rows of an item's -LSE, read a whole item ahead of their use
    auto load_lse = [&](int n, float (&v)[4]) {
      const int i0 = sq.first + (qt_a + n / p.G) * 128, hq = hkv * p.G + n % p.G;
      const float* src = p.cu_q != nullptr ? p.lse + static_cast<size_t>(hq) * p.total_q + sq.q_off
                                           : p.lse + (static_cast<size_t>(b) * p.Hq + hq) * sq.Lq;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * 32 + lane;
        v[e] = i < sq.Lq ? __ldg(src + i) : 0.f;
      }
    };
    float cur[4], nxt[4];
    load_lse(0, cur);
    int issued = 0;
    for (int n = 0; n < N; ++n) {
      const int st = n % NQ;
      if (n + 1 < N) load_lse(n + 1, nxt);
      if (n >= NQ && !mbar_wait_warp(&q_empty[st], ((n / NQ) - 1) & 1, fs)) break;
      if (lane == 0) {
        const int i0 = sq.first + (qt_a + n / p.G) * 128, hq = hkv * p.G + n % p.G;
        mbar_arrive_expect_tx(&q_full[st], Lay::Q_BYTES);
        for (int h = 0; h < D / 64; ++h)
          tma_load_4d(&tm_q, &q_full[st], sQ + st * Lay::Q_BYTES + h * 16384, h * 64, hq, sq.q_off + i0, bt);
      }
      issued = n + 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) sLse[st * 128 + e * 32 + lane] = cur[e] * -1.4426950408889634f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[st]);
#pragma unroll
      for (int e = 0; e < 4; ++e) cur[e] = nxt[e];
    }
    if (lane == 0)
      for (int n = max(0, issued - NQ); n < issued; ++n) mbar_wait_drain(&q_full[n % NQ], (n / NQ) & 1);
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
      bool ok = mbar_wait(k_ready, 0, fs);
      tc_fence_after();
      for (int n = 0; ok && n < N; ++n) {
        const int st = n % NQ;
        // test hook: wait on a barrier only this thread completes (after the
        // loop), so the bounded wait expires and the CTA takes its abort path
        if (n == p.stall_tile && !mbar_wait(mma_final, 0, fs)) break;
        if (!mbar_wait(&q_full[st], (n / NQ) & 1, fs)) break;
        for (int y = 0; y < 2; ++y) {
          if (n > 0 && !mbar_wait(&s_empty[y], (n - 1) & 1, fs)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_f16_ts(tmem + Lay::COL_S + y * 128, tmem + Lay::COL_K + y * (D / 2) + kk * 8,
                        sdesc_add(dQ, st * Lay::Q_BYTES + (kk >> 2) * 16384 + (kk & 3) * 32), IDESC,
                        kk > 0 ? 1u : 0u);
          umma_commit(&s_full[y]);
        }
        if (ok) umma_commit(&q_empty[st]);
      }
      umma_commit(mma_final);  // completes once every MMA above has finished
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute warps
    const int wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    {  // this key's row into tensor memory (A operand: two values to a column)
      const uint32_t tK = tmem + Lay::COL_K + x * (D / 2) + lane_base;
      const uint4* src = nullptr;
      if (key < sq.Lk) {
        const size_t row = p.cu_q != nullptr ? static_cast<size_t>(sq.k_off) + key
                                             : static_cast<size_t>(b) * sq.Lk + key;
        src = reinterpret_cast<const uint4*>(p.k + (row * p.Hkv + hkv) * D);
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 v = src != nullptr ? __ldg(src + c * 8 + e) : make_uint4(0u, 0u, 0u, 0u);
          w[4 * e] = v.x;
          w[4 * e + 1] = v.y;
          w[4 * e + 2] = v.z;
          w[4 * e + 3] = v.w;
        }
        tmem_st32(tK + c * 32, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(k_ready);
    }
    const uint32_t tS = tmem + Lay::COL_S + x * 128 + lane_base;
    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2);
    const int kw0 = k0 + x * 128 + wq * 32;  // the warp's first key
    const uint32_t lse_s = smem_u32(sLse);
    float sum = 0.f, comp = 0.f;  // compensated over the tiles: a key may be seen by 10^5 queries
    bool aborted = false;
    for (int n = 0; n < N; ++n) {
      const int st = n % NQ;
      const int i0 = sq.first + (qt_a + n / p.G) * 128;
      if (!mbar_wait_warp(&s_full[x], n & 1, fs)) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const int pos0 = sq.P0 + i0;                                   // position of the tile's first row
      const bool none = kw0 > pos0 + 127 || kw0 >= sq.Lk;            // no row sees a key of the warp
      const bool plain = kw0 + 31 <= pos0 && i0 + 128 <= sq.Lq;      // every row sees every key of the warp
      uint32_t sv[128];
      if (!none) {
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_at(tS + c * 32, sv + c * 32);
        tmem_ld_wait();
      }
      tc_fence_before();
      mbar_arrive(&s_empty[x]);
      // the tile's LSEs: written before this phase of q_full completed, which the
      // MMA thread waited for before the scores; the wait makes them visible here
      if (!mbar_wait_warp(&q_full[st], (n / NQ) & 1, fs)) {
        aborted = true;
        break;
      }
      float tile = 0.f;
      if (!none) {
        const uint32_t la = lse_s + st * 512;
        if (plain) {
          uint64_t acc[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = 0ull;  // (+0, +0)
#pragma unroll
          for (int j = 0; j < 128; j += 16) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              uint64_t l0, l1;
              ld_shared_2f2(la + (j + 2 * e) * 4, l0, l1);
              const uint64_t x0 = f2_fma(f2_pack(__uint_as_float(sv[j + 2 * e]), __uint_as_float(sv[j + 2 * e + 1])),
                                         sl2, l0);
              const uint64_t x1 = f2_fma(
                  f2_pack(__uint_as_float(sv[j + 2 * e + 2]), __uint_as_float(sv[j + 2 * e + 3])), sl2, l1);
              auto ex = [](uint64_t v, bool poly) {
                if (poly) return exp2_poly2(v);
                float lo, hi;
                f2_unpack(v, lo, hi);
                return f2_pack(ex2_approx(lo), ex2_approx(hi));
              };
              // spread over the eight pairs: e < 2 * kMassPoly picks the even ones first
              acc[e] = f2_add(acc[e], ex(x0, e < 2 * kMassPoly));
              acc[e + 1] = f2_add(acc[e + 1], ex(x1, e < 2 * (kMassPoly - 4)));
            }
          }
#pragma unroll
          for (int e = 4; e > 0; e >>= 1)
#pragma unroll
            for (int i = 0; i < e; ++i) acc[i] = f2_add(acc[i], acc[i + e]);
          float lo, hi;
          f2_unpack(acc[0], lo, hi);
          tile = lo + hi;
        } else {
          // columns c with key <= pos0 + c and i0 + c < Lq; what is masked may be
          // anything (the next sequence's rows), so it is replaced, not multiplied
          const int c_lo = key - pos0, c_hi = sq.Lq - i0;
          const float s = p.scale_log2;
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 128; j += 4) {
            const float4 l = ld_shared_f4(la + j * 4);
            const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool live = j + e >= c_lo && j + e < c_hi;
              part[e] += ex2_approx(live ? fmaf(__uint_as_float(sv[j + e]), s, lv[e]) : -INFINITY);
            }
          }
          tile = (part[0] + part[1]) + (part[2] + part[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[st]);  // this warp has read the LSEs
      const float y = tile - comp, t = sum + y;
      comp = (t - sum) - y;
      sum = t;
    }
    if (!aborted) finish(sum);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    if (lane == 0) mbar_wait_drain(mma_final, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Lay::TMEM_COLS);
  }
}

// Adds the chunks' partial sums of each key, in order, and the earlier mass.
// (A template only so that every translation unit may include this file.)
template <int kThreads>
__global__ void __launch_bounds__(kThreads) mala_key_mass_join_kernel(const KeyMassParams p) {
  const int bk = blockIdx.y, b = bk / p.Hkv;
  const int key = blockIdx.x * kThreads + threadIdx.x;
  const KeyMassSeq sq = key_mass_seq(p, b);
  if (!sq.ok || key >= p.ld) return;
  float sum = 0.f;
  if (key < sq.Lk) {
    const int tiles = sq.n_qt - key_mass_qt0(sq, key & ~255);
    const int n = tiles > 0 ? (tiles + p.chunk_q - 1) / p.chunk_q : 0;
    const float* src = p.part + static_cast<size_t>(bk) * p.n_chunks * (p.n_pairs * 256) + key;
    for (int c = 0; c < n; ++c) sum += src[static_cast<size_t>(c) * (p.n_pairs * 256)];
    if (p.mass_in != nullptr && p.decay != 0.f && key < sq.P0)
      sum = fmaf(p.decay, p.mass_in[static_cast<size_t>(bk) * p.ld + key], sum);
  }
  p.mass_out[static_cast<size_t>(bk) * p.ld + key] = sum;
}

}  // namespace mala
