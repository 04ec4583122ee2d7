// mala_evict.cuh -- eviction from a paged cache by collected attention weight.
//
// mala_evict_select_kernel: which rows of a sequence's cache remain, for every
// (sequence, KV head). With L rows and a budget of K < L, the first n_sink and
// the last n_recent rows remain, and of the rows between them the
// need = K - n_sink - n_recent heaviest, ties to the lowest row. The kernel
// finds the need-th largest mass by a radix select over the masses' ordered bit
// patterns (11, 11 and 10 bits, most significant first), then lists the rows
// above it and the first of those equal to it in ascending order. One cluster of
// kCluster CTAs works on one row of masses, each CTA on a contiguous part: the
// digit counts are joined through distributed shared memory, and the parts'
// output offsets are the counts of the CTAs before them, so nothing depends on
// the order of atomics. Where a thread meets at most 32 rows (kKeep) their keys stay
// in shared memory and two bit masks say which of them remain for sure and which
// still share the threshold's digits, so that only the first digit's count and the
// listing walk over all rows; in longer parts the masses are read five times, from
// L2 after the first. 64 rows of 32K masses to 4K: 13.4 us (16.7 with all five walks
// over values in registers).
//
// mala_evict_gather_kernel: copies the K and V of the remaining rows into other
// pages. Bound by HBM: each kept row of a head is read and written once, in
// pieces of D * 2 bytes on the reading side (rows of the other heads lie
// between) and whole lines on the writing side.
#pragma once

#include <cooperative_groups.h>

#include "mala_ptx.cuh"

namespace mala {

struct EvictParams {
  const float* mass;  // [B, Hkv, ld]
  const int32_t* seqlens;
  int32_t* index;     // [B, Hkv, budget]
  int32_t* new_lens;  // [B]
  float* mass_out;    // [B, Hkv, ld_out], nullable
  int B, Hkv, ld, budget, n_sink, n_recent, ld_out;
  unsigned* status;
};

constexpr int kEvictThreads = 1024;
constexpr int kEvictBins = 2048;

constexpr uint32_t kNanKey = 0x007fffffu;  // -infinity's

// Bit pattern whose unsigned order is the masses' order: -0 equals +0, and NaN
// ranks with -infinity.
__device__ __forceinline__ uint32_t mass_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return kNanKey;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the warps before this one (wsum: a value per warp, in shared memory).
template <int NW>
__device__ __forceinline__ uint32_t before_warp(const uint32_t* wsum, int warp, int lane) {
  static_assert(NW == 32, "one value per lane");
  return __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u);
}

template <int kCluster, int kKeep>
__global__ void __launch_bounds__(kEvictThreads) mala_evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  constexpr int NT = kEvictThreads, NW = NT / 32;
  static_assert(kEvictBins == 2 * NT, "two bins per thread");
  __shared__ __align__(16) uint32_t hist[3][kEvictBins];  // one per pass: no pass waits for the last one's readers
  __shared__ uint32_t wsum[NW], w_gt[NW], w_eq[NW];
  __shared__ uint32_t s_digit, s_above, s_count;
  __shared__ uint32_t cta_cnt[2];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
  const int b = row / p.Hkv, h = row % p.Hkv;
  int L = __ldg(p.seqlens + b);
  if (L < 0 || L > p.ld) {  // an invalid length is reported, and nothing of the sequence remains
    if (h == 0 && rank == 0 && tid == 0) atomicOr(p.status, kStatusSeqTable);
    L = 0;
  }
  const int n_new = min(L, p.budget);
  const float* mass = p.mass + static_cast<size_t>(row) * p.ld;
  int32_t* index = p.index + static_cast<size_t>(row) * p.budget;
  float* mass_out = p.mass_out ? p.mass_out + static_cast<size_t>(row) * p.ld_out : nullptr;
  const int gt = rank * NT + tid, gn = kCluster * NT;
  if (h == 0 && gt == 0) p.new_lens[b] = n_new;
  for (int r = n_new + gt; r < p.budget; r += gn) index[r] = -1;
  if (mass_out)
    for (int r = n_new + gt; r < p.ld_out; r += gn) mass_out[r] = 0.f;
  if (L <= p.budget) {  // everything remains (the same for every CTA of the cluster)
    for (int r = gt; r < L; r += gn) {
      index[r] = r;
      if (mass_out) mass_out[r] = mass[r];
    }
    return;
  }

  const int lo = p.n_sink, hi = L - p.n_recent;  // L > budget >= n_sink + n_recent
  const int need = p.budget - p.n_sink - p.n_recent;
  for (int r = gt; r < lo; r += gn) {
    index[r] = r;
    if (mass_out) mass_out[r] = mass[r];
  }
  for (int r = hi + gt; r < L; r += gn) {
    const int at = p.budget - (L - r);
    index[at] = r;
    if (mass_out) mass_out[at] = mass[r];
  }
  if (need == 0) return;  // uniform over the cluster

  cg::cluster_group cluster = cg::this_cluster();
  auto sync_all = [&]() {
    if constexpr (kCluster == 1) __syncthreads();
    else cluster.sync();
  };
  // this warp's part of the rows between: whole runs of 32 rows
  const int mid = hi - lo;
  const int per_warp = ((mid + kCluster * NW - 1) / (kCluster * NW) + 31) & ~31;
  const int w0 = lo + min((rank * NW + warp) * per_warp, mid);
  const int w1 = min(w0 + per_warp, hi);
  const uint32_t below = (1u << lane) - 1u;

#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(&hist[i][2 * tid]) = make_uint2(0u, 0u);
  __syncthreads();
  uint32_t remaining = static_cast<uint32_t>(need);
  // the threshold's digit of a pass, from the counts of all CTAs; what is still needed of its rows.
  // True: no further digit has to be read, as all of this digit's rows remain (the same for every CTA)
  auto find_digit = [&](const int pass) {
    sync_all();
    // counts of this thread's two bins over the cluster; thread 0 takes the highest
    const int top = kEvictBins - 2 - 2 * tid;
    uint2 cnt = make_uint2(0u, 0u);
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      const uint32_t* other = kCluster == 1 ? hist[pass] : cluster.map_shared_rank(&hist[pass][0], c);
      const uint2 v = *reinterpret_cast<const uint2*>(other + top);
      cnt.x += v.x;
      cnt.y += v.y;
    }
    const uint32_t sum = cnt.x + cnt.y;
    uint32_t incl = sum;  // inclusive scan over the threads, from the highest bin down
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    const uint32_t above = before_warp<NW>(wsum, warp, lane) + incl - sum;
    if (above < remaining && above + sum >= remaining) {  // one thread: the digit is one of its bins
      const bool high = above + cnt.y >= remaining;
      s_digit = static_cast<uint32_t>(high ? top + 1 : top);
      s_above = high ? above : above + cnt.y;
      s_count = high ? cnt.y : cnt.x;
    }
    __syncthreads();
    remaining -= s_above;
    return s_count == remaining;
  };
  // where this warp's rows above the threshold and its rows equal to it (by the digits read) begin
  auto begin_at = [&](uint32_t n_gt, uint32_t n_eq, uint32_t& base_gt, uint32_t& base_eq) {
    n_gt = __reduce_add_sync(0xffffffffu, n_gt);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
      w_gt[warp] = n_gt;
      w_eq[warp] = n_eq;
    }
    __syncthreads();
    base_gt = before_warp<NW>(w_gt, warp, lane);
    base_eq = before_warp<NW>(w_eq, warp, lane);
    if constexpr (kCluster > 1) {
      if (warp == NW - 1 && lane == 0) {
        cta_cnt[0] = base_gt + n_gt;
        cta_cnt[1] = base_eq + n_eq;
      }
      cluster.sync();
      for (int c = 0; c < rank; ++c) {
        const uint32_t* other = cluster.map_shared_rank(cta_cnt, c);
        base_gt += other[0];
        base_eq += other[1];
      }
    }
  };
  auto digit_of = [](uint32_t key, int pass) {
    return pass == 0 ? key >> 21 : pass == 1 ? key >> 10 & 2047u : key & 1023u;
  };

  if constexpr (kKeep > 0) {
    extern __shared__ uint32_t keep[];  // [kKeep][threads]: keys of the rows w0 + lane + 32 i
    const int n_in = max(0, min(kKeep, (w1 - w0 - lane + 31) / 32));
    uint32_t open = n_in >= 32 ? 0xffffffffu : (1u << n_in) - 1u;  // rows with the threshold's digits so far
    uint32_t over = 0;                                             // rows above it
    float x[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) x[i] = open >> i & 1 ? mass[w0 + lane + 32 * i] : 0.f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (open >> i & 1) {
        const uint32_t key = mass_key(x[i]);
        keep[i * NT + tid] = key;
        atomicAdd(&hist[0][digit_of(key, 0)], 1u);
      }
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const bool done = find_digit(pass);
      auto classify = [&](int i) {
        const uint32_t key = keep[i * NT + tid], digit = digit_of(key, pass);
        if (digit != s_digit) {
          open &= ~(1u << i);
          if (digit > s_digit) over |= 1u << i;
        } else if (pass < 2 && !done) {
          atomicAdd(&hist[pass < 2 ? pass + 1 : 0][digit_of(key, pass + 1)], 1u);
        }
      };
      if (pass == 0 || kKeep <= 4) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
          if (open >> i & 1) classify(i);
      } else {
        for (uint32_t left = open; left != 0; left &= left - 1) classify(__ffs(left) - 1);
      }
      if (done) break;
    }
    uint32_t base_gt, base_eq;
    begin_at(__popc(over), __popc(open), base_gt, base_eq);
    int at = lo + static_cast<int>(base_gt + min(base_eq, remaining));
    if (__any_sync(0xffffffffu, open != 0)) {  // of the rows equal to the threshold the first `remaining`
      for (int i = 0; i < kKeep; ++i) {
        const uint32_t be = __ballot_sync(0xffffffffu, open >> i & 1);
        if ((open >> i & 1) && base_eq + __popc(be & below) < remaining) over |= 1u << i;
        base_eq += __popc(be);
      }
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const uint32_t b = __ballot_sync(0xffffffffu, over >> i & 1);
      if (over >> i & 1) {
        const int r = w0 + lane + 32 * i, to = at + __popc(b & below);
        index[to] = r;
        if (mass_out) {
          const uint32_t key = keep[i * NT + tid];
          // from the key, as a load here would wait for the stores before it (-0 comes out as +0)
          mass_out[to] = key == kNanKey ? mass[r] : __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
        }
      }
      at += __popc(b);
    }
  } else {
    // every row of the part, in order: f(row, mass, whether the row is there)
    auto for_part = [&](auto&& f) {
#pragma unroll 8
      for (int r0 = w0; r0 < w1; r0 += 32) {
        const int r = r0 + lane;
        f(r, r < w1 ? mass[r] : 0.f, r < w1);
      }
    };
    uint32_t prefix = 0, mask = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      for_part([&](int, float x, bool there) {
        const uint32_t key = mass_key(x);
        if (there && (key & mask) == prefix) atomicAdd(&hist[pass][digit_of(key, pass)], 1u);
      });
      const bool done = find_digit(pass);
      constexpr int kShift[3] = {21, 10, 0};
      prefix |= s_digit << kShift[pass];
      mask |= (pass == 2 ? 1023u : 2047u) << kShift[pass];
      if (done) break;
    }
    uint32_t n_gt = 0, n_eq = 0;
    for_part([&](int, float x, bool there) {
      const uint32_t key = mass_key(x) & mask;
      n_gt += there && key > prefix ? 1u : 0u;
      n_eq += there && key == prefix ? 1u : 0u;
    });
    uint32_t base_gt, base_eq;
    begin_at(n_gt, n_eq, base_gt, base_eq);
    for_part([&](int r, float x, bool there) {
      const uint32_t key = mass_key(x) & mask;
      const bool is_gt = there && key > prefix, is_eq = there && key == prefix;
      const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
      const uint32_t eq_rank = base_eq + __popc(be & below);
      if (is_gt || (is_eq && eq_rank < remaining)) {
        const int at = lo + static_cast<int>(base_gt + __popc(bg & below) + min(eq_rank, remaining));
        index[at] = r;
        if (mass_out) mass_out[at] = x;
      }
      base_gt += __popc(bg);
      base_eq += __popc(be);
    });
  }
  if constexpr (kCluster > 1) cluster.sync();  // no CTA leaves while another may read its counts
}

struct GatherParams {
  const uint4* k;  // [num_pages, page, Hkv, d]
  const uint4* v;
  uint4* k_out;    // [num_out_pages, page, Hkv, d]
  uint4* v_out;
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* out_table;    // [B, max_out_pages]
  const int32_t* index;        // [B, Hkv, budget]
  const int32_t* lens;         // [B] rows that remain
  int B, Hkv, budget, num_pages, max_pages, num_out_pages, max_out_pages, page_shift;
  unsigned* status;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 4;  // rows of a head a thread copies 16 bytes of, K and V

template <int D>
__global__ void __launch_bounds__(kGatherThreads) mala_evict_gather_kernel(const GatherParams p) {
  cudaGridDependencySynchronize();
  constexpr int LPR = D / 8, SLOTS = kGatherThreads / LPR;
  const int b = blockIdx.y;
  const int len = min(__ldg(p.lens + b), p.budget);
  const int c = threadIdx.x % LPR;
  const long long n = static_cast<long long>(max(len, 0)) * p.Hkv;  // (row, head) pairs, heads fastest
  const long long first = static_cast<long long>(blockIdx.x) * SLOTS * kGatherRows + threadIdx.x / LPR;
  const int page_mask = (1 << p.page_shift) - 1;
  long long src[kGatherRows], dst[kGatherRows];
  uint4 kv[kGatherRows], vv[kGatherRows];
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    const long long i = first + u * SLOTS;
    src[u] = -1;
    if (i >= n) continue;
    const int r = static_cast<int>(i / p.Hkv), h = static_cast<int>(i % p.Hkv);
    const int from = __ldg(p.index + (static_cast<long long>(b) * p.Hkv + h) * p.budget + r);
    const int to_pg = __ldg(p.out_table + static_cast<long long>(b) * p.max_out_pages + (r >> p.page_shift));
    int pg = -1;
    if (from >= 0 && (from >> p.page_shift) < p.max_pages)
      pg = __ldg(p.block_table + static_cast<long long>(b) * p.max_pages + (from >> p.page_shift));
    if (pg < 0 || pg >= p.num_pages || to_pg < 0 || to_pg >= p.num_out_pages) {
      if (c == 0) atomicOr(p.status, kStatusSeqTable);
      continue;
    }
    src[u] = (((static_cast<long long>(pg) << p.page_shift) + (from & page_mask)) * p.Hkv + h) * LPR + c;
    dst[u] = (((static_cast<long long>(to_pg) << p.page_shift) + (r & page_mask)) * p.Hkv + h) * LPR + c;
  }
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u)
    if (src[u] >= 0) {
      kv[u] = p.k[src[u]];
      vv[u] = p.v[src[u]];
    }
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u)
    if (src[u] >= 0) {
      p.k_out[dst[u]] = kv[u];
      p.v_out[dst[u]] = vv[u];
    }
}

}  // namespace mala
