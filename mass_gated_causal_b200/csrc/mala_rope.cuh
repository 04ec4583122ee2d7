// mala_rope.cuh -- rotary positions with several axes, and their form that
// writes the new keys and values of a step straight into a paged cache.
//
// Mathematics: the first 2n values of a head form n pairs; pair i of a token
// turns by theta_i = pos[axis(i)] * inv_freq[i]:
//   y1 = x1 cos theta - x2 sin theta,   y2 = x2 cos theta + x1 sin theta.
// The rotation is orthogonal, so its gradient is the rotation by -theta. The
// values past the pairs, and V, are copied.
//
// Angles: pos * inv_freq / (2 pi) is formed in fp64 and reduced to a fraction
// of a turn in [-1/2, 1/2] there (a position of 10^6 would leave an fp32 angle
// an error of 0.06 radians); the sine and cosine of the fraction are fp32. They
// are computed here rather than read from a table: a thread does it once for
// its pairs and uses it for all of its heads.
//
// Layout: a row is one head of one token. A unit is the 16 values of a row that
// hold eight pairs (or 16 copied values), two 16-byte chunks; D / 16 lanes
// cover a row, and neighbouring rows go to neighbouring lanes, so a warp's
// loads are whole lines. A thread keeps its token and its unit and walks the
// rows hg, hg + groups, ... of the token, four loads ahead. Bound by HBM: every
// value is read once and written once. 32K tokens of 48 heads of 128 (805 MB): 124
// us, 6.5 TB/s, as fast as a plain copy; 8K tokens 37.5 us, of which about 7 are
// the launch and its ends; 8 tokens 3.4 us, all of it latency.
#pragma once

#include "mala_ptx.cuh"

namespace mala {

struct RopeParams {
  const uint16_t* src[3];  // q, k, v (null with zero heads)
  uint16_t* dst[3];
  long long src_tok[3], src_head[3];  // strides in elements
  long long dst_tok[3], dst_head[3];
  int heads[3];
  const int32_t* pos;  // [n_axes, T]
  const float* inv_freq;
  uint64_t axis_lo, axis_hi;  // two bits a pair: its axis
  int T, pairs, groups;       // groups: threads that share a token's rows
  float sign;                 // -1: the transposed rotation
  // paged destination of k and v (kPaged)
  const int32_t* block_table;  // [num_seqs, max_pages]
  const int32_t* seqlens;      // [num_seqs] lengths with the new tokens
  const int32_t* cu;           // [num_seqs + 1] token offsets, or null: per_seq tokens each
  int num_seqs, per_seq, max_pages, num_pages, page_shift;
  unsigned* status;
};

constexpr int kRopeThreads = 128;

// Row (in its sequence's cache) and sequence of new token t. Returns 1: there
// is one; 0: the token belongs to no sequence, or to an idle one (length 0);
// -1: its sequence's tables are invalid.
__device__ __forceinline__ int rope_cache_row(const RopeParams& p, int t, int& seq, int& row) {
  int first, n;
  if (p.cu != nullptr) {
    // the last sequence whose offset is <= t (a bad table still ends the search in range)
    int lo = 0, hi = p.num_seqs;
    while (lo + 1 < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= t) lo = mid; else hi = mid;
    }
    seq = lo;
    first = __ldg(p.cu + lo);
    const int end = __ldg(p.cu + lo + 1);
    if (first > t || end <= t) return 0;
    if (first < 0 || end > p.T) return -1;
    n = end - first;
  } else {
    seq = t / p.per_seq;
    first = seq * p.per_seq;
    n = p.per_seq;
  }
  const int len = __ldg(p.seqlens + seq);
  if (len == 0) return 0;
  if (len < n || static_cast<long long>(len) > (static_cast<long long>(p.max_pages) << p.page_shift)) return -1;
  row = len - n + (t - first);
  return 1;
}

template <int D, bool kAdjacent, bool kPaged, int U>
__global__ void __launch_bounds__(kRopeThreads) mala_rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 16;  // lanes per row
  const int unit = threadIdx.x % LPR;
  const long long slot = static_cast<long long>(blockIdx.x) * (kRopeThreads / LPR) + threadIdx.x / LPR;
  const int t = static_cast<int>(slot / p.groups);
  const int hg = static_cast<int>(slot % p.groups);
  if (t >= p.T) return;

  long long page_row = -1;  // paged: row of the pools ([num_pages * page] rows), -1 for no such row
  if (kPaged) {
    int seq = 0, row = 0;
    const int ok = rope_cache_row(p, t, seq, row);
    if (ok == 0) return;  // no sequence's token: nothing of it is touched
    if (ok > 0) {
      const int pg = __ldg(p.block_table + static_cast<long long>(seq) * p.max_pages + (row >> p.page_shift));
      if (pg >= 0 && pg < p.num_pages)
        page_row = (static_cast<long long>(pg) << p.page_shift) + (row & ((1 << p.page_shift) - 1));
    }
    if (page_row < 0 && hg == 0 && unit == 0) atomicOr(p.status, kStatusSeqTable);
  }

  // this thread's chunks: of a rotated row, and of a copied one
  const bool turns = unit * 8 < p.pairs;
  const int plain_a = 16 * unit;
  const int rest = 2 * p.pairs + 16 * (unit - p.pairs / 8);  // units past the pairs
  const int a_off = turns ? (kAdjacent ? 16 * unit : 8 * unit) : rest;
  const int b_off = turns ? (kAdjacent ? 16 * unit + 8 : p.pairs + 8 * unit) : rest + 8;

  float cs[8], sn[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = unit * 8 + i;
      const int axis = static_cast<int>((pair < 32 ? p.axis_lo >> (2 * pair) : p.axis_hi >> (2 * (pair - 32))) & 3u);
      const double turn = static_cast<double>(__ldg(p.pos + static_cast<long long>(axis) * p.T + t)) *
                          static_cast<double>(__ldg(p.inv_freq + pair)) * 0.15915494309189533577;
      const float f = static_cast<float>(2.0 * (turn - rint(turn)));  // half turns, in [-1, 1]
      sincospif(f, &sn[i], &cs[i]);
      sn[i] *= p.sign;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
  }

  const int h_k = p.heads[0], h_v = h_k + p.heads[1], h_end = h_v + p.heads[2];
  for (int h0 = hg; h0 < h_end; h0 += p.groups * U) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * p.groups;
      if (h >= h_end) break;
      const int w = h < h_k ? 0 : h < h_v ? 1 : 2;
      const int hh = w == 0 ? h : w == 1 ? h - h_k : h - h_v;
      const uint16_t* row = p.src[w] + t * p.src_tok[w] + hh * p.src_head[w];
      a[u] = *reinterpret_cast<const uint4*>(row + (w == 2 ? plain_a : a_off));
      b[u] = *reinterpret_cast<const uint4*>(row + (w == 2 ? plain_a + 8 : b_off));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * p.groups;
      if (h >= h_end) break;
      const int w = h < h_k ? 0 : h < h_v ? 1 : 2;
      const int hh = w == 0 ? h : w == 1 ? h - h_k : h - h_v;
      if (w != 2 && turns) {
        uint32_t x[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
        uint32_t y[8];
        if (kAdjacent) {  // word i holds pair i
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x1 = bf16lo_to_f32(x[i]), x2 = bf16hi_to_f32(x[i]);
            y[i] = pack_bf16x2(x1 * cs[i] - x2 * sn[i], x2 * cs[i] + x1 * sn[i]);
          }
        } else {  // words i and i + 4 hold pairs 2i and 2i + 1
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p1 = bf16lo_to_f32(x[i]), p2 = bf16lo_to_f32(x[i + 4]);
            const float q1 = bf16hi_to_f32(x[i]), q2 = bf16hi_to_f32(x[i + 4]);
            y[i] = pack_bf16x2(p1 * cs[2 * i] - p2 * sn[2 * i], q1 * cs[2 * i + 1] - q2 * sn[2 * i + 1]);
            y[i + 4] = pack_bf16x2(p2 * cs[2 * i] + p1 * sn[2 * i], q2 * cs[2 * i + 1] + q1 * sn[2 * i + 1]);
          }
        }
        a[u] = make_uint4(y[0], y[1], y[2], y[3]);
        b[u] = make_uint4(y[4], y[5], y[6], y[7]);
      }
      uint16_t* row;
      if (kPaged && w != 0) {
        if (page_row < 0) continue;
        row = p.dst[w] + (page_row * p.heads[w] + hh) * D;
      } else {
        row = p.dst[w] + t * p.dst_tok[w] + hh * p.dst_head[w];
      }
      *reinterpret_cast<uint4*>(row + (w == 2 ? plain_a : a_off)) = a[u];
      *reinterpret_cast<uint4*>(row + (w == 2 ? plain_a + 8 : b_off)) = b[u];
    }
  }
}

}  // namespace mala
