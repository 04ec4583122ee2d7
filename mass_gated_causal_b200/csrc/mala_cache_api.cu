// mala_cache_api.cu -- C ABI of the operators beside attention that a cache
// needs: rotary positions (training, and into a paged cache) and eviction by
// collected attention weight. Host side only; the kernels are included below.
#include <algorithm>

#include "mala_evict.cuh"
#include "mala_evict_check.h"
#include "mala_host.h"
#include "mala_rope.cuh"

using namespace mala::host;

namespace {

// ------------------------------------------------------------------- rope
// The axis of every pair, two bits each. Returns a status.
int rope_axes(int rotary_dim, const int32_t* sections, int n_axes, bool cyclic, uint64_t* lo, uint64_t* hi) {
  if (!sections || n_axes < 1 || n_axes > 4) return MALA_ERR_INVALID_ARG;
  const int pairs = rotary_dim / 2;
  int sum = 0, count[4] = {0, 0, 0, 0};
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0 || sections[a] > pairs) return MALA_ERR_INVALID_ARG;
    sum += sections[a];
  }
  if (sum != pairs) return MALA_ERR_INVALID_ARG;
  *lo = *hi = 0;
  for (int i = 0; i < pairs; ++i) {
    int a = 0;
    if (cyclic) {
      a = i % n_axes;
      if (i >= n_axes * sections[a]) a = 0;
    } else {
      for (int end = sections[0]; i >= end;) end += sections[++a];
    }
    ++count[a];
    (i < 32 ? *lo : *hi) |= static_cast<uint64_t>(a) << (2 * (i & 31));
  }
  for (int a = 0; a < n_axes; ++a)
    if (count[a] != sections[a]) return MALA_ERR_INVALID_ARG;  // sections that do not interleave
  return MALA_OK;
}

int check_rope(int T, int Hq, int Hkv, int d, int rotary_dim, unsigned flags, unsigned known) {
  if (T < 0 || Hq < 1 || Hkv < 1 || (flags & ~known)) return MALA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return MALA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > d || rotary_dim % 16 != 0) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(Hq) + 2ll * Hkv >= (1ll << 20)) return MALA_ERR_UNSUPPORTED;
  return MALA_OK;
}

// One strided tensor of rows: 16-byte chunks of every row aligned, and, for a
// destination, rows that do not overlap (all heads of a token before the next
// token, or all tokens of a head before the next head).
int check_rows(const void* x, long long tok, long long head, int T, int heads, int d, bool written) {
  if (!aligned16(x) || tok % 8 != 0 || head % 8 != 0) return MALA_ERR_UNSUPPORTED;
  if (tok < 0 || head < 0) return MALA_ERR_INVALID_ARG;
  if (static_cast<double>(T - 1) * tok + static_cast<double>(heads - 1) * head >= static_cast<double>(1ll << 40))
    return MALA_ERR_UNSUPPORTED;
  if (written) {
    if ((T > 1 && tok < d) || (heads > 1 && head < d)) return MALA_ERR_INVALID_ARG;
    if (T > 1 && heads > 1 && tok < (heads - 1) * head + d && head < (T - 1) * tok + d) return MALA_ERR_INVALID_ARG;
  }
  return MALA_OK;
}

template <int D, bool kAdjacent, bool kPaged>
int launch_rope_u(const mala::RopeParams& p, int rows, cudaStream_t st) {
  constexpr int SLOTS = mala::kRopeThreads / (D / 16);
  const long long slots = static_cast<long long>(p.T) * p.groups;
  const long long grid = (slots + SLOTS - 1) / SLOTS;
  if (grid >= (1ll << 31)) return MALA_ERR_UNSUPPORTED;
  const unsigned g = static_cast<unsigned>(grid);
  if (rows >= 4) mala::mala_rope_kernel<D, kAdjacent, kPaged, 4><<<g, mala::kRopeThreads, 0, st>>>(p);
  else if (rows >= 2) mala::mala_rope_kernel<D, kAdjacent, kPaged, 2><<<g, mala::kRopeThreads, 0, st>>>(p);
  else mala::mala_rope_kernel<D, kAdjacent, kPaged, 1><<<g, mala::kRopeThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

template <bool kPaged>
int launch_rope(mala::RopeParams p, int d, bool adjacent, cudaStream_t st) {
  // Rows (heads) per thread: one while the rows of all tokens do not fill the
  // GPU (768 threads to an SM, by their registers), then up to 12 so that a
  // thread's sines serve several heads, in whole groups of the loads a thread has
  // in flight (1, 2, 4, 8, 12). 8K tokens of 48 heads: 37.5 us with 12 rows a
  // thread, 41 with 4, 72 with 1; 16 rows are no better (32K tokens 127 against 124).
  const long long rows = p.heads[0] + p.heads[1] + p.heads[2];
  const long long threads = p.T * rows * (d / 16);
  const long long fill = static_cast<long long>(sm_count()) * 768;
  int per = static_cast<int>(std::min<long long>(std::max<long long>(threads / fill, 1), 12));
  per = per >= 4 ? per / 4 * 4 : per >= 2 ? 2 : 1;
  p.groups = static_cast<int>((rows + per - 1) / per);
  if (d == 128)
    return adjacent ? launch_rope_u<128, true, kPaged>(p, per, st) : launch_rope_u<128, false, kPaged>(p, per, st);
  return adjacent ? launch_rope_u<64, true, kPaged>(p, per, st) : launch_rope_u<64, false, kPaged>(p, per, st);
}

// ------------------------------------------------------------------ evict
// Whether two arrays (their bytes) share any.
bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<unsigned long long>(nb) && y < x + static_cast<unsigned long long>(na);
}

template <int C, int kKeep>
int launch_select_keep(const mala::EvictParams& p, cudaStream_t st) {
  auto kern = mala::mala_evict_select_kernel<C, kKeep>;
  constexpr int kBytes = kKeep * mala::kEvictThreads * 4;
  // (beside the 24 KB of counts it passes the 48 KB that need no leave)
  if (kBytes > 20 * 1024 && set_smem(kern, kBytes) != MALA_OK) return MALA_ERR_CUDA;
  if constexpr (C == 1) {
    kern<<<static_cast<unsigned>(p.B) * p.Hkv, mala::kEvictThreads, kBytes, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * C);
  cfg.blockDim = dim3(mala::kEvictThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return MALA_ERR_CUDA;
  }
  return MALA_OK;
}

template <int C>
int launch_select(const mala::EvictParams& p, cudaStream_t st) {
  // masses a thread meets in the longest row
  const int each = (p.ld + C * mala::kEvictThreads - 1) / (C * mala::kEvictThreads);
  // (keys kept for 1, 4, 16 or 32 of them: 1K rows of masses 3.7 us with one, 4.0 with room for four;
  // 64 rows of 64K masses 18.4 us with 32, 48 with every pass reading the masses again)
  if constexpr (C == 1)  // (a cluster's threads meet two at least: it is chosen for more than 1024 C masses)
    if (each <= 1) return launch_select_keep<C, 1>(p, st);
  if (each <= 4) return launch_select_keep<C, 4>(p, st);
  if (each <= 16) return launch_select_keep<C, 16>(p, st);
  if (each <= 32) return launch_select_keep<C, 32>(p, st);
  return launch_select_keep<C, 0>(p, st);
}

}  // namespace

extern "C" {

int mala_rope(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* v_out,
              const int64_t* strides, const int32_t* positions, const float* inv_freq, int T, int Hq, int Hkv, int d,
              int rotary_dim, const int32_t* sections, int n_axes, unsigned flags, void* stream) {
  int rc = check_rope(T, Hq, Hkv, d, rotary_dim, flags,
                      MALA_ROPE_ADJACENT | MALA_ROPE_CYCLIC | MALA_ROPE_INVERSE);
  if (rc != MALA_OK) return rc;
  mala::RopeParams p = {};
  rc = rope_axes(rotary_dim, sections, n_axes, (flags & MALA_ROPE_CYCLIC) != 0, &p.axis_lo, &p.axis_hi);
  if (rc != MALA_OK) return rc;
  if (!strides) return MALA_ERR_INVALID_ARG;
  if (T == 0) return MALA_OK;
  if (!positions || !inv_freq) return MALA_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr) || (k != nullptr) != (k_out != nullptr) ||
      (v != nullptr) != (v_out != nullptr) || (!q && !k && !v))
    return MALA_ERR_INVALID_ARG;
  const void* src[3] = {q, k, v};
  void* dst[3] = {q_out, k_out, v_out};
  for (int w = 0; w < 3; ++w) {
    if (!src[w]) continue;
    p.heads[w] = w == 0 ? Hq : Hkv;
    p.src[w] = static_cast<const uint16_t*>(src[w]);
    p.dst[w] = static_cast<uint16_t*>(dst[w]);
    p.src_tok[w] = strides[2 * w];
    p.src_head[w] = strides[2 * w + 1];
    p.dst_tok[w] = strides[6 + 2 * w];
    p.dst_head[w] = strides[6 + 2 * w + 1];
    rc = check_rows(src[w], p.src_tok[w], p.src_head[w], T, p.heads[w], d, false);
    if (rc == MALA_OK) rc = check_rows(dst[w], p.dst_tok[w], p.dst_head[w], T, p.heads[w], d, true);
    if (rc != MALA_OK) return rc;
  }
  p.pos = positions;
  p.inv_freq = inv_freq;
  p.T = T;
  p.pairs = rotary_dim / 2;
  p.sign = (flags & MALA_ROPE_INVERSE) ? -1.f : 1.f;
  return launch_rope<false>(p, d, (flags & MALA_ROPE_ADJACENT) != 0, static_cast<cudaStream_t>(stream));
}

int mala_rope_append(const void* q, const void* k, const void* v, void* q_out, const int64_t* strides,
                     const int32_t* positions, const float* inv_freq, void* k_pages, void* v_pages,
                     const int32_t* block_table, const int32_t* seqlens_k, const int32_t* cu_seqlens, int num_seqs,
                     int T, int Hq, int Hkv, int num_pages, int page_size, int max_pages_per_seq, int d,
                     int rotary_dim, const int32_t* sections, int n_axes, unsigned flags, void* stream) {
  int rc = check_rope(T, Hq, Hkv, d, rotary_dim, flags, MALA_ROPE_ADJACENT | MALA_ROPE_CYCLIC);
  if (rc != MALA_OK) return rc;
  mala::RopeParams p = {};
  rc = rope_axes(rotary_dim, sections, n_axes, (flags & MALA_ROPE_CYCLIC) != 0, &p.axis_lo, &p.axis_hi);
  if (rc != MALA_OK) return rc;
  if (!strides || num_seqs < 1 || num_pages < 1 || max_pages_per_seq < 1) return MALA_ERR_INVALID_ARG;
  if (page_size != 64 && page_size != 128) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages_per_seq) * page_size >= (1ll << 31) ||
      static_cast<long long>(num_pages) * page_size >= (1ll << 31) ||
      static_cast<long long>(num_pages) * page_size * Hkv * d >= (1ll << 40))
    return MALA_ERR_UNSUPPORTED;
  if (!cu_seqlens && T % num_seqs != 0) return MALA_ERR_INVALID_ARG;
  if (T == 0) return MALA_OK;
  if (!k || !v || !k_pages || !v_pages || !positions || !inv_freq || !block_table || !seqlens_k ||
      (q != nullptr) != (q_out != nullptr))
    return MALA_ERR_INVALID_ARG;
  const void* src[3] = {q, k, v};
  void* dst[3] = {q_out, k_pages, v_pages};
  for (int w = 0; w < 3; ++w) {
    if (!src[w]) continue;
    p.heads[w] = w == 0 ? Hq : Hkv;
    p.src[w] = static_cast<const uint16_t*>(src[w]);
    p.dst[w] = static_cast<uint16_t*>(dst[w]);
    p.src_tok[w] = strides[2 * w];
    p.src_head[w] = strides[2 * w + 1];
    rc = check_rows(src[w], p.src_tok[w], p.src_head[w], T, p.heads[w], d, false);
    if (rc != MALA_OK) return rc;
    if (w == 0) {
      p.dst_tok[0] = strides[6];
      p.dst_head[0] = strides[7];
      rc = check_rows(q_out, p.dst_tok[0], p.dst_head[0], T, Hq, d, true);
      if (rc != MALA_OK) return rc;
    } else if (!aligned16(dst[w])) {
      return MALA_ERR_UNSUPPORTED;
    }
  }
  p.pos = positions;
  p.inv_freq = inv_freq;
  p.T = T;
  p.pairs = rotary_dim / 2;
  p.sign = 1.f;
  p.block_table = block_table;
  p.seqlens = seqlens_k;
  p.cu = cu_seqlens;
  p.num_seqs = num_seqs;
  p.per_seq = cu_seqlens ? 0 : T / num_seqs;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  p.page_shift = page_size == 64 ? 6 : 7;
  p.status = status_ptr();
  if (!p.status) return MALA_ERR_CUDA;
  return launch_rope<true>(p, d, (flags & MALA_ROPE_ADJACENT) != 0, static_cast<cudaStream_t>(stream));
}

int mala_evict_select(const float* mass, const int32_t* seqlens_k, int32_t* index, int32_t* new_seqlens,
                      float* mass_out, int B, int Hkv, int ld_mass, int budget, int n_sink, int n_recent,
                      int ld_mass_out, void* stream) {
  if (!mass || !seqlens_k || !index || !new_seqlens) return MALA_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || ld_mass < 1 || budget < 1 || n_sink < 0 || n_recent < 0) return MALA_ERR_INVALID_ARG;
  if (static_cast<long long>(n_sink) + n_recent > budget) return MALA_ERR_INVALID_ARG;
  if (new_seqlens == seqlens_k || mass_out == mass) return MALA_ERR_INVALID_ARG;
  if (mass_out && ld_mass_out < budget) return MALA_ERR_INVALID_ARG;
  if (!aligned16(mass) || !aligned16(index) || (mass_out && !aligned16(mass_out))) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv >= (1ll << 24) || ld_mass > (1 << 30) || budget > (1 << 30) ||
      (mass_out && ld_mass_out > (1 << 30)))
    return MALA_ERR_UNSUPPORTED;
  // what one block writes, another may still read
  const long long rows = static_cast<long long>(B) * Hkv;
  if (overlap(new_seqlens, 4ll * B, seqlens_k, 4ll * B) ||
      (mass_out && overlap(mass_out, 4 * rows * ld_mass_out, mass, 4 * rows * ld_mass)))
    return MALA_ERR_INVALID_ARG;
  mala::EvictParams p = {};
  p.mass = mass;
  p.seqlens = seqlens_k;
  p.index = index;
  p.new_lens = new_seqlens;
  p.mass_out = mass_out;
  p.B = B;
  p.Hkv = Hkv;
  p.ld = ld_mass;
  p.budget = budget;
  p.n_sink = n_sink;
  p.n_recent = n_recent;
  p.ld_out = ld_mass_out;
  p.status = status_ptr();
  if (!p.status) return MALA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // CTAs per row of masses: as many as keep all rows on the GPU at once (one
  // CTA to an SM), but no more than leave each 2K masses
  int cluster = 1;
  while (cluster < 8 && rows * cluster * 2 <= sm_count() && ld_mass > 2048 * cluster) cluster *= 2;
  switch (cluster) {
    case 1: return launch_select<1>(p, st);
    case 2: return launch_select<2>(p, st);
    case 4: return launch_select<4>(p, st);
    default: return launch_select<8>(p, st);
  }
}

int mala_evict_gather(const void* k_pages, const void* v_pages, const int32_t* block_table, const int32_t* index,
                      const int32_t* new_seqlens, void* k_out_pages, void* v_out_pages, const int32_t* out_table,
                      int B, int Hkv, int budget, int num_pages, int num_out_pages, int page_size,
                      int max_pages_per_seq, int max_out_pages_per_seq, int d, void* stream) {
  const int rc = mala::check_gather(k_pages, v_pages, block_table, index, new_seqlens, k_out_pages, v_out_pages,
                                    out_table, B, Hkv, budget, num_pages, num_out_pages, page_size, max_pages_per_seq,
                                    max_out_pages_per_seq, d);
  if (rc != MALA_OK) return rc;
  mala::GatherParams p = {};
  p.k = static_cast<const uint4*>(k_pages);
  p.v = static_cast<const uint4*>(v_pages);
  p.k_out = static_cast<uint4*>(k_out_pages);
  p.v_out = static_cast<uint4*>(v_out_pages);
  p.block_table = block_table;
  p.out_table = out_table;
  p.index = index;
  p.lens = new_seqlens;
  p.B = B;
  p.Hkv = Hkv;
  p.budget = budget;
  p.num_pages = num_pages;
  p.max_pages = max_pages_per_seq;
  p.num_out_pages = num_out_pages;
  p.max_out_pages = max_out_pages_per_seq;
  p.page_shift = page_size == 64 ? 6 : 7;
  p.status = status_ptr();
  if (!p.status) return MALA_ERR_CUDA;
  const int per_block = mala::kGatherThreads / (d / 8) * mala::kGatherRows;
  const long long gx = (static_cast<long long>(budget) * Hkv + per_block - 1) / per_block;
  if (gx >= (1ll << 31)) return MALA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(B));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto kern = d == 128 ? mala::mala_evict_gather_kernel<128> : mala::mala_evict_gather_kernel<64>;
  return launch_second(kern, grid, mala::kGatherThreads, st, p);  // usually mala_evict_select's second half
}

}  // extern "C"
