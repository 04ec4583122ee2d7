// mala_decode_mass_api.cu -- C ABI of the paged decode that also collects each
// key's attention weight (host side; the kernels are included below).
#include <algorithm>

#include "mala_decode.cuh"
#include "mala_decode_mass.cuh"
#include "mala_host.h"

using namespace mala::host;

namespace {

struct Layout {
  size_t scores, o_part, lse_part, total;
};

Layout layout(int B, int Hq, long long keys, int d, int n_splits) {
  Layout w;
  const size_t rows = static_cast<size_t>(B) * Hq;
  w.scores = 0;
  w.o_part = align256(rows * keys * 4);
  w.lse_part = w.o_part + align256(rows * n_splits * d * 4);
  w.total = w.lse_part + align256(rows * n_splits * 4);
  return w;
}

template <int D, int BK, int GP, bool G>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const mala::DecParams& p, cudaStream_t st) {
  using Lay = mala::DecLayout<D, BK, GP>;
  auto kern = mala::mala_decode_split_kernel<D, BK, GP, G, true, true>;
  if (set_smem(kern, Lay::ALLOC_BYTES) != MALA_OK) return MALA_ERR_CUDA;
  kern<<<static_cast<unsigned>(p.B) * p.Hkv * p.n_splits, 320, Lay::ALLOC_BYTES, st>>>(mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

template <int D, int BK, bool G>
int launch_g(const CUtensorMap& mk, const CUtensorMap& mv, const mala::DecParams& p, cudaStream_t st) {
  if (p.G <= 1) return launch<D, BK, 1, G>(mk, mv, p, st);
  if (p.G <= 2) return launch<D, BK, 2, G>(mk, mv, p, st);
  if (p.G <= 4) return launch<D, BK, 4, G>(mk, mv, p, st);
  return launch<D, BK, 8, G>(mk, mv, p, st);
}

template <int D, int BK>
int launch_gate(bool gate, const CUtensorMap& mk, const CUtensorMap& mv, const mala::DecParams& p, cudaStream_t st) {
  return gate ? launch_g<D, BK, true>(mk, mv, p, st) : launch_g<D, BK, false>(mk, mv, p, st);
}

}  // namespace

extern "C" {

size_t mala_decode_mass_workspace_size(int B, int Hq, int d, int page_size, int max_pages_per_seq, int n_splits) {
  if (B < 1 || Hq < 1 || max_pages_per_seq < 1 || n_splits < 1 || (d != 64 && d != 128) ||
      (page_size != 64 && page_size != 128))
    return 0;
  return layout(B, Hq, static_cast<long long>(max_pages_per_seq) * page_size, d, n_splits).total;
}

int mala_decode_paged_mass(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                           const int32_t* seqlens_k, void* o, float* lse, const float* mass_in, float* mass_out,
                           int B, int Hq, int Hkv, int num_pages, int page_size, int max_pages_per_seq, int d,
                           float scale, float tau, float decay, int ld_mass, int n_splits, void* workspace,
                           size_t workspace_bytes, int32_t* kept_tiles, uint8_t* keep_map, void* stream) {
  if (!block_table || !seqlens_k || !mass_out || num_pages < 1 || max_pages_per_seq < 1) return MALA_ERR_INVALID_ARG;
  if (page_size != 64 && page_size != 128) return MALA_ERR_UNSUPPORTED;
  const long long max_lk = static_cast<long long>(max_pages_per_seq) * page_size;
  if (max_lk >= (1ll << 31) || static_cast<long long>(num_pages) * page_size >= (1ll << 31))
    return MALA_ERR_UNSUPPORTED;
  const int Lk = static_cast<int>(max_lk);
  int rc = check_decode_args(q, k_pages, v_pages, o, lse, B, Hq, Hkv, Lk, d, scale, tau, page_size, n_splits,
                             kept_tiles);
  if (rc != MALA_OK) return rc;
  if (!(decay >= 0.f) || !std::isfinite(decay) || ld_mass < Lk) return MALA_ERR_INVALID_ARG;
  if (!aligned16(mass_out) || (mass_in && !aligned16(mass_in))) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size * Hkv * d >= (1ll << 40)) return MALA_ERR_UNSUPPORTED;
  if (n_splits == 0) n_splits = mala_decode_default_splits(B, Hkv, Lk, page_size);
  if (n_splits > 65535) return MALA_ERR_UNSUPPORTED;
  const Layout lay = layout(B, Hq, max_lk, d, n_splits);
  if (!workspace || workspace_bytes < lay.total || !aligned256(workspace)) return MALA_ERR_WORKSPACE;
  const int key_blocks = (ld_mass + mala::kDecMassKeys - 1) / mala::kDecMassKeys;
  const int merge_blocks = (B * Hq + mala::kDecMassThreads / 32 - 1) / (mala::kDecMassThreads / 32);
  const long long blocks = merge_blocks + static_cast<long long>(B) * Hkv * key_blocks;
  if (blocks >= (1ll << 31) || static_cast<long long>(B) * Hkv * n_splits >= (1ll << 31)) return MALA_ERR_UNSUPPORTED;
  CUtensorMap mk, mv;
  if (!make_bshd_map(&mk, k_pages, num_pages, page_size, Hkv, d, page_size) ||
      !make_bshd_map(&mv, v_pages, num_pages, page_size, Hkv, d, page_size))
    return MALA_ERR_CUDA;
  unsigned* status = status_ptr();
  if (!status) return MALA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);

  mala::DecParams p = {};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lk = Lk; p.G = Hq / Hkv;
  p.nk = max_pages_per_seq;
  p.n_splits = n_splits;
  p.tiles_per_split = (p.nk + n_splits - 1) / n_splits;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.log2_tau = tau > 0.f ? std::log2(tau) : 0.f;
  p.seqlens = seqlens_k;
  p.block_table = block_table;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  p.q = static_cast<const uint16_t*>(q);
  p.o_part = reinterpret_cast<float*>(ws + lay.o_part);
  p.lse_part = reinterpret_cast<float*>(ws + lay.lse_part);
  p.kept_tiles = kept_tiles;
  p.keep_map = keep_map;
  p.status = status;
  p.wait_ns = wait_limit_ns();
  p.stall_tile = stall_tile();
  p.scores = reinterpret_cast<float*>(ws + lay.scores);
  if (cudaMemsetAsync(kept_tiles, 0, sizeof(int32_t) * B * Hq, st) != cudaSuccess) return MALA_ERR_CUDA;
  const bool gate = tau > 0.f;
  if (d == 128 && page_size == 128) rc = launch_gate<128, 128>(gate, mk, mv, p, st);
  else if (d == 64 && page_size == 128) rc = launch_gate<64, 128>(gate, mk, mv, p, st);
  else if (d == 128) rc = launch_gate<128, 64>(gate, mk, mv, p, st);
  else rc = launch_gate<64, 64>(gate, mk, mv, p, st);
  if (rc != MALA_OK) return rc;

  mala::DecMassParams m = {};
  m.o_part = p.o_part;
  m.lse_part = p.lse_part;
  m.o = static_cast<uint16_t*>(o);
  m.lse = lse;
  m.scores = p.scores;
  m.seqlens = seqlens_k;
  m.mass_in = mass_in;
  m.mass_out = mass_out;
  m.B = B; m.Hq = Hq; m.Hkv = Hkv; m.G = p.G;
  m.n_splits = n_splits;
  m.ld = ld_mass;
  m.ld_scores = Lk;
  m.max_len = Lk;
  m.merge_blocks = merge_blocks;
  m.key_blocks = key_blocks;
  m.decay = decay;
  if (d == 128)
    mala::mala_decode_mass_kernel<128><<<static_cast<unsigned>(blocks), mala::kDecMassThreads, 0, st>>>(m);
  else
    mala::mala_decode_mass_kernel<64><<<static_cast<unsigned>(blocks), mala::kDecMassThreads, 0, st>>>(m);
  return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

}  // extern "C"
