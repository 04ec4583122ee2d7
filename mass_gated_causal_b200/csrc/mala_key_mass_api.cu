// mala_key_mass_api.cu -- C ABI of the attention weight that a prompt's keys
// collected (host side; the kernels are included below).
#include <algorithm>

#include "mala_host.h"
#include "mala_key_mass.cuh"
#include "mala_key_mass_window.cuh"

using namespace mala::host;

namespace {

// Columns of Q that mala_key_mass_window_kernel holds (rows of all heads, each
// head's rounded up to 8), or 0 if it does not take the call.
int window_cols(int G, int Lq, int window) {
  const int rows = window > 0 ? std::min(window, Lq) : Lq;
  const int pad = (std::min(rows, 512) + 7) & ~7;
  return pad <= 256 && static_cast<long long>(pad) * G <= mala::kWinMaxCols ? pad * G : 0;
}

struct Plan {
  int chunk_q, n_chunks;  // query tiles a CTA takes; chunks of the longest walk
  int blocks;             // key blocks of the longest sequence
  size_t part_bytes;
};

// How the walks over the query tiles are cut. `units` (b, KV head) pairs, in
// units of the longest sequence; `slots` of them have room in the partials.
//
// A CTA's walk is one key block's query tiles. While the longest walk is at most
// 0.6 of an SM's share of all walks, the walks are whole: they start longest
// first and the shorter ones even the SMs out. Above that, an SM that got the
// longest walk would still run when the others are done, so the walks are cut
// into chunks of half a share: 8K keys, 8 heads over 2 KV heads, 93 us against 288
// with whole walks. Chunks of a quarter share cost more in starts than they even
// out (105 us there; 8K keys of 16 heads, which the rule leaves whole, 152 us, 165 in
// halves of a share and 174 in quarters).
Plan plan(double units, long long slots, int G, int Lq, int Lk, int window) {
  Plan w = {};
  if (window_cols(G, Lq, window) > 0) return w;  // Q fits in shared memory: the keys stream past it
  const int first = window > 0 && window < Lq ? Lq - window : 0;
  const long long n_qt = (Lq - first + 127) / 128;
  w.blocks = (Lk + mala::kMassKeys - 1) / mala::kMassKeys;
  const long long seen = static_cast<long long>(Lk) - Lq + first;  // position of the first row that counts
  const long long whole = std::min<long long>(w.blocks, seen / mala::kMassKeys + 1), rest = w.blocks - whole;
  const double walks =
      static_cast<double>(whole) * n_qt + std::max(0.0, static_cast<double>(rest) * (n_qt - (rest + 1)));
  const double share = walks * units * G / sm_count();
  long long chunk = n_qt;
  if (static_cast<double>(n_qt) * G > 0.6 * share)
    chunk = std::max<long long>(1, std::min<long long>(n_qt, static_cast<long long>(std::ceil(0.5 * share / G))));
  w.chunk_q = static_cast<int>(chunk);
  w.n_chunks = static_cast<int>((n_qt + chunk - 1) / chunk);
  w.part_bytes =
      w.n_chunks > 1 ? align256(static_cast<size_t>(slots) * w.n_chunks * w.blocks * mala::kMassKeys * sizeof(float)) : 0;
  return w;
}

template <int D>
int launch(const CUtensorMap& mq, const mala::KeyMassParams& p, unsigned grid, cudaStream_t st) {
  using Lay = mala::KeyMassLayout<D>;
  auto kern = mala::mala_key_mass_kernel<D>;
  if (set_smem(kern, Lay::ALLOC_BYTES) != MALA_OK) return MALA_ERR_CUDA;
  kern<<<grid, Lay::THREADS, Lay::ALLOC_BYTES, st>>>(mq, p);
  if (cudaGetLastError() != cudaSuccess) return MALA_ERR_CUDA;
  if (p.n_chunks > 1) {
    const dim3 jg(static_cast<unsigned>((p.ld + 255) / 256), static_cast<unsigned>(p.B) * p.Hkv);
    return launch_second(mala::mala_key_mass_join_kernel<256>, jg, 256, st, p);
  }
  return MALA_OK;
}

template <int D, int kCols, int kBlocks>
int launch_window(const CUtensorMap& mq, const CUtensorMap& mk, mala::WinParams wp, cudaStream_t st) {
  using Lay = mala::WinLayout<D, kCols, kBlocks>;
  wp.k_stages = std::min(Lay::MAX_STAGES, (232448 - Lay::bytes(0)) / Lay::K_BYTES);
  const int bytes = Lay::bytes(wp.k_stages);
  auto kern = mala::mala_key_mass_window_kernel<D, kCols, kBlocks>;
  if (set_smem(kern, bytes) != MALA_OK) return MALA_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(wp.m.B) * wp.m.Hkv * wp.parts;
  kern<<<grid, Lay::THREADS, bytes, st>>>(mq, mk, wp);
  return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

template <int D>
int run_window(const void* q, const void* k, const mala::KeyMassParams& p, int cols, cudaStream_t st) {
  const bool packed = p.cu_q != nullptr;
  const int tb = packed ? 1 : p.B, tq = packed ? p.total_q : p.Lq, tk = packed ? p.total_k : p.Lk;
  mala::WinParams wp = {};
  wp.m = p;
  wp.rows_pad = cols / p.G;
  // CTAs per (b, KV head): the count whose waves of one CTA per SM take the fewest key tiles in all
  const long long units = static_cast<long long>(p.B) * p.Hkv, tiles = (p.Lk + 127) / 128;
  const long long sms = sm_count();
  long long best = -1;
  for (long long s = 1; s <= std::min(tiles, sms); ++s) {
    const long long per = (tiles + s - 1) / s, waves = (units * s + sms - 1) / sms;
    const long long cost = waves * (per + 3);  // a CTA's start takes about as long as three tiles
    if (best < 0 || cost < best) {
      best = cost;
      wp.parts = static_cast<int>(s);
    }
  }
  CUtensorMap mq, mk;
  if (!make_bshd_map(&mq, q, tb, tq, p.Hq, D, wp.rows_pad) || !make_bshd_map(&mk, k, tb, tk, p.Hkv, D, 128))
    return MALA_ERR_CUDA;
  if (cols > 384) return launch_window<D, 256, 2>(mq, mk, wp, st);
  if (cols > 256) return launch_window<D, 192, 2>(mq, mk, wp, st);
  if (cols > 192) return launch_window<D, 256, 1>(mq, mk, wp, st);
  if (cols > 128) return launch_window<D, 192, 1>(mq, mk, wp, st);
  if (cols > 64) return launch_window<D, 128, 1>(mq, mk, wp, st);
  return launch_window<D, 64, 1>(mq, mk, wp, st);
}

int check(int B, int Hq, int Hkv, int Lq, int Lk, int d, float scale, int window, float decay, int ld) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk < Lq || Hq % Hkv != 0) return MALA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || !(decay >= 0.f) || !std::isfinite(decay)) return MALA_ERR_INVALID_ARG;
  if (window < 0 || ld < Lk) return MALA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return MALA_ERR_UNSUPPORTED;
  // (LSE / scale and its bf16 parts stay within fp32's range; so does every score)
  if (scale < 0x1p-64f || scale > 0x1p64f) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv >= (1ll << 16) || ld > (1 << 30)) return MALA_ERR_UNSUPPORTED;
  return MALA_OK;
}

int run(const void* q, const void* k, const float* lse, const float* mass_in, float* mass_out, int B, int Hq, int Hkv,
        int Lq, int Lk, int d, float scale, int window, float decay, int ld, void* workspace, size_t workspace_bytes,
        void* stream, const int32_t* cu_q, const int32_t* cu_k, int total_q, int total_k) {
  const void* ptrs[] = {q, k, lse, mass_out};
  for (const void* x : ptrs)
    if (!aligned16(x)) return MALA_ERR_UNSUPPORTED;
  if (mass_in && !aligned16(mass_in)) return MALA_ERR_UNSUPPORTED;
  const bool packed = cu_q != nullptr;
  const long long slots = static_cast<long long>(B) * Hkv;
  const double units = packed ? Hkv * std::max(1.0, static_cast<double>(total_q) / Lq) : static_cast<double>(slots);
  const Plan w = plan(units, slots, Hq / Hkv, Lq, Lk, window);
  if (w.part_bytes > 0 && (!workspace || workspace_bytes < w.part_bytes || !aligned256(workspace)))
    return MALA_ERR_WORKSPACE;
  mala::KeyMassParams p = {};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.Lq = Lq;
  p.Lk = Lk;
  p.window = window;
  p.chunk_q = w.chunk_q;
  p.n_chunks = w.n_chunks;
  // whole walks write the result, up to the end of its rows; chunks write partials
  p.n_blocks = w.n_chunks > 1 ? w.blocks : (ld + mala::kMassKeys - 1) / mala::kMassKeys;
  p.part_ld = w.blocks * mala::kMassKeys;
  p.k = static_cast<const uint16_t*>(k);
  p.lse = lse;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.total_q = total_q;
  p.total_k = total_k;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const double inv = 1.0 / static_cast<double>(scale);
  p.inv_hi = static_cast<float>(inv);
  p.inv_lo = static_cast<float>(inv - p.inv_hi);
  p.decay = decay;
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.ld = ld;
  p.part = static_cast<float*>(workspace);
  p.status = status_ptr();
  if (!p.status) return MALA_ERR_CUDA;
  p.wait_ns = wait_limit_ns();
  p.stall_tile = stall_tile();
  if (const int cols = window_cols(p.G, Lq, window)) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d == 128 ? run_window<128>(q, k, p, cols, st) : run_window<64>(q, k, p, cols, st);
  }
  const long long grid = static_cast<long long>(p.n_blocks) * slots * w.n_chunks;
  if (grid >= (1ll << 31)) return MALA_ERR_UNSUPPORTED;
  CUtensorMap mq;
  if (!make_bshd_map(&mq, q, packed ? 1 : B, packed ? total_q : Lq, Hq, d, 128)) return MALA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned g = static_cast<unsigned>(grid);
  return d == 128 ? launch<128>(mq, p, g, st) : launch<64>(mq, p, g, st);
}

}  // namespace

extern "C" {

size_t mala_key_mass_workspace_size(int B, int Hq, int Hkv, int Lq, int Lk, int window) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk < Lq || Hq % Hkv != 0 || window < 0) return 0;
  const long long slots = static_cast<long long>(B) * Hkv;
  return plan(static_cast<double>(slots), slots, Hq / Hkv, Lq, Lk, window).part_bytes;
}

size_t mala_key_mass_varlen_workspace_size(int num_seqs, int Hq, int Hkv, int max_seqlen_q, int max_seqlen_k,
                                           int total_q, int window) {
  max_seqlen_q = std::min(max_seqlen_q, max_seqlen_k);  // no sequence has more queries than keys
  if (num_seqs < 1 || Hq < 1 || Hkv < 1 || max_seqlen_q < 1 || total_q < 1 || Hq % Hkv != 0 || window < 0) return 0;
  return plan(Hkv * std::max(1.0, static_cast<double>(total_q) / max_seqlen_q), static_cast<long long>(num_seqs) * Hkv,
              Hq / Hkv, max_seqlen_q, max_seqlen_k, window)
      .part_bytes;
}

int mala_key_mass(const void* q, const void* k, const float* lse, const float* mass_in, float* mass_out, int B, int Hq,
                  int Hkv, int Lq, int Lk, int d, float scale, int window, float decay, int ld_mass, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (!q || !k || !lse || !mass_out) return MALA_ERR_INVALID_ARG;
  int rc = check(B, Hq, Hkv, Lq, Lk, d, scale, window, decay, ld_mass);
  if (rc != MALA_OK) return rc;
  if (static_cast<long long>(B) * Lk * Hq * d >= (1ll << 40)) return MALA_ERR_UNSUPPORTED;
  return run(q, k, lse, mass_in, mass_out, B, Hq, Hkv, Lq, Lk, d, scale, window, decay, ld_mass, workspace,
             workspace_bytes, stream, nullptr, nullptr, 0, 0);
}

int mala_key_mass_varlen(const void* q, const void* k, const float* lse, const int32_t* cu_seqlens_q,
                         const int32_t* cu_seqlens_k, const float* mass_in, float* mass_out, int num_seqs,
                         int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int Hq, int Hkv, int d,
                         float scale, int window, float decay, int ld_mass, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (!q || !k || !lse || !mass_out || !cu_seqlens_q || !cu_seqlens_k) return MALA_ERR_INVALID_ARG;
  if (num_seqs < 1 || total_q < 1 || total_k < 1 || max_seqlen_q > total_q || max_seqlen_k > total_k)
    return MALA_ERR_INVALID_ARG;
  max_seqlen_q = std::min(max_seqlen_q, max_seqlen_k);  // no sequence has more queries than keys
  int rc = check(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, scale, window, decay, ld_mass);
  if (rc != MALA_OK) return rc;
  if (static_cast<long long>(std::max(total_q, total_k)) * Hq * d >= (1ll << 40)) return MALA_ERR_UNSUPPORTED;
  return run(q, k, lse, mass_in, mass_out, num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, scale, window, decay,
             ld_mass, workspace, workspace_bytes, stream, cu_seqlens_q, cu_seqlens_k, total_q, total_k);
}

}  // extern "C"
