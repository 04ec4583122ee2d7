// mala_decode_mass_api.cu -- C ABI of the paged decode that also collects each
// key's attention weight (host side; the kernels are included below).
#include <algorithm>
#include <atomic>

#include "mala_decode.cuh"
#include "mala_decode_mass.cuh"
#include "mala_host.h"

using namespace mala::host;

namespace {

struct Layout {
  size_t scores, o_part, lse_part, plan, total;
  int slots;  // partial results of a (b, query head)
};

// CTAs of the ungated kernel: two to an SM.
int flat_grid() { return 2 * sm_count(); }

// n_splits > 0: the gated kernel's partials; 0: the ungated kernel's. Its runs are at
// least kFlatLeastRun tiles and at least an even share of all tiles, of which one
// (b, KV head) holds at most a 1 / Hkv part, so it meets at most that many runs.
Layout layout(int B, int Hq, int Hkv, long long keys, int d, int n_splits) {
  Layout w;
  const long long tiles = (keys + mala::kFlatTile - 1) / mala::kFlatTile;
  const long long shared = (flat_grid() + Hkv - 1) / Hkv;
  w.slots = n_splits > 0 ? n_splits
                         : static_cast<int>(std::min((tiles + mala::kFlatLeastRun - 1) / mala::kFlatLeastRun, shared)) + 1;
  const size_t rows = static_cast<size_t>(B) * Hq;
  w.scores = 0;
  w.o_part = align256(rows * keys * 4);
  w.lse_part = w.o_part + align256(rows * w.slots * d * 4);
  w.plan = w.lse_part + align256(rows * w.slots * 4);
  w.total = w.plan + align256((static_cast<size_t>(B) + 1) * 4);
  return w;
}

template <int D>
int launch_flat(const CUtensorMap& mk, const CUtensorMap& mv, const mala::FlatParams& p, cudaStream_t st) {
  using Lay = mala::FlatLayout<D>;
  auto kern = mala::mala_decode_flat_kernel<D, false>;
  if (set_smem(kern, Lay::ALLOC_BYTES) != MALA_OK) return MALA_ERR_CUDA;
  kern<<<flat_grid(), mala::kFlatThreads, Lay::ALLOC_BYTES, st>>>(mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

// Readies the kernel of short caches for clusters of this size. The limit on shared memory is
// the kernel's, shared by all host threads: always the most any call takes, never this call's
// size, or another thread's smaller call could lower it between here and the launch.
template <int D>
int ready_short(int cluster) {
  auto kern = mala::mala_decode_flat_kernel<D, true>;
  if (set_smem(kern, mala::FlatLayout<D>::short_bytes(kMaxDecodeGroup, mala::kShortTiles)) != MALA_OK)
    return MALA_ERR_CUDA;
  if (cluster > 8 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return MALA_ERR_CUDA;
  return MALA_OK;
}

template <int D>
cudaLaunchConfig_t short_config(unsigned grid, int cluster, int bytes, cudaLaunchAttribute* attr, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(mala::kFlatThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of the short kernel that the current device holds at once (0: none, or the
// question failed), with two of its CTAs to an SM (`pair`) or one. Asked once per device,
// for the most shared memory that either takes.
template <int D>
int short_room(int cluster, bool pair) {
  using Lay = mala::FlatLayout<D>;
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][2][5];  // clusters + 1, by log2 of the size
  int dev = 0, lg = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  while ((1 << lg) < cluster) ++lg;
  std::atomic<int>* slot = dev < kDevices ? &known[dev][pair ? 1 : 0][lg] : nullptr;
  if (slot && slot->load() > 0) return slot->load() - 1;
  cudaLaunchAttribute attr;
  constexpr int kMost = Lay::short_bytes(kMaxDecodeGroup, mala::kShortTiles);
  const int bytes = pair ? std::min(Lay::PAIR_BYTES, kMost) : kMost;
  const cudaLaunchConfig_t cfg = short_config<D>(cluster, cluster, bytes, &attr, nullptr);
  int n = 0;
  if (ready_short<D>(cluster) != MALA_OK ||
      cudaOccupancyMaxActiveClusters(&n, mala::mala_decode_flat_kernel<D, true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (slot) slot->store(n + 1);
  return n;
}

template <int D>
int pick_short(long long units, long long keys, int G) {
  using Lay = mala::FlatLayout<D>;
  const long long tiles = (keys + mala::kFlatTile - 1) / mala::kFlatTile;
  return mala::short_cluster(units, tiles, 2ll * sm_count(), [&](int c, int each) {
    return short_room<D>(c, Lay::short_bytes(G, each) <= Lay::PAIR_BYTES);
  });
}

template <int D>
int launch_short(const CUtensorMap& mk, const CUtensorMap& mv, mala::FlatParams p, cudaStream_t st) {
  using Lay = mala::FlatLayout<D>;
  const int tiles = (p.max_len + mala::kFlatTile - 1) / mala::kFlatTile, each = (tiles + p.cluster - 1) / p.cluster;
  p.pitch = Lay::short_pitch(each);
  if (ready_short<D>(p.cluster) != MALA_OK) return MALA_ERR_CUDA;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = short_config<D>(static_cast<unsigned>(p.B) * p.Hkv * p.cluster, p.cluster,
                                                 Lay::short_bytes(p.G, each), &attr, st);
  if (cudaLaunchKernelEx(&cfg, mala::mala_decode_flat_kernel<D, true>, mk, mv, p) != cudaSuccess) {
    cudaGetLastError();
    return MALA_ERR_CUDA;
  }
  return MALA_OK;
}

template <int D>
int launch_mass(const mala::DecMassParams& m, unsigned grid, cudaStream_t st) {
  auto kern = m.G <= 1   ? mala::mala_decode_mass_kernel<D, 1>
              : m.G <= 2 ? mala::mala_decode_mass_kernel<D, 2>
              : m.G <= 4 ? mala::mala_decode_mass_kernel<D, 4>
                         : mala::mala_decode_mass_kernel<D, 8>;
  return launch_second(kern, dim3(grid), mala::kDecMassThreads, st, m);
}

template <int D, int BK, int GP>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const mala::DecParams& p, cudaStream_t st) {
  using Lay = mala::DecLayout<D, BK, GP>;
  auto kern = mala::mala_decode_split_kernel<D, BK, GP, true, true, true>;
  if (set_smem(kern, Lay::ALLOC_BYTES) != MALA_OK) return MALA_ERR_CUDA;
  kern<<<static_cast<unsigned>(p.B) * p.Hkv * p.n_splits, 320, Lay::ALLOC_BYTES, st>>>(mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

template <int D, int BK>
int launch_g(const CUtensorMap& mk, const CUtensorMap& mv, const mala::DecParams& p, cudaStream_t st) {
  if (p.G <= 1) return launch<D, BK, 1>(mk, mv, p, st);
  if (p.G <= 2) return launch<D, BK, 2>(mk, mv, p, st);
  if (p.G <= 4) return launch<D, BK, 4>(mk, mv, p, st);
  return launch<D, BK, 8>(mk, mv, p, st);
}

}  // namespace

extern "C" {

size_t mala_decode_mass_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages_per_seq,
                                       int n_splits) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages_per_seq < 1 || n_splits < 0 || (d != 64 && d != 128) ||
      (page_size != 64 && page_size != 128))
    return 0;
  return layout(B, Hq, Hkv, static_cast<long long>(max_pages_per_seq) * page_size, d, n_splits).total;
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
  if (ld_mass > (1 << 30)) return MALA_ERR_UNSUPPORTED;  // keys are counted in 32 bits, in blocks past the end too
  if (static_cast<long long>(num_pages) * page_size * Hkv * d >= (1ll << 40)) return MALA_ERR_UNSUPPORTED;
  // without a gate the tiles are dealt evenly over the GPU, whatever n_splits says
  const bool gate = tau > 0.f;
  if (!gate) n_splits = 0;
  else if (n_splits == 0) n_splits = mala_decode_default_splits(B, Hkv, Lk, page_size);
  if (n_splits > 65535) return MALA_ERR_UNSUPPORTED;
  if (B * (max_lk / mala::kFlatTile) * Hkv >= (1ll << 31)) return MALA_ERR_UNSUPPORTED;
  const Layout lay = layout(B, Hq, Hkv, max_lk, d, n_splits);
  if (!workspace || workspace_bytes < lay.total || !aligned256(workspace)) return MALA_ERR_WORKSPACE;
  const int key_blocks = (ld_mass + mala::kDecMassKeys - 1) / mala::kDecMassKeys;
  const int merge_blocks = (B * Hq + mala::kDecMassThreads / 32 - 1) / (mala::kDecMassThreads / 32);
  const long long blocks = merge_blocks + static_cast<long long>(B) * Hkv * key_blocks;
  if (blocks >= (1ll << 31) || static_cast<long long>(B) * Hkv * n_splits >= (1ll << 31)) return MALA_ERR_UNSUPPORTED;
  const int rows = gate ? page_size : mala::kFlatTile;
  CUtensorMap mk, mv;
  if (!make_bshd_map(&mk, k_pages, num_pages, page_size, Hkv, d, rows) ||
      !make_bshd_map(&mv, v_pages, num_pages, page_size, Hkv, d, rows))
    return MALA_ERR_CUDA;
  unsigned* status = status_ptr();
  if (!status) return MALA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);

  float* scores = reinterpret_cast<float*>(ws + lay.scores);
  float* o_part = reinterpret_cast<float*>(ws + lay.o_part);
  float* lse_part = reinterpret_cast<float*>(ws + lay.lse_part);
  int* plan = reinterpret_cast<int*>(ws + lay.plan);
  const int G = Hq / Hkv;
  if (gate) {
    mala::DecParams p = {};
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lk = Lk; p.G = G;
    p.nk = max_pages_per_seq;
    p.n_splits = n_splits;
    p.tiles_per_split = (p.nk + n_splits - 1) / n_splits;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.log2_tau = std::log2(tau);
    p.seqlens = seqlens_k;
    p.block_table = block_table;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    p.q = static_cast<const uint16_t*>(q);
    p.o_part = o_part;
    p.lse_part = lse_part;
    p.kept_tiles = kept_tiles;
    p.keep_map = keep_map;
    p.status = status;
    p.wait_ns = wait_limit_ns();
    p.stall_tile = stall_tile();
    p.scores = scores;
    if (cudaMemsetAsync(kept_tiles, 0, sizeof(int32_t) * B * Hq, st) != cudaSuccess) return MALA_ERR_CUDA;
    if (d == 128 && page_size == 128) rc = launch_g<128, 128>(mk, mv, p, st);
    else if (d == 64 && page_size == 128) rc = launch_g<64, 128>(mk, mv, p, st);
    else if (d == 128) rc = launch_g<128, 64>(mk, mv, p, st);
    else rc = launch_g<64, 64>(mk, mv, p, st);
  } else {
    mala::FlatParams p = {};
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = G;
    p.seqlens = seqlens_k;
    p.block_table = block_table;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    p.page_shift = page_size == 64 ? 6 : 7;
    p.max_len = Lk;
    p.q = static_cast<const uint16_t*>(q);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = status;
    p.wait_ns = wait_limit_ns();
    p.stall_tile = stall_tile();
    const long long units = static_cast<long long>(B) * Hkv;
    p.cluster = d == 128 ? pick_short<128>(units, max_lk, G) : pick_short<64>(units, max_lk, G);
    if (p.cluster > 0) {
      p.o = static_cast<uint16_t*>(o);
      p.lse = lse;
      p.mass_in = mass_in;
      p.mass_out = mass_out;
      p.kept_tiles = kept_tiles;
      p.keep_map = keep_map;
      p.decay = decay;
      p.ld = ld_mass;
      return d == 128 ? launch_short<128>(mk, mv, p, st) : launch_short<64>(mk, mv, p, st);
    }
    p.o_part = o_part;
    p.lse_part = lse_part;
    p.scores = scores;
    p.plan = plan;
    p.slots = lay.slots;
    rc = d == 128 ? launch_flat<128>(mk, mv, p, st) : launch_flat<64>(mk, mv, p, st);
  }
  if (rc != MALA_OK) return rc;

  mala::DecMassParams m = {};
  m.o_part = o_part;
  m.lse_part = lse_part;
  m.o = static_cast<uint16_t*>(o);
  m.lse = lse;
  m.scores = scores;
  m.seqlens = seqlens_k;
  m.mass_in = mass_in;
  m.mass_out = mass_out;
  m.plan = gate ? nullptr : plan;
  m.kept_tiles = kept_tiles;
  m.keep_map = keep_map;
  m.B = B; m.Hq = Hq; m.Hkv = Hkv; m.G = G;
  m.slots = lay.slots;
  m.ld = ld_mass;
  m.max_len = Lk;
  m.max_pages = max_pages_per_seq;
  m.page = page_size;
  m.merge_blocks = merge_blocks;
  m.key_blocks = key_blocks;
  m.decay = decay;
  const unsigned grid = static_cast<unsigned>(blocks);
  return d == 128 ? launch_mass<128>(m, grid, st) : launch_mass<64>(m, grid, st);
}

}  // extern "C"
