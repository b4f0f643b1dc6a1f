// Host side of the operators around the layer (include/deco_moe.h, "the block
// around the layer"): argument checks and launches.  Included by api.cu.
#pragma once

#include "norm_kernels.cuh"
#include "q4_kernels.cuh"
#include "sort_kernels.cuh"

namespace deco {
namespace {

bool is_dtype(int d) { return d == DECO_F32 || d == DECO_BF16; }
bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a row stride: 0 stands for the width; nothing below the width (rows would
// overlap)
bool resolve_ld(long long& ld, int width) {
  if (ld == 0) ld = width;
  return ld >= width;
}
bool resolve_ld(long long& ld, int width, const void* p) { return !p || resolve_ld(ld, width); }

// a launch that may start while the kernel before it on the stream leaves
template <typename A>
cudaError_t launch_behind(void (*k)(A), dim3 grid, int threads, const A& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

// ---- norms ------------------------------------------------------------------

struct NormGrid {
  int cl, threads, clusters;
};

// CTAs of at most `most` threads, `per_sm` of which an SM holds with that many
NormGrid norm_grid(int T, int D, int most, int per_sm, bool partial_sums) {
  NormGrid g{};
  g.cl = 1;
  while (g.cl * most * nrm::kCols < D) g.cl *= 2;
  const int width = ((D + g.cl - 1) / g.cl + 7) / 8 * 8;
  g.threads = (width / 8 + 31) / 32 * 32;
  const int sms = num_sms();
  const int per = std::min(32, per_sm * most / g.threads);
  g.clusters = std::max(1, std::min(T, sms * per / g.cl));
  // every cluster leaves a row of partial sums: at least 8 rows each beyond one CTA per SM
  if (partial_sums) g.clusters = std::min(g.clusters, std::max(std::max(1, sms / g.cl), T / 8));
  return g;
}

// most: the dynamic shared memory that any call of this kernel takes.  Every
// call opts in to that much, so that calls of other sizes from other threads
// leave the limit where it is.
template <typename A>
cudaError_t norm_launch(void (*k)(A), const NormGrid& g, int smem, int most, const A& a, cudaStream_t st) {
  // the sums' static buffers count too: opt in well below 48 KB
  const cudaError_t err = most > 40 * 1024 ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most) : cudaSuccess;
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.clusters * g.cl);
  cfg.blockDim = dim3(g.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = g.cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = g.cl > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, a);
}

deco_status_t check_norm(const deco_block_norm_t* s) {
  if (!s || s->T < 0 || s->d_model <= 0 || !is_dtype(s->dtype)) return DECO_ERR_INVALID_ARG;
  if (!(s->rms_eps >= 0.f) || !std::isfinite(s->rms_eps) || !std::isfinite(s->branch_scale)) return DECO_ERR_INVALID_ARG;
  if (s->gate < DECO_GATE_NONE || s->gate > DECO_GATE_FULL) return DECO_ERR_INVALID_ARG;
  if (s->d_model > nrm::kMaxD || s->T > (1 << 20)) return DECO_ERR_UNSUPPORTED;
  return DECO_OK;
}

// the kernels' row strides are bytes in 32 bits
bool stride_ok(long long ld, int dtype) { return ld * (long long)elem_size(dtype) <= 0xffffffffll; }
uint32_t stride_of(long long ld, int dtype) { return (uint32_t)(ld * (long long)elem_size(dtype)); }

// rows of 8-column accesses: D, the stride and the base allow them
bool rows8(const void* p, long long ld, int dtype) { return !p || (aligned16(p) && ld * elem_size(dtype) % 16 == 0); }

NormGrid norm_bwd_grid(int T, int D) { return norm_grid(std::max(T, 1), D, nrm::kBwdCta, nrm::kBwdPerSm, true); }

size_t norm_partials(const deco_block_norm_t& s) {
  const NormGrid g = norm_bwd_grid(s.T, s.d_model);
  return align256((size_t)2 * g.clusters * s.d_model * 4);
}

constexpr int norm_smem(bool vec, int pieces, int threads) { return vec ? nrm::ring_rows(pieces) * pieces * threads * 16 : 0; }

template <typename T, int VEC, bool FULL>
cudaError_t norm_fwd(nrm::FwdArgs& a, cudaStream_t st) {
  const NormGrid g = norm_grid(a.T, a.D, nrm::kFwdCta<T, VEC>, nrm::kFwdPerSm<T, VEC>, false);
  a.cl = g.cl;
  constexpr int pieces = nrm::kFwdPieces<T, FULL>;
  return norm_launch(nrm::kn_forward<T, VEC, FULL>, g, norm_smem(VEC == 8, pieces, g.threads), norm_smem(VEC == 8, pieces, nrm::kFwdCta<T, VEC>),
                     a, st);
}
template <typename T>
cudaError_t norm_fwd_any(bool vec, nrm::FwdArgs& a, cudaStream_t st) {
  if (a.gate_kind == nrm::kFull) return vec ? norm_fwd<T, 8, true>(a, st) : norm_fwd<T, 1, true>(a, st);
  return vec ? norm_fwd<T, 8, false>(a, st) : norm_fwd<T, 1, false>(a, st);
}

template <typename T, typename TH, typename TR, int VEC, bool FULL>
cudaError_t norm_bwd(const NormGrid& g, const nrm::BwdArgs& a, cudaStream_t st) {
  constexpr int pieces = nrm::kBwdPieces<T, TH, TR, FULL>;
  const auto smem = [](int threads) { return norm_smem(VEC == 8, pieces, threads) + 64 * threads; };   // the ring, two vectors
  return norm_launch(nrm::kn_backward<T, TH, TR, VEC, FULL>, g, smem(g.threads), smem(nrm::kBwdCta), a, st);
}
template <typename T, typename TH, typename TR>
cudaError_t norm_bwd_any(bool vec, const NormGrid& g, const nrm::BwdArgs& a, cudaStream_t st) {
  if (a.gate_kind == nrm::kFull) return vec ? norm_bwd<T, TH, TR, 8, true>(g, a, st) : norm_bwd<T, TH, TR, 1, true>(g, a, st);
  return vec ? norm_bwd<T, TH, TR, 8, false>(g, a, st) : norm_bwd<T, TH, TR, 1, false>(g, a, st);
}

// ---- sorting ------------------------------------------------------------------

struct SortPlan {
  bool small;
  int tile, n_tiles;
  size_t bytes;
};

// One launch sorts up to kSmallSlots slots, each of its CTAs all of them; but
// it copies rows in sorted order and so reads x once a pair.  Three launches
// read it once: 19 us against 27 at 2048 x 8 rows of 4 KB, 9 against 10 at half
// of kSmallBytes, for 8 us more of the host's time.
constexpr long long kSmallBytes = 32 << 20;

SortPlan sort_plan(int T, int S, int E, bool mask, long long row_bytes) {
  SortPlan p{};
  const long long n = (long long)T * S;
  p.small = n <= srt::kSmallSlots && n * row_bytes <= kSmallBytes;
  if (p.small) return p;
  // a tile an SM at most: of tokens (a few a thread, as every tile reads the
  // histograms of all), or of slots in steps of 32 a warp
  const long long unit = mask ? 4 * (srt::kSortThreads / E) : srt::kSortThreads, all = mask ? T : n;
  p.tile = (int)(((all + srt::kMaxTiles - 1) / srt::kMaxTiles + unit - 1) / unit * unit);
  p.n_tiles = (int)((all + p.tile - 1) / p.tile);
  p.bytes = align256((size_t)srt::kMaxTiles * E * 4);
  return p;
}

deco_status_t check_sort(int T, int S, int E) {
  if (T < 0 || S <= 0 || E <= 0) return DECO_ERR_INVALID_ARG;
  if (S > srt::kMaxS || E > srt::kMaxE || T > (1 << 20)) return DECO_ERR_UNSUPPORTED;
  return DECO_OK;
}

template <typename V>
cudaError_t run_dispatch(const SortPlan& p, const srt::Args& a, cudaStream_t st) {
  if (p.small) {
    const long long n = (long long)a.T * a.S;   // pairs at most; a CTA for every few of them
    const int ctas = a.xs ? (int)std::max<long long>(1, std::min<long long>(num_sms(), n)) : 1;
    const auto k = a.active ? srt::ks_small_mask<V> : n <= srt::kSmallThreads * 4 ? srt::ks_small<V, 4> : srt::ks_small<V, 16>;
    const int smem = (int)(2 * n);
    // static shared memory counts too: opt in well below 48 KB
    const cudaError_t err =
        smem > 24 * 1024 ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * srt::kSmallSlots) : cudaSuccess;
    if (err != cudaSuccess) return err;
    k<<<ctas, srt::kSmallThreads, smem, st>>>(a);
    return cudaGetLastError();
  }
  (a.active ? srt::ks_count_mask : srt::ks_count)<<<p.n_tiles, srt::kSortThreads, 0, st>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) err = launch_behind(a.active ? srt::ks_tables_mask : srt::ks_tables, dim3(p.n_tiles), srt::kSortThreads, a, st);
  const int threads = std::min(srt::kThreads, (a.row_bytes / (int)sizeof(V) + 31) / 32 * 32);
  if (err == cudaSuccess && a.xs) err = launch_behind(srt::ks_copy<V>, dim3(a.T), threads, a, st);
  return err;
}

template <typename T, typename TY, int VEC>
cudaError_t launch_combine(const srt::CombineArgs& a, cudaStream_t st) {
  const int threads = std::min(srt::kCombThreads, (((a.D + 7) / 8) + 31) / 32 * 32);
  srt::ks_combine<T, TY, VEC><<<dim3(a.T, (a.D + threads * 8 - 1) / (threads * 8)), threads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_combine_bwd(const srt::CombineBwdArgs& a, cudaStream_t st) {
  const int threads = std::min(srt::kThreads, (((a.D + 7) / 8) + 31) / 32 * 32);
  // few tokens: several CTAs share one's rows, until there are two an SM
  const int parts = std::max(1, std::min({(2 * num_sms() + a.T - 1) / a.T, (a.S + srt::kBwdRows - 1) / srt::kBwdRows, 16}));
  srt::ks_combine_bwd<T, VEC><<<dim3(a.T, parts), threads, 0, st>>>(a);
  return cudaGetLastError();
}

// ---- 4-bit weights --------------------------------------------------------------

deco_status_t check_q4(long long rows, int K, int group) {
  if (rows <= 0 || K <= 0) return DECO_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return DECO_ERR_UNSUPPORTED;
  if (K > (1 << 20) || rows > (1ll << 31) / 8) return DECO_ERR_UNSUPPORTED;
  return DECO_OK;
}

int q4_padded(int K) { return (K + q4::kBlock - 1) / q4::kBlock * q4::kBlock; }

bool q4_blocks_ok(long long rows, int K, unsigned* ctas) {
  const long long n = (rows * (q4_padded(K) / q4::kBlock) + q4::kPackWarps - 1) / q4::kPackWarps;
  *ctas = (unsigned)n;
  return n <= 0x7fffffffll;
}

// at most 2^this warps share a row's K
template <typename T> constexpr int kQ4MostSplit = sizeof(T) == 4 ? 3 : 4;

struct Q4Plan {
  int m, split, cluster;      // row tiles a warp; warps a row, CTAs a row (log2)
  long long units;
};

template <typename T, int NT, int M, int G>
cudaError_t q4_launch(q4::Args& a, const Q4Plan& p, cudaStream_t st) {
  using S = q4::Smem<T, NT, M>;
  static_assert(S::kMaxBlocks >= 1 << kQ4MostSplit<T>, "the largest split has room for a block of x a warp");
  const int blocks = (a.Kp / q4::kBlock + (1 << p.cluster) - 1) >> p.cluster, bpw = (blocks + (1 << p.split) - 1) >> p.split;
  a.split_log2 = p.split;
  a.cluster_log2 = p.cluster;
  a.chunk = std::max(1, std::min(bpw, S::kMaxBlocks >> p.split));
  const int bytes = S::kRing + S::kPart + S::x_bytes(a.chunk << p.split);
  const auto kernel = a.zero ? q4::kq_matvec<T, NT, M, G, true> : q4::kq_matvec<T, NT, M, G, false>;
  const cudaError_t err = allow_smem(kernel, S::kRing + S::kPart + S::kX);
  if (err != cudaSuccess) return err;
  const long long most = num_sms() >> p.cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<long long>(1, std::min(p.units, most)) << p.cluster);
  cfg.blockDim = dim3(q4::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1 << p.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// How a product of N x (128 blocks) weights against `items` tiles of rows of x,
// `likely` of them there, is cut: the fewest steps (blocks of a row tile) of
// the busiest SM.  A step of two row tiles costs about 1.8 of one (the operands
// of x are shared), a unit's sums and barriers about one step, a cluster's two;
// fetching x again for a part of K that did not fit about two.
// (T = 1, K = 2048, N = 512 to 139264 in us: 3.4 to 40; T = 16: 4.4 to 57.)
template <typename T>
Q4Plan q4_plan(int N, int blocks, int nt, long long items, long long likely, int sms) {
  constexpr bool kF32 = sizeof(T) == 4;
  const auto room = [&](int m) {   // blocks of x that fit
    if (kF32) return nt == 1 ? q4::Smem<T, 1, 1>::kMaxBlocks : q4::Smem<T, 2, 1>::kMaxBlocks;
    if (nt == 4) return q4::Smem<T, 4, 1>::kMaxBlocks;
    if (nt == 2) return m == 1 ? q4::Smem<T, 2, 1>::kMaxBlocks : q4::Smem<T, 2, 2>::kMaxBlocks;
    return m == 1 ? q4::Smem<T, 1, 1>::kMaxBlocks : q4::Smem<T, 1, 2>::kMaxBlocks;
  };
  Q4Plan best{1, 0, 0, 0};
  double least = 1e30;
  for (int m = 1; m <= (nt == 4 || kF32 ? 1 : 2); ++m)
    for (int s = 0; s <= kQ4MostSplit<T> && (s == 0 || (1 << s) <= blocks); ++s) {
      const int width = (q4::kWarps >> s) * 16 * m;
      const long long tiles = (N + width - 1) / width;
      for (int c = 0; (1 << c) <= (width <= q4::kClusterWidth ? q4::kMaxCluster : 1) && (c == 0 || (1 << (s + c)) <= blocks); ++c) {
        const int mine = (blocks + (1 << c) - 1) >> c, bpw = (mine + (1 << s) - 1) >> s, chunk = std::max(1, std::min(bpw, room(m) >> s));
        const long long clusters = std::max(1, sms >> c);
        const double cost = (double)((tiles * likely + clusters - 1) / clusters) *
                            ((m == 1 ? 1.0 : 1.8) * bpw + (c ? 2.0 : 1.0) + 2.0 * ((bpw + chunk - 1) / chunk - 1));
        if (cost < least) {
          least = cost;
          best = {m, s, c, tiles * items};
        }
      }
    }
  return best;
}

// The launch of a product: `most` is the largest number of rows one matrix can
// meet as far as the call tells: a batch, or, by expert, the smaller of x's and
// y's rows.  Sorted rows in order say T x E there where an expert has T at most,
// and so take wider tiles than they fill: 16 tokens on 64 experts of 2048 x 256
// 15.3 us, by perm 13.5.
template <typename T, int G>
cudaError_t q4_run(q4::Args& a, long long most, cudaStream_t st) {
  constexpr bool kF32 = sizeof(T) == 4;   // three pieces of x: two tiles of rows of x, one of W at most, by shared memory
  const int nt = most <= 8 ? 1 : most <= 16 || kF32 ? 2 : 4;
  const long long rows = 8 * nt;
  const long long items = a.E ? std::min<long long>(a.E, a.rows_y) + a.rows_y / rows : (a.rows_y + rows - 1) / rows;
  const long long likely = a.E ? std::min<long long>(a.E, a.rows_y) : items;
  a.x_vec = a.K % 8 == 0 && aligned16(a.x) && a.ld_x * sizeof(T) % 16 == 0;
  const Q4Plan p = q4_plan<T>(a.N, a.Kp / q4::kBlock, nt, items, likely, num_sms());
  if constexpr (!kF32) {
    if (nt == 4) return q4_launch<T, 4, 1, G>(a, p, st);
    if (p.m == 2) return nt == 2 ? q4_launch<T, 2, 2, G>(a, p, st) : q4_launch<T, 1, 2, G>(a, p, st);
  }
  return nt == 2 ? q4_launch<T, 2, 1, G>(a, p, st) : q4_launch<T, 1, 1, G>(a, p, st);
}

template <typename T>
cudaError_t q4_group(q4::Args& a, int group, long long most, cudaStream_t st) {
  return group == 32 ? q4_run<T, 32>(a, most, st) : group == 64 ? q4_run<T, 64>(a, most, st) : q4_run<T, 128>(a, most, st);
}

deco_status_t q4_product(int N, int K, int group, int dtype, int out_dtype, int rows_x, const void* x, long long ld_x, const void* q,
                         const void* scale, const uint8_t* zero, int E, const int* offsets, const int* perm, long long rows_y, void* y,
                         long long ld_y, void* stream, const char* what) {
  deco_status_t st = check_q4((long long)N * std::max(E, 1), K, group);
  if (st != DECO_OK) return st;
  if (rows_x < 0 || rows_y < 0 || N <= 0 || !is_dtype(dtype) || !is_dtype(out_dtype)) return DECO_ERR_INVALID_ARG;
  if (dtype == DECO_F32 && out_dtype != DECO_F32) return DECO_ERR_UNSUPPORTED;
  if (rows_x > (1 << 28) || rows_y > (1ll << 28)) return DECO_ERR_UNSUPPORTED;
  // the kernel counts its units of at least 16 x 8 in 32 bits
  const long long units = (long long)(N / 16 + 1) * (std::min<long long>(E, rows_y) + rows_y / 8 + 1);
  if (units > 0x7fffffffll || units * (q4_padded(K) / q4::kBlock) > (1ll << 36)) return DECO_ERR_UNSUPPORTED;   // also a CTA's steps
  if (!resolve_ld(ld_x, K) || !resolve_ld(ld_y, N)) return DECO_ERR_INVALID_ARG;
  // perm into an x of no rows asks for zero rows
  if (rows_y == 0 || (rows_x == 0 && !perm)) return DECO_OK;
  if ((!x && rows_x) || !q || !scale || !y || x == y) return DECO_ERR_INVALID_ARG;
  if (!aligned_to(x, elem_size(dtype)) || !aligned_to(y, elem_size(out_dtype)) || !aligned16(q) || !aligned_to(scale, 8) ||
      (zero && !aligned_to(zero, 4)))
    return DECO_ERR_INVALID_ARG;
  if (E && (!offsets || !aligned_to(offsets, 4) || (perm && !aligned_to(perm, 4)))) return DECO_ERR_INVALID_ARG;
  q4::Args a{};
  a.N = N;
  a.K = K;
  a.Kp = q4_padded(K);
  a.rows_x = rows_x;
  a.rows_y = rows_y;
  a.q = static_cast<const unsigned char*>(q);
  a.scale = static_cast<const unsigned char*>(scale);
  a.zero = zero;
  a.x = rows_x ? x : q;   // an address even where there is nothing to read: copies of zeros name one
  a.y = y;
  a.ld_x = ld_x;
  a.ld_y = ld_y;
  a.y_f32 = out_dtype == DECO_F32;
  a.E = E;
  a.offsets = offsets;
  a.perm = perm;
  const long long most = E ? std::min<long long>(rows_x, rows_y) : rows_y;
  cudaStream_t cs = as_stream(stream);
  return cuda_status(dtype == DECO_F32 ? q4_group<float>(a, group, most, cs) : q4_group<bf16>(a, group, most, cs), what);
}

}  // namespace
}  // namespace deco

extern "C" {

using namespace deco;

deco_status_t deco_block_norm_forward(const deco_block_norm_t* shape, const void* x, const void* y, const float* g_post,
                                      const void* gate, const float* g_pre, void* out, void* h, void* stream) {
  deco_status_t st = check_norm(shape);
  if (st != DECO_OK) return st;
  deco_block_norm_t s = *shape;
  const int D = s.d_model;
  if (s.T == 0) return DECO_OK;   // tensors without elements may have no address
  if ((y == nullptr) != (out == nullptr) || (g_pre == nullptr) != (h == nullptr) || (!y && !h)) return DECO_ERR_INVALID_ARG;
  if (!y && (g_post || s.gate != DECO_GATE_NONE)) return DECO_ERR_INVALID_ARG;
  if ((gate != nullptr) != (s.gate != DECO_GATE_NONE)) return DECO_ERR_INVALID_ARG;
  if (!resolve_ld(s.ld_x, D) || !resolve_ld(s.ld_y, D, y) || !resolve_ld(s.ld_out, D, out) || !resolve_ld(s.ld_h, D, h) ||
      !resolve_ld(s.ld_gate, D, s.gate == DECO_GATE_FULL ? gate : nullptr))
    return DECO_ERR_INVALID_ARG;
  const size_t es = elem_size(s.dtype);
  if (!x || !aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(out, es) || !aligned_to(h, es) || !aligned_to(g_post, 4) ||
      !aligned_to(g_pre, 4) || !aligned_to(gate, s.gate == DECO_GATE_FULL ? es : 4))
    return DECO_ERR_INVALID_ARG;
  // out may be x (an update in place, the same stride); nothing else aliases
  if (out == x && s.ld_out != s.ld_x) return DECO_ERR_INVALID_ARG;
  if ((h && (h == x || h == y || h == out || h == gate)) || (out && (out == y || out == gate))) return DECO_ERR_INVALID_ARG;
  const long long lds[] = {s.ld_x, s.ld_y, s.ld_gate, s.ld_out, s.ld_h};
  for (long long ld : lds)
    if (!stride_ok(ld, s.dtype)) return DECO_ERR_UNSUPPORTED;
  nrm::FwdArgs a{s.T, D, s.gate, 1, s.rms_eps, s.branch_scale, stride_of(s.ld_x, s.dtype), stride_of(s.ld_y, s.dtype),
                 stride_of(s.ld_gate, s.dtype), stride_of(s.ld_out, s.dtype), stride_of(s.ld_h, s.dtype),
                 x, y, gate, g_post, g_pre, out, h};
  const bool vec = D % 8 == 0 && rows8(x, s.ld_x, s.dtype) && rows8(y, s.ld_y, s.dtype) && rows8(out, s.ld_out, s.dtype) &&
                   rows8(h, s.ld_h, s.dtype) && aligned16(g_post) && aligned16(g_pre) &&
                   (s.gate == DECO_GATE_FULL ? rows8(gate, s.ld_gate, s.dtype) : s.gate == DECO_GATE_TOKEN || aligned16(gate));
  cudaStream_t cs = as_stream(stream);
  cudaError_t err;
  err = s.dtype == DECO_F32 ? norm_fwd_any<float>(vec, a, cs) : norm_fwd_any<bf16>(vec, a, cs);
  return cuda_status(err, "block_norm_forward");
}

deco_status_t deco_block_norm_backward_workspace_size(const deco_block_norm_t* shape, size_t* bytes) {
  const deco_status_t st = check_norm(shape);
  if (st != DECO_OK) return st;
  if (!bytes) return DECO_ERR_INVALID_ARG;
  *bytes = norm_partials(*shape);
  return DECO_OK;
}

deco_status_t deco_block_norm_backward(const deco_block_norm_t* shape, const void* x, const void* y, const float* g_post,
                                       const void* gate, const float* g_pre, const void* dout, const void* dh,
                                       const deco_block_norm_grads_t* grads, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  deco_status_t st = check_norm(shape);
  if (st != DECO_OK) return st;
  deco_block_norm_t s = *shape;
  const int D = s.d_model;
  if (!grads || !is_dtype(s.dh_dtype) || !is_dtype(s.dout_dtype)) return DECO_ERR_INVALID_ARG;
  if (s.dtype == DECO_F32 && (s.dh_dtype != DECO_F32 || s.dout_dtype != DECO_F32)) return DECO_ERR_UNSUPPORTED;
  const deco_block_norm_grads_t& g = *grads;
  if (!aligned_to(g.dg_pre, 4) || !aligned_to(g.dg_post, 4)) return DECO_ERR_INVALID_ARG;
  cudaStream_t cs = as_stream(stream);
  if (s.T == 0) {   // sums over no rows
    cudaError_t err = cudaSuccess;
    float* zs[] = {g.dg_pre, g.dg_post, s.gate == DECO_GATE_CHANNEL ? static_cast<float*>(g.dgate) : nullptr};
    for (float* z : zs)
      if (z && err == cudaSuccess) err = cudaMemsetAsync(z, 0, (size_t)D * 4, cs);
    return cuda_status(err, "block_norm_backward");
  }
  if ((!dout && !dh) || (dh != nullptr) != (g_pre != nullptr)) return DECO_ERR_INVALID_ARG;
  if (!y && (g_post || s.gate != DECO_GATE_NONE)) return DECO_ERR_INVALID_ARG;
  if ((gate != nullptr) != (s.gate != DECO_GATE_NONE)) return DECO_ERR_INVALID_ARG;
  if ((g.dg_pre != nullptr) != (dh != nullptr) || (g.dg_post != nullptr) != (g_post != nullptr) || (g.dgate != nullptr) != (gate != nullptr))
    return DECO_ERR_INVALID_ARG;
  if (!resolve_ld(s.ld_x, D) || !resolve_ld(s.ld_y, D, y) || !resolve_ld(s.ld_out, D, dout) || !resolve_ld(s.ld_h, D, dh) ||
      !resolve_ld(s.ld_gate, D, s.gate == DECO_GATE_FULL ? gate : nullptr))
    return DECO_ERR_INVALID_ARG;
  const size_t es = elem_size(s.dtype), eh = elem_size(s.dh_dtype), er = elem_size(s.dout_dtype);
  if (!g.dx || (g.dy != nullptr) != (y != nullptr) || (dh && !x)) return DECO_ERR_INVALID_ARG;
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(dh, eh) || !aligned_to(dout, er) || !aligned_to(g.dx, er) ||
      !aligned_to(g.dy, es) || !aligned_to(g_post, 4) || !aligned_to(g_pre, 4) ||
      !aligned_to(gate, s.gate == DECO_GATE_FULL ? es : 4) || !aligned_to(g.dgate, s.gate == DECO_GATE_FULL ? es : 4))
    return DECO_ERR_INVALID_ARG;
  if (!stride_ok(s.ld_x, s.dtype) || !stride_ok(s.ld_y, s.dtype) || !stride_ok(s.ld_gate, s.dtype) || !stride_ok(s.ld_out, s.dout_dtype) ||
      !stride_ok(s.ld_h, s.dh_dtype))
    return DECO_ERR_UNSUPPORTED;
  // dx may be dout (both [T][D] without gaps); nothing else aliases
  if (g.dx == dout && s.ld_out != D) return DECO_ERR_INVALID_ARG;
  const void* ins[] = {x, y, gate, dh};
  const void* outs[] = {g.dx, g.dy, g.dgate};
  for (const void* o : outs)
    for (const void* i : ins)
      if (o && o == i) return DECO_ERR_INVALID_ARG;
  if (g.dx == g.dy || g.dx == g.dgate || (g.dy && (g.dy == g.dgate || g.dy == dout)) || (g.dgate && g.dgate == dout)) return DECO_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < norm_partials(s)) return DECO_ERR_WORKSPACE;
  const bool vec = D % 8 == 0 && rows8(x, s.ld_x, s.dtype) && rows8(y, s.ld_y, s.dtype) && rows8(dout, s.ld_out, s.dout_dtype) &&
                   rows8(dh, s.ld_h, s.dh_dtype) && rows8(g.dx, D, s.dout_dtype) && rows8(g.dy, D, s.dtype) &&
                   aligned16(g_post) && aligned16(g_pre) &&
                   (s.gate == DECO_GATE_FULL ? rows8(gate, s.ld_gate, s.dtype) && rows8(g.dgate, D, s.dtype)
                                             : s.gate == DECO_GATE_TOKEN || aligned16(gate));
  const NormGrid ng = norm_bwd_grid(s.T, D);
  nrm::BwdArgs a{s.T, D, s.gate, ng.cl, s.rms_eps, s.branch_scale, stride_of(s.ld_x, s.dtype), stride_of(s.ld_y, s.dtype),
                 stride_of(s.ld_gate, s.dtype), stride_of(s.ld_out, s.dout_dtype), stride_of(s.ld_h, s.dh_dtype),
                 x, y, gate, dout, dh, g_post, g_pre, g.dx, g.dy, g.dgate, static_cast<float*>(workspace)};
  cudaError_t err;
  const bool h32 = s.dh_dtype == DECO_F32, r32 = s.dout_dtype == DECO_F32;
  if (s.dtype == DECO_F32) err = norm_bwd_any<float, float, float>(vec, ng, a, cs);
  else if (h32) err = r32 ? norm_bwd_any<bf16, float, float>(vec, ng, a, cs) : norm_bwd_any<bf16, float, bf16>(vec, ng, a, cs);
  else err = r32 ? norm_bwd_any<bf16, bf16, float>(vec, ng, a, cs) : norm_bwd_any<bf16, bf16, bf16>(vec, ng, a, cs);
  if (err != cudaSuccess) return cuda_status(err, "block_norm_backward");
  const bool channel = s.gate == DECO_GATE_CHANNEL;
  const nrm::RedArgs r{D, ng.clusters, a.part, g.dg_pre, g.dg_post, channel ? static_cast<float*>(g.dgate) : nullptr, g_post,
                       channel ? static_cast<const float*>(gate) : nullptr};
  if (!r.dg_pre && !r.dg_post && !r.dgate) return DECO_OK;
  return cuda_status(launch_behind(nrm::kn_reduce, dim3((D + 31) / 32, 2), nrm::kRedWarps * 32, r, cs), "block_norm_backward: sums");
}

deco_status_t deco_moe_dispatch_workspace_size(int T, int slots, int E, int d_model, int dtype, size_t* bytes) {
  const deco_status_t st = check_sort(T, slots, E);
  if (st != DECO_OK) return st;
  if (!bytes || d_model <= 0 || !is_dtype(dtype)) return DECO_ERR_INVALID_ARG;
  *bytes = sort_plan(T, slots, E, false, (long long)d_model * elem_size(dtype)).bytes;   // the same under a mask
  return DECO_OK;
}

deco_status_t deco_moe_dispatch(int T, int slots, int E, int d_model, int dtype, const int* experts, const uint8_t* active,
                                const void* x, long long ld_x, const deco_dispatch_t* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
  deco_status_t st = check_sort(T, slots, E);
  if (st != DECO_OK) return st;
  if (!out || d_model <= 0 || !is_dtype(dtype) || out->capacity < 0) return DECO_ERR_INVALID_ARG;
  if (T && ((experts == nullptr) == (active == nullptr) || (active && slots != E) || !aligned_to(experts, 4))) return DECO_ERR_INVALID_ARG;
  if (d_model > (1 << 20) || out->capacity > 0x7fffffffll || (long long)T * slots > (1 << 28)) return DECO_ERR_UNSUPPORTED;
  const int* tabs[] = {out->counts, out->offsets, out->n_pairs};
  for (const int* p : tabs)
    if (!p || !aligned_to(p, 4)) return DECO_ERR_INVALID_ARG;
  if (T && (!out->row_of || !aligned_to(out->row_of, 4) || (out->capacity && (!out->slot_of || !aligned_to(out->slot_of, 4))))) return DECO_ERR_INVALID_ARG;
  long long ld_xs = out->ld_xs;
  const size_t es = elem_size(dtype);
  if (out->xs) {
    if (!resolve_ld(ld_x, d_model) || !resolve_ld(ld_xs, d_model)) return DECO_ERR_INVALID_ARG;
    if (T && (!x || x == out->xs || !aligned_to(x, es) || !aligned_to(out->xs, es))) return DECO_ERR_INVALID_ARG;
  }
  const SortPlan p = sort_plan(T, slots, E, active != nullptr, (long long)d_model * es);
  if (p.bytes && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bytes)) return DECO_ERR_WORKSPACE;
  srt::Args a{};
  a.T = T;
  a.S = slots;
  a.E = E;
  a.D = d_model;
  while ((1 << a.bits) <= E) ++a.bits;
  a.experts = experts;
  a.active = active;
  a.cap = out->capacity;
  a.counts = out->counts;
  a.offsets = out->offsets;
  a.slot_of = out->slot_of;
  a.row_of = out->row_of;
  a.n_pairs = out->n_pairs;
  a.x = x;
  a.xs = out->xs;
  a.ld_x = ld_x * es;
  a.ld_xs = ld_xs * es;
  a.row_bytes = (int)(d_model * es);
  a.tile = p.tile;
  a.n_tiles = p.n_tiles;
  a.hist = static_cast<int*>(workspace);
  // the widest copy that the rows' bytes, strides and bases allow
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.xs) | a.ld_x | a.ld_xs | a.row_bytes;
  cudaStream_t cs = as_stream(stream);
  const cudaError_t err = all % 16 == 0 ? run_dispatch<uint4>(p, a, cs) : all % 4 == 0 ? run_dispatch<uint32_t>(p, a, cs)
                                                                                       : run_dispatch<uint16_t>(p, a, cs);
  return cuda_status(err, "dispatch");
}

deco_status_t deco_moe_combine(int T, int slots, int d_model, int dtype, int out_dtype, const int* row_of, const float* w,
                               const void* ys, long long n_rows, long long ld_ys, const void* base, long long ld_base, void* y,
                               long long ld_y, void* stream) {
  deco_status_t st = check_sort(T, slots, 1);
  if (st != DECO_OK) return st;
  if (d_model <= 0 || !is_dtype(dtype) || !is_dtype(out_dtype) || n_rows < 0) return DECO_ERR_INVALID_ARG;
  if (dtype == DECO_F32 && out_dtype != DECO_F32) return DECO_ERR_UNSUPPORTED;
  if (d_model > (1 << 20)) return DECO_ERR_UNSUPPORTED;
  if (!resolve_ld(ld_ys, d_model) || !resolve_ld(ld_base, d_model, base) || !resolve_ld(ld_y, d_model)) return DECO_ERR_INVALID_ARG;
  if (T == 0) return DECO_OK;
  const size_t es = elem_size(dtype);
  if (!row_of || !y || (n_rows && !ys) || y == ys || !aligned_to(row_of, 4) || !aligned_to(w, 4) || !aligned_to(ys, es) ||
      !aligned_to(base, es) || !aligned_to(y, elem_size(out_dtype)))
    return DECO_ERR_INVALID_ARG;
  if (y == base && (ld_y != ld_base || out_dtype != dtype)) return DECO_ERR_INVALID_ARG;
  const srt::CombineArgs a{T, slots, d_model, n_rows, row_of, w, ys, base, y, ld_ys, ld_base, ld_y};
  const bool vec = d_model % 8 == 0 && rows8(ys, ld_ys, dtype) && rows8(base, ld_base, dtype) && rows8(y, ld_y, out_dtype);
  cudaStream_t cs = as_stream(stream);
  cudaError_t err;
  if (dtype == DECO_F32) err = vec ? launch_combine<float, float, 8>(a, cs) : launch_combine<float, float, 1>(a, cs);
  else if (out_dtype == DECO_F32) err = vec ? launch_combine<bf16, float, 8>(a, cs) : launch_combine<bf16, float, 1>(a, cs);
  else err = vec ? launch_combine<bf16, bf16, 8>(a, cs) : launch_combine<bf16, bf16, 1>(a, cs);
  return cuda_status(err, "combine");
}

deco_status_t deco_moe_combine_backward(int T, int slots, int d_model, int dtype, const int* row_of, const float* w, const void* ys,
                                        long long n_rows, long long ld_ys, const void* dy, long long ld_dy, void* dys,
                                        long long ld_dys, float* dw, void* stream) {
  deco_status_t st = check_sort(T, slots, 1);
  if (st != DECO_OK) return st;
  if (d_model <= 0 || !is_dtype(dtype) || n_rows < 0) return DECO_ERR_INVALID_ARG;
  if (d_model > (1 << 20)) return DECO_ERR_UNSUPPORTED;
  if (!resolve_ld(ld_ys, d_model) || !resolve_ld(ld_dy, d_model) || !resolve_ld(ld_dys, d_model)) return DECO_ERR_INVALID_ARG;
  if (T == 0) return DECO_OK;
  const size_t es = elem_size(dtype);
  if (!row_of || !dy || (n_rows && (!ys || !dys || dys == ys)) || dys == dy || !aligned_to(row_of, 4) || !aligned_to(w, 4) ||
      !aligned_to(dw, 4) || !aligned_to(ys, es) || !aligned_to(dy, es) || !aligned_to(dys, es))
    return DECO_ERR_INVALID_ARG;
  const srt::CombineBwdArgs a{T, slots, d_model, n_rows, row_of, w, ys, dy, dys, dw, ld_ys, ld_dy, ld_dys};
  const bool vec = d_model % 8 == 0 && rows8(ys, ld_ys, dtype) && rows8(dy, ld_dy, dtype) && rows8(dys, ld_dys, dtype);
  cudaStream_t cs = as_stream(stream);
  const cudaError_t err = dtype == DECO_F32 ? (vec ? launch_combine_bwd<float, 8>(a, cs) : launch_combine_bwd<float, 1>(a, cs))
                                            : (vec ? launch_combine_bwd<bf16, 8>(a, cs) : launch_combine_bwd<bf16, 1>(a, cs));
  return cuda_status(err, "combine_backward");
}

deco_status_t deco_q4_quantize(long long rows, int K, int group, int dtype, const void* W, void* q, void* scale, uint8_t* zero,
                               void* stream) {
  deco_status_t st = check_q4(rows, K, group);
  if (st != DECO_OK) return st;
  if (!is_dtype(dtype) || !W || !q || !scale || !aligned_to(W, elem_size(dtype)) || !aligned16(q) || !aligned_to(scale, 8))
    return DECO_ERR_INVALID_ARG;
  unsigned ctas = 0;
  if (!q4_blocks_ok(rows, K, &ctas)) return DECO_ERR_UNSUPPORTED;
  const q4::PackArgs a{rows, K, q4_padded(K), group, W, static_cast<uint32_t*>(q), static_cast<bf16*>(scale), zero};
  cudaStream_t cs = as_stream(stream);
  if (dtype == DECO_F32) q4::kq_quantize<float><<<ctas, q4::kPackThreads, 0, cs>>>(a);
  else q4::kq_quantize<bf16><<<ctas, q4::kPackThreads, 0, cs>>>(a);
  return cuda_status(cudaGetLastError(), "q4_quantize");
}

deco_status_t deco_q4_pack(long long rows, int K, const uint8_t* codes, void* q, void* stream) {
  deco_status_t st = check_q4(rows, K, 128);
  if (st != DECO_OK) return st;
  if (!codes || !q || codes == q || !aligned16(q)) return DECO_ERR_INVALID_ARG;
  unsigned ctas = 0;
  if (!q4_blocks_ok(rows, K, &ctas)) return DECO_ERR_UNSUPPORTED;
  const q4::PackArgs a{rows, K, q4_padded(K), 128, codes, static_cast<uint32_t*>(q), nullptr, nullptr};
  q4::kq_pack<<<ctas, q4::kPackThreads, 0, as_stream(stream)>>>(a);
  return cuda_status(cudaGetLastError(), "q4_pack");
}

deco_status_t deco_q4_dequantize(long long rows, int K, int group, int dtype, const void* q, const void* scale, const uint8_t* zero,
                                 void* W, void* stream) {
  deco_status_t st = check_q4(rows, K, group);
  if (st != DECO_OK) return st;
  if (!is_dtype(dtype) || !W || !q || !scale || !aligned_to(W, elem_size(dtype)) || !aligned16(q) || !aligned_to(scale, 2))
    return DECO_ERR_INVALID_ARG;
  unsigned ctas = 0;
  if (!q4_blocks_ok(rows, K, &ctas)) return DECO_ERR_UNSUPPORTED;
  const q4::PackArgs a{rows, K, q4_padded(K), group, nullptr, const_cast<uint32_t*>(static_cast<const uint32_t*>(q)),
                       const_cast<bf16*>(static_cast<const bf16*>(scale)), const_cast<uint8_t*>(zero)};
  cudaStream_t cs = as_stream(stream);
  if (dtype == DECO_F32) q4::kq_dequantize<float><<<ctas, q4::kPackThreads, 0, cs>>>(a, static_cast<float*>(W));
  else q4::kq_dequantize<bf16><<<ctas, q4::kPackThreads, 0, cs>>>(a, static_cast<bf16*>(W));
  return cuda_status(cudaGetLastError(), "q4_dequantize");
}

deco_status_t deco_q4_matvec(int T, int N, int K, int group, int dtype, int out_dtype, const void* x, long long ld_x, const void* q,
                             const void* scale, const uint8_t* zero, void* y, long long ld_y, void* stream) {
  return q4_product(N, K, group, dtype, out_dtype, T, x, ld_x, q, scale, zero, 0, nullptr, nullptr, T, y, ld_y, stream, "q4_matvec");
}

deco_status_t deco_q4_expert_matvec(int E, int N, int K, int group, int dtype, int out_dtype, const int* offsets, const int* perm,
                                    int rows_x, const void* x, long long ld_x, const void* q, const void* scale, const uint8_t* zero,
                                    long long rows_y, void* y, long long ld_y, void* stream) {
  if (E <= 0) return DECO_ERR_INVALID_ARG;
  if (E > srt::kMaxE) return DECO_ERR_UNSUPPORTED;
  return q4_product(N, K, group, dtype, out_dtype, rows_x, x, ld_x, q, scale, zero, E, offsets, perm, rows_y, y, ld_y, stream,
                    "q4_expert_matvec");
}

}  // extern "C"
