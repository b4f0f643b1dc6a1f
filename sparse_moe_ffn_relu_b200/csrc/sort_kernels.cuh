// Tokens sorted by expert and back.
//
// A batch has T x S slots (t, k); slot i = t S + k holds an expert (k itself
// under a mask [T][E], S = E; the k-th expert number of the token otherwise)
// or nothing.  The pairs (token, expert) in stable order of expert, token, k
// are the sorted rows:
//   counts[e], offsets[E+1]   rows of each expert, their first row
//   slot_of[row] = i, row_of[i] = row (-1: no expert, or no room)
//   dispatch   xs[row] = x[t]
//   combine    y[t] = base[t] + sum_k w[t,k] ys[row_of[t,k]]   (k ascending, fp32)
//   backward   dys[row] = w[t,k] dy[t],  dw[t,k] = dy[t] . ys[row]
//              (dispatch's own backward is combine without weights)
//
// All of it moves rows and is bound by DRAM; the tables are a few bytes per
// slot.  Sorting is a counting sort, and no atomics order anything.  Under a
// mask a thread walks an expert's tokens, and a scan over (expert, run of
// tokens) gives each walk its first row.  Of lists of experts a warp takes 32
// consecutive slots at a time, lanes of the same expert find each other by a
// ballot on each bit of its number (a match instruction took about 35 cycles of
// the whole SM: 34 us instead of 27 for 2048 x 8 slots in one launch), and their
// ranks are population counts.
//   ks_small     all of it in one launch: every CTA sorts the whole batch in
//                shared memory (kSmallSlots slots at most) and copies its
//                share of the rows, a warp a row
//                (16 tokens of 2048 columns on 64 experts: 4.4 us)
//   ks_count, ks_tables, ks_copy   the same over tiles of slots: histograms,
//                ranks over the histograms of the tiles before, rows token by
//                token (x is read once); each starts as the one before leaves
#pragma once

#include "norm_kernels.cuh"

namespace deco {
namespace srt {

constexpr int kThreads = 256;          // of a token's CTA
constexpr int kWarps = kThreads / 32;
constexpr int kSortThreads = 512;      // of a tile's CTA
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSmallThreads = 1024;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kMaxE = 256;
constexpr int kMaxS = 256;
constexpr int kSmallSlots = 16384;     // sixteen 32-slot steps a warp
constexpr int kMaxTiles = 148;         // a tile an SM

struct Args {
  int T, S, E, D;             // S slots a token
  int bits;                   // of an expert's number, -1 apart
  const int* experts;         // [T][S], or null
  const uint8_t* active;      // [T][E], or null (S = E)
  long long cap;              // rows of xs
  int *counts, *offsets, *slot_of, *row_of, *n_pairs;
  const void* x;
  void* xs;                   // null: tables only
  long long ld_x, ld_xs;      // bytes
  int row_bytes;
  int tile, n_tiles;          // slots a tile, a multiple of kSortThreads; under a mask: tokens a tile
  int* hist;                  // [n_tiles][E]
};

// expert of slot i of the lists, -1 if none
__device__ __forceinline__ int expert_of(const Args& a, int i) {
  const int e = a.experts[i];
  return (unsigned)e < (unsigned)a.E ? e : -1;
}

// exclusive prefix sum over the CTA's WARPS x 32 threads; *total gets the sum
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

constexpr int kAhead = 4;   // 32-slot steps whose experts are loaded together

// the experts of slots i0 + lane + 32 k, k < N, -1 from i1 on
template <int N>
__device__ __forceinline__ void load_experts(const Args& a, int i0, int i1, int (&e)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = i0 + 32 * k + (threadIdx.x & 31);
    e[k] = i < i1 ? expert_of(a, i) : -1;
  }
}

// lanes whose experts are the same as this lane's, by a ballot on each bit of
// the numbers (-1 is all ones, which `bits` bits leave to no expert)
__device__ __forceinline__ unsigned same_expert(const Args& a, int e) {
  unsigned same = kFull;
#pragma unroll
  for (int b = 0; b < 9; ++b) {
    if (b >= a.bits) break;
    const bool on = (e >> b) & 1;
    const unsigned m = __ballot_sync(kFull, on);
    same &= on ? m : ~m;
  }
  return same;
}

// adds a warp's 32 experts to its own histogram
template <typename H>
__device__ __forceinline__ void add_step(int e, unsigned same, H* hist) {
  const int lane = threadIdx.x & 31;
  if (e >= 0 && (same & ((1u << lane) - 1)) == 0) hist[e] += (H)__popc(same);
  __syncwarp();
}

// the row of a warp's 32 slots, given the first row of each expert in `next`
// (the warp's own; left at the first row behind them); -1: no expert, no room
template <typename H>
__device__ __forceinline__ int rank_step(long long cap, int e, unsigned same, H* next) {
  const int lane = threadIdx.x & 31;
  const int before = __popc(same & ((1u << lane) - 1));
  const int row = e >= 0 ? (int)next[e] + before : -1;
  __syncwarp();
  if (e >= 0 && before == 0) next[e] += (H)__popc(same);
  __syncwarp();
  return row < cap ? row : -1;
}

// A mask's tokens [t0, t1) dealt to a CTA's threads: thread q E + e walks the
// q-th run of `per` tokens of expert e.
struct Walk {
  int e, q, runs, t0, t1;   // t0 >= t1: nothing
  __device__ __forceinline__ Walk(const Args& a, int first, int end, int threads) {
    runs = threads / a.E;
    q = threadIdx.x / a.E;
    e = threadIdx.x - q * a.E;
    const int per = (end - first + runs - 1) / runs;
    t0 = first + q * per;
    t1 = q < runs ? min(end, t0 + per) : t0;
  }
  __device__ __forceinline__ int count(const Args& a) const {
    int n = 0;
#pragma unroll 8
    for (int t = t0; t < t1; ++t) n += a.active[(size_t)t * a.E + e] != 0;
    return n;
  }
};

// The sum of the walks' counts before this one, in order of expert, then run;
// s: a word a thread.  Afterwards s[e * runs] is the sum before expert e.
template <int WARPS>
__device__ __forceinline__ int walk_scan(const Args& a, const Walk& w, int count, int* s, int* wsum, int* total) {
  const int mine = w.q < w.runs ? w.e * w.runs + w.q : (int)threadIdx.x;   // threads without a walk: behind the others
  s[mine] = count;
  __syncthreads();
  const int before = block_scan<WARPS>(s[threadIdx.x], wsum, total);
  s[threadIdx.x] = before;
  __syncthreads();
  return s[mine];
}

__device__ __forceinline__ void write_offsets(const Args& a, int e, int first, int count, int total) {
  const long long cap = a.cap;
  const int f = (int)min((long long)first, cap), l = (int)min((long long)first + count, cap);
  if (e < a.E) {
    a.counts[e] = l - f;
    a.offsets[e] = f;
  }
  if (e == 0) {
    a.offsets[a.E] = (int)min((long long)total, cap);
    *a.n_pairs = total;
  }
}

// copies n bytes; V: the widest access that pointers, strides and n allow
template <typename V>
__device__ __forceinline__ void copy_row(const char* src, char* dst, int n, int lane) {
  const int m = n / (int)sizeof(V);
  int j = lane;
  for (; j + 96 < m; j += 128) {
    V v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = reinterpret_cast<const V*>(src)[j + 32 * q];
#pragma unroll
    for (int q = 0; q < 4; ++q) reinterpret_cast<V*>(dst)[j + 32 * q] = v[q];
  }
  for (; j < m; j += 32) reinterpret_cast<V*>(dst)[j] = reinterpret_cast<const V*>(src)[j];
}

// the rows of the batch, a warp a row, over all CTAs
template <typename V>
__device__ __forceinline__ void copy_rows(const Args& a, const uint16_t* slot, int rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < rows; r += kSmallThreads) a.slot_of[r] = slot[r];
  if (!a.xs) return;
  for (int r = blockIdx.x + warp * gridDim.x; r < rows; r += gridDim.x * kSmallWarps)
    copy_row<V>(static_cast<const char*>(a.x) + (long long)(slot[r] / a.S) * a.ld_x,
                static_cast<char*>(a.xs) + (long long)r * a.ld_xs, a.row_bytes, lane);
}

// STEPS: 32-slot steps of a warp at most
template <typename V, int STEPS>
__global__ void __launch_bounds__(kSmallThreads) ks_small(const Args a) {
  __shared__ __align__(4) uint16_t whist[kSmallWarps][kMaxE];   // counts and rows up to 16384
  static_assert(__alignof__(whist) >= alignof(uint32_t), "zeroed by words");
  extern __shared__ uint16_t s_slot[];             // [slots]
  __shared__ int wsum[kSmallWarps];
  const int n = a.T * a.S, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = ((n + kSmallWarps - 1) / kSmallWarps + 31) / 32 * 32, steps = per / 32;
  const int i0 = warp * per, i1 = min(n, i0 + per);
  int e[STEPS];
  unsigned same[STEPS];
  load_experts(a, i0, i1, e);
  for (int j = threadIdx.x; j < kSmallWarps * kMaxE / 2; j += kSmallThreads) reinterpret_cast<uint32_t*>(&whist[0][0])[j] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    if (k < steps) {
      same[k] = same_expert(a, e[k]);
      add_step(e[k], same[k], whist[warp]);
    }
  __syncthreads();
  const int ex = threadIdx.x;
  int count = 0, total;
  if (ex < kMaxE)
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) count += whist[w][ex];
  const int first = block_scan<kSmallWarps>(count, wsum, &total);
  if (ex < kMaxE) {
    int f = first;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      const int c = whist[w][ex];
      whist[w][ex] = (uint16_t)f;
      f += c;
    }
  }
  __syncthreads();
  const bool writer = blockIdx.x == 0;
  if (writer) write_offsets(a, ex, first, count, total);
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    if (k < steps) {
      const int row = rank_step(a.cap, e[k], same[k], whist[warp]), i = i0 + 32 * k + lane;
      if (row >= 0) s_slot[row] = (uint16_t)i;
      if (writer && i < i1) a.row_of[i] = row;
    }
  __syncthreads();
  copy_rows<V>(a, s_slot, (int)min((long long)total, a.cap));
}

// the same of a mask
template <typename V>
__global__ void __launch_bounds__(kSmallThreads) ks_small_mask(const Args a) {
  __shared__ int s_walk[kSmallThreads], wsum[kSmallWarps];
  extern __shared__ uint16_t s_slot[];
  const Walk w(a, 0, a.T, kSmallThreads);
  // at most kSmallSlots / (kSmallThreads - kMaxE) + 1 = 22 tokens a walk: their bits
  unsigned bits = 0;
#pragma unroll 8
  for (int t = w.t0; t < w.t1; ++t) bits |= (a.active[(size_t)t * a.E + w.e] != 0 ? 1u : 0u) << (t - w.t0);
  int total;
  int row = walk_scan<kSmallWarps>(a, w, __popc(bits), s_walk, wsum, &total);
  const bool writer = blockIdx.x == 0;
  if (writer && (int)threadIdx.x < a.E) {
    const int first = s_walk[threadIdx.x * w.runs], end = (int)threadIdx.x + 1 < a.E ? s_walk[(threadIdx.x + 1) * w.runs] : total;
    write_offsets(a, threadIdx.x, first, end - first, total);
  }
  for (int t = w.t0; t < w.t1; ++t) {
    const int slot = t * a.E + w.e, r = (bits >> (t - w.t0)) & 1 && row < a.cap ? row : -1;
    if ((bits >> (t - w.t0)) & 1) ++row;
    if (r >= 0) s_slot[r] = (uint16_t)slot;
    if (writer) a.row_of[slot] = r;
  }
  __syncthreads();
  copy_rows<V>(a, s_slot, (int)min((long long)total, a.cap));
}

// a warp's part of a tile: its histogram
__device__ __forceinline__ void tile_hist(const Args& a, int i0, int i1, int* hist) {
  for (int i = i0; i < i1; i += 32 * kAhead) {
    int e[kAhead];
    load_experts(a, i, i1, e);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + 32 * k < i1) add_step(e[k], same_expert(a, e[k]), hist);
  }
}

// histogram of each tile of slots
__global__ void __launch_bounds__(kSortThreads) ks_count(const Args a) {
  __shared__ int whist[kSortWarps][kMaxE];
  cudaTriggerProgrammaticLaunchCompletion();
  const int n = a.T * a.S, warp = threadIdx.x >> 5, per = a.tile / kSortWarps;
  for (int j = threadIdx.x; j < kSortWarps * kMaxE; j += kSortThreads) (&whist[0][0])[j] = 0;
  __syncthreads();
  const int i0 = min(n, blockIdx.x * a.tile + warp * per), i1 = min(n, i0 + per);
  tile_hist(a, i0, i1, whist[warp]);
  __syncthreads();
  const int e = threadIdx.x;
  if (e >= a.E) return;
  int count = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) count += whist[w][e];
  a.hist[(size_t)blockIdx.x * a.E + e] = count;
}

// Rows of expert e = threadIdx.x in the tiles before this one (*before) and the
// first row of that expert (returned); CTA 0 writes the offsets.
__device__ __forceinline__ int first_row(const Args& a, int* wsum, int* s_before, int* s_all, int* before) {
  // a few threads an expert, each every so many tiles
  const int parts = min(kSortThreads / a.E, 32);
  int b4 = 0, all = 0;
  const int ex = threadIdx.x % a.E, part = threadIdx.x / a.E;
  if (part < parts)
    for (int b0 = part; b0 < a.n_tiles; b0 += 16 * parts) {   // 16 loads on the way (a loop's remainder would wait for each)
      int v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = b0 + i * parts;
        v[i] = b < a.n_tiles ? a.hist[(size_t)b * a.E + ex] : 0;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        all += v[i];
        if (b0 + i * parts < (int)blockIdx.x) b4 += v[i];
      }
    }
  s_before[threadIdx.x] = b4;
  s_all[threadIdx.x] = all;
  __syncthreads();
  const int e = threadIdx.x;
  b4 = all = 0;
  if (e < a.E)
    for (int p = 0; p < parts; ++p) {
      b4 += s_before[p * a.E + e];
      all += s_all[p * a.E + e];
    }
  int total;
  const int first = block_scan<kSortWarps>(all, wsum, &total);
  if (blockIdx.x == 0) write_offsets(a, e, first, all, total);
  *before = b4;
  return first;
}

__global__ void __launch_bounds__(kSortThreads) ks_tables(const Args a) {
  __shared__ int whist[kSortWarps][kMaxE];
  __shared__ int wsum[kSortWarps];
  __shared__ int s_before[kSortThreads], s_all[kSortThreads];
  cudaTriggerProgrammaticLaunchCompletion();
  const int n = a.T * a.S, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = a.tile / kSortWarps;
  for (int j = threadIdx.x; j < kSortWarps * kMaxE; j += kSortThreads) (&whist[0][0])[j] = 0;
  __syncthreads();
  const int i0 = min(n, blockIdx.x * a.tile + warp * per), i1 = min(n, i0 + per);
  tile_hist(a, i0, i1, whist[warp]);
  cudaGridDependencySynchronize();   // ks_count's histograms are there
  int before;
  const int first = first_row(a, wsum, s_before, s_all, &before);
  const int e = threadIdx.x;
  if (e < kMaxE) {
    int f = first + before;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = whist[w][e];
      whist[w][e] = f;
      f += c;
    }
  }
  __syncthreads();
  for (int i = i0; i < i1; i += 32 * kAhead) {
    int x[kAhead];
    load_experts(a, i, i1, x);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + 32 * k < i1) {
        const int row = rank_step(a.cap, x[k], same_expert(a, x[k]), whist[warp]), slot = i + 32 * k + lane;
        if (slot < i1) a.row_of[slot] = row;
        if (row >= 0) a.slot_of[row] = slot;
      }
  }
}

// the same of a mask; a tile is a.tile tokens
__global__ void __launch_bounds__(kSortThreads) ks_count_mask(const Args a) {
  __shared__ int s_n[kSortThreads];
  cudaTriggerProgrammaticLaunchCompletion();
  const Walk w(a, min(a.T, (int)blockIdx.x * a.tile), min(a.T, ((int)blockIdx.x + 1) * a.tile), kSortThreads);
  s_n[threadIdx.x] = w.count(a);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = warp; e < a.E; e += kSortWarps) {
    int n = 0;
    for (int q = lane; q < w.runs; q += 32) n += s_n[q * a.E + e];
    n = __reduce_add_sync(kFull, n);
    if (lane == 0) a.hist[(size_t)blockIdx.x * a.E + e] = n;
  }
}

__global__ void __launch_bounds__(kSortThreads) ks_tables_mask(const Args a) {
  __shared__ int s_walk[kSortThreads], wsum[kSortWarps];
  __shared__ int s_before[kSortThreads], s_all[kSortThreads], s_row[kMaxE];
  cudaTriggerProgrammaticLaunchCompletion();
  const Walk w(a, min(a.T, (int)blockIdx.x * a.tile), min(a.T, ((int)blockIdx.x + 1) * a.tile), kSortThreads);
  int total, row = walk_scan<kSortWarps>(a, w, w.count(a), s_walk, wsum, &total);
  cudaGridDependencySynchronize();   // ks_count_mask's histograms are there
  int before;
  const int first = first_row(a, wsum, s_before, s_all, &before);
  if ((int)threadIdx.x < a.E) s_row[threadIdx.x] = first + before - s_walk[threadIdx.x * w.runs];   // walks before this expert's do not count
  __syncthreads();
  row += s_row[w.e];
  for (int t = w.t0; t < w.t1; ++t) {
    const int slot = t * a.E + w.e;
    const bool on = a.active[slot] != 0;
    const int r = on && row < a.cap ? row : -1;
    row += on;
    a.row_of[slot] = r;
    if (r >= 0) a.slot_of[r] = slot;
  }
}

// The slots of token t that have a row, in order: their rows and weights, s_k
// their numbers (CTA of any size; barriers inside).  Returns how many there are.
__device__ __forceinline__ int token_rows(const int* row_of, const float* w, long long t, int S, long long n_rows, int* s_row, float* s_w,
                                          int* s_k, int* s_n) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int n = 0;
    for (int k0 = 0; k0 < S; k0 += 32 * kAhead) {
      int row[kAhead];
      float f[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int k = k0 + 32 * q + lane;
        row[q] = k < S ? row_of[t * S + k] : -1;
        f[q] = w && k < S ? w[t * S + k] : 1.f;
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const bool ok = row[q] >= 0 && row[q] < n_rows;
        const unsigned m = __ballot_sync(kFull, ok);
        if (ok) {
          const int at = n + __popc(m & ((1u << lane) - 1));
          s_row[at] = row[q];
          s_w[at] = f[q];
          s_k[at] = k0 + 32 * q + lane;
        }
        n += __popc(m);
      }
    }
    if (lane == 0) *s_n = n;
  }
  __syncthreads();
  return *s_n;
}

// x[t] into the rows of token t; one CTA a token.  Measured: 4096 tokens of 4 KB
// into 13 rows each 38 us, 6.2 TB/s (95 % of a copy's rate); with the histograms
// and tables before it 44 us, or 46 us by a mask of as many pairs (4096 x 64).
template <typename V>
__global__ void __launch_bounds__(kThreads) ks_copy(const Args a) {
  __shared__ int s_row[kMaxS], s_k[kMaxS], s_n;
  __shared__ float s_w[kMaxS];
  const long long t = blockIdx.x;
  const V* x = reinterpret_cast<const V*>(static_cast<const char*>(a.x) + t * a.ld_x);
  const int m = a.row_bytes / (int)sizeof(V);
  V v;
  if ((int)threadIdx.x < m) v = x[threadIdx.x];   // on its way while the table is read
  cudaGridDependencySynchronize();                // ks_tables' rows are there
  const int n = token_rows(a.row_of, nullptr, t, a.S, a.cap, s_row, s_w, s_k, &s_n);
  for (int j = threadIdx.x; j < m;) {
#pragma unroll 4
    for (int r = 0; r < n; ++r) reinterpret_cast<V*>(static_cast<char*>(a.xs) + (long long)s_row[r] * a.ld_xs)[j] = v;
    j += blockDim.x;
    if (j < m) v = x[j];
  }
}

struct CombineArgs {
  int T, S, D;
  long long n_rows;
  const int* row_of;     // [T][S]
  const float* w;        // [T][S] or null (1)
  const void* ys;
  const void* base;      // [T][D] or null
  void* y;
  long long ld_ys, ld_base, ld_y;
};

// y[t] = base[t] + sum_k w ys[row]; grid (T, column blocks), a thread owns 8
// columns.  The sums are in the slots' order, so only loads overlap: 8 rows of
// bf16 at a time (4 at a time 78 us, 8 74 us for 2048 tokens of 26 rows of 8 KB:
// 6.4 TB/s, 98 % of a copy's rate).
constexpr int kCombThreads = 128;
template <typename T, typename TY, int VEC>
__global__ void __launch_bounds__(kCombThreads) ks_combine(const CombineArgs a) {
  __shared__ int s_row[kMaxS], s_k[kMaxS], s_n;
  __shared__ float s_w[kMaxS];
  const long long t = blockIdx.x;
  const nrm::Cols c = nrm::cols_from<T, VEC>(blockIdx.y * blockDim.x * 8, a.D);
  nrm::Seg<T, VEC> sb;
  if (a.base) sb.load(static_cast<const T*>(a.base) + t * a.ld_base, c);   // on its way while the table is read
  const int n = token_rows(a.row_of, a.w, t, a.S, a.n_rows, s_row, s_w, s_k, &s_n);
  float acc[8], v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (a.base) sb.get(acc);
  int r = 0;
  constexpr int kRows = VEC == 8 ? 16 / (int)sizeof(T) : 4;   // rows' loads in flight: 32 registers of them
  for (; r + kRows <= n; r += kRows) {
    nrm::Seg<T, VEC> s[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) s[q].load(static_cast<const T*>(a.ys) + (long long)s_row[r + q] * a.ld_ys, c);
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const float f = s_w[r + q];
      s[q].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f, v[i], acc[i]);
    }
  }
  if (r < n) {                   // the rest, together as well
    nrm::Seg<T, VEC> s[kRows - 1];
#pragma unroll
    for (int q = 0; q < kRows - 1; ++q)
      if (r + q < n) s[q].load(static_cast<const T*>(a.ys) + (long long)s_row[r + q] * a.ld_ys, c);
#pragma unroll
    for (int q = 0; q < kRows - 1; ++q)
      if (r + q < n) {
        const float f = s_w[r + q];
        s[q].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(f, v[i], acc[i]);
      }
  }
  nrm::store8<TY, VEC>(static_cast<TY*>(a.y) + t * a.ld_y, c, acc);
}

struct CombineBwdArgs {
  int T, S, D;
  long long n_rows;
  const int* row_of;
  const float* w;
  const void* ys;
  const void* dy;
  void* dys;
  float* dw;             // [T][S] or null
  long long ld_ys, ld_dy, ld_dys;
};

// dys[row] = w dy[t], dw = dy[t] . ys[row].  One CTA a token, or gridDim.y of
// them that share its rows; a thread holds 8 columns of dy[t] and goes through
// the rows, four at a time.  The four rows' dot products share a butterfly
// (each quarter of the warp ends with one of them); the warps' parts are added
// in warp order.  Measured: 1021 fp32 tokens of 2048 columns with about 13 rows
// each 40 us, 5.6 TB/s (86 % of a copy's rate: a CTA waits for its row table,
// then for its first rows); a warp a row, dy from L1, took 51 us.  2048 bf16
// tokens of 4096 columns with 26 rows each 145 us (95 %).
constexpr int kBwdRows = 4;
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) ks_combine_bwd(const CombineBwdArgs a) {
  __shared__ int s_row[kMaxS], s_k[kMaxS], s_n;
  __shared__ float s_w[kMaxS], s_dot[kMaxS][kWarps + 1];
  const long long t = blockIdx.x;
  nrm::Seg<T, VEC> sd;
  sd.load(static_cast<const T*>(a.dy) + t * a.ld_dy, nrm::cols_from<T, VEC>(0, a.D));   // on its way while the table is read
  const int n = token_rows(a.row_of, a.w, t, a.S, a.n_rows, s_row, s_w, s_k, &s_n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int per = (n + gridDim.y - 1) / gridDim.y, r0 = min(n, (int)blockIdx.y * per), r1 = min(n, r0 + per);
  if (a.dw && blockIdx.y == 0)
    for (int k = threadIdx.x; k < a.S; k += blockDim.x) {   // slots without a row
      const int row = a.row_of[t * a.S + k];
      if (row < 0 || row >= a.n_rows) a.dw[t * a.S + k] = 0.f;
    }
  for (int c0 = 0; c0 < a.D; c0 += blockDim.x * 8) {
    const nrm::Cols c = nrm::cols_from<T, VEC>(c0, a.D);
    float d[8];
    if (c0 > 0) sd.load(static_cast<const T*>(a.dy) + t * a.ld_dy, c);
    sd.get(d);
    for (int r = r0; r < r1; r += kBwdRows) {
      nrm::Seg<T, VEC> sy[kBwdRows];
#pragma unroll
      for (int q = 0; q < kBwdRows; ++q)
        if (r + q < r1) sy[q].load(static_cast<const T*>(a.ys) + (long long)s_row[r + q] * a.ld_ys, c);
      float dot[kBwdRows];
#pragma unroll
      for (int q = 0; q < kBwdRows; ++q) {
        dot[q] = 0.f;
        if (r + q >= r1) continue;
        float y[8];
        sy[q].get(y);
        const float w = s_w[r + q];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[q] = fmaf(d[i], y[i], dot[q]);
          y[i] = w * d[i];
        }
        nrm::store8<T, VEC>(static_cast<T*>(a.dys) + (long long)s_row[r + q] * a.ld_dys, c, y);
      }
      const bool b16 = lane & 16, b8 = lane & 8;
      const float u = (b16 ? dot[2] : dot[0]) + __shfl_xor_sync(kFull, b16 ? dot[0] : dot[2], 16);
      const float v = (b16 ? dot[3] : dot[1]) + __shfl_xor_sync(kFull, b16 ? dot[1] : dot[3], 16);
      float s = (b8 ? v : u) + __shfl_xor_sync(kFull, b8 ? u : v, 8);   // of row 2 b16 + b8
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      const int row = r + (lane >> 3);
      if ((lane & 7) == 0 && row < r1) s_dot[row][warp] = c0 == 0 ? s : s_dot[row][warp] + s;
    }
  }
  __syncthreads();
  if (!a.dw) return;
  for (int r = r0 + threadIdx.x; r < r1; r += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += s_dot[r][w];
    a.dw[t * a.S + s_k[r]] = s;
  }
}

}  // namespace srt
}  // namespace deco
