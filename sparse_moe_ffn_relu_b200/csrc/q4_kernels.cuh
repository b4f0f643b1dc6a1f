// Products with 4-bit weights and group scales:
//   y[t][n] = sum_k x[t][k] W[n][k],  W[n][k] = scale[n][k / G] (code[n][k] - zero[n][k / G])
// (zero = 8 without zero points), for the few rows of a decode batch, plain or
// with each row's own expert's matrix.
//
// The bound is reading the codes: N K / 2 bytes.  The multiply-adds go to the
// tensor cores as m16n8k16 tiles with 16 rows of W and 8 rows of x: a code
// minus its zero is an integer of magnitude <= 15, exact in bf16, made two at
// a time by one logic operation (the code in the low bits of 128.0's
// significand) and one subtraction (128 + zero).  A group's products are
// summed by the tensor core in fp32 and scaled by one fp32 multiply-add per
// group, so the only roundings are those of fp32 sums.  fp32 x enters as three
// bf16 pieces whose sum is exact.
//
// Measured (codes from L2): one token, 2048 x 1024: 3.5 us, the launch and three
// dependent latencies.  16 tokens, 17408 x 2048: 11 us, 1.7 TB/s of weights (26 %
// of a copy's rate), and 16 tokens on the 63 experts of 256 x 2048 that a router
// activates 12 us.  What bounds these is what surrounds the steps (32 rows x 128
// codes a warp): a warp makes four in its life, and of the 678 warp instructions
// that come to each about 250 unpack (112 shifts and logic operations, 64
// subtractions), multiply (32 tensor operations, 8 loads of x) and scale; the
// others make the table of units, stage x, form addresses and add the warps'
// sums.  1 and 8 tokens, 139264 x 2048: 40 and 43 us, 3.5 TB/s (54 %), at 374
// instructions a step: about 25 us of the busiest scheduler's issue slots and 22
// of its integer pipe, neither full, as four warps a scheduler do not cover each
// other's waits.  Every 8 NT rows of x (32 in bf16, 16 in fp32) read and unpack
// all of W again: 64, 256 and 2048 rows of 17408 x 2048 take 29, 103 and 754 us.
//
// Layout: rows padded to Kp, a multiple of 128.  A block of 128 codes is 16
// words of 8; word w sits at place 4 (w % 4) + w / 4, so that the 16 bytes
// that lane t of a quad loads are words t, t + 4, t + 8 and t + 12, and each
// tensor-core step takes 32 consecutive columns from the quad: whole groups
// of 32, 64 or 128.  In a word, code 2 i is in bits 4 i and code 2 i + 1 in
// bits 16 + 4 i: the pair that one operand register holds.
#pragma once

#include <cooperative_groups.h>

#include "norm_kernels.cuh"

namespace deco {
namespace q4 {

constexpr int kBlock = 128;            // codes of a block
constexpr int kWarps = 16;             // of a product's CTA, one CTA an SM
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;             // steps of codes in the ring: two on the way, one in use
constexpr int kMaxE = 256;
constexpr int kMaxCluster = 8;
constexpr int kClusterWidth = 32;      // rows of W in a unit of a cluster, at most
constexpr int kPackWarps = 8;          // making and reading the layout
constexpr int kPackThreads = kPackWarps * 32;

struct Args {
  int N, K, Kp;
  int rows_x;                // rows of x
  long long rows_y;          // rows of y
  const unsigned char* q;    // [E][N][Kp / 2]
  const unsigned char* scale;   // [E][N][Kp / G] bf16
  const uint8_t* zero;       // [E][N][Kp / G], or null
  const void* x;
  void* y;
  long long ld_x, ld_y;
  int x_vec;                 // rows of x allow 8-column loads
  int y_f32;
  int split_log2;            // 2^this warps share a row's K
  int cluster_log2;          // 2^this CTAs share K before that, as a cluster
  int chunk;                 // blocks of K whose x is in shared memory, a warp's (all warps': << split_log2)
  // by expert
  int E;                     // 0: one matrix, row i of y from row i of x
  const int* offsets;        // [E + 1] sorted rows of each expert
  const int* perm;           // row of x of each sorted row, or null
};

// d = a b + c of a 16 x 16 and a 16 x 8 tile; first: c = 0
template <bool kFirst>
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFirst)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// codes 2 i and 2 i + 1 of a word, minus their zero: 128 + code by one logic
// operation, plus bias = -(128 + zero) twice (exact: all are integers below 256)
__device__ __forceinline__ uint32_t dequant(uint32_t word, int i, uint32_t bias) {
  uint32_t v, d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));   // (a & b) | c
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0x3f803f80u), "r"(bias));
  return d;
}

// 8 consecutive columns of a row of x as bf16 pairs: kPieces<T> terms
template <typename T> constexpr int kPieces = 1;
template <> constexpr int kPieces<float> = 3;

__device__ __forceinline__ uint32_t pair_hi(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }

// x = hi + mid + lo exactly, each with at most 8 significant bits; the lower
// terms of an infinity or NaN are 0
__device__ __forceinline__ void split3(float x, uint32_t (&p)[3]) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7f800000u) == 0x7f800000u) {
    p[0] = (u & 0x007fffffu) ? 0x7fff0000u : u;
    p[1] = p[2] = 0;
    return;
  }
  p[0] = u & 0xffff0000u;
  const float r = x - __uint_as_float(p[0]);
  p[1] = __float_as_uint(r) & 0xffff0000u;
  p[2] = __float_as_uint(r - __uint_as_float(p[1]));
}

// columns k .. k + 7 of a row (null: zeros) as operand pairs
__device__ __forceinline__ void load_x(const bf16* row, int k, int K, bool vec, uint32_t (&b)[1][4]) {
  if (vec) {
    const uint4 q = row && k < K ? *reinterpret_cast<const uint4*>(row + k) : uint4{0, 0, 0, 0};
    b[0][0] = q.x; b[0][1] = q.y; b[0][2] = q.z; b[0][3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = row && k + 2 * i < K ? __bfloat16_as_ushort(row[k + 2 * i]) : 0u;
      const uint32_t hi = row && k + 2 * i + 1 < K ? __bfloat16_as_ushort(row[k + 2 * i + 1]) : 0u;
      b[0][i] = lo | hi << 16;
    }
  }
}
__device__ __forceinline__ void load_x(const float* row, int k, int K, bool vec, uint32_t (&b)[3][4]) {
  float v[8];
  if (vec) {
    if (row && k < K) load8(row + k, v);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = row && k + i < K ? row[k + i] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p0[3], p1[3];
    split3(v[2 * i], p0);
    split3(v[2 * i + 1], p1);
#pragma unroll
    for (int p = 0; p < 3; ++p) b[p][i] = pair_hi(p0[p], p1[p]);
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// copy16, or 16 zero bytes
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0) : "memory");
}

// Work is dealt in units: a tile of rows of W (16 M a warp, kWarps / split
// warps side by side) against an item, up to 8 NT rows of x (of one expert).
// Units go item by item; a cursor walks them.
struct Cursor {
  int e, item, row;   // row: the tile's first row of this lane's warp, plus g
};

template <typename T, int NT, int M>
struct Smem {
  static constexpr int kPitch = 16 * M + 4;                       // floats: stores of a warp meet every bank once
  static constexpr int kRing = kThreads * M * 2 * 16 * kStages;   // bytes
  static constexpr int kPart = kWarps * 8 * NT * kPitch * 4;      // partial sums
  static constexpr int kX = 232448 - 4096 - 8 * NT * kClusterWidth * 4 - kRing - kPart;   // what is left for x
  // x: [pieces][8 NT rows] of some blocks of K; rows lie 64 bytes off a
  // multiple of 128 apart, so that a quarter warp's 16-byte loads meet every bank once
  static constexpr int row_bytes(int blocks) { return blocks * kBlock * 2 + 64; }
  static constexpr int x_bytes(int blocks) { return kPieces<T> * 8 * NT * row_bytes(blocks); }
  static constexpr int kMaxBlocks = (kX / (kPieces<T> * 8 * NT) - 64) / (kBlock * 2);
};

// the scales (bf16 pairs) of a block's groups
template <int G>
__device__ __forceinline__ void load_scales(const unsigned char* p, uint32_t (&s)[G == 32 ? 2 : 1]) {
  if constexpr (G == 32) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    s[0] = v.x;
    s[1] = v.y;
  } else if constexpr (G == 64) {
    s[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    s[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}
template <int G>
__device__ __forceinline__ uint32_t load_zeros(const uint8_t* p) {
  if constexpr (G == 32) return *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (G == 64) return *reinterpret_cast<const uint16_t*>(p);
  else return *p;
}

// One CTA an SM walks its share of the units.  The rows of x of the current
// item lie in shared memory, as bf16 pieces.  The codes come through a ring
// there, by asynchronous copies two steps ahead: each lane fetches the 16-byte
// pieces that it multiplies itself, so that waiting for its own copies is all
// the synchronisation they need.  The split warps of a row take consecutive
// parts of K (bpw blocks each) and add their sums in warp order.  A matrix of
// few rows and many columns is shared by the CTAs of a cluster in the same way.
template <typename T, int NT, int M, int G, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) kq_matvec(const Args a) {
  constexpr int kTile = 8 * NT, kWords = G / 32, kS = G == 32 ? 2 : 1, kP = kPieces<T>, kGroups = kBlock / G;
  constexpr int kUnroll = kP * NT * M < 4 ? 2 : 1;   // more would spill
  using S = Smem<T, NT, M>;
  extern __shared__ __align__(16) unsigned char smem[];
  float* part = reinterpret_cast<float*>(smem + S::kRing);
  unsigned char* xs = smem + S::kRing + S::kPart;
  __shared__ int s_first[kMaxE + 1], s_begin[kMaxE], s_end[kMaxE], s_warp[kWarps];
  __shared__ float s_sum[kTile * kClusterWidth];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int split = 1 << a.split_log2;
  const int width_log2 = (M == 1 ? 8 : 9) - a.split_log2, width = 1 << width_log2;   // rows of W in a unit
  const int row0 = (warp >> a.split_log2) * 16 * M + g, part_k = warp & (split - 1);
  const int tiles = (a.N + width - 1) >> width_log2, blocks = a.Kp / kBlock;
  // this CTA's blocks of K, and in them this warp's
  namespace cg = cooperative_groups;
  const int ctas = 1 << a.cluster_log2, rank = a.cluster_log2 ? (int)cg::this_cluster().block_rank() : 0;
  const int cta_blocks = (blocks + ctas - 1) >> a.cluster_log2, cta_block = rank * cta_blocks;
  const int bpw = (cta_blocks + split - 1) >> a.split_log2, first_block = cta_block + part_k * bpw;
  // the items of each expert: s_first, their prefix sums
  int items;
  if (a.E) {
    int n = 0;
    if (tid < a.E) {
      const long long lo = max(a.offsets[tid], 0), hi = min((long long)a.offsets[tid + 1], a.rows_y);
      s_begin[tid] = (int)lo;
      s_end[tid] = (int)hi;
      n = (int)max(hi - lo, 0ll);
    }
    int c = (n + kTile - 1) / kTile, s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) s_warp[warp] = s;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    if (tid < a.E) s_first[tid + 1] = before + s;
    if (tid == 0) s_first[0] = 0;
    __syncthreads();
    items = s_first[a.E];
  } else {
    items = (int)((a.rows_y + kTile - 1) / kTile);
  }
  // this cluster's units: an even share, the first few of the clusters one more
  const unsigned clusters = gridDim.x >> a.cluster_log2, cluster = blockIdx.x >> a.cluster_log2;
  const unsigned units = (unsigned)items * (unsigned)tiles, each = units / clusters, more = units % clusters;
  const unsigned u0 = cluster * each + min(cluster, more);
  const int count = (int)(each + (cluster < more ? 1 : 0));
  if (count == 0) return;
  const int steps = count * bpw;   // a warp's, the ones behind its last block included

  auto next = [&](Cursor& c) {
    c.row += width;
    if (c.row - row0 >= a.N) {
      c.row = row0;
      ++c.item;
      if (a.E && c.item < items)
        while (s_first[c.e + 1] <= c.item) ++c.e;
    }
  };

  Cursor now{0, (int)(u0 / (unsigned)tiles), 0};
  now.row = (int)(u0 - (unsigned)now.item * (unsigned)tiles) * width + row0;
  if (a.E)
    while (s_first[now.e + 1] <= now.item) ++now.e;

  // This lane's rows are row, row + 8, ... of the tile; off(i): from the first of
  // them to the i-th, in strides, no further than the matrix.
  auto first_row = [&](const Cursor& c) { return (uint32_t)min(c.row, a.N - 1); };
  auto off = [&](const Cursor& c, int i) { return (uint32_t)min(8 * i, max(a.N - 1 - c.row, 0) & ~7); };

  // the codes of the next step to fetch
  Cursor ahead = now;
  const uint32_t stride = (uint32_t)a.Kp / 2, ng = (uint32_t)a.Kp / G;
  const unsigned char* q_at;
  uint32_t q_off[2 * M];
  int q_b, left = steps;
  auto aim = [&]() {
    q_at = a.q + (uint64_t)((uint32_t)ahead.e * (uint32_t)a.N + first_row(ahead)) * stride + (uint32_t)(first_block * 64 + t * 16);
#pragma unroll
    for (int i = 1; i < 2 * M; ++i) q_off[i] = off(ahead, i) * stride;
    q_b = 0;
  };
  aim();
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + tid * 16, ring_end = ring + S::kRing;
  const int my_blocks = min(bpw, min(blocks, cta_block + cta_blocks) - first_block);   // of this warp; 0 or less: none
  uint32_t dst = ring;
  auto fetch = [&]() {
    if (left > 0) {
      if (q_b < my_blocks) {
        copy16(dst, q_at);
#pragma unroll
        for (int i = 1; i < 2 * M; ++i) copy16(dst + i * (kThreads * 16), q_at + q_off[i]);
      }
      --left;
      dst += 2 * M * kThreads * 16;
      if (dst == ring_end) dst = ring;
      q_at += 64;
      if (++q_b == bpw) {
        next(ahead);
        aim();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch();

  const int chunks = (bpw + a.chunk - 1) / a.chunk, pitch = S::row_bytes(a.chunk << a.split_log2);
  int item = -1, rows = 0;
  long long r0 = 0;
  // the scales and zeros of the next step
  uint32_t sc[2 * M][kS], zp[2 * M], s_off[2 * M];
  const unsigned char* s_at;
  const uint8_t* z_at;
  auto scales_at = [&](const Cursor& c) {
    const uint64_t at = (uint64_t)((uint32_t)c.e * (uint32_t)a.N + first_row(c)) * ng + (uint32_t)(first_block * kGroups);
    s_at = a.scale + 2 * at;
    if constexpr (ZERO) z_at = a.zero + at;
#pragma unroll
    for (int i = 1; i < 2 * M; ++i) s_off[i] = off(c, i) * ng;
  };
  auto scales = [&](int b) {
    if (b < my_blocks) {
#pragma unroll
      for (int i = 0; i < 2 * M; ++i) {
        load_scales<G>(i ? s_at + 2 * (uint64_t)s_off[i] : s_at, sc[i]);
        if constexpr (ZERO) zp[i] = load_zeros<G>(i ? z_at + s_off[i] : z_at);
      }
      s_at += 2 * kGroups;
      if constexpr (ZERO) z_at += kGroups;
    }
  };
  // x of the item for the steps b0 .. b0 + chunk - 1 of every part of K into
  // shared memory; a row by 512 / 2^ceil(log2 rows) threads
  auto stage = [&](int b0) {
    const int log2 = rows > 1 ? 32 - __clz(rows - 1) : 0, per = kThreads >> log2, row = tid / per;
    if (row >= rows) return;
    const long long r = a.perm ? a.perm[r0 + row] : r0 + row;
    const T* src = r >= 0 && r < a.rows_x ? static_cast<const T*>(a.x) + r * a.ld_x : nullptr;
    const int end = kBlock * (chunks == 1 ? cta_blocks : a.chunk << a.split_log2);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(xs + row * pitch);
#pragma unroll 4
    for (int k = (tid & (per - 1)) * 8; k < end; k += per * 8) {
      int from = cta_block * kBlock + k;
      if (chunks > 1) {                                 // place of K of a column of the chunk
        const int blk = k / kBlock;
        from = (cta_block + blk / a.chunk * bpw + b0 + blk % a.chunk) * kBlock + k % kBlock;
      }
      if (kP == 1 && a.x_vec) {                         // as it is
        const bool in = src && from < a.K;
        copy16_or_zero(to + k * 2, in ? static_cast<const void*>(src + from) : a.x, in);
        continue;
      }
      uint32_t v[kP][4];
      load_x(src, from, a.K, a.x_vec, v);
#pragma unroll
      for (int p = 0; p < kP; ++p) *reinterpret_cast<uint4*>(xs + (p * kTile + row) * pitch + k * 2) = make_uint4(v[p][0], v[p][1], v[p][2], v[p][3]);
    }
  };
  scales_at(now);
  scales(0);
  const bool padded = a.Kp - a.K >= G;
  const uint32_t xw = (uint32_t)__cvta_generic_to_shared(xs) + g * pitch + part_k * a.chunk * (kBlock * 2) + t * 16;
  uint32_t src = ring;
#pragma unroll 1
  for (int u = 0; u < count; ++u) {
    const bool other = now.item != item;                // other rows of x
    if (other) {
      item = now.item;
      if (a.E) {
        r0 = s_begin[now.e] + (long long)(item - s_first[now.e]) * kTile;
        rows = min(kTile, (int)(s_end[now.e] - r0));
      } else {
        r0 = (long long)item * kTile;
        rows = (int)min((long long)kTile, a.rows_y - r0);
      }
    }
    const int nt = (rows + 7) / 8;
    float tot[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[m][n][i] = 0.f;
    uint32_t xk = xw;
#pragma unroll(kUnroll)
    for (int b = 0, in = 0; b < bpw; ++b) {
      if (in == 0 && (other || chunks > 1)) {
        __syncthreads();                                // nobody reads the x before
        stage(b);
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncthreads();
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      uint4 q[2 * M];
      uint32_t s[2 * M][kS], z[2 * M];
#pragma unroll
      for (int i = 0; i < 2 * M; ++i) {
        q[i] = shared16(src + i * (kThreads * 16));
#pragma unroll
        for (int k = 0; k < kS; ++k) s[i][k] = sc[i][k];
        if constexpr (ZERO) z[i] = zp[i];
        else z[i] = 0x08080808u;
      }
      src += 2 * M * kThreads * 16;
      if (src == ring_end) src = ring;
      const uint32_t xb = xk;
      xk += kBlock * 2;
      if (++in == a.chunk) {
        in = 0;
        xk = xw;
      }
      fetch();                                          // into the slot read a step ago
      if (b + 1 < bpw) {                                // the scales one step ahead
        scales(b + 1);
      } else if (u + 1 < count) {
        Cursor then = now;
        next(then);
        scales_at(then);
        scales(0);
      }
      if (b >= my_blocks) continue;
      if (padded && first_block + b + 1 == blocks) {    // groups that are padding: their x is 0, their scales are not used
#pragma unroll
        for (int k = 1; k < kGroups; ++k)
          if ((blocks - 1) * kBlock + k * G >= a.K)
#pragma unroll
            for (int i = 0; i < 2 * M; ++i) s[i][k / 2] &= k & 1 ? 0x0000ffffu : 0u;
      }
      float acc[M][NT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int grp = j / kWords;
        uint32_t f[M][2][4];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const uint32_t wa = j == 0 ? q[2 * m].x : j == 1 ? q[2 * m].y : j == 2 ? q[2 * m].z : q[2 * m].w;
          const uint32_t wb = j == 0 ? q[2 * m + 1].x : j == 1 ? q[2 * m + 1].y : j == 2 ? q[2 * m + 1].z : q[2 * m + 1].w;
          // bytes (zero, 0xc3, zero, 0xc3): -(128 + zero) twice
          const uint32_t ba = __byte_perm(z[2 * m], 0xc3u, 0x4040u + 0x0101u * grp), bb = __byte_perm(z[2 * m + 1], 0xc3u, 0x4040u + 0x0101u * grp);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[m][h][0] = dequant(wa, 2 * h, ba);
            f[m][h][1] = dequant(wb, 2 * h, bb);
            f[m][h][2] = dequant(wa, 2 * h + 1, ba);
            f[m][h][3] = dequant(wb, 2 * h + 1, bb);
          }
        }
        const bool first = j % kWords == 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= nt) break;
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            const uint4 v = shared16(xb + (p * kTile + 8 * n) * pitch + j * 64);
#pragma unroll
            for (int m = 0; m < M; ++m) {
              if (first && p == 0) mma_bf16<true>(acc[m][n], f[m][0], v.x, v.y);
              else mma_bf16<false>(acc[m][n], f[m][0], v.x, v.y);
              mma_bf16<false>(acc[m][n], f[m][1], v.z, v.w);
            }
          }
          if (j % kWords == kWords - 1) {               // the group's scale
#pragma unroll
            for (int m = 0; m < M; ++m) {
              const uint32_t ua = s[2 * m][grp / 2], ub = s[2 * m + 1][grp / 2];
              const float fa = __uint_as_float(grp & 1 ? ua & 0xffff0000u : ua << 16);
              const float fb = __uint_as_float(grp & 1 ? ub & 0xffff0000u : ub << 16);
              tot[m][n][0] = fmaf(fa, acc[m][n][0], tot[m][n][0]);
              tot[m][n][1] = fmaf(fa, acc[m][n][1], tot[m][n][1]);
              tot[m][n][2] = fmaf(fb, acc[m][n][2], tot[m][n][2]);
              tot[m][n][3] = fmaf(fb, acc[m][n][3], tot[m][n][3]);
            }
          }
        }
      }
    }
    float* mine = part + (warp * kTile + 2 * t) * S::kPitch + g;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n >= nt) break;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float* p = mine + 8 * n * S::kPitch + 16 * m;
        p[0] = tot[m][n][0];
        p[S::kPitch] = tot[m][n][1];
        p[8] = tot[m][n][2];
        p[S::kPitch + 8] = tot[m][n][3];
      }
    }
    __syncthreads();
    const int n0 = now.row - row0;
    auto store = [&](int col, int n, float sum) {
      const long long at = (r0 + col) * a.ld_y + n;
      if (a.y_f32) static_cast<float*>(a.y)[at] = sum;
      else static_cast<bf16*>(a.y)[at] = __float2bfloat16_rn(sum);
    };
#pragma unroll 1
    for (int o = tid; o < rows << width_log2; o += kThreads) {
      const int col = o >> width_log2, c = o & (width - 1), n = n0 + c;
      if (n >= a.N) continue;
      const float* p = part + (((c / (16 * M)) << a.split_log2) * kTile + col) * S::kPitch + c % (16 * M);
      float sum = p[0];
#pragma unroll 4
      for (int w = 1; w < split; ++w) sum += p[w * (kTile * S::kPitch)];
      if (a.cluster_log2) s_sum[o] = sum;
      else store(col, n, sum);
    }
    if (a.cluster_log2) {                               // the CTAs' sums, added by the first in rank order
      cg::this_cluster().sync();
      if (rank == 0)
        for (int o = tid; o < rows << width_log2; o += kThreads) {
          const int col = o >> width_log2, n = n0 + (o & (width - 1));
          if (n >= a.N) continue;
          float sum = s_sum[o];
          for (int r = 1; r < ctas; ++r) sum += *cg::this_cluster().map_shared_rank(&s_sum[o], r);
          store(col, n, sum);
        }
      cg::this_cluster().sync();                        // nobody overwrites or leaves before
    }
    if (u + 1 < count) __syncthreads();   // the next unit's sums go to the same place
    next(now);
  }
}

// ---- making and reading the layout: a warp takes a block of 128 codes of a
// row, lane l its columns l, l + 32, l + 64 and l + 96

struct PackArgs {
  long long rows;
  int K, Kp, group;
  const void* src;        // weights [rows][K], or codes (bytes)
  uint32_t* q;
  bf16* scale;
  uint8_t* zero;          // null: symmetric
};

// words from this lane's codes of the four 32-column parts; lanes l % 8 == 0 store
__device__ __forceinline__ void store_codes(uint32_t* block, const uint32_t (&code)[4]) {
  const int lane = threadIdx.x & 31, c = lane & 7, shift = 4 * (c >> 1) + 16 * (c & 1);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = code[i] << shift;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) w[i] |= __shfl_xor_sync(kFull, w[i], o);
  }
  if (c == 0) *reinterpret_cast<uint4*>(block + (lane >> 3) * 4) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Symmetric: scale = max |w| / 7 rounded to bf16, code = round(w / scale) + 8.
// With zero points: lo = min(w, 0), hi = max(w, 0), scale = (hi - lo) / 15,
// zero = round(-lo / scale), code = round(w / scale) + zero.  All in fp32,
// rounded to nearest even and clamped to 0..15; scale 0 gives code = zero.
template <typename T>
__global__ void __launch_bounds__(kPackThreads) kq_quantize(const PackArgs a) {
  const int lane = threadIdx.x & 31, blocks = a.Kp / kBlock;
  const long long id = (long long)blockIdx.x * kPackWarps + (threadIdx.x >> 5);
  if (id >= a.rows * blocks) return;
  const long long row = id / blocks;
  const int k0 = (int)(id % blocks) * kBlock;
  float v[4], lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + 32 * i + lane;
    v[i] = k < a.K ? to_f32(static_cast<const T*>(a.src)[row * a.K + k]) : 0.f;
    lo[i] = fminf(v[i], 0.f);
    hi[i] = fmaxf(v[i], 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo[i] = fminf(lo[i], __shfl_xor_sync(kFull, lo[i], o));
      hi[i] = fmaxf(hi[i], __shfl_xor_sync(kFull, hi[i], o));
    }
  }
  const int per = a.group / 32;   // 32-column parts of a group
  if (per > 1) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      lo[i] = lo[i + 1] = fminf(lo[i], lo[i + 1]);
      hi[i] = hi[i + 1] = fmaxf(hi[i], hi[i + 1]);
    }
  }
  if (per > 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[i] = lo[i + 2] = fminf(lo[i], lo[i + 2]);
      hi[i] = hi[i + 2] = fmaxf(hi[i], hi[i + 2]);
    }
  }
  uint32_t code[4];
  const long long g0 = row * (a.Kp / a.group) + k0 / a.group;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16 sb = __float2bfloat16_rn(a.zero ? __fdiv_rn(hi[i] - lo[i], 15.f) : __fdiv_rn(fmaxf(hi[i], -lo[i]), 7.f));
    const float s = to_f32(sb);
    const float z = !a.zero ? 8.f : s > 0.f ? fminf(rintf(__fdiv_rn(-lo[i], s)), 15.f) : 0.f;
    const int k = k0 + 32 * i + lane;
    code[i] = k < a.K ? (uint32_t)fminf(fmaxf((s > 0.f ? rintf(__fdiv_rn(v[i], s)) : 0.f) + z, 0.f), 15.f) : 0u;
    if (lane == 0 && i % per == 0) {
      a.scale[g0 + i / per] = sb;
      if (a.zero) a.zero[g0 + i / per] = (uint8_t)z;
    }
  }
  store_codes(a.q + id * (kBlock / 8), code);
}

__global__ void __launch_bounds__(kPackThreads) kq_pack(const PackArgs a) {
  const int lane = threadIdx.x & 31, blocks = a.Kp / kBlock;
  const long long id = (long long)blockIdx.x * kPackWarps + (threadIdx.x >> 5);
  if (id >= a.rows * blocks) return;
  const long long row = id / blocks;
  const int k0 = (int)(id % blocks) * kBlock;
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + 32 * i + lane;
    code[i] = k < a.K ? static_cast<const uint8_t*>(a.src)[row * a.K + k] & 15u : 0u;
  }
  store_codes(a.q + id * (kBlock / 8), code);
}

template <typename T>
__global__ void __launch_bounds__(kPackThreads) kq_dequantize(const PackArgs a, T* out) {
  const int lane = threadIdx.x & 31, blocks = a.Kp / kBlock;
  const long long id = (long long)blockIdx.x * kPackWarps + (threadIdx.x >> 5);
  if (id >= a.rows * blocks) return;
  const long long row = id / blocks;
  const int k0 = (int)(id % blocks) * kBlock;
  const uint4 q = *reinterpret_cast<const uint4*>(a.q + id * (kBlock / 8) + (lane >> 3) * 4);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  const int c = lane & 7, shift = 4 * (c >> 1) + 16 * (c & 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + 32 * i + lane;
    if (k >= a.K) continue;
    const long long grp = row * (a.Kp / a.group) + k / a.group;
    const float z = a.zero ? (float)a.zero[grp] : 8.f;
    out[row * a.K + k] = from_f32<T>(to_f32(a.scale[grp]) * ((float)((w[i] >> shift) & 15u) - z));
  }
}

}  // namespace q4
}  // namespace deco
