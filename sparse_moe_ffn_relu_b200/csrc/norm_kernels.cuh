// The norms around a block, with the block's gate and residual scale.
//
// With n(v) = v / sqrt(mean v^2 + eps) per row, forward:
//   out = x + c gate * n(y) * g_post          (y the block's output)
//   h   = n(out as stored) * g_pre            (the next block's input)
// and backward, from dout and dh, with o the stored out, a = dh * g_pre,
// r_o = 1 / sqrt(mean o^2 + eps) and r_y likewise:
//   dx      = dout + r_o a - o r_o^3 mean(a o)
//   dg_pre  = sum_t dh o r_o
//   dy      = r_y b - y r_y^3 mean(b y),      b = c dx * gate * g_post
//   dg_post = sum_t c dx * gate * y r_y
//   dgate   = c dx * y r_y * g_post, summed over the axes it is broadcast on
// Without g_post the norm behind the block is left out (n(y) g_post -> y),
// without g_pre the one before the next block, without y the sum.
//
// One row is held in registers between its sums, so every tensor is read once
// and written once: the bound is DRAM.  A thread owns 8 columns, a CTA of up to
// 512 threads (256 in fp32's forward pass) 4096 (2048), a cluster of 2, 4 or 8
// CTAs (sums joined through distributed shared memory) the rows that are wider.
// A row's two norms need two sums after one another forward; backward one round
// of six sums serves both.  CTAs are persistent and walk the rows; the parameter gradients are per-thread fp32 sums over a CTA's rows,
// written once per CTA and added in CTA order by kn_reduce, so they are
// bitwise reproducible.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace deco {
namespace nrm {

constexpr int kMaxThreads = 512;
constexpr int kBwdCta = 512;                          // of the backward pass
constexpr int kCols = 8;                              // columns a thread owns
constexpr int kMaxCluster = 8;
constexpr int kMaxD = 256 * kCols * kMaxCluster;      // 16384

enum Gate { kNone = 0, kChannel = 1, kToken = 2, kFull = 3 };

// 16 bytes read once: not kept in L1.  (Not the read-only path: x may be out.)
__device__ __forceinline__ uint4 ld_once16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The columns a thread owns within its row.  VEC = 8 (D, strides and pointers
// allow 16-byte accesses): two quads of 4, consecutive in a 16-bit row, a
// block's width apart in an fp32 row, so that a warp's 16-byte accesses are
// consecutive.  VEC = 1: single columns a block's width apart, for every other
// D, stride or alignment.
struct Cols {
  int first, step, end;   // VEC = 1: first + i step; VEC = 8: first + (i / 4) step + i % 4; i < 8, while < end
  template <int VEC>
  __device__ __forceinline__ int col(int i) const { return VEC == 8 ? first + (i / 4) * step + i % 4 : first + i * step; }
};

// row `row` of a tensor whose rows are `stride` bytes apart: one multiply-add
__device__ __forceinline__ const char* row_at(const void* base, int row, uint32_t stride) {
  return static_cast<const char*>(base) + (uint64_t)(uint32_t)row * stride;
}
__device__ __forceinline__ char* row_at(void* base, int row, uint32_t stride) { return static_cast<char*>(base) + (uint64_t)(uint32_t)row * stride; }

// 8 columns of a row as loaded
template <typename T, int VEC>
struct Seg;

template <typename T>
struct Seg<T, 8> {
  static constexpr int kQ = (int)sizeof(T) / 2;
  uint4 q[kQ];
  __device__ __forceinline__ void load(const void* row, const Cols& c) {
#pragma unroll
    for (int i = 0; i < kQ; ++i)
      q[i] = c.first + i * c.step < c.end ? ld_once16(static_cast<const T*>(row) + c.first + i * c.step) : uint4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      unpack16(q[0], v);
    } else {
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
};

template <typename T>
struct Seg<T, 1> {
  float v_[8];
  __device__ __forceinline__ void load(const void* row, const Cols& c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = c.first + i * c.step;
      v_[i] = col < c.end ? to_f32(static_cast<const T*>(row)[col]) : 0.f;
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v_[i];
  }
};

// rounds v to T in place and stores it
template <typename T, int VEC>
__device__ __forceinline__ void store8(void* row, const Cols& c, float (&v)[8]) {
  T* p = static_cast<T*>(row);
  if constexpr (VEC == 8) {
    if constexpr (sizeof(T) == 2) {
      if (c.first >= c.end) return;
      uint4 q;
      uint32_t* w = &q.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
      *reinterpret_cast<uint4*>(p + c.first) = q;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (c.first + i * c.step < c.end)
          *reinterpret_cast<float4*>(p + c.first + i * c.step) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = c.first + i * c.step;
      if (col < c.end) {
        const T r = from_f32<T>(v[i]);
        p[col] = r;
        v[i] = to_f32(r);
      }
    }
  }
}

// 8 columns of an fp32 vector [D], 0 where the thread owns none
template <int VEC>
__device__ __forceinline__ void load_vec(const float* g, const Cols& c, float (&v)[8]) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = c.first + i * c.step;
      const float4 f = at < c.end ? *reinterpret_cast<const float4*>(g + at) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * i] = f.x;
      v[4 * i + 1] = f.y;
      v[4 * i + 2] = f.z;
      v[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = c.first + i * c.step;
      v[i] = col < c.end ? g[col] : 0.f;
    }
  }
}

// ---- pairs of fp32 values: one instruction computes both

typedef unsigned long long f2;

__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum_of(const f2 (&v)[2]) {   // of two accumulators
  const float2 a = halves(v[0]), b = halves(v[1]);
  return (a.x + b.x) + (a.y + b.y);
}
template <typename S>
__device__ __forceinline__ void get2(const S& seg, f2 (&v)[4]) {
  float f[8];
  seg.get(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}
// stores v rounded to T; kKeep: v becomes the rounded values
template <typename T, int VEC, bool kKeep>
__device__ __forceinline__ void put2(void* row, const Cols& c, f2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = halves(v[i]);
    f[2 * i] = h.x;
    f[2 * i + 1] = h.y;
  }
  store8<T, VEC>(row, c, f);
  if constexpr (kKeep)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}

// Sums over a row: within a warp, over the warps through shared memory and, in
// a cluster of more than one CTA, over the CTAs in rank order.  Several values
// share the butterflies: where two halves of a warp would add the same two
// values, each half goes on with one of them.  Two buffers in turn, so that one
// barrier per sum is enough: a buffer is written again only after the next
// sum's barrier, which every thread reaches after its last read.
template <int NV>
struct SumBuffers {
  float warp[2][NV][kMaxThreads / 32];  // [buffer][value][warp]; 0 where there is no warp
  float cta[2][NV][kMaxCluster];        // [buffer][value][rank], filled by the peers
};
template <int NV>
struct RowSum {
  SumBuffers<NV>* s;
  int buf, cl;
  __device__ __forceinline__ RowSum(SumBuffers<NV>* buffers, int cluster) : s(buffers), buf(0), cl(cluster) {
    for (int i = threadIdx.x; i < (int)(sizeof(s->warp) / 4); i += blockDim.x) (&s->warp[0][0][0])[i] = 0.f;
    __syncthreads();
    if (cl > 1) cooperative_groups::this_cluster().sync();   // every CTA of the cluster runs before its memory is written
  }
  __device__ __forceinline__ static float half(bool upper, float a, float b, int o) {   // a's sum over the pair in the lower lane, b's in the upper
    return (upper ? b : a) + __shfl_xor_sync(kFull, upper ? a : b, o);
  }
  __device__ __forceinline__ void operator()(float (&v)[NV]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if constexpr (NV == 1) {
      float x = v[0];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
      if (nw > 1) {
        if (lane == 0) s->warp[buf][0][warp] = x;
        __syncthreads();
        x = s->warp[buf][0][lane & 15];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
      }
      v[0] = x;
    } else {
      static_assert(NV == 6, "one value or six");
      const bool b16 = lane & 16, b8 = lane & 8, b4 = lane & 4;
      const float u0 = half(b16, v[0], v[1], 16), u1 = half(b16, v[2], v[3], 16);
      float u2 = half(b16, v[4], v[5], 16);
      u2 += __shfl_xor_sync(kFull, u2, 8);
      float x = half(b4, half(b8, u0, u1, 8), u2, 4);
      x += __shfl_xor_sync(kFull, x, 2);
      x += __shfl_xor_sync(kFull, x, 1);
      const int mine = b4 ? 4 + b16 : 2 * b8 + b16;   // the value that this group of four lanes has (4 and 5: two groups)
      if (nw > 1) {
        static_assert(kMaxThreads / 32 == 16, "four warps' sums a lane");
        if ((lane & 3) == 0) s->warp[buf][mine][warp] = x;   // the second group writes the same
        __syncthreads();
        const float4 w = *reinterpret_cast<const float4*>(&s->warp[buf][mine][4 * (lane & 3)]);
        x = (w.x + w.y) + (w.z + w.w);
        x += __shfl_xor_sync(kFull, x, 2);
        x += __shfl_xor_sync(kFull, x, 1);
      }
      constexpr int kFrom[6] = {0, 16, 8, 24, 4, 20};
#pragma unroll
      for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(kFull, x, kFrom[i]);
    }
    if (cl > 1) {
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      const int rank = (int)cluster.block_rank();
      if ((int)threadIdx.x < cl)
#pragma unroll
        for (int i = 0; i < NV; ++i) *cluster.map_shared_rank(&s->cta[buf][i][rank], (int)threadIdx.x) = v[i];
      cluster.sync();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = 0.f;
        for (int r = 0; r < cl; ++r) v[i] += s->cta[buf][i][r];
      }
    }
    buf ^= 1;
  }
};

// Rows on their way.  VEC = 8: a ring of kRows rows in shared memory, filled by
// asynchronous copies ROWS - 1 rows ahead; a thread fetches the columns that
// it reads itself, so waiting for its own copies is enough.  (Loads into
// registers a row ahead did not help: the compiler moves them down to their
// uses.)  VEC = 1 loads a row when it is needed.
constexpr int ring_rows(int pieces) { return pieces <= 6 ? 3 : 2; }   // with 256 threads: 72 KB at most, 82 KB with two rows
template <int VEC, int PIECES>
struct Ring {
  static constexpr int kRows = ring_rows(PIECES);
  uint32_t begin, end, at;   // shared addresses of this thread's first piece: of the first slot, behind the last, of the next to use
  uint32_t piece;            // bytes from a piece to the next
  __device__ __forceinline__ explicit Ring(unsigned char* smem) {
    piece = blockDim.x * 16;
    begin = at = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    end = begin + kRows * PIECES * piece;
  }
  template <typename T>
  __device__ __forceinline__ void fetch(int p, const char* row, const Cols& c) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      if (c.first + i * c.step < c.end)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + (p + i) * piece),
                     "l"(row + (uint32_t)(c.first + i * c.step) * (uint32_t)sizeof(T))
                     : "memory");
  }
  // zeros where the thread's columns are beyond the row's end: never fetched
  template <typename T>
  __device__ __forceinline__ void clear(int p, const Cols& c) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      if (c.first + i * c.step >= c.end)
        for (int r = 0; r < kRows; ++r)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(begin + (r * PIECES + p + i) * piece), "r"(0) : "memory");
  }
  template <typename T>
  __device__ __forceinline__ void read(int p, Seg<T, 8>& s) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(s.q[i].x), "=r"(s.q[i].y), "=r"(s.q[i].z), "=r"(s.q[i].w)
                   : "r"(at + (p + i) * piece)
                   : "memory");
  }
  __device__ __forceinline__ void turn() {
    at += PIECES * piece;
    if (at == end) at = begin;
  }
  __device__ __forceinline__ void sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kRows - 2) : "memory"); }
};

// the calling thread's columns of the blockDim.x x 8 from `first` on, below `end`
template <typename T, int VEC>
__device__ __forceinline__ Cols cols_from(int first, int end) {
  constexpr int kRun = VEC == 1 ? 1 : 16 / (int)sizeof(T);   // consecutive columns
  Cols c;
  c.first = first + kRun * (int)threadIdx.x;
  c.step = VEC == 1 ? (int)blockDim.x : sizeof(T) == 2 ? 4 : 4 * (int)blockDim.x;
  c.end = min(end, first + (int)blockDim.x * 8);
  return c;
}

template <typename T, int VEC>
__device__ __forceinline__ Cols own_cols(int D, int cl) {
  const int width = ((D + cl - 1) / cl + 7) / 8 * 8;   // columns of a CTA of the cluster
  const int rank = cl > 1 ? (int)cooperative_groups::this_cluster().block_rank() : 0;
  return cols_from<T, VEC>(rank * width, min(D, (rank + 1) * width));
}

struct FwdArgs {
  int T, D, gate_kind, cl;
  float eps, c;
  uint32_t st_x, st_y, st_gate, st_out, st_h;   // bytes from a row to the next
  const void *x, *y, *gate;
  const float *g_post, *g_pre;
  void *out, *h;
};

// Forward.  Measured: 4096 x 4096 bf16 with a full gate 27.6 us, 6.1 TB/s of the
// 168 MB it has to move (94 % of a copy's rate); 8192 x 2048 with a gate per
// channel 24 us in bf16, 47 us in fp32 (86 and 88 %); one token of 2048 columns
// 2.7 us, which is the launch and four dependent latencies.  VEC = 1 waits for
// each row's own loads: 8192 x 2047 bf16 84 us, fp32 64 us.
// pieces of 16 bytes a thread has in a slot of the ring
template <typename T, bool FULL>
constexpr int kFwdPieces = (FULL ? 3 : 2) * (int)sizeof(T) / 2;
// threads of a CTA at most, CTAs an SM (64 registers a thread, 85 or 128)
template <typename T, int VEC>
constexpr int kFwdCta = sizeof(T) == 2 && VEC == 8 ? 512 : 256;
template <typename T, int VEC>
constexpr int kFwdPerSm = sizeof(T) == 4 && VEC == 8 ? 3 : 2;

template <typename T, int VEC, bool FULL>
__global__ void __launch_bounds__(kFwdCta<T, VEC>, kFwdPerSm<T, VEC>) kn_forward(const FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) SumBuffers<1> buffers;
  RowSum<1> sum(&buffers, a.cl);
  const Cols c = own_cols<T, VEC>(a.D, a.cl);
  const float inv_d = 1.f / (float)a.D;
  const int step = gridDim.x / a.cl;
  constexpr int kP = (int)sizeof(T) / 2;
  Ring<VEC, kFwdPieces<T, FULL>> in(smem), out(smem);
  int t = blockIdx.x / a.cl, ahead = t;
  auto fetch = [&]() {
    if (ahead < a.T) {
      in.template fetch<T>(0, row_at(a.x, ahead, a.st_x), c);
      if (a.y) in.template fetch<T>(kP, row_at(a.y, ahead, a.st_y), c);
      if (FULL) in.template fetch<T>(2 * kP, row_at(a.gate, ahead, a.st_gate), c);
      ahead += step;
      in.turn();
    }
    in.sent();
  };
  if constexpr (VEC == 8) {
    in.template clear<T>(0, c);
    in.template clear<T>(kP, c);
    if (FULL) in.template clear<T>(2 * kP, c);
    for (int i = 0; i < in.kRows - 1; ++i) fetch();
  }
  f2 fp[4], fh[4];   // g_post and the channels' gate; g_pre
  {
    float u[8], v[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[i] = w[i] = 1.f;
    if (a.g_post) load_vec<VEC>(a.g_post, c, u);
    if (a.gate_kind == kChannel) load_vec<VEC>(static_cast<const float*>(a.gate), c, v);
    if (a.h) load_vec<VEC>(a.g_pre, c, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fp[i] = pair(u[2 * i] * v[2 * i], u[2 * i + 1] * v[2 * i + 1]);
      fh[i] = pair(w[2 * i], w[2 * i + 1]);
    }
  }
  for (; t < a.T; t += step) {
    Seg<T, VEC> sx, sy, sg;
    if constexpr (VEC == 8) {
      out.wait();
      out.read(0, sx);
      if (a.y) out.read(kP, sy);
      if (FULL) out.read(2 * kP, sg);
      out.turn();
      fetch();       // into the slot read a row ago
    } else {
      sx.load(row_at(a.x, t, a.st_x), c);
      if (a.y) sy.load(row_at(a.y, t, a.st_y), c);
      if (FULL) sg.load(row_at(a.gate, t, a.st_gate), c);
    }
    f2 o[4];
    get2(sx, o);
    if (a.y) {
      f2 y[4];
      get2(sy, y);
      float scale = a.c;
      if (a.g_post) {
        f2 s2[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) s2[i & 1] = fma2(y[i], y[i], s2[i & 1]);
        float ss[1] = {sum_of(s2)};
        sum(ss);
        scale *= rsqrtf(ss[0] * inv_d + a.eps);
      }
      if (a.gate_kind == kToken) scale *= static_cast<const float*>(a.gate)[t];
      if (FULL) {
        f2 g[4];
        get2(sg, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], g[i]);
      }
      const f2 sc = both(scale);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fma2(sc, mul2(y[i], fp[i]), o[i]);
      put2<T, VEC, true>(row_at(a.out, t, a.st_out), c, o);   // o is what was stored from here on
    }
    if (a.h) {
      f2 s2[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) s2[i & 1] = fma2(o[i], o[i], s2[i & 1]);
      float ss[1] = {sum_of(s2)};
      sum(ss);
      const f2 r = both(rsqrtf(ss[0] * inv_d + a.eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mul2(mul2(o[i], r), fh[i]);
      put2<T, VEC, false>(row_at(a.h, t, a.st_h), c, o);
    }
  }
}

struct BwdArgs {
  int T, D, gate_kind, cl;
  float eps, c;
  uint32_t st_x, st_y, st_gate, st_dout, st_dh;   // bytes from a row to the next
  const void *x, *y, *gate, *dout, *dh;      // x: the stored sum
  const float *g_post, *g_pre;
  void *dx, *dy, *dgate;
  float* part;                               // [2][clusters][D]: dg_pre; S (below)
};

// TH: type of dh.  TR: type of dout and dx.
// With a gate per channel, S = sum_t c dx y r_y serves two gradients:
// dg_post = S gate, dgate = S g_post; otherwise S = sum_t c dx gate y r_y = dg_post.
// Backward.  Measured: 8192 x 2048 bf16 with a gate per channel 48 us with
// kn_reduce, of which 35 us grow with the rows (5.7 TB/s, 89 % of a copy's rate;
// 32768 rows take 156 us) and 13 us do not.  Seen of those: kn_reduce, about 4 us,
// and the partial sums, which leave as single floats 32 bytes apart; the rings'
// filling and draining is the likely rest.  In fp32 68 us (91 % of a copy's rate).
// VEC = 1 has no rows on their way: 8192 x 2047 bf16 146 us, fp32 83 us.
template <typename T, typename TH, typename TR, bool FULL>
constexpr int kBwdPieces = ((FULL ? 3 : 2) * (int)sizeof(T) + (int)sizeof(TH) + (int)sizeof(TR)) / 2;

constexpr int kBwdPerSm = 1;   // 128 registers a thread; 768 threads of 80: 51 us instead of 48 at 8192 x 2048
template <typename T, typename TH, typename TR, int VEC, bool FULL>
__global__ void __launch_bounds__(kBwdCta, kBwdPerSm) kn_backward(const BwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) SumBuffers<6> buffers;
  RowSum<6> sum(&buffers, a.cl);
  cudaTriggerProgrammaticLaunchCompletion();   // kn_reduce's blocks may come up as this grid's leave
  const Cols c = own_cols<T, VEC>(a.D, a.cl);
  const float inv_d = 1.f / (float)a.D;
  const int n_clusters = gridDim.x / a.cl, cluster = blockIdx.x / a.cl;
  constexpr int kX = 0, kY = (int)sizeof(T) / 2, kH = 2 * kY, kD = kH + (int)sizeof(TH) / 2, kG = kD + (int)sizeof(TR) / 2;   // pieces
  Ring<VEC, kBwdPieces<T, TH, TR, FULL>> in(smem), out(smem);
  int t = cluster, ahead = t;
  auto fetch = [&]() {
    if (ahead < a.T) {
      if (a.dh) {
        in.template fetch<T>(kX, row_at(a.x, ahead, a.st_x), c);
        in.template fetch<TH>(kH, row_at(a.dh, ahead, a.st_dh), c);
      }
      if (a.y) in.template fetch<T>(kY, row_at(a.y, ahead, a.st_y), c);
      if (a.dout) in.template fetch<TR>(kD, row_at(a.dout, ahead, a.st_dout), c);   // dx may be dout: rows not written yet
      if (FULL) in.template fetch<T>(kG, row_at(a.gate, ahead, a.st_gate), c);
      ahead += n_clusters;
      in.turn();
    }
    in.sent();
  };
  if constexpr (VEC == 8) {
    in.template clear<T>(kX, c);
    in.template clear<T>(kY, c);
    in.template clear<TH>(kH, c);
    in.template clear<TR>(kD, c);
    if (FULL) in.template clear<T>(kG, c);
    for (int i = 0; i < in.kRows - 1; ++i) fetch();
  }
  f2 acc_pre[4], acc[4];
  // g_pre, then g_post and the channels' gate: in shared memory, this thread's 2 x 32 bytes
  f2* const vec = reinterpret_cast<f2*>(smem + (VEC == 8 ? in.end - in.begin : 0)) + 2 * threadIdx.x;
  auto vector_at = [&](int which, f2 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(vec + (2 * which + i) * 2 * blockDim.x);
      v[2 * i] = q.x;
      v[2 * i + 1] = q.y;
    }
  };
  {
    float u[8], v[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[i] = w[i] = 1.f;
    if (a.g_post) load_vec<VEC>(a.g_post, c, u);
    if (a.gate_kind == kChannel) load_vec<VEC>(static_cast<const float*>(a.gate), c, v);
    if (a.dh) load_vec<VEC>(a.g_pre, c, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc_pre[i] = acc[i] = 0;
      vec[(i / 2) * 2 * blockDim.x + i % 2] = pair(w[2 * i], w[2 * i + 1]);
      vec[(2 + i / 2) * 2 * blockDim.x + i % 2] = pair(u[2 * i] * v[2 * i], u[2 * i + 1] * v[2 * i + 1]);
    }
  }
  for (; t < a.T; t += n_clusters) {
    Seg<T, VEC> sx, sy, sg;
    Seg<TH, VEC> sh;
    Seg<TR, VEC> sd;
    if constexpr (VEC == 8) {
      out.wait();
      if (a.dh) {
        out.read(kX, sx);
        out.read(kH, sh);
      }
      if (a.y) out.read(kY, sy);
      if (a.dout) out.read(kD, sd);
      if (FULL) out.read(kG, sg);
      out.turn();
      fetch();
    } else {
      if (a.dh) {
        sx.load(row_at(a.x, t, a.st_x), c);
        sh.load(row_at(a.dh, t, a.st_dh), c);
      }
      if (a.y) sy.load(row_at(a.y, t, a.st_y), c);
      if (a.dout) sd.load(row_at(a.dout, t, a.st_dout), c);
      if (FULL) sg.load(row_at(a.gate, t, a.st_gate), c);
    }
    f2 dx[4], o[4], dh[4], y[4], g[4], f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dx[i] = o[i] = dh[i] = y[i] = 0;
    if (a.dout) get2(sd, dx);
    if (a.dh) {
      get2(sx, o);
      get2(sh, dh);
    }
    if (a.y) get2(sy, y);
    if (FULL) get2(sg, g);
    // One round of sums serves both norms: with a = dh g_pre and z = y gate
    // g_post, sum dx z = sum dout z + r sum a z - r k sum o z.
    float s[6];
    {
      f2 q[6] = {0, 0, 0, 0, 0, 0}, z[4];   // o o, a o, y y, dout z, a z, o z
      vector_at(1, z);
      vector_at(0, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[i] = mul2(z[i], y[i]);
        if (FULL) z[i] = mul2(z[i], g[i]);
        const f2 h = mul2(dh[i], f[i]);
        q[0] = fma2(o[i], o[i], q[0]);
        q[1] = fma2(h, o[i], q[1]);
        q[2] = fma2(y[i], y[i], q[2]);
        q[3] = fma2(dx[i], z[i], q[3]);
        q[4] = fma2(h, z[i], q[4]);
        q[5] = fma2(o[i], z[i], q[5]);
      }
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        const float2 p = halves(q[i]);
        s[i] = p.x + p.y;
      }
    }
    sum(s);
    float dz = s[3];                        // sum dx z (without the token's gate)
    if (a.dh) {
      const float r = rsqrtf(s[0] * inv_d + a.eps), k = s[1] * inv_d * r * r;
      dz = fmaf(r, fmaf(-k, s[5], s[4]), dz);
      const f2 r2 = both(r), k2 = both(-k);
      vector_at(0, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {         // dx += r (dh g_pre - o k)
        const f2 n = mul2(o[i], r2);
        acc_pre[i] = fma2(dh[i], n, acc_pre[i]);
        dx[i] = fma2(r2, mul2(dh[i], f[i]), fma2(n, k2, dx[i]));
      }
    }
    if (a.y) {
      const float gt = a.gate_kind == kToken ? static_cast<const float*>(a.gate)[t] : 1.f;
      const float r = a.g_post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
      const float k = a.g_post ? -dz * inv_d * r * r : 0.f;
      if (a.gate_kind == kToken && threadIdx.x == 0 && c.first == 0) static_cast<float*>(a.dgate)[t] = a.c * r * dz;
      const f2 scale = both(a.c * gt * r), k2 = both(k), cr = both(a.c * r), gt2 = both(gt);
      vector_at(1, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 dm = mul2(mul2(cr, y[i]), dx[i]);      // c dx n(y)
        acc[i] = fma2(dm, FULL ? g[i] : gt2, acc[i]);
        f2 b = mul2(dx[i], f[i]);
        if (FULL) {
          b = mul2(b, g[i]);
          g[i] = mul2(dm, f[i]);
        }
        y[i] = mul2(scale, fma2(y[i], k2, b));
      }
      if (FULL) put2<T, VEC, false>(row_at(a.dgate, t, a.D * (uint32_t)sizeof(T)), c, g);
      put2<T, VEC, false>(row_at(a.dy, t, a.D * (uint32_t)sizeof(T)), c, y);
    }
    put2<TR, VEC, false>(row_at(a.dx, t, a.D * (uint32_t)sizeof(TR)), c, dx);
  }
  const size_t at = (size_t)cluster * a.D;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = c.template col<VEC>(i);
    if (col >= c.end) continue;
    const float2 p = halves(acc_pre[i / 2]), s = halves(acc[i / 2]);
    if (a.dh) a.part[at + col] = i & 1 ? p.y : p.x;
    if (a.g_post || a.gate_kind == kChannel) a.part[(size_t)n_clusters * a.D + at + col] = i & 1 ? s.y : s.x;
  }
}

// The clusters' partial sums added in a fixed order: grid (ceil(D / 32), 2),
// 32 warps of 32 columns each taking every 32nd cluster, then the warps' sums
// by a warp's butterfly per column.
constexpr int kRedWarps = 32;
struct RedArgs {
  int D, n;
  const float* part;
  float *dg_pre, *dg_post, *dgate;   // null: not wanted; dgate: of a gate per channel
  const float *g_post, *gate;        // null: 1
};
__global__ void __launch_bounds__(kRedWarps * 32) kn_reduce(const RedArgs a) {
  const bool pre = blockIdx.y == 0;
  cudaGridDependencySynchronize();   // launched while kn_backward still runs
  if (pre ? !a.dg_pre : !a.dg_post && !a.dgate) return;
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < a.D) {
    const float* p = a.part + (size_t)(pre ? 0 : a.n) * a.D + col;
#pragma unroll 8
    for (int g = warp; g < a.n; g += kRedWarps) s += p[(size_t)g * a.D];
  }
  sm[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sm[lane][warp]);
  const int out = blockIdx.x * 32 + warp;
  if (lane != 0 || out >= a.D) return;
  if (pre) {
    a.dg_pre[out] = s;
  } else {
    if (a.dg_post) a.dg_post[out] = s * (a.dgate ? a.gate[out] : 1.f);
    if (a.dgate) a.dgate[out] = s * (a.g_post ? a.g_post[out] : 1.f);
  }
}

}  // namespace nrm
}  // namespace deco
