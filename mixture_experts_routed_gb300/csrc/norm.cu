// norm.cu - the root-mean-square norms that stand before and after a block,
// fused with the block's gate and the residual scale, and their backward.
// With rstd(v) = 1 / sqrt(mean(v^2) + eps) over the d values of a row:
//
//   out = alpha x + beta g * (b rstd(b) w_post)      (post: b the block's output)
//   n   = out rstd(out) w_pre                        (pre: the next block's input)
//
// g is absent (1), one value per token, per channel or per element. Either
// half may be left out; without the post half, out is x. n takes the
// unrounded fp32 out; sums and statistics are fp32, and each output is
// rounded once, when it is stored.
//
// Backward, with yh = out rstd_pre, bh = b rstd_post, u = bh w_post, given
// dout (the residual's gradient at out) and dn:
//   v = dn w_pre        D  = dout + rstd_pre (v - yh mean(v yh))
//   dw_pre = sum_t dn yh                 dx = alpha D
//   G = beta D          dg = G u (summed over what g spans)
//   dw_post = sum_t G g bh
//   v' = G g w_post     db = rstd_post (v' - bh mean(v' bh))
//
// A channel gate keeps one sum, A = sum_t G bh: dw_post = g A, dg = w_post A.
//
// yh wants out as the forward had it, not as bf16 rounded it (each term of
// dw_pre would be off by up to 2^-9): the backward reads x in its place and
// forms out again, in fp32, from x and the b that it reads anyway.
//
// Both directions are bound by HBM: every tensor is read or written once.
// A row is shared by a warp or by a block; each thread copies the vectors of
// its own columns into a ring of rows in shared memory (cp.async: a thread
// waits for its own copies only, so the ring needs no barrier) and reads
// them as often as the sums in between require, while the next rows are on
// their way. Loads into registers instead left too little in flight beside
// the column sums and weights (16384 x 5120 forward: 173 us, now 109, 6.1
// TB/s; 8191 x 7168 backward: 250 us, now 174, 4.7 TB/s).
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kGateToken = 1, kGateChannel = 2, kGateElement = 3;  // (0: none)

// 16 bytes of a row: VEC elements, widened to fp32.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ void widen(const uint4& r, float (&v)[Vec<T>::N]) {
  if constexpr (std::is_same<T, float>::value) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  } else {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Rounded once, to nearest even, into the tensor's type.
template <typename T>
__device__ __forceinline__ void store(T* p, const float (&v)[Vec<T>::N]) {
  if constexpr (std::is_same<T, float>::value) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint4 r;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r.x = w[0];
    r.y = w[1];
    r.z = w[2];
    r.w = w[3];
    *reinterpret_cast<uint4*>(p) = r;
  }
}

// N consecutive fp32 values (16-byte aligned), through L1.
template <int N>
__device__ __forceinline__ void ld_f32(const float* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p + i));
    v[i] = f.x;
    v[i + 1] = f.y;
    v[i + 2] = f.z;
    v[i + 3] = f.w;
  }
}
template <int N>
__device__ __forceinline__ void ld_f32_stream(const float* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint4 f = ld_stream(p + i);
    v[i] = __uint_as_float(f.x);
    v[i + 1] = __uint_as_float(f.y);
    v[i + 2] = __uint_as_float(f.z);
    v[i + 3] = __uint_as_float(f.w);
  }
}

// Two fp32 values in one 64-bit register, and the packed operations on them:
// half the instructions of a row's arithmetic, which with them no longer
// outlasts its bytes.
typedef unsigned long long f2;
__device__ __forceinline__ f2 mk2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f2 dup2(float a) { return mk2(a, a); }
__device__ __forceinline__ float2 un2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <typename T>
__device__ __forceinline__ void widen2(const uint4& r, f2 (&v)[Vec<T>::N / 2]) {
  if constexpr (std::is_same<T, float>::value) {
    v[0] = mk2(__uint_as_float(r.x), __uint_as_float(r.y));
    v[1] = mk2(__uint_as_float(r.z), __uint_as_float(r.w));
  } else {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = mk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ void store2(T* p, const f2 (&v)[Vec<T>::N / 2]) {
  constexpr int N = Vec<T>::N;
  float u[N];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 f = un2(v[i]);
    u[2 * i] = f.x;
    u[2 * i + 1] = f.y;
  }
  store<T>(p, u);
}

template <int N>
__device__ __forceinline__ void store2f(float* p, const f2 (&v)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 2; i += 2) {
    const float2 a = un2(v[i]), b = un2(v[i + 1]);
    reinterpret_cast<float4*>(p)[i / 2] = make_float4(a.x, a.y, b.x, b.y);
  }
}

// Sums of two values over the threads of a row (a warp, or the block), in a
// fixed order; every thread gets them. `buf`: 2 x 32 pairs, `turn` alternates
// so that one barrier is enough.
template <bool WARP>
__device__ __forceinline__ float2 row_sums(float2 v, float2* buf, int& turn) {
  const int lane = threadIdx.x & 31;
  // the lower half of the warp takes the first value, the upper the second
  auto warp_pair = [&](float2 u) {
    const bool up = lane >= 16;
    const float give = up ? u.x : u.y, keep = up ? u.y : u.x;
    float w = keep + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w;
  };
  float w = warp_pair(v);
  if constexpr (!WARP) {
    float2* b = buf + turn * 32;
    turn ^= 1;
    if (lane == 0) b[threadIdx.x >> 5].x = w;
    if (lane == 16) b[threadIdx.x >> 5].y = w;
    __syncthreads();
    w = warp_pair(lane < (blockDim.x >> 5) ? b[lane] : float2{0.f, 0.f});
  }
  return float2{__shfl_sync(0xffffffffu, w, 0), __shfl_sync(0xffffffffu, w, 16)};
}
// one value, over the block
__device__ __forceinline__ float row_sum(float v, float2* buf, int& turn) {
  return row_sums<false>(float2{v, 0.f}, buf, turn).x;
}

struct NormArgs {
  int T, d, gate;
  float eps, alpha, beta;
};

// The gate's N values at (row t, column c).
template <typename T, int N>
__device__ __forceinline__ void gate_at(const void* gate, int kind, float gt, size_t t, int d, int c,
                                        float (&g)[N]) {
  if (kind == kGateChannel) {
    ld_f32<N>(static_cast<const float*>(gate) + c, g);
  } else if (kind == kGateElement) {
    widen<T>(ld_stream(static_cast<const T*>(gate) + t * d + c), g);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = gt;
  }
}

// The weight of the branch at column c: w_post, times a channel gate.
template <int N>
__device__ __forceinline__ void branch_weight(const float* w_post, const void* gate, int kind,
                                              int c, float (&w)[N]) {
  ld_f32<N>(w_post + c, w);
  if (kind == kGateChannel) {
    float g[N];
    ld_f32<N>(static_cast<const float*>(gate) + c, g);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] *= g[i];
  }
}
template <int N>
__device__ __forceinline__ void pack2(const float (&w)[N], f2 (&v)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[i] = mk2(w[2 * i], w[2 * i + 1]);
}

// Threads of a block that takes rows by the warp; other blocks are one row's
// threads, at most two vectors each forward (two small blocks to an SM do
// better there than one wide one, 111 us for 125 at 16384 x 5120), one
// backward.
constexpr int kWarpBlock = 128;
constexpr int kFwdVecs = 2, kBwdVecs = 1;
constexpr int kRowVecs = 1024;  // vectors of the longest row a ring takes

// This thread's copies of one tensor's row.
template <typename T, int V>
__device__ __forceinline__ void ring_fill(uint4* dst, const T* row, int nvec, int tid, int tpr) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * tpr;
    if (i < nvec)
      ptx::cp_async16(ptx::smem_u32(dst + i), row + static_cast<size_t>(i) * Vec<T>::N);
  }
}

// Forward: S rows in flight.
template <typename T, bool WARP, int S, bool POST, bool PRE>
__global__ void __launch_bounds__(WARP ? kWarpBlock : kRowVecs / kFwdVecs, WARP ? 4 : 1)
    norm_ring_kernel(const NormArgs a, const T* __restrict__ x, const T* __restrict__ b,
                     const float* __restrict__ w_post, const void* __restrict__ gate,
                     const float* __restrict__ w_pre, T* __restrict__ out, T* __restrict__ n,
                     float* __restrict__ rstd_post, float* __restrict__ rstd_pre) {
  constexpr int N = Vec<T>::N, H = N / 2, RPB = WARP ? kWarpBlock / 32 : 1;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 buf[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int tpr = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int sub = WARP ? threadIdx.x >> 5 : 0;  // the block's row group
  const int d = a.d, nvec = d / N;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool elem = POST && a.gate == kGateElement;
  const int size = nvec * (1 + (POST ? 1 : 0) + (elem ? 1 : 0));  // a ring slot: x, b, gate
  uint4* mine = ring + static_cast<size_t>(sub) * S * size;
  const int step = gridDim.x * RPB, t0 = blockIdx.x * RPB + sub;
  auto fill = [&](int t, int slot) {
    if (t < a.T) {
      uint4* dst = mine + slot * size;
      const size_t at = static_cast<size_t>(t) * d;
      ring_fill<T, kFwdVecs>(dst, x + at, nvec, tid, tpr);
      if (POST) ring_fill<T, kFwdVecs>(dst + nvec, b + at, nvec, tid, tpr);
      if (elem) ring_fill<T, kFwdVecs>(dst + 2 * nvec, static_cast<const T*>(gate) + at, nvec, tid, tpr);
    }
    ptx::cp_async_commit();
  };
  f2 wb[kFwdVecs][H], wn[kFwdVecs][H];
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fill(t0 + s * step, s);
#pragma unroll
  for (int j = 0; j < kFwdVecs; ++j) {
    const int c = (tid + j * tpr) * N;
    if (c < d) {
      float w[N];
      if constexpr (POST) {
        branch_weight<N>(w_post, gate, a.gate, c, w);
        pack2<N>(w, wb[j]);
      }
      if constexpr (PRE) {
        ld_f32<N>(w_pre + c, w);
        pack2<N>(w, wn[j]);
      }
    }
  }
  const f2 alpha = dup2(a.alpha);
  const bool token = POST && a.gate == kGateToken;
  float gt_next = token && t0 < a.T ? __ldg(static_cast<const float*>(gate) + t0) : 1.f;
  // this thread's part of a row's sum of b^2
  auto b_square = [&](const uint4* in) {
    f2 ss = 0;
    if constexpr (POST) {
#pragma unroll
      for (int j = 0; j < kFwdVecs; ++j) {
        const int i = tid + j * tpr;
        if (i < nvec) {
          f2 v[H];
          widen2<T>(in[nvec + i], v);
#pragma unroll
          for (int q = 0; q < H; ++q) ss = fma2(v[q], v[q], ss);
        }
      }
    }
    const float2 h = un2(ss);
    return h.x + h.y;
  };
  float sum_b = 0.f;
  ptx::cp_async_wait<S - 2>();  // the first row
  if (POST && t0 < a.T) {
    sum_b = row_sums<WARP>(float2{b_square(mine), 0.f}, buf, turn).x;
  }
  int slot = 0;
  for (int t = t0; t < a.T; t += step) {
    // the slot that the row before this one was read from is filled again
    fill(t + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
    ptx::cp_async_wait<S - 2>();  // this row and the next
    const uint4* in = mine + slot * size;
    slot = slot + 1 == S ? 0 : slot + 1;
    const uint4* in_next = mine + slot * size;
    const float gt = gt_next;
    if (token && t + step < a.T) gt_next = __ldg(static_cast<const float*>(gate) + t + step);
    const float rb = POST ? 1.f / sqrtf(fmaf(sum_b, inv_d, a.eps)) : 0.f;
    if (POST && rstd_post != nullptr && tid == 0) rstd_post[t] = rb;
    const size_t at = static_cast<size_t>(t) * d;
    const f2 scale = dup2(a.beta * gt * rb);
    f2 ss = 0;
    f2 y[kFwdVecs][H];
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j) {
      const int i = tid + j * tpr;
      if (i < nvec) {
        widen2<T>(in[i], y[j]);
        if constexpr (POST) {
          f2 v[H];
          widen2<T>(in[nvec + i], v);
#pragma unroll
          for (int q = 0; q < H; ++q) v[q] = mul2(v[q], scale);  // (first: scale may be 0)
          if (elem) {
            f2 g[H];
            widen2<T>(in[2 * nvec + i], g);
#pragma unroll
            for (int q = 0; q < H; ++q) v[q] = mul2(v[q], g[q]);
          }
#pragma unroll
          for (int q = 0; q < H; ++q) y[j][q] = fma2(v[q], wb[j][q], mul2(alpha, y[j][q]));
          store2<T>(out + at + i * N, y[j]);
        }
        if constexpr (PRE) {
#pragma unroll
          for (int q = 0; q < H; ++q) ss = fma2(y[j][q], y[j][q], ss);
        }
      }
    }
    const float2 h = un2(ss);
    const float mine_b = t + step < a.T ? b_square(in_next) : 0.f;
    const float2 sums = row_sums<WARP>(float2{mine_b, h.x + h.y}, buf, turn);
    sum_b = sums.x;
    if constexpr (PRE) {
      const float ro = 1.f / sqrtf(fmaf(sums.y, inv_d, a.eps));
      if (rstd_pre != nullptr && tid == 0) rstd_pre[t] = ro;
      const f2 r2 = dup2(ro);
#pragma unroll
      for (int j = 0; j < kFwdVecs; ++j) {
        const int i = tid + j * tpr;
        if (i < nvec) {
#pragma unroll
          for (int q = 0; q < H; ++q) y[j][q] = mul2(mul2(y[j][q], r2), wn[j][q]);
          store2<T>(n + at + i * N, y[j]);
        }
      }
    }
  }
  ptx::cp_async_wait<0>();
}

// Half a vector, in pairs, from its raw 16 bytes.
template <typename T>
__device__ __forceinline__ void widen_half(const uint4& r, int half, f2 (&v)[Vec<T>::N / 4]) {
  const uint32_t lo = half == 0 ? r.x : r.z, hi = half == 0 ? r.y : r.w;
  if constexpr (std::is_same<T, float>::value) {
    v[0] = mk2(__uint_as_float(lo), __uint_as_float(hi));
  } else {
    v[0] = mk2(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u));
    v[1] = mk2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  }
}
// ... and rounded back into them.
template <typename T>
__device__ __forceinline__ void round_half(uint4& r, int half, const f2 (&v)[Vec<T>::N / 4]) {
  uint32_t w[2];
  if constexpr (std::is_same<T, float>::value) {
    const float2 a = un2(v[0]);
    w[0] = __float_as_uint(a.x);
    w[1] = __float_as_uint(a.y);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = un2(v[i]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  if (half == 0) {
    r.x = w[0];
    r.y = w[1];
  } else {
    r.z = w[0];
    r.w = w[1];
  }
}

// Backward. Each row group walks rows g, g + groups, ... and keeps its rows'
// column sums (of dw_pre; of dw_post, or A of a channel gate) in registers,
// written once to part[group][2][d]; reduce_columns adds the groups in
// order. Factors that a row shares (rstd, beta, a token gate) are taken out
// of the per-element terms, in an order in which no square or cube of rstd
// stands alone: it is up to 1 / sqrt(eps) where the row is all but zero, and
// its cube passes the range at rows of 1e13 and at an eps of 1e-26. A row with
// rstd 0 (its sum of squares passed the range) is zeroed in the ring. The
// first sum of a row is taken a row ahead of the rest; S rows are in the ring,
// each part of a slot filled again as soon as its row is done with it.
// A thread takes one vector, half by half: its sums and weights are 32
// registers, and what a half needs fits beside them at 28 warps to the SM
// (two vectors at 14 warps: 201 us for the 8191 x 7168 backward).
template <typename T, int MAXT, int S, bool POST, bool PRE, bool ELEM>
__global__ void __launch_bounds__(MAXT, MAXT == kWarpBlock ? 4 : 1)
    norm_ring_bwd_kernel(const NormArgs a, const T* __restrict__ dout,
                         const float* __restrict__ dn, const T* __restrict__ x,
                         const T* __restrict__ b, const float* __restrict__ w_post,
                         const void* __restrict__ gate, const float* __restrict__ w_pre,
                         const float* __restrict__ rstd_post, const float* __restrict__ rstd_pre,
                         T* __restrict__ dx, T* __restrict__ db, void* __restrict__ dgate,
                         float* __restrict__ part) {
  constexpr bool WARP = MAXT == kWarpBlock;
  constexpr int N = Vec<T>::N, H = N / 2, Q = N / 4, RPB = WARP ? kWarpBlock / 32 : 1;
  constexpr int P = N / 4;  // 16-byte pieces of dn to a vector
  static_assert(S == 2 || S == 3, "rows in the first ring");
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 buf[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, sub = WARP ? threadIdx.x >> 5 : 0;
  const int d = a.d, nvec = d / N;
  const bool mine = tid < nvec;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool token = POST && a.gate == kGateToken;
  // a slot: dout, x and dn, b, an element gate
  const int off_x = nvec, off_b = PRE ? (2 + P) * nvec : nvec, off_g = off_b + nvec;
  const int size = off_b + (POST ? nvec : 0) + (ELEM ? nvec : 0);
  uint4* slots = ring + static_cast<size_t>(sub) * S * size + tid;
  const int group = blockIdx.x * RPB + sub, step = gridDim.x * RPB;
  auto copy = [&](uint4* dst, const void* src) { ptx::cp_async16(ptx::smem_u32(dst), src); };
  // a row's copies: what a row at work is done with first, and b
  auto fill_rest = [&](int t, uint4* dst) {
    if (t < a.T && mine) {
      const size_t at = static_cast<size_t>(t) * d + tid * N;
      copy(dst, dout + at);
      if constexpr (PRE) {
        copy(dst + off_x, x + at);
#pragma unroll
        for (int q = 0; q < P; ++q) copy(dst + off_x + (1 + q) * nvec, dn + at + q * 4);
      }
      if constexpr (ELEM) copy(dst + off_g, static_cast<const T*>(gate) + at);
    }
  };
  auto fill_b = [&](int t, uint4* dst) {
    if constexpr (POST)
      if (t < a.T && mine) copy(dst + off_b, b + static_cast<size_t>(t) * d + tid * N);
    ptx::cp_async_commit();
  };
  f2 wb[H], wn[H], apre[H] = {}, apost[H] = {};
#pragma unroll
  for (int i = 0; i < S; ++i) {
    fill_rest(group + i * step, slots + i * size);
    fill_b(group + i * step, slots + i * size);
  }
  if (mine) {
    float w[N];
    if constexpr (POST) {
      branch_weight<N>(w_post, gate, a.gate, tid * N, w);
      pack2<N>(w, wb);
    }
    if constexpr (PRE) {
      ld_f32<N>(w_pre + tid * N, w);
      pack2<N>(w, wn);
    }
  }
  // statistics and token gate of a row, the next and, on its way, the one after
  struct Stats {
    float ro, rb, gt;
  };
  auto fetch = [&](int t) {
    Stats r{0.f, 0.f, 1.f};
    if (t < a.T) {
      if (PRE) r.ro = __ldg(rstd_pre + t);
      if (POST) r.rb = __ldg(rstd_post + t);
      if (token) r.gt = __ldg(static_cast<const float*>(gate) + t);
    }
    return r;
  };
  // half h of dn
  auto half_dn = [&](const uint4* in, int h, f2 (&v)[Q]) {
    if constexpr (Q == 2) {
      const uint4 r = in[off_x + (1 + h) * nvec];
      v[0] = mk2(__uint_as_float(r.x), __uint_as_float(r.y));
      v[1] = mk2(__uint_as_float(r.z), __uint_as_float(r.w));
    } else {
      widen_half<T>(in[off_x + nvec], h, v);
    }
  };
  // what a row with rstd 0 has in its norm counts as 0 (each thread reads its
  // own columns only)
  auto drop = [&](uint4* in, const Stats& st) {
    if (POST && st.rb == 0.f && mine) in[off_b] = uint4{};
    if (PRE && st.ro == 0.f && mine) {
#pragma unroll
      for (int q = 0; q <= P; ++q) in[off_x + q * nvec] = uint4{};
    }
  };
  const f2 al = dup2(POST ? a.alpha : 1.f);
  // a row's part of mean(v y), and its terms of dw_pre
  auto first = [&](const uint4* in, const Stats& st) {
    f2 ss = 0;
    if constexpr (PRE) {
      if (mine) {
        const f2 r2 = dup2(st.ro), k = dup2(st.gt * a.beta * st.rb);
        const uint4 xr = in[off_x];
        uint4 br = {}, gr = {};
        if constexpr (POST) br = in[off_b];
        if constexpr (ELEM) gr = in[off_g];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f2 y[Q], v[Q];
          widen_half<T>(xr, h, y);
          if constexpr (POST) {
            f2 u[Q], g[Q];
            widen_half<T>(br, h, u);
            if constexpr (ELEM) widen_half<T>(gr, h, g);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              u[q] = mul2(u[q], wb[h * Q + q]);
              if constexpr (ELEM) u[q] = mul2(u[q], g[q]);
              y[q] = fma2(k, u[q], mul2(al, y[q]));
            }
          }
          half_dn(in, h, v);
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const f2 p = mul2(v[q], y[q]);
            apre[h * Q + q] = fma2(p, r2, apre[h * Q + q]);
            ss = fma2(p, wn[h * Q + q], ss);
          }
        }
      }
    }
    const float2 f = un2(ss);
    return f.x + f.y;
  };
  Stats now = fetch(group), next = fetch(group + step);
  float s1 = 0.f;
  ptx::cp_async_wait<S - 1>();  // the first row
  if (group < a.T) drop(slots, now);
  if (PRE && group < a.T)
    s1 = row_sums<WARP>(float2{first(slots, now), 0.f}, buf, turn).x;
  int slot = 0;
  for (int t = group; t < a.T; t += step) {
    uint4* in = slots + slot * size;
    slot = slot + 1 == S ? 0 : slot + 1;
    uint4* in_next = slots + slot * size;
    const size_t at = static_cast<size_t>(t) * d + tid * N;
    const Stats after = fetch(t + 2 * step);
    const float k = now.gt * a.beta * now.rb;
    // D = dout + ro (v - yh mean(v yh)), dx = alpha D and, of the branch, D w
    f2 v2[H], ss = 0;
    if (mine) {
      const float c = now.ro * s1 * inv_d * now.ro;  // (ro s1 / d is the mean)
      const f2 r2 = dup2(now.ro), cx = dup2(-c * (POST ? a.alpha : 1.f)), cu = dup2(-c * k),
               k2 = dup2(k);
      const uint4 dr = in[0];
      uint4 xr = {}, brr = {}, gr = {}, od, og = {};
      if constexpr (PRE) xr = in[off_x];
      if constexpr (POST) brr = in[off_b];
      if constexpr (ELEM) gr = in[off_g];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f2 D[Q], u[Q], bb[Q], g[Q];
        widen_half<T>(dr, h, D);
        if constexpr (POST) {
          widen_half<T>(brr, h, bb);
          if constexpr (ELEM) widen_half<T>(gr, h, g);
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            u[q] = mul2(bb[q], wb[h * Q + q]);
            if constexpr (ELEM) u[q] = mul2(u[q], g[q]);
          }
        }
        if constexpr (PRE) {
          f2 y[Q], v[Q];
          widen_half<T>(xr, h, y);
          half_dn(in, h, v);
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            v[q] = fma2(y[q], cx, mul2(v[q], wn[h * Q + q]));
            if constexpr (POST) v[q] = fma2(u[q], cu, v[q]);
            D[q] = fma2(v[q], r2, D[q]);
          }
        }
        f2 o[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) o[q] = mul2(al, D[q]);
        round_half<T>(od, h, o);
        if constexpr (POST) {
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            ss = fma2(D[q], u[q], ss);
            bb[q] = mul2(bb[q], k2);
            if constexpr (ELEM) {
              o[q] = mul2(D[q], mul2(bb[q], wb[h * Q + q]));
              D[q] = mul2(D[q], g[q]);
            }
            apost[h * Q + q] = fma2(D[q], bb[q], apost[h * Q + q]);
            v2[h * Q + q] = mul2(D[q], wb[h * Q + q]);
          }
          if constexpr (ELEM) round_half<T>(og, h, o);
        }
      }
      *reinterpret_cast<uint4*>(dx + at) = od;
      if constexpr (ELEM) *reinterpret_cast<uint4*>(static_cast<T*>(dgate) + at) = og;
    }
    fill_rest(t + S * step, in);  // (of this row only b is read again)
    ptx::cp_async_wait<S - 2>();  // the next row
    const float2 f = un2(ss);
    if (t + step < a.T) drop(in_next, next);
    const float ahead = t + step < a.T ? first(in_next, next) : 0.f;
    const float2 sums = row_sums<WARP>(float2{ahead, f.x + f.y}, buf, turn);
    s1 = sums.x;
    if constexpr (POST) {
      // sum of D w b: beta rb of it is a token gate's gradient
      if (token && tid == 0) static_cast<float*>(dgate)[t] = a.beta * now.rb * sums.y;
      if (mine) {
        const f2 kv = dup2(k), mb = dup2(-(now.rb * sums.y * inv_d) * now.rb);
        const uint4 brr = in[off_b];
        uint4 o;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f2 bb[Q];
          widen_half<T>(brr, h, bb);
#pragma unroll
          for (int q = 0; q < Q; ++q) bb[q] = mul2(kv, fma2(mb, bb[q], v2[h * Q + q]));
          round_half<T>(o, h, bb);
        }
        *reinterpret_cast<uint4*>(db + at) = o;
      }
    }
    fill_b(t + S * step, in);
    now = next;
    next = after;
  }
  ptx::cp_async_wait<0>();
  if (mine) {
    float* o = part + static_cast<size_t>(group) * 2 * d + tid * N;
    if (PRE) store2f<N>(o, apre);
    if (POST) store2f<N>(o + d, apost);
  }
}

// Rows too wide for the ring (more than 1024 vectors): 512 threads a row,
// which is read again (from L2) after each sum.
constexpr int kWideThreads = 512;

template <typename T, bool POST, bool PRE>
__global__ void __launch_bounds__(kWideThreads)
    norm_wide_kernel(const NormArgs a, const T* __restrict__ x, const T* __restrict__ b,
                     const float* __restrict__ w_post, const void* __restrict__ gate,
                     const float* __restrict__ w_pre, T* __restrict__ out, T* __restrict__ n,
                     float* __restrict__ rstd_post, float* __restrict__ rstd_pre) {
  constexpr int N = Vec<T>::N, TPR = kWideThreads;
  __shared__ float2 buf[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, d = a.d, nvec = d / N;
  const float inv_d = 1.f / static_cast<float>(d);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t at = static_cast<size_t>(t) * d;
    float rb = 0.f, gt = 1.f, ss = 0.f;
    if constexpr (POST) {
      if (a.gate == kGateToken) gt = __ldg(static_cast<const float*>(gate) + t);
      for (int i = tid; i < nvec; i += TPR) {
        float v[N];
        widen<T>(ld_stream(b + at + i * N), v);
#pragma unroll
        for (int q = 0; q < N; ++q) ss = fmaf(v[q], v[q], ss);
      }
      ss = row_sum(ss, buf, turn);
      rb = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
      if (rstd_post != nullptr && tid == 0) rstd_post[t] = rb;
    }
    auto row_y = [&](int i, float (&y)[N]) {
      widen<T>(ld_stream(x + at + i * N), y);
      if constexpr (POST) {
        float v[N], w[N], g[N];
        widen<T>(ld_stream(b + at + i * N), v);
        ld_f32<N>(w_post + i * N, w);
        gate_at<T, N>(gate, a.gate, gt, t, d, i * N, g);
#pragma unroll
        for (int q = 0; q < N; ++q)
          y[q] = fmaf(a.alpha, y[q], a.beta * g[q] * (v[q] * rb * w[q]));
      }
    };
    ss = 0.f;
    for (int i = tid; i < nvec; i += TPR) {
      float y[N];
      row_y(i, y);
      if (POST) store<T>(out + at + i * N, y);
#pragma unroll
      for (int q = 0; q < N; ++q) ss = fmaf(y[q], y[q], ss);
    }
    if constexpr (PRE) {
      ss = row_sum(ss, buf, turn);
      const float ro = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
      if (rstd_pre != nullptr && tid == 0) rstd_pre[t] = ro;
      for (int i = tid; i < nvec; i += TPR) {
        float y[N], w[N];
        row_y(i, y);
        ld_f32<N>(w_pre + i * N, w);
#pragma unroll
        for (int q = 0; q < N; ++q) y[q] = y[q] * ro * w[q];
        store<T>(n + at + i * N, y);
      }
    }
  }
}

// The column sums of a block live in its part[block][2][d].
template <typename T, bool POST, bool PRE>
__global__ void __launch_bounds__(kWideThreads)
    norm_wide_bwd_kernel(const NormArgs a, const T* __restrict__ dout,
                         const float* __restrict__ dn, const T* __restrict__ x,
                         const T* __restrict__ b, const float* __restrict__ w_post,
                         const void* __restrict__ gate, const float* __restrict__ w_pre,
                         const float* __restrict__ rstd_post, const float* __restrict__ rstd_pre,
                         T* __restrict__ dx, T* __restrict__ db, void* __restrict__ dgate,
                         float* __restrict__ part) {
  constexpr int N = Vec<T>::N, TPR = kWideThreads;
  __shared__ float2 buf[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, d = a.d, nvec = d / N;
  const float inv_d = 1.f / static_cast<float>(d);
  float* part_pre = part + static_cast<size_t>(blockIdx.x) * 2 * d;
  float* part_post = part_pre + d;
  const bool elem = POST && a.gate == kGateElement;
  bool fresh = true;  // this block's first row: the sums start
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, fresh = false) {
    const size_t at = static_cast<size_t>(t) * d;
    const float ro = PRE ? __ldg(rstd_pre + t) : 0.f;
    const float rb = POST ? __ldg(rstd_post + t) : 0.f;
    const bool token = POST && a.gate == kGateToken;
    const float gt = token ? __ldg(static_cast<const float*>(gate) + t) : 1.f;
    auto pre_at = [&](int i, float (&yh)[N], float (&v)[N], float (&w)[N]) {
      widen<T>(ld_stream(x + at + i * N), yh);
      if constexpr (POST) {
        float u[N], wp[N], g[N];
        widen<T>(ld_stream(b + at + i * N), u);
        ld_f32<N>(w_post + i * N, wp);
        gate_at<T, N>(gate, a.gate, gt, t, d, i * N, g);
#pragma unroll
        for (int q = 0; q < N; ++q)
          yh[q] = fmaf(a.alpha, yh[q], a.beta * g[q] * (u[q] * rb * wp[q]));
      }
      ld_f32_stream<N>(dn + at + i * N, v);
      ld_f32<N>(w_pre + i * N, w);
#pragma unroll
      for (int q = 0; q < N; ++q) yh[q] *= ro;
    };
    float s1 = 0.f;
    if constexpr (PRE) {
      for (int i = tid; i < nvec; i += TPR) {
        float yh[N], v[N], w[N];
        pre_at(i, yh, v, w);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          float* o = part_pre + i * N + q;
          *o = fmaf(v[q], yh[q], fresh ? 0.f : *o);
          s1 = fmaf(v[q] * w[q], yh[q], s1);
        }
      }
      s1 = row_sum(s1, buf, turn) * inv_d;
    }
    auto d_at = [&](int i, float (&D)[N]) {
      widen<T>(ld_stream(dout + at + i * N), D);
      if constexpr (PRE) {
        float yh[N], v[N], w[N];
        pre_at(i, yh, v, w);
#pragma unroll
        for (int q = 0; q < N; ++q) D[q] += ro * (v[q] * w[q] - yh[q] * s1);
      }
    };
    // of the branch: G, the element gate's part of it, bh and the weight
    auto branch_at = [&](int i, float (&D)[N], float (&bh)[N], float (&w)[N], float (&g)[N]) {
      widen<T>(ld_stream(b + at + i * N), bh);
      branch_weight<N>(w_post, gate, a.gate, i * N, w);
#pragma unroll
      for (int q = 0; q < N; ++q) g[q] = 1.f;
      if (elem) widen<T>(ld_stream(static_cast<const T*>(gate) + at + i * N), g);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        bh[q] *= rb;
        D[q] *= a.beta;
      }
    };
    const float al = POST ? a.alpha : 1.f;
    float s2 = 0.f;
    for (int i = tid; i < nvec; i += TPR) {
      float D[N], o[N];
      d_at(i, D);
#pragma unroll
      for (int q = 0; q < N; ++q) o[q] = al * D[q];
      store<T>(dx + at + i * N, o);
      if constexpr (POST) {
        float bh[N], w[N], g[N];
        branch_at(i, D, bh, w, g);
        if (elem) {
#pragma unroll
          for (int q = 0; q < N; ++q) o[q] = D[q] * (bh[q] * w[q]);
          store<T>(static_cast<T*>(dgate) + at + i * N, o);
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
          float* s = part_post + i * N + q;
          *s = fmaf(gt * g[q] * D[q], bh[q], fresh ? 0.f : *s);
          s2 = fmaf(D[q] * g[q] * w[q], bh[q], s2);
        }
      }
    }
    if constexpr (POST) {
      s2 = row_sum(s2, buf, turn);
      if (token && tid == 0) static_cast<float*>(dgate)[t] = s2;
      s2 *= inv_d;
      for (int i = tid; i < nvec; i += TPR) {
        float D[N], bh[N], w[N], g[N], o[N];
        d_at(i, D);
        branch_at(i, D, bh, w, g);
#pragma unroll
        for (int q = 0; q < N; ++q) o[q] = rb * gt * (D[q] * g[q] * w[q] - bh[q] * s2);
        store<T>(db + at + i * N, o);
      }
    }
  }
}

// The groups' column sums, in order: 8 slices of the groups, each added in
// order, then the slices in order. z 0: dw_pre; 1: dw_post, or with a channel
// gate A, whence dw_post = g A and dgate = w_post A.
__global__ void __launch_bounds__(256)
    reduce_columns_kernel(const float* __restrict__ part, int groups, int d, int which0,
                          const float* __restrict__ w_post, const float* __restrict__ gate,
                          float* __restrict__ dw_pre, float* __restrict__ dw_post,
                          float* __restrict__ dgate) {
  __shared__ float sm[8][32];
  pdl_wait();
  pdl_trigger();
  const int which = which0 + blockIdx.y;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  const int per = (groups + 7) / 8;
  const int p1 = min(groups, (sl + 1) * per);
  float s = 0.f;
  const float* src = part + static_cast<size_t>(which) * d + c;
#pragma unroll 8
  for (int p = sl * per; p < p1; ++p) s += src[static_cast<size_t>(p) * 2 * d];
  sm[sl][threadIdx.x & 31] = s;
  __syncthreads();
  if (sl == 0) {
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) r += sm[i][threadIdx.x];
    if (which == 0) {
      dw_pre[c] = r;
    } else if (dgate != nullptr) {
      dw_post[c] = __ldg(gate + c) * r;
      dgate[c] = __ldg(w_post + c) * r;
    } else {
      dw_post[c] = r;
    }
  }
}

// Threads to a row of nvec vectors, at most `vecs` each (0: too wide for the
// ring): a warp for short rows, one vector a thread while those are enough.
int threads_of(int nvec, int vecs) {
  if (nvec > kRowVecs) return 0;
  return ceil_div(nvec <= kRowVecs / vecs ? nvec : ceil_div(nvec, vecs), 32) * 32;
}

// Bytes of a row's tensors in the ring.
size_t fwd_slot(int dtype, int d, bool post, bool elem) {
  return static_cast<size_t>(d) * (dtype == 0 ? 4 : 2) * (1 + (post ? 1 : 0) + (elem ? 1 : 0));
}
size_t bwd_slot(int dtype, int d, bool post, bool pre, bool elem) {
  const int es = dtype == 0 ? 4 : 2;
  return static_cast<size_t>(d) *
         (es + (pre ? es + 4 : 0) + (post ? es * (1 + (elem ? 1 : 0)) : 0));
}
constexpr size_t kRingMost = 225 * 1024;  // shared memory an SM has for its blocks' rings
constexpr int kStages = 3;

// Blocks an SM is to hold: what their registers (96 a thread forward, 64
// backward) and rings leave room for.
int blocks_per_sm(int tpr, int regs, size_t ring) {
  const int threads = tpr == 32 ? kWarpBlock : tpr, by_regs = 65536 / (regs * threads);
  const int by_ring = static_cast<int>(kRingMost / ring);
  const int n = by_regs < by_ring ? by_regs : by_ring;
  return n < 1 ? 1 : n;
}

// Backward row groups (each writes its column sums): one wave of blocks of
// the form with both halves, each group with a row of its own where T allows.
int bwd_groups(int dtype, int d, bool elem, int T) {
  const int tpr = threads_of(d / (dtype == 0 ? 4 : 8), kBwdVecs);
  if (tpr == 0) return T < 152 ? T : 152;
  const int rpb = tpr == 32 ? kWarpBlock / 32 : 1;
  const size_t ring = bwd_slot(dtype, d, true, true, elem) * kStages * rpb;
  const int most = 152 * blocks_per_sm(tpr, 64, ring) * rpb;
  return ceil_div(T < most ? T : most, rpb) * rpb;
}

template <typename K, typename... Args>
cudaError_t launch_ring(K kernel, int blocks, int threads, size_t smem, cudaStream_t s,
                        Args... args) {
  if (smem > 47 * 1024) {  // (the default limit is 48 KB, of which the sums take some)
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(blocks), dim3(threads), smem, s, args...);
}

template <typename T, bool POST, bool PRE>
struct Fwd {
  template <typename... Args>
  static cudaError_t go(const NormArgs& a, int num_sms, cudaStream_t s, Args... args) {
    const int tpr = threads_of(a.d / Vec<T>::N, kFwdVecs);
    if (tpr == 0)
      return launch_pdl(norm_wide_kernel<T, POST, PRE>, dim3(a.T < num_sms * 4 ? a.T : num_sms * 4),
                        dim3(kWideThreads), 0, s, a, args...);
    const bool elem = POST && a.gate == kGateElement;
    const int rpb = tpr == 32 ? kWarpBlock / 32 : 1;
    const size_t ring = fwd_slot(sizeof(T) == 4 ? 0 : 1, a.d, POST, elem) * kStages * rpb;
    const int most = num_sms * blocks_per_sm(tpr, 96, ring), blocks = ceil_div(a.T, rpb);
    const int grid = blocks < most ? blocks : most;
    return tpr == 32 ? launch_ring(norm_ring_kernel<T, true, kStages, POST, PRE>, grid, kWarpBlock,
                                   ring, s, a, args...)
                     : launch_ring(norm_ring_kernel<T, false, kStages, POST, PRE>, grid, tpr, ring,
                                   s, a, args...);
  }
};

template <typename T, bool POST, bool PRE>
struct Bwd {
  template <typename... Args>
  static cudaError_t go(const NormArgs& a, int groups, cudaStream_t s, Args... args) {
    const int tpr = threads_of(a.d / Vec<T>::N, kBwdVecs);
    if (tpr == 0)
      return launch_pdl(norm_wide_bwd_kernel<T, POST, PRE>, dim3(groups), dim3(kWideThreads), 0, s,
                        a, args...);
    const int rpb = tpr == 32 ? kWarpBlock / 32 : 1;
    auto ring = [&](int rows) {
      return bwd_slot(sizeof(T) == 4 ? 0 : 1, a.d, POST, PRE, a.gate == kGateElement) * rows * rpb;
    };
    auto run = [&](auto elem) {
      constexpr bool ELEM = POST && decltype(elem)::value;
      if (tpr == 32)
        return launch_ring(norm_ring_bwd_kernel<T, kWarpBlock, kStages, POST, PRE, ELEM>,
                           groups / rpb, kWarpBlock, ring(kStages), s, a, args...);
      // the longest rows leave room for two
      return ring(kStages) <= kRingMost
                 ? launch_ring(norm_ring_bwd_kernel<T, kRowVecs, kStages, POST, PRE, ELEM>, groups,
                               tpr, ring(kStages), s, a, args...)
                 : launch_ring(norm_ring_bwd_kernel<T, kRowVecs, 2, POST, PRE, ELEM>, groups, tpr,
                               ring(2), s, a, args...);
    };
    return a.gate == kGateElement ? run(std::true_type()) : run(std::false_type());
  }
};

template <typename T, template <typename, bool, bool> class K, typename F>
cudaError_t by_halves(bool post, bool pre, F f) {
  if (post && pre) return f(K<T, true, true>());
  if (post) return f(K<T, true, false>());
  return f(K<T, false, true>());
}

template <typename T>
cudaError_t forward_of(const NormArgs& a, int num_sms, cudaStream_t s, const void* x,
                       const void* b, const float* w_post, const void* gate, const float* w_pre,
                       void* out, void* n, float* rstd_post, float* rstd_pre) {
  return by_halves<T, Fwd>(b != nullptr, w_pre != nullptr, [&](auto k) {
    return decltype(k)::go(a, num_sms, s, static_cast<const T*>(x), static_cast<const T*>(b),
                           w_post, gate, w_pre, static_cast<T*>(out), static_cast<T*>(n),
                           rstd_post, rstd_pre);
  });
}
template <typename T>
cudaError_t backward_of(const NormArgs& a, int groups, cudaStream_t s, const void* dout,
                        const float* dn, const void* x, const void* b, const float* w_post,
                        const void* gate, const float* w_pre, const float* rstd_post,
                        const float* rstd_pre, void* dx, void* db, void* dgate, float* part) {
  return by_halves<T, Bwd>(b != nullptr, w_pre != nullptr, [&](auto k) {
    return decltype(k)::go(a, groups, s, static_cast<const T*>(dout), dn,
                           static_cast<const T*>(x), static_cast<const T*>(b), w_post, gate,
                           w_pre, rstd_post, rstd_pre, static_cast<T*>(dx), static_cast<T*>(db),
                           dgate, part);
  });
}

}  // namespace

cudaError_t launch_block_norm(int dtype, int gate_kind, float eps, float alpha, float beta, int T,
                              int d, const void* x, const void* b, const float* w_post,
                              const void* gate, const float* w_pre, void* out, void* n,
                              float* rstd_post, float* rstd_pre, int num_sms, cudaStream_t s) {
  const NormArgs a{T, d, gate_kind, eps, alpha, beta};
  return dtype == 0 ? forward_of<float>(a, num_sms, s, x, b, w_post, gate, w_pre, out, n,
                                        rstd_post, rstd_pre)
                    : forward_of<__nv_bfloat16>(a, num_sms, s, x, b, w_post, gate, w_pre, out, n,
                                                rstd_post, rstd_pre);
}

size_t block_norm_bwd_ws(int dtype, int gate_kind, int T, int d) {
  return static_cast<size_t>(bwd_groups(dtype, d, gate_kind == kGateElement, T)) * 2 * d *
         sizeof(float);
}

cudaError_t launch_block_norm_bwd(int dtype, int gate_kind, float eps, float alpha, float beta,
                                  int T, int d, const void* dout, const float* dn, const void* x,
                                  const void* b, const float* w_post, const void* gate,
                                  const float* w_pre, const float* rstd_post,
                                  const float* rstd_pre, void* dx, void* db, float* dw_post,
                                  void* dgate, float* dw_pre, float* part, cudaStream_t s) {
  const NormArgs a{T, d, gate_kind, eps, alpha, beta};
  const int groups = T > 0 ? bwd_groups(dtype, d, gate_kind == kGateElement, T) : 0;
  if (T > 0) {
    const cudaError_t e =
        dtype == 0 ? backward_of<float>(a, groups, s, dout, dn, x, b, w_post, gate, w_pre,
                                        rstd_post, rstd_pre, dx, db, dgate, part)
                   : backward_of<__nv_bfloat16>(a, groups, s, dout, dn, x, b, w_post, gate, w_pre,
                                                rstd_post, rstd_pre, dx, db, dgate, part);
    if (e != cudaSuccess) return e;
  }
  const bool post = b != nullptr, pre = w_pre != nullptr;
  const bool chan = post && gate_kind == kGateChannel;
  return launch_pdl(reduce_columns_kernel, dim3(d / 32, (post ? 1 : 0) + (pre ? 1 : 0)), dim3(256),
                    0, s, static_cast<const float*>(part), groups, d, pre ? 0 : 1, w_post,
                    chan ? static_cast<const float*>(gate) : nullptr, dw_pre, dw_post,
                    chan ? static_cast<float*>(dgate) : nullptr);
}

}  // namespace moe
