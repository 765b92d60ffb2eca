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
// Both directions are bound by HBM: every tensor is read or written once,
// a row held in registers between the two reductions it needs.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateElement = 3;

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

// Sum over the TPR threads of a row, in a fixed order; every thread gets it.
// `buf`: the row's 2 x 32 floats, `turn` alternates so that one barrier per
// sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* b = buf + turn * 32;
    turn ^= 1;
    if (lane == 0) b[w] = v;
    __syncthreads();
    v = lane < W ? b[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
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

constexpr int block_of(int tpr) { return tpr < 128 ? 128 : tpr; }

// A row is shared by TPR threads, each holding up to NV vectors of it.
// NV = 0: rows too wide for registers; the row is read again (from L2) after
// each sum.
template <typename T, int TPR, int NV, bool POST, bool PRE>
__global__ void __launch_bounds__(block_of(TPR))
    block_norm_kernel(const NormArgs a, const T* __restrict__ x, const T* __restrict__ b,
                      const float* __restrict__ w_post, const void* __restrict__ gate,
                      const float* __restrict__ w_pre, T* __restrict__ out, T* __restrict__ n,
                      float* __restrict__ rstd_post, float* __restrict__ rstd_pre) {
  constexpr int N = Vec<T>::N;
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float buf[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int tid = RPB == 1 ? threadIdx.x : threadIdx.x % TPR;
  const int d = a.d, nvec = d / N;
  const float inv_d = 1.f / static_cast<float>(d);
  for (size_t t = static_cast<size_t>(blockIdx.x) * RPB + threadIdx.x / TPR; t < a.T;
       t += static_cast<size_t>(gridDim.x) * RPB) {
    const T* xr = x + t * d;
    const T* br = POST ? b + t * d : nullptr;
    constexpr int M = NV > 0 ? NV : 1;
    uint4 xv[M], bv[M];
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * TPR;
        if (i < nvec) {
          if (POST) bv[j] = ld_stream(br + i * N);
          xv[j] = ld_stream(xr + i * N);
        }
      }
    }
    float rb = 0.f, gt = 1.f;
    if constexpr (POST) {
      if (a.gate == kGateToken) gt = __ldg(static_cast<const float*>(gate) + t);
      float ss = 0.f;
      auto square = [&](const uint4& raw) {
        float v[N];
        widen<T>(raw, v);
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(v[i], v[i], ss);
      };
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (tid + j * TPR < nvec) square(bv[j]);
      } else {
        for (int i = tid; i < nvec; i += TPR) square(ld_stream(br + static_cast<size_t>(i) * N));
      }
      ss = row_sum<TPR>(ss, buf, turn);
      rb = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
      if (rstd_post != nullptr && tid == 0) rstd_post[t] = rb;
    }
    // y = alpha x + beta g (b rb w_post) at vector i
    auto row_y = [&](int i, const uint4& xraw, const uint4& braw, float (&y)[N]) {
      widen<T>(xraw, y);
      if constexpr (POST) {
        float bb[N], w[N], g[N];
        widen<T>(braw, bb);
        ld_f32<N>(w_post + i * N, w);
        gate_at<T, N>(gate, a.gate, gt, t, d, i * N, g);
#pragma unroll
        for (int q = 0; q < N; ++q)
          y[q] = fmaf(a.alpha, y[q], a.beta * g[q] * (bb[q] * rb * w[q]));
      }
    };
    float ss = 0.f;
    float y[M][N];
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * TPR;
        if (i < nvec) {
          row_y(i, xv[j], bv[j], y[j]);
          if (POST) store<T>(out + t * d + i * N, y[j]);
          if (PRE) {
#pragma unroll
            for (int q = 0; q < N; ++q) ss = fmaf(y[j][q], y[j][q], ss);
          }
        }
      }
    } else {
      for (int i = tid; i < nvec; i += TPR) {
        row_y(i, ld_stream(xr + static_cast<size_t>(i) * N),
              POST ? ld_stream(br + static_cast<size_t>(i) * N) : uint4{}, y[0]);
        if (POST) store<T>(out + t * d + static_cast<size_t>(i) * N, y[0]);
        if (PRE) {
#pragma unroll
          for (int q = 0; q < N; ++q) ss = fmaf(y[0][q], y[0][q], ss);
        }
      }
    }
    if constexpr (PRE) {
      ss = row_sum<TPR>(ss, buf, turn);
      const float ro = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
      if (rstd_pre != nullptr && tid == 0) rstd_pre[t] = ro;
      auto put = [&](int i, float (&v)[N]) {
        float w[N];
        ld_f32<N>(w_pre + i * N, w);
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = v[q] * ro * w[q];
        store<T>(n + t * d + static_cast<size_t>(i) * N, v);
      };
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (tid + j * TPR < nvec) put(tid + j * TPR, y[j]);
      } else {
        for (int i = tid; i < nvec; i += TPR) {
          row_y(i, ld_stream(xr + static_cast<size_t>(i) * N),
                POST ? ld_stream(br + static_cast<size_t>(i) * N) : uint4{}, y[0]);
          put(i, y[0]);
        }
      }
    }
  }
}

// Backward. Each group of TPR threads walks rows g, g + groups, ... and keeps
// its rows' column sums (dw_pre, dw_post, a channel gate's dgate) in
// registers, written once to part[group][3][d]; reduce_columns adds the
// groups in order. NV = 0: the sums live in part itself.
template <typename T, int TPR, int NV, bool POST, bool PRE>
__global__ void __launch_bounds__(block_of(TPR))
    block_norm_bwd_kernel(const NormArgs a, const T* __restrict__ dout,
                          const float* __restrict__ dn, const T* __restrict__ yo,
                          const T* __restrict__ b, const float* __restrict__ w_post,
                          const void* __restrict__ gate, const float* __restrict__ w_pre,
                          const float* __restrict__ rstd_post,
                          const float* __restrict__ rstd_pre, T* __restrict__ dx,
                          T* __restrict__ db, void* __restrict__ dgate,
                          float* __restrict__ part) {
  constexpr int N = Vec<T>::N;
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float buf[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int tid = RPB == 1 ? threadIdx.x : threadIdx.x % TPR;
  const int d = a.d, nvec = d / N;
  const float inv_d = 1.f / static_cast<float>(d);
  const size_t group = static_cast<size_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  float* part_pre = part + group * 3 * d;
  float* part_post = part_pre + d;
  float* part_gate = part_post + d;
  const bool chan = POST && a.gate == kGateChannel;
  constexpr int M = NV > 0 ? NV : 1;
  float apre[M][N] = {}, apost[M][N] = {}, agate[M][N] = {};
  if constexpr (NV == 0) {
    for (int c = tid; c < 3 * d; c += TPR) part_pre[c] = 0.f;
    __syncthreads();
  }
  for (size_t t = group; t < a.T; t += static_cast<size_t>(gridDim.x) * RPB) {
    const size_t row = t * d;
    const float ro = PRE ? __ldg(rstd_pre + t) : 0.f;
    const float rb = POST ? __ldg(rstd_post + t) : 0.f;
    const float gt = POST && a.gate == kGateToken ? __ldg(static_cast<const float*>(gate) + t)
                                                  : 1.f;
    // D (in place of dout) and, first, sum of v yh
    float s1 = 0.f;
    float D[M][N], yh[M][N], v[M][N], bh[M][N];
    auto load = [&](int i, float (&D_)[N], float (&yh_)[N], float (&v_)[N]) {
      widen<T>(ld_stream(dout + row + static_cast<size_t>(i) * N), D_);
      if constexpr (PRE) {
        float w[N];
        widen<T>(ld_stream(yo + row + static_cast<size_t>(i) * N), yh_);
        ld_f32_stream<N>(dn + row + static_cast<size_t>(i) * N, v_);
        ld_f32<N>(w_pre + i * N, w);
#pragma unroll
        for (int q = 0; q < N; ++q) yh_[q] *= ro;
      }
    };
    auto first = [&](int i, float (&yh_)[N], float (&v_)[N], float (&acc)[N]) {
      float w[N];
      ld_f32<N>(w_pre + i * N, w);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        acc[q] = fmaf(v_[q], yh_[q], acc[q]);
        v_[q] *= w[q];
        s1 = fmaf(v_[q], yh_[q], s1);
      }
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * TPR;
        if (i < nvec) {
          load(i, D[j], yh[j], v[j]);
          if constexpr (POST) widen<T>(ld_stream(b + row + static_cast<size_t>(i) * N), bh[j]);
        }
      }
      if constexpr (PRE) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (tid + j * TPR < nvec) first(tid + j * TPR, yh[j], v[j], apre[j]);
      }
    } else if constexpr (PRE) {
      for (int i = tid; i < nvec; i += TPR) {
        load(i, D[0], yh[0], v[0]);
        float acc[N];
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] = part_pre[i * N + q];
        first(i, yh[0], v[0], acc);
#pragma unroll
        for (int q = 0; q < N; ++q) part_pre[i * N + q] = acc[q];
      }
    }
    if constexpr (PRE) s1 = row_sum<TPR>(s1, buf, turn) * inv_d;
    // dx = alpha D (D itself without the post half); then the branch: G = beta D
    float s2 = 0.f, sg = 0.f;
    const float al = POST ? a.alpha : 1.f;
    auto second = [&](int i, float (&D_)[N], float (&yh_)[N], float (&v_)[N], float (&bh_)[N],
                      float (&ap)[N], float (&ag)[N], bool put) {
      float o[N];
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if constexpr (PRE) D_[q] += ro * (v_[q] - yh_[q] * s1);
        o[q] = al * D_[q];
      }
      if (put) store<T>(dx + row + static_cast<size_t>(i) * N, o);
      if constexpr (POST) {
        float w[N], g[N], e[N];
        ld_f32<N>(w_post + i * N, w);
        gate_at<T, N>(gate, a.gate, gt, t, d, i * N, g);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const float G = a.beta * D_[q];
          bh_[q] *= rb;
          const float gu = G * (bh_[q] * w[q]);
          const float gg = G * g[q];
          e[q] = gu;
          sg += gu;
          ap[q] = fmaf(gg, bh_[q], ap[q]);
          ag[q] += gu;
          D_[q] = gg * w[q];  // v'
          s2 = fmaf(D_[q], bh_[q], s2);
        }
        if (a.gate == kGateElement && put)
          store<T>(static_cast<T*>(dgate) + row + static_cast<size_t>(i) * N, e);
      }
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (tid + j * TPR < nvec)
          second(tid + j * TPR, D[j], yh[j], v[j], bh[j], apost[j], agate[j], true);
    } else {
      for (int i = tid; i < nvec; i += TPR) {
        load(i, D[0], yh[0], v[0]);
        if constexpr (PRE) {
          float none[N] = {}, keep = s1;
          first(i, yh[0], v[0], none);
          s1 = keep;
        }
        float ap[N] = {}, ag[N] = {};
        if constexpr (POST) widen<T>(ld_stream(b + row + static_cast<size_t>(i) * N), bh[0]);
        second(i, D[0], yh[0], v[0], bh[0], ap, ag, true);
        if constexpr (POST) {
#pragma unroll
          for (int q = 0; q < N; ++q) {
            part_post[i * N + q] += ap[q];
            if (chan) part_gate[i * N + q] += ag[q];
          }
        }
      }
    }
    if constexpr (POST) {
      s2 = row_sum<TPR>(s2, buf, turn) * inv_d;
      if (a.gate == kGateToken) {
        sg = row_sum<TPR>(sg, buf, turn);
        if (tid == 0) static_cast<float*>(dgate)[t] = sg;
      }
      auto third = [&](int i, float (&v2)[N], float (&bh_)[N]) {
        float o[N];
#pragma unroll
        for (int q = 0; q < N; ++q) o[q] = rb * (v2[q] - bh_[q] * s2);
        store<T>(db + row + static_cast<size_t>(i) * N, o);
      };
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (tid + j * TPR < nvec) third(tid + j * TPR, D[j], bh[j]);
      } else {
        for (int i = tid; i < nvec; i += TPR) {
          load(i, D[0], yh[0], v[0]);
          if constexpr (PRE) {
            float none[N] = {}, keep = s1;
            first(i, yh[0], v[0], none);
            s1 = keep;
          }
          float ap[N] = {}, ag[N] = {};
          widen<T>(ld_stream(b + row + static_cast<size_t>(i) * N), bh[0]);
          const float mean = s2;
          second(i, D[0], yh[0], v[0], bh[0], ap, ag, false);
          s2 = mean;
          third(i, D[0], bh[0]);
        }
      }
    }
  }
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * TPR;
      if (i >= nvec) continue;
#pragma unroll
      for (int q = 0; q < N; q += 4) {
        if (PRE)
          *reinterpret_cast<float4*>(part_pre + i * N + q) =
              make_float4(apre[j][q], apre[j][q + 1], apre[j][q + 2], apre[j][q + 3]);
        if (POST)
          *reinterpret_cast<float4*>(part_post + i * N + q) =
              make_float4(apost[j][q], apost[j][q + 1], apost[j][q + 2], apost[j][q + 3]);
        if (chan)
          *reinterpret_cast<float4*>(part_gate + i * N + q) =
              make_float4(agate[j][q], agate[j][q + 1], agate[j][q + 2], agate[j][q + 3]);
      }
    }
  }
}

// o[c] = sum over groups p of part[p][which][c], in order: 8 slices of the
// groups, each added in order, then the slices in order.
__global__ void __launch_bounds__(256)
    reduce_columns_kernel(const float* __restrict__ part, int groups, int d,
                          float* __restrict__ o_pre, float* __restrict__ o_post,
                          float* __restrict__ o_gate) {
  __shared__ float sm[8][32];
  pdl_wait();
  pdl_trigger();
  float* outs[3] = {o_pre, o_post, o_gate};
  float* o = outs[blockIdx.y];
  if (o == nullptr) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  const int per = (groups + 7) / 8;
  const int p1 = min(groups, (sl + 1) * per);
  float s = 0.f;
  const float* src = part + static_cast<size_t>(blockIdx.y) * d + c;
#pragma unroll 8
  for (int p = sl * per; p < p1; ++p) s += src[static_cast<size_t>(p) * 3 * d];
  sm[sl][threadIdx.x & 31] = s;
  __syncthreads();
  if (sl == 0) {
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) r += sm[i][threadIdx.x];
    o[c] = r;
  }
}

// How a row of nvec vectors is shared: the narrowest group that holds it
// with at most `most` vectors a thread; few rows take wider groups, so that
// the one wave they are runs with as much memory in flight as it can.
struct Shape {
  int tpr, nv;
};
Shape shape_of(int nvec, int T, int most) {
  static const int widths[4] = {32, 128, 256, 512};
  if (T <= kNormFewRows) {
    for (int w : {32, 128, 256, 512})
      if (nvec <= w) return {w, 1};
    if (nvec <= 1024) return {512, 2};
  }
  for (int w : widths)
    if (nvec <= w * most) {
      const int nv = ceil_div(nvec, w);
      return {w, nv > 2 ? 4 : nv};
    }
  return {512, 0};
}

template <typename T, bool POST, bool PRE>
struct Fwd {
  static constexpr int kMost = 4;  // vectors a thread holds
  template <int TPR, int NV>
  static cudaError_t go(const NormArgs& a, int groups, const void* x, const void* b,
                        const float* w_post, const void* gate, const float* w_pre, void* out,
                        void* n, float* rstd_post, float* rstd_pre, cudaStream_t s) {
    constexpr int RPB = block_of(TPR) / TPR;
    return launch_pdl(block_norm_kernel<T, TPR, NV, POST, PRE>, dim3(ceil_div(groups, RPB)),
                      dim3(block_of(TPR)), 0, s, a, static_cast<const T*>(x),
                      static_cast<const T*>(b), w_post, gate, w_pre, static_cast<T*>(out),
                      static_cast<T*>(n), rstd_post, rstd_pre);
  }
};
template <typename T, bool POST, bool PRE>
struct Bwd {
  static constexpr int kMost = 2;
  template <int TPR, int NV>
  static cudaError_t go(const NormArgs& a, int groups, const void* dout, const float* dn,
                        const void* yo, const void* b, const float* w_post, const void* gate,
                        const float* w_pre, const float* rstd_post, const float* rstd_pre,
                        void* dx, void* db, void* dgate, float* part, cudaStream_t s) {
    constexpr int RPB = block_of(TPR) / TPR;
    return launch_pdl(block_norm_bwd_kernel<T, TPR, NV, POST, PRE>, dim3(groups / RPB),
                      dim3(block_of(TPR)), 0, s, a, static_cast<const T*>(dout), dn,
                      static_cast<const T*>(yo), static_cast<const T*>(b), w_post, gate, w_pre,
                      rstd_post, rstd_pre, static_cast<T*>(dx), static_cast<T*>(db), dgate, part);
  }
};

template <template <typename, bool, bool> class K, typename T, bool POST, bool PRE,
          typename... Args>
cudaError_t by_shape(Shape sh, Args&&... args) {
  using F = K<T, POST, PRE>;
  switch (sh.tpr * 8 + sh.nv) {
    case 32 * 8 + 1: return F::template go<32, 1>(args...);
    case 32 * 8 + 2: return F::template go<32, 2>(args...);
    case 128 * 8 + 1: return F::template go<128, 1>(args...);
    case 128 * 8 + 2: return F::template go<128, 2>(args...);
    case 256 * 8 + 1: return F::template go<256, 1>(args...);
    case 256 * 8 + 2: return F::template go<256, 2>(args...);
    case 512 * 8 + 1: return F::template go<512, 1>(args...);
    case 512 * 8 + 2: return F::template go<512, 2>(args...);
    case 512 * 8 + 0: return F::template go<512, 0>(args...);
  }
  if constexpr (F::kMost == 4) {
    switch (sh.tpr) {
      case 32: return F::template go<32, 4>(args...);
      case 128: return F::template go<128, 4>(args...);
      case 256: return F::template go<256, 4>(args...);
      case 512: return F::template go<512, 4>(args...);
    }
  }
  return cudaErrorInvalidValue;
}

template <template <typename, bool, bool> class K, typename... Args>
cudaError_t by_kind(int dtype, bool post, bool pre, Shape sh, Args&&... args) {
  if (dtype == 0) {
    if (post && pre) return by_shape<K, float, true, true>(sh, args...);
    if (post) return by_shape<K, float, true, false>(sh, args...);
    return by_shape<K, float, false, true>(sh, args...);
  }
  if (post && pre) return by_shape<K, __nv_bfloat16, true, true>(sh, args...);
  if (post) return by_shape<K, __nv_bfloat16, true, false>(sh, args...);
  return by_shape<K, __nv_bfloat16, false, true>(sh, args...);
}

// Backward row groups: a multiple of the rows per block, at most
// kNormGroups(tpr), each with at least one row of its own where T allows.
int bwd_groups(Shape sh, int T) {
  const int rpb = block_of(sh.tpr) / sh.tpr;
  const int most = sh.tpr == 32 ? 2432 : (sh.tpr == 128 ? 608 : (sh.nv == 0 ? 152 : 304));
  const int g = T < most ? T : most;
  return ceil_div(g, rpb) * rpb;
}

}  // namespace

cudaError_t launch_block_norm(int dtype, int gate_kind, float eps, float alpha, float beta, int T,
                              int d, const void* x, const void* b, const float* w_post,
                              const void* gate, const float* w_pre, void* out, void* n,
                              float* rstd_post, float* rstd_pre, int num_sms, cudaStream_t s) {
  const int vec = dtype == 0 ? 4 : 8;
  const Shape sh = shape_of(d / vec, T, 4);  // Fwd::kMost
  const NormArgs a{T, d, gate_kind, eps, alpha, beta};
  // a few rows a group, so that the channel weights stay in L1
  const int resident = num_sms * (2048 / block_of(sh.tpr)) * (block_of(sh.tpr) / sh.tpr);
  return by_kind<Fwd>(dtype, b != nullptr, w_pre != nullptr, sh, a, T < resident ? T : resident, x,
                      b, w_post, gate, w_pre, out, n, rstd_post, rstd_pre, s);
}

size_t block_norm_bwd_ws(int dtype, int T, int d) {
  const Shape sh = shape_of(d / (dtype == 0 ? 4 : 8), T, 2);
  return static_cast<size_t>(bwd_groups(sh, T)) * 3 * d * sizeof(float);
}

cudaError_t launch_block_norm_bwd(int dtype, int gate_kind, float eps, float alpha, float beta,
                                  int T, int d, const void* dout, const float* dn, const void* yo,
                                  const void* b, const float* w_post, const void* gate,
                                  const float* w_pre, const float* rstd_post,
                                  const float* rstd_pre, void* dx, void* db, float* dw_post,
                                  void* dgate, float* dw_pre, float* part, cudaStream_t s) {
  const Shape sh = shape_of(d / (dtype == 0 ? 4 : 8), T, 2);
  const NormArgs a{T, d, gate_kind, eps, alpha, beta};
  const int groups = bwd_groups(sh, T);
  if (T > 0) {
    const cudaError_t e =
        by_kind<Bwd>(dtype, b != nullptr, w_pre != nullptr, sh, a, groups, dout, dn, yo, b,
                     w_post, gate, w_pre, rstd_post, rstd_pre, dx, db, dgate, part, s);
    if (e != cudaSuccess) return e;
  }
  float* cg = b != nullptr && gate_kind == kGateChannel ? static_cast<float*>(dgate) : nullptr;
  return launch_pdl(reduce_columns_kernel, dim3(d / 32, 3), dim3(256), 0, s,
                    static_cast<const float*>(part), T > 0 ? groups : 0, d,
                    w_pre != nullptr ? dw_pre : nullptr, b != nullptr ? dw_post : nullptr, cg);
}

}  // namespace moe
