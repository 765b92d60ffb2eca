// fp8.cu - 8-bit floating point for the expert products, forward and
// backward: the quantisation of rows and of expert weights, and the
// expert-grouped products of the two.
//
// Format: E4M3 codes (S.EEEE.MMM, largest 448, no infinities) and one
// power-of-two scale 2^(s - 127), a byte s, per block:
//   s - 127 = the least e >= -127 with amax <= 448 2^e (s = 127 for a block of
//   zeros; 255, which stands for NaN, for one with an infinity or a NaN)
//   code = E4M3(v / 2^(s - 127)), to nearest even
// so nothing saturates, and (scaling by a power of two being exact) the form
// is a function of the input bits alone.
//
//   rows      blocks of 128 along a row: codes [R][C], scales [R][pitch],
//             pitch = ceil(C / 128) rounded up to 4 (padding: any bytes)
//   columns   blocks of 128 rows of one expert, its segment cut into tiles:
//             codes [tile * 128 + row][C] (zeros past a segment's end), scales
//             [tile][C]
//   weights   blocks of 128 x 128 of W[e]: codes [E][K][N] as W lies, scales
//             [E][ceil(K / 128)][ceil(N / 128)]
//
//   Y[r]  = sum_k x[r][k] W[e][k]          rows, weights
//   dX[r] = sum_n dy[r][n] W[e][.][n]      rows, the same weights
//   dW[e] = sum_r x[r]^T dy[r]             columns, columns
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "grouped.cuh"
#include "moe.h"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t scale_code(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  if (amax_bits == 0u) return 127u;
  // 448 = 1.75 2^8: one more where the mantissa passes 1.75
  const int s = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return static_cast<uint32_t>(max(s, 0));
}
// 1 / scale = 2^(127 - s): exact for s in 0..253
__device__ __forceinline__ float inv_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (254u - s) << 23);
}
// the scale 2^(s - 127) (s = 0: 2^-127, subnormal)
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (s == 0u ? 0x00400000u : s << 23));
}

// four scaled values to four codes, a lowest
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// two codes to the values they stand for before their scale (exact in fp16)
__device__ __forceinline__ float2 code_values(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h)
      : "r"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// SiLU'(z) = g (1 + z (1 - g)), g the sigmoid, by t = exp(-|z|); its limits 0
// and 1 where t is 0
__device__ __forceinline__ float silu_slope(float z) {
  const float t = expf(-fabsf(z));
  if (t == 0.f) return z > 0.f ? 1.f : 0.f;
  const float y = 1.f / (1.f + t);
  const float g = z >= 0.f ? y : t * y, o = z >= 0.f ? t * y : y;
  return g * fmaf(z, o, 1.f);
}

// 16 bytes of T in fp32
template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[16 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) {
    if constexpr (sizeof(T) == 4)
      v[i] = __uint_as_float(w[i]);
    else
      v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
}
// V scaled codes
template <int V>
__device__ __forceinline__ void st_codes(uint8_t* p, const float (&v)[V]) {
  if constexpr (V == 8)
    *reinterpret_cast<uint2*>(p) =
        make_uint2(pack4(v[0], v[1], v[2], v[3]), pack4(v[4], v[5], v[6], v[7]));
  else
    *reinterpret_cast<uint32_t*>(p) = pack4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// ---------------------------------------------------------------- rows
// A block takes tiles of 128 rows of one expert x 128 columns, a thread 16
// bytes of every 16th (fp32: 8th) row, all loaded before the first is used; a
// row's lanes agree on its amax by shuffles, the columns' amax goes through
// shared memory. Both forms come out of the one read.
// Bound by HBM: bf16 in, one byte a form out.
constexpr int kRowThreads = 256;

template <typename T, int ACT, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kRowThreads)
    fp8_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ src, int x_rows,
                    const float* __restrict__ weight, const T* __restrict__ z,
                    const int32_t* __restrict__ offsets, int E, int R, int C,
                    uint8_t* __restrict__ q, uint8_t* __restrict__ sc, uint8_t* __restrict__ cq,
                    uint8_t* __restrict__ csc, uint32_t* err) {
  constexpr int V = 16 / sizeof(T), LPR = 128 / V, RPP = kRowThreads / LPR, PASS = 128 / RPP;
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  __shared__ uint32_t top[COLS ? kRowThreads / 32 : 1][128];
  __shared__ float inv[128];
  pdl_wait();
  pdl_trigger();
  if (!load_segments(offsets, E, R, seg, base, &ok, err)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = up_div(C, 128), pitch = (nb + 3) & ~3;
  const int c0 = tid % LPR * V, r0 = tid / LPR;
  // (at most 2^17 + 256 row tiles of 512 blocks)
  const int tiles = base[E] * nb;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int rt = t / nb, cb = t - rt * nb;
    const int e = last_at_most(base, E - 1, rt);
    const int row0 = seg[e] + (rt - base[e]) * 128, rows = min(128, seg[e + 1] - row0);
    const int col = cb * 128 + c0;
    const bool in = col < C;
    uint4 raw[PASS];
    uint4 zr[ACT == MOE_ACT_SILU_GRAD ? PASS : 1];
    float w[PASS];
#pragma unroll
    for (int j = 0; j < PASS; ++j) {
      const int r = r0 + j * RPP;
      raw[j] = uint4{0, 0, 0, 0};
      w[j] = 1.f;
      if constexpr (ACT == MOE_ACT_SILU_GRAD) zr[j] = uint4{0, 0, 0, 0};
      if (r >= rows || !in) continue;
      int xr = row0 + r;
      if (src != nullptr) {
        xr = __ldg(src + xr);
        if (xr < 0 || xr >= x_rows) {
          atomicOr(err, kErrBadIndex);
          continue;
        }
      }
      raw[j] = ld_once(x + static_cast<size_t>(xr) * C + col);
      if (weight != nullptr) w[j] = __ldg(weight + row0 + r);
      if constexpr (ACT == MOE_ACT_SILU_GRAD)
        zr[j] = ld_once(z + static_cast<size_t>(row0 + r) * C + col);
    }
    // (a form that takes long to compute is kept in fp32; else the raw words are)
    float held[ACT != MOE_ACT_NONE ? PASS : 1][V];
    auto value = [&](int j, float (&v)[V]) {
      if constexpr (ACT != MOE_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = held[j][i];
      } else {
        unpack<T>(raw[j], v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= w[j];
      }
    };
    if constexpr (ACT != MOE_ACT_NONE) {
#pragma unroll
      for (int j = 0; j < PASS; ++j) {
        float zv[V];
        unpack<T>(raw[j], held[j]);
        if constexpr (ACT == MOE_ACT_SILU_GRAD) unpack<T>(zr[j], zv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if constexpr (ACT == MOE_ACT_SILU)
            held[j][i] = silu_of<float>(held[j][i]) * w[j];
          else
            held[j][i] *= silu_slope(zv[i]) * w[j];
        }
      }
    }
    uint32_t cm[COLS ? V : 1] = {};
#pragma unroll
    for (int j = 0; j < PASS; ++j) {
      const int r = r0 + j * RPP;
      float v[V];
      value(j, v);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t a = mag(v[i]);
        if constexpr (ROWS) m = max(m, a);
        if constexpr (COLS) cm[i] = max(cm[i], a);
      }
      if constexpr (ROWS) {
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t s = scale_code(m);
        const float f = inv_scale(s);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= f;
        if (r < rows && in) {
          st_codes(q + static_cast<size_t>(row0 + r) * C + col, v);
          if (c0 == 0) sc[static_cast<size_t>(row0 + r) * pitch + cb] = static_cast<uint8_t>(s);
        }
      }
    }
    if constexpr (COLS) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if constexpr (LPR == 16) cm[i] = max(cm[i], __shfl_xor_sync(0xffffffffu, cm[i], 16));
      if (lane < LPR)
#pragma unroll
        for (int i = 0; i < V; ++i) top[warp][c0 + i] = cm[i];
      __syncthreads();
      if (tid < 128) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kRowThreads / 32; ++k) m = max(m, top[k][tid]);
        const uint32_t s = scale_code(m);
        inv[tid] = inv_scale(s);
        if (cb * 128 + tid < C)
          csc[static_cast<size_t>(rt) * C + cb * 128 + tid] = static_cast<uint8_t>(s);
      }
      __syncthreads();
      if (in) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = inv[c0 + i];
#pragma unroll
        for (int j = 0; j < PASS; ++j) {
          const int r = r0 + j * RPP;
          float v[V];
          value(j, v);
          // (past the segment: zeros, also in a column whose scale is NaN)
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = r < rows ? v[i] * f[i] : 0.f;
          st_codes(cq + (static_cast<size_t>(rt) * 128 + r) * C + col, v);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- weights
// A block takes 128 x 128 of one expert. Bound by HBM.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    fp8_weights_kernel(const T* __restrict__ W, int K, int N, uint8_t* __restrict__ q,
                       uint8_t* __restrict__ sc) {
  constexpr int V = 16 / sizeof(T), LPR = 128 / V, RPP = kRowThreads / LPR, PASS = 128 / RPP;
  __shared__ uint32_t top[kRowThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, e = blockIdx.z;
  const int n = blockIdx.x * 128 + tid % LPR * V, k0 = blockIdx.y * 128 + tid / LPR;
  const size_t at = static_cast<size_t>(e) * K * N;
  uint4 raw[PASS];
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int k = k0 + j * RPP;
    raw[j] = n < N && k < K ? ld_once(W + at + static_cast<size_t>(k) * N + n) : uint4{0, 0, 0, 0};
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    float v[V];
    unpack<T>(raw[j], v);
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, mag(v[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) top[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) m = max(m, top[i]);
  const uint32_t s = scale_code(m);
  const float f = inv_scale(s);
  if (tid == 0)
    sc[(static_cast<size_t>(e) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] =
        static_cast<uint8_t>(s);
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int k = k0 + j * RPP;
    float v[V];
    unpack<T>(raw[j], v);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= f;
    if (n < N && k < K) st_codes(q + at + static_cast<size_t>(k) * N + n, v);
  }
}

// ---------------------------------------------------------------- and back
// [rows][cols] codes whose scale lies at sc[(row / per) * pitch + col / 128]
// (rows: per 1; weights: 128, each expert's K rows by themselves), 8 codes a
// thread and step.
template <typename T>
__global__ void __launch_bounds__(256)
    fp8_back_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc, int experts,
                    int rows, int cols, int per, int pitch, T* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int words = cols / 8, high = up_div(rows, per);
  const long long all = static_cast<long long>(experts) * rows * words;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < all;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long row = i / words;
    const int c = static_cast<int>(i - row * words) * 8;
    const int e = static_cast<int>(row / rows), r = static_cast<int>(row - static_cast<long long>(e) * rows);
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + i * 8));
    const float s = scale_value(
        __ldg(sc + (static_cast<size_t>(e) * high + r / per) * pitch + (c >> 7)));
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = code_values((j < 2 ? w.x : w.y) >> (j & 1) * 16);
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
    T* o = out + i * 8;
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        p[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(p[0], p[1], p[2], p[3]);
    }
  }
}

// ---------------------------------------------------------------- products
// MODE 0: Y, 1: dX, 2: dW. 64 x 64 outputs a block, 4 x 4 a thread, fp32 FMA
// over 16 steps of the contraction at a time.
struct Params {
  const uint8_t *a, *as, *b, *bs;
  const int32_t* offsets;
  void* out;
  uint32_t* err;
  int E, R, K, N, silu;
};
__device__ __forceinline__ float value_of(uint32_t code, uint32_t s) {
  return code_values(code).x * scale_value(s);
}

template <int MODE, typename TO>
__global__ void __launch_bounds__(256) fp8_product_kernel(const Params p) {
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  __shared__ float As[16][65], Bs[16][65];
  pdl_wait();
  pdl_trigger();
  if (!load_segments(p.offsets, p.E, p.R, seg, base, &ok, p.err)) return;
  const int tid = threadIdx.x, K = p.K, N = p.N;
  const int width = MODE == 1 ? K : N;  // of the output
  const int c0 = blockIdx.x * 64;
  int e, row0, rows, len, tile0 = 0;  // output rows; the contraction
  size_t out0;
  if constexpr (MODE == 2) {
    const int mt = up_div(K, 64);
    e = blockIdx.y / mt;
    row0 = (blockIdx.y - e * mt) * 64;
    rows = K - row0;
    len = (base[e + 1] - base[e]) * 128;
    tile0 = base[e];
    out0 = static_cast<size_t>(e) * K + row0;
  } else {
    const int rt = blockIdx.y >> 1;
    if (rt >= base[p.E]) return;
    e = last_at_most(base, p.E - 1, rt);
    row0 = seg[e] + (rt - base[e]) * 128 + (blockIdx.y & 1) * 64;
    rows = seg[e + 1] - row0;
    len = MODE == 1 ? N : K;
    out0 = row0;
  }
  if (rows <= 0) return;
  rows = min(rows, 64);
  const int nbk = up_div(K, 128), nbn = up_div(N, 128), pitch = (up_div(len, 128) + 3) & ~3;
  float acc[4][4] = {};
  const int ty = tid / 16, tx = tid % 16;
  for (int k0 = 0; k0 < len; k0 += 16) {
    for (int i = tid; i < 1024; i += 256) {
      const int r = i / 16, k = k0 + i % 16;
      float a = 0.f, b = 0.f;
      if (MODE != 2 && r < rows)
        a = value_of(p.a[static_cast<size_t>(row0 + r) * len + k],
                     p.as[static_cast<size_t>(row0 + r) * pitch + k / 128]);
      if (MODE == 2 && r < rows)
        a = value_of(p.a[(static_cast<size_t>(tile0) * 128 + k) * K + row0 + r],
                     p.as[(static_cast<size_t>(tile0) + k / 128) * K + row0 + r]);
      const int c = c0 + r;
      if (MODE == 0 && c < N)
        b = value_of(p.b[(static_cast<size_t>(e) * K + k) * N + c],
                     p.bs[(static_cast<size_t>(e) * nbk + k / 128) * nbn + c / 128]);
      if (MODE == 1 && c < K)
        b = value_of(p.b[(static_cast<size_t>(e) * K + c) * N + k],
                     p.bs[(static_cast<size_t>(e) * nbk + c / 128) * nbn + k / 128]);
      if (MODE == 2 && c < N)
        b = value_of(p.b[(static_cast<size_t>(tile0) * 128 + k) * N + c],
                     p.bs[(static_cast<size_t>(tile0) + k / 128) * N + c]);
      As[i % 16][r] = a;
      Bs[i % 16][r] = b;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  TO* out = static_cast<TO*>(p.out);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = ty * 4 + i, c = c0 + tx * 4 + j;
      if (r < rows && c < width)
        out[(out0 + r) * width + c] = static_cast<TO>(p.silu ? silu_of<TO>(acc[i][j]) : acc[i][j]);
    }
}

template <int MODE, typename TO>
cudaError_t launch_mode(const Params& p, cudaStream_t s) {
  const int width = MODE == 1 ? p.K : p.N;
  const int tall = MODE == 2 ? p.E * up_div(p.K, 64) : 2 * static_cast<int>(row_tiles(p.R, p.E));
  return launch_pdl(fp8_product_kernel<MODE, TO>, dim3(up_div(width, 64), tall), dim3(256), 0, s, p);
}

template <typename T, int ACT>
cudaError_t launch_rows(const void* x, const int32_t* src, int x_rows, const float* weight,
                        const void* z, const int32_t* offsets, int E, int R, int C, uint8_t* q,
                        uint8_t* sc, uint8_t* cq, uint8_t* csc, uint32_t* err, int num_sms,
                        cudaStream_t s) {
  const long long tiles = static_cast<long long>(row_tiles(R, E)) * up_div(C, 128);
  const long long most = static_cast<long long>(num_sms) * 4;
  const dim3 grid(static_cast<unsigned>(tiles < most ? tiles : most)), block(kRowThreads);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, s, static_cast<const T*>(x), src, x_rows, weight,
                      static_cast<const T*>(z), offsets, E, R, C, q, sc, cq, csc, err);
  };
  if (cq == nullptr) return go(fp8_rows_kernel<T, ACT, true, false>);
  return q == nullptr ? go(fp8_rows_kernel<T, ACT, false, true>)
                      : go(fp8_rows_kernel<T, ACT, true, true>);
}

template <typename T>
cudaError_t launch_rows_act(int act, const void* x, const int32_t* src, int x_rows,
                            const float* weight, const void* z, const int32_t* offsets, int E,
                            int R, int C, uint8_t* q, uint8_t* sc, uint8_t* cq, uint8_t* csc,
                            uint32_t* err, int num_sms, cudaStream_t s) {
  return act == MOE_ACT_NONE
             ? launch_rows<T, MOE_ACT_NONE>(x, src, x_rows, weight, z, offsets, E, R, C, q, sc, cq,
                                            csc, err, num_sms, s)
         : act == MOE_ACT_SILU
             ? launch_rows<T, MOE_ACT_SILU>(x, src, x_rows, weight, z, offsets, E, R, C, q, sc, cq,
                                            csc, err, num_sms, s)
             : launch_rows<T, MOE_ACT_SILU_GRAD>(x, src, x_rows, weight, z, offsets, E, R, C, q, sc,
                                                 cq, csc, err, num_sms, s);
}

template <typename T>
cudaError_t launch_back(const uint8_t* q, const uint8_t* sc, int experts, int rows, int cols,
                        int per, int pitch, void* out, int num_sms, cudaStream_t s) {
  const long long blocks = (static_cast<long long>(experts) * rows * (cols / 8) + 255) / 256;
  const long long most = static_cast<long long>(num_sms) * 8;
  return launch_pdl(fp8_back_kernel<T>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                    dim3(256), 0, s, q, sc, experts, rows, cols, per, pitch, static_cast<T*>(out));
}

}  // namespace

cudaError_t launch_fp8_rows(int dtype, int act, const void* x, const int32_t* src, int x_rows,
                            const float* weight, const void* z, const int32_t* offsets, int E,
                            int R, int C, uint8_t* q, uint8_t* sc, uint8_t* cq, uint8_t* csc,
                            uint32_t* err, int num_sms, cudaStream_t s) {
  return dtype == 0 ? launch_rows_act<float>(act, x, src, x_rows, weight, z, offsets, E, R, C, q,
                                             sc, cq, csc, err, num_sms, s)
                    : launch_rows_act<__nv_bfloat16>(act, x, src, x_rows, weight, z, offsets, E, R,
                                                     C, q, sc, cq, csc, err, num_sms, s);
}

cudaError_t launch_fp8_weights(int dtype, const void* W, int E, int K, int N, uint8_t* q,
                               uint8_t* sc, cudaStream_t s) {
  const dim3 grid(up_div(N, 128), up_div(K, 128), E), block(kRowThreads);
  return dtype == 0 ? launch_pdl(fp8_weights_kernel<float>, grid, block, 0, s,
                                 static_cast<const float*>(W), K, N, q, sc)
                    : launch_pdl(fp8_weights_kernel<__nv_bfloat16>, grid, block, 0, s,
                                 static_cast<const __nv_bfloat16*>(W), K, N, q, sc);
}

cudaError_t launch_fp8_back(int dtype, const uint8_t* q, const uint8_t* sc, int experts, int rows,
                            int cols, int per, int pitch, void* out, int num_sms, cudaStream_t s) {
  return dtype == 0
             ? launch_back<float>(q, sc, experts, rows, cols, per, pitch, out, num_sms, s)
             : launch_back<__nv_bfloat16>(q, sc, experts, rows, cols, per, pitch, out, num_sms, s);
}

cudaError_t launch_fp8_product(int mode, const uint8_t* a, const uint8_t* as, const uint8_t* b,
                               const uint8_t* bs, const int32_t* offsets, int E, int R, int K,
                               int N, int out_f32, int silu, void* out, uint32_t* err,
                               cudaStream_t s) {
  const Params p{a, as, b, bs, offsets, out, err, E, R, K, N, silu};
  if (mode == 2) return launch_mode<2, float>(p, s);
  if (mode == 1)
    return out_f32 ? launch_mode<1, float>(p, s) : launch_mode<1, __nv_bfloat16>(p, s);
  return out_f32 ? launch_mode<0, float>(p, s) : launch_mode<0, __nv_bfloat16>(p, s);
}

}  // namespace moe
