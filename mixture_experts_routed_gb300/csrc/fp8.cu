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
//             [tile][ceil(C / 128)][128], column i of 128 at (i % 32) 4 + i / 32
//   weights   blocks of 128 x 128 of W[e]: codes [E][K][N] as W lies, scales
//             [E][ceil(K / 128)][ceil(N / 128)]
//
//   Y[r]  = sum_k x[r][k] W[e][k]          rows, weights
//   dX[r] = sum_n dy[r][n] W[e][.][n]      rows, the same weights
//   dW[e] = sum_r x[r]^T dy[r]             columns, columns
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "grouped.cuh"
#include "moe.h"
#include "ptx.cuh"
#include "range.cuh"
#include "tmap.cuh"

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

// What is quantised: 16 bytes of x (and of z) through the activation, times a
// row's weight.
template <typename T, int ACT>
__device__ __forceinline__ void input(const uint4& x, const uint4& z, float w,
                                      float (&v)[16 / sizeof(T)]) {
  constexpr int V = 16 / sizeof(T);
  unpack<T>(x, v);
  float zv[V];
  if constexpr (ACT == MOE_ACT_SILU_GRAD) unpack<T>(z, zv);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (ACT == MOE_ACT_NONE)
      v[i] *= w;
    else if constexpr (ACT == MOE_ACT_SILU)
      v[i] = silu_of<float>(v[i]) * w;
    else
      v[i] *= silu_slope(zv[i]) * w;
  }
}

// Eight bf16 values as they are, two to an instruction: their scaling by powers
// of two in bf16 (exact, but for results below 2^-126, whose code is 0 either
// way), their amax as 16-bit whole numbers.
__device__ __forceinline__ uint2 scaled_codes(const uint4& u, const uint32_t (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w[i]), "r"(f[i]));
    v[2 * i] = __uint_as_float(r << 16);
    v[2 * i + 1] = __uint_as_float(r & 0xffff0000u);
  }
  return make_uint2(pack4(v[0], v[1], v[2], v[3]), pack4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ uint32_t amax2(const uint4& u) {
  return __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                  __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
}
__device__ __forceinline__ uint32_t of_two(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
// the bf16 factors of two scales in one word
__device__ __forceinline__ uint32_t inv_pair(uint32_t lo, uint32_t hi) {
  return __byte_perm(__float_as_uint(inv_scale(lo)), __float_as_uint(inv_scale(hi)), 0x7632);
}

// ---------------------------------------------------------------- rows
// A warp quantises groups of four spans (256 bf16 or 128 fp32 values each) of
// a row: a lane loads 16 bytes of a span, a block's 16 (32) lanes agree on its
// amax. The groups of all rows are shared out evenly, each warp's one after
// the other, and a group is loaded while the one before it is quantised.
// Bound by HBM: the row is read once, a byte a value written. 16384 rows of
// 7168 bf16 values: 59 us, 6.0 TB/s; 2047 rows of 2048 of 64 experts 3.9 us (by
// tiles of one expert's rows, as below, 97 and 12 us). kRowBlocks: blocks of 256
// threads for each SM, which holds four at once (3, 4, 5 held at once, 8: 64.0,
// 60.3, 65.3, 58.7 us). 16384 rows of 5120 bf16 values, 6.0 TB/s as they are,
// gathered or weighted (42 us), 88 us as SiLU and 165 as SiLU' of two tensors
// (2.9 and 2.6 TB/s); of fp32 67, 101 and 184 us.
constexpr int kRowBlocks = 8;

// PLAIN: bf16 values as they are (no activation, no weights)
template <typename T, int ACT, bool PLAIN>
__global__ void __launch_bounds__(256)
    fp8_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ src, int x_rows,
                    const float* __restrict__ weight, const T* __restrict__ z,
                    const int32_t* __restrict__ offsets, int E, int R, int C,
                    uint8_t* __restrict__ q, uint8_t* __restrict__ sc, uint32_t* err) {
  constexpr int V = 16 / sizeof(T), LPB = 128 / V, SPAN = 32 * V, F = 4;
  constexpr bool Z = ACT == MOE_ACT_SILU_GRAD;
  __shared__ int bad;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += 256) {
    const int o = __ldg(offsets + e);
    if (o < 0 || o > R || (e > 0 && o < __ldg(offsets + e - 1))) bad = 1;
  }
  __syncthreads();
  if (bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kErrBadIndex);
    return;
  }
  const int first = __ldg(offsets), end = __ldg(offsets + E);
  const int lane = threadIdx.x & 31;
  const int groups = up_div(C, F * SPAN), pitch = up_div(up_div(C, 128), 4) * 4;
  // (at most 2^24 rows of 128 groups)
  const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
  const uint32_t total = static_cast<uint32_t>(end - first) * groups;
  const uint32_t share = total / warps, more = total - share * warps;
  const uint32_t g0 = share * warp + min(warp, more);
  int left = share + (warp < more ? 1 : 0);
  if (left == 0) return;
  int r = first + static_cast<int>(g0 / groups), g = static_cast<int>(g0 % groups);
  const T *row, *zrow;
  bool in;
  float w;
  auto find = [&](int r) {
    const int xr = src != nullptr ? __ldg(src + r) : r;
    in = xr >= 0 && xr < x_rows;
    if (!in && lane == 0) atomicOr(err, kErrBadIndex);
    row = x + static_cast<size_t>(in ? xr : 0) * C;
    if constexpr (Z) zrow = z + static_cast<size_t>(r) * C;
    // (no row: zeros, whatever its weight)
    w = weight != nullptr && in ? __ldg(weight + r) : 1.f;
  };
  uint4 raw[F], zr[Z ? F : 1];
  auto load = [&](int kb) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const bool some = in && kb + f * SPAN < C;
      raw[f] = some ? ld_once(row + kb + f * SPAN) : uint4{0, 0, 0, 0};
      if constexpr (Z) zr[f] = some ? ld_once(zrow + kb + f * SPAN) : uint4{0, 0, 0, 0};
    }
  };
  find(r);
  load(g * F * SPAN + lane * V);
  while (true) {
    uint8_t* qr = q + static_cast<size_t>(r) * C;
    uint8_t* sr = sc + static_cast<size_t>(r) * pitch;
    const int kb = g * F * SPAN + lane * V;
    uint4 now[F], znow[Z ? F : 1];
    const float wnow = w;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      now[f] = raw[f];
      if constexpr (Z) znow[f] = zr[f];
    }
    if (--left > 0) {
      if (++g == groups) {
        g = 0;
        find(++r);
      }
      load(g * F * SPAN + lane * V);
    }
    uint32_t word = 0;  // four blocks' scales
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int k = kb + f * SPAN;
      uint32_t s;
      if constexpr (PLAIN) {
        uint32_t m = amax2(now[f]);
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = scale_code(of_two(m));
        const uint32_t inv = inv_pair(s, s), f4[4] = {inv, inv, inv, inv};
        if (k < C) *reinterpret_cast<uint2*>(qr + k) = scaled_codes(now[f], f4);
      } else {
        float v[V];
        input<T, ACT>(now[f], znow[Z ? f : 0], wnow, v);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, mag(v[i]));
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = scale_code(m);
        const float inv = inv_scale(s);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= inv;
        if (k < C) st_codes(qr + k, v);
      }
      // (the scales' lines are padded to four)
      if constexpr (V == 8) {
        word |= (s | __shfl_sync(0xffffffffu, s, 16) << 8) << (f & 1) * 16;
        if ((f & 1) && lane == 0 && k - SPAN < C)
          *reinterpret_cast<uint32_t*>(sr + ((k - SPAN) >> 7)) = word;
        if (f & 1) word = 0;
      } else {
        word |= s << f * 8;
        if (f == F - 1 && lane == 0 && kb < C) *reinterpret_cast<uint32_t*>(sr + (kb >> 7)) = word;
      }
    }
    if (left == 0) return;
  }
}

// ---------------------------------------------------------------- columns
// A block takes tiles of 128 rows of one expert x 128 columns, a thread 16
// bytes of every 16th (fp32: 8th) row, which it copies to a place of its own in
// shared memory (cp.async) DEPTH tiles ahead. The columns' amax goes over
// shared memory, a row's (where the rows' form is wanted too) by shuffles:
// both forms come out of the one read. (What this cost for bf16 as they are,
// before the kernel below took them: 88 us for 16384 x 5120.) Both forms of as
// many bf16 values: weighted and gathered 117 us, SiLU 128, SiLU' 316 (2.9, 2.6
// and 1.6 TB/s); of fp32, as they are, 168, with a weight and gathered 389, SiLU
// 212, SiLU' 436. Bound by latency, SiLU near issue (0.7 of the slots, SiLU'
// 0.36): each row's amax takes shuffles of its own,
// and 128 registers, or the ring of two tensors or of fp32, leave two blocks or
// one to an SM.
constexpr int kColThreads = 256, kColWarps = kColThreads / 32, kTileBytes = 128 * 128;

// T's tiles, TENSORS of them (x, or x and z), in at most BUFS buffers
template <typename T, int TENSORS, int MOST>
struct ColRing {
  static constexpr int V = 16 / sizeof(T), LPR = 128 / V, RPP = kColThreads / LPR,
                       PASS = 128 / RPP;
  static_assert(PASS <= 32, "a bit for each row of a thread");
  static constexpr int BYTES = kTileBytes * sizeof(T) * TENSORS;
  static constexpr int FIT = BYTES <= 32768 ? 3 : BYTES <= 65536 ? 2 : 1;
  static constexpr int BUFS = FIT < MOST ? FIT : MOST, DEPTH = BUFS - 1, SMEM = BUFS * BYTES;
  static_assert(SMEM <= 200 * 1024, "shared memory");
  struct At {
    int rt, cb, row0, rows;  // (rows 0: no such tile)
    uint32_t none;           // bit j: this thread's row j has no source
  };
  const T *x, *z;
  const int32_t* src;
  int x_rows, E, C, nb, tiles;
  const int *seg, *base;
  uint4* buf;  // [BUFS][TENSORS][PASS][threads]
  uint32_t* err;
  int c0, r0;

  __device__ uint4* piece(int b, int h, int j) const {
    return buf + ((b * TENSORS + h) * PASS + j) * kColThreads + threadIdx.x;
  }
  // Tile t's place, its values on their way to buffer b. A thread reads only
  // what it copied: no barrier, and a buffer is free once its thread is
  // through with it.
  __device__ At fetch(int t, int b) const {
    At a{0, 0, 0, 0, 0u};
    if (t < tiles) {
      a.rt = t / nb;
      a.cb = t - a.rt * nb;
      const int e = last_at_most(base, E - 1, a.rt);
      a.row0 = seg[e] + (a.rt - base[e]) * 128;
      a.rows = min(128, seg[e + 1] - a.row0);
      const int col = a.cb * 128 + c0;
      const size_t at = static_cast<size_t>(a.row0 + r0) * C + col;
      if (a.rows == 128 && a.cb * 128 + 128 <= C && src == nullptr) {
#pragma unroll
        for (int j = 0; j < PASS; ++j) {
          const size_t on = at + static_cast<size_t>(j) * RPP * C;
          ptx::cp_async16(ptx::smem_u32(piece(b, 0, j)), x + on);
          if constexpr (TENSORS > 1) ptx::cp_async16(ptx::smem_u32(piece(b, 1, j)), z + on);
        }
      } else {
#pragma unroll
        for (int j = 0; j < PASS; ++j) {
          const int r = a.row0 + r0 + j * RPP;
          bool some = r0 + j * RPP < a.rows;
          int xr = r;
          if (some && src != nullptr) {
            xr = __ldg(src + r);
            if (xr < 0 || xr >= x_rows) {
              atomicOr(err, kErrBadIndex);
              a.none |= 1u << j;
              some = false;
            }
          }
          if (some && col < C) {
            ptx::cp_async16(ptx::smem_u32(piece(b, 0, j)), x + static_cast<size_t>(xr) * C + col);
            if constexpr (TENSORS > 1)
              ptx::cp_async16(ptx::smem_u32(piece(b, 1, j)), z + static_cast<size_t>(r) * C + col);
          } else {
            *piece(b, 0, j) = uint4{0, 0, 0, 0};
            if constexpr (TENSORS > 1) *piece(b, 1, j) = uint4{0, 0, 0, 0};
          }
        }
      }
    }
    ptx::cp_async_commit();
    return a;
  }
  // f(tile's place, its buffer) for every tile of this block, in turn; all its
  // threads take part
  template <typename F>
  __device__ void walk(F f) const {
    At at[DEPTH + 1];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) at[i] = fetch(blockIdx.x + i * gridDim.x, i);
    int b = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int ahead = b + DEPTH >= BUFS ? b + DEPTH - BUFS : b + DEPTH;
      at[DEPTH] = fetch(t + DEPTH * gridDim.x, ahead);
      ptx::cp_async_wait<DEPTH>();
      f(at[0], b);
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) at[i] = at[i + 1];
      if (++b == BUFS) b = 0;
    }
    ptx::cp_async_wait<0>();
  }
};

struct ColOut {
  uint8_t *q, *sc, *cq, *csc;
};

template <typename T, int ACT, bool ROWS>
__global__ void __launch_bounds__(kColThreads)
    fp8_columns_kernel(const T* __restrict__ x, const int32_t* __restrict__ src, int x_rows,
                       const float* __restrict__ weight, const T* __restrict__ z,
                       const int32_t* __restrict__ offsets, int E, int R, int C, const ColOut o,
                       uint32_t* err) {
  constexpr bool Z = ACT == MOE_ACT_SILU_GRAD;
  using K = ColRing<T, Z ? 2 : 1, 3>;
  constexpr int V = K::V, LPR = K::LPR, RPP = K::RPP, PASS = K::PASS;
  extern __shared__ __align__(16) uint8_t buf[];
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  __shared__ __align__(16) uint32_t top[kColWarps][128];
  __shared__ float inv[128];
  pdl_wait();
  pdl_trigger();
  if (!load_segments(offsets, E, R, seg, base, &ok, err)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = up_div(C, 128), pitch = (nb + 3) & ~3;
  const int c0 = tid % LPR * V, r0 = tid / LPR;
  // (at most 2^17 + 256 row tiles of 512 blocks)
  const K ring{x, z, src, x_rows, E, C, nb, base[E] * nb, seg, base,
               reinterpret_cast<uint4*>(buf), err, c0, r0};
  ring.walk([&](const typename K::At& a, int b) {
    const int col = a.cb * 128 + c0;
    const bool in = col < C;
    float held[PASS][V];
    uint32_t cm[V] = {};
#pragma unroll
    for (int j = 0; j < PASS; ++j) {
      const int r = r0 + j * RPP;
      // (no source: zeros, whatever its weight)
      const bool weighed = weight != nullptr && r < a.rows && (a.none >> j & 1) == 0;
      const float w = weighed ? __ldg(weight + a.row0 + r) : 1.f;
      input<T, ACT>(*ring.piece(b, 0, j), *ring.piece(b, Z ? 1 : 0, j), w, held[j]);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t g = mag(held[j][i]);
        if constexpr (ROWS) m = max(m, g);
        cm[i] = max(cm[i], g);
      }
      if constexpr (ROWS) {
#pragma unroll
        for (int k = 1; k < LPR; k <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
        const uint32_t s = scale_code(m);
        const float f = inv_scale(s);
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = held[j][i] * f;
        if (r < a.rows && in) {
          st_codes(o.q + static_cast<size_t>(a.row0 + r) * C + col, v);
          if (c0 == 0)
            o.sc[static_cast<size_t>(a.row0 + r) * pitch + a.cb] = static_cast<uint8_t>(s);
        }
      }
    }
    if constexpr (LPR == 16) {
#pragma unroll
      for (int i = 0; i < V; ++i) cm[i] = max(cm[i], __shfl_xor_sync(0xffffffffu, cm[i], 16));
    }
    if (lane < LPR) {
#pragma unroll
      for (int i = 0; i < V; i += 4)
        *reinterpret_cast<uint4*>(&top[warp][c0 + i]) =
            make_uint4(cm[i], cm[i + 1], cm[i + 2], cm[i + 3]);
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kColWarps; ++k) m = max(m, top[k][tid]);
      const uint32_t s = scale_code(m);
      inv[tid] = inv_scale(s);
      o.csc[(static_cast<size_t>(a.rt) * nb + a.cb) * 128 + (tid & 31) * 4 + (tid >> 5)] =
          static_cast<uint8_t>(s);
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
        // (past the segment: zeros, also in a column whose scale is NaN)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = r < a.rows ? held[j][i] * f[i] : 0.f;
        st_codes(o.cq + (static_cast<size_t>(a.rt) * 128 + r) * C + col, v);
      }
    }
  });
}

// The same for bf16 values as they are (no activation, no weights). The eight
// rows' amax of a thread are reduced together, two to a word: a lane gives away
// half of its words at each step, ends with two rows', makes their scales, and
// hands the factors back. Bound by HBM: 16384 x 5120 values to both forms in 59
// us, 5.7 TB/s (with every row's amax reduced by itself 83); gathered 74.
template <bool ROWS>
__global__ void __launch_bounds__(kColThreads, 3)
    fp8_columns_bf16_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ src,
                            int x_rows, const int32_t* __restrict__ offsets, int E, int R, int C,
                            const ColOut o, uint32_t* err) {
  using K = ColRing<__nv_bfloat16, 1, 2>;
  static_assert(K::PASS == 8 && K::LPR == 16, "a thread's rows");
  extern __shared__ __align__(16) uint8_t buf[];
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  __shared__ __align__(16) uint32_t top[kColWarps][64], inv[64];
  pdl_wait();
  pdl_trigger();
  if (!load_segments(offsets, E, R, seg, base, &ok, err)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = up_div(C, 128), pitch = (nb + 3) & ~3;
  const int c0 = tid % 16 * 8, r0 = tid / 16;
  // (at most 2^17 + 256 row tiles of 512 blocks)
  const K ring{x, nullptr, src, x_rows, E, C, nb, base[E] * nb, seg, base,
               reinterpret_cast<uint4*>(buf), err, c0, r0};
  ring.walk([&](const typename K::At& a, int b) {
    const int col = a.cb * 128 + c0;
    const bool in = col < C;
    uint4 raw[8];
    uint32_t cm[4] = {}, rm[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      raw[j] = *ring.piece(b, 0, j);
      const uint32_t u[4] = {raw[j].x & 0x7fff7fffu, raw[j].y & 0x7fff7fffu,
                             raw[j].z & 0x7fff7fffu, raw[j].w & 0x7fff7fffu};
#pragma unroll
      for (int i = 0; i < 4; ++i) cm[i] = __vmaxu2(cm[i], u[i]);
      rm[j] = __vmaxu2(__vmaxu2(u[0], u[1]), __vmaxu2(u[2], u[3]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) cm[i] = __vmaxu2(cm[i], __shfl_xor_sync(0xffffffffu, cm[i], 16));
    if (lane < 16)
      *reinterpret_cast<uint4*>(&top[warp][c0 / 2]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    if constexpr (ROWS) {
      uint32_t p[4];  // rows j and j + 4
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[j] = __vmaxu2(__byte_perm(rm[j], rm[j + 4], 0x5410), __byte_perm(rm[j], rm[j + 4], 0x7632));
      const bool up8 = lane & 8, up4 = lane & 4;
      uint32_t m0 = up8 ? p[2] : p[0], m1 = up8 ? p[3] : p[1];
      m0 = __vmaxu2(m0, __shfl_xor_sync(0xffffffffu, up8 ? p[0] : p[2], 8));
      m1 = __vmaxu2(m1, __shfl_xor_sync(0xffffffffu, up8 ? p[1] : p[3], 8));
      uint32_t m = __vmaxu2(up4 ? m1 : m0, __shfl_xor_sync(0xffffffffu, up4 ? m0 : m1, 4));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const uint32_t lo = scale_code(m << 16), hi = scale_code(m & 0xffff0000u);
      const uint32_t both = inv_pair(lo, hi);
      // (two of the four lanes that hold a pair of rows write its scales)
      const int r = r0 + ((lane >> 2 & 3) >> 1) * 32 + (lane >> 2 & 1) * 16 + (lane & 1) * 64;
      if ((lane & 2) == 0 && r < a.rows)
        o.sc[static_cast<size_t>(a.row0 + r) * pitch + a.cb] =
            static_cast<uint8_t>(lane & 1 ? hi : lo);
      uint8_t* to = o.q + static_cast<size_t>(a.row0 + r0) * C + col;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t f = __shfl_sync(0xffffffffu, both, (lane & 16) | j << 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t g = __byte_perm(f, 0, h ? 0x3232 : 0x1010);
          const uint32_t f4[4] = {g, g, g, g};
          const int i = j + h * 4;
          if (r0 + i * 16 < a.rows && in)
            *reinterpret_cast<uint2*>(to + static_cast<size_t>(i) * 16 * C) =
                scaled_codes(raw[i], f4);
        }
      }
    }
    __syncthreads();
    if (tid < 64) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kColWarps; ++k) m = __vmaxu2(m, top[k][tid]);
      const uint32_t lo = scale_code(m << 16), hi = scale_code(m & 0xffff0000u);
      inv[tid] = inv_pair(lo, hi);
      // columns 2 tid and 2 tid + 1 of the block
      uint8_t* to = o.csc + (static_cast<size_t>(a.rt) * nb + a.cb) * 128 + (tid & 15) * 8 + (tid >> 4);
      to[0] = static_cast<uint8_t>(lo);
      to[4] = static_cast<uint8_t>(hi);
    }
    __syncthreads();
    if (in) {
      const uint4 f = *reinterpret_cast<const uint4*>(&inv[c0 / 2]);
      const uint32_t f4[4] = {f.x, f.y, f.z, f.w};
      uint8_t* to = o.cq + (static_cast<size_t>(a.rt) * 128 + r0) * C + col;
      // (past the segment: zeros, also in a column whose scale is NaN)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint2*>(to + static_cast<size_t>(j) * 16 * C) =
            r0 + j * 16 < a.rows ? scaled_codes(raw[j], f4) : make_uint2(0, 0);
    }
  });
}

// ---------------------------------------------------------------- weights
// A block takes 128 x 128 of one expert. Bound by HBM: 16 x 1536 x 5120 bf16
// values in 55 us, 6.9 TB/s, fp32 96 us, 6.5 TB/s.
template <typename T>
__global__ void __launch_bounds__(kColThreads)
    fp8_weights_kernel(const T* __restrict__ W, int K, int N, uint8_t* __restrict__ q,
                       uint8_t* __restrict__ sc) {
  constexpr int V = 16 / sizeof(T), LPR = 128 / V, RPP = kColThreads / LPR, PASS = 128 / RPP;
  __shared__ uint32_t top[kColThreads / 32];
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
    if constexpr (V == 8) {
      m = __vmaxu2(m, amax2(raw[j]));
    } else {
      m = max(m, max(max(raw[j].x & 0x7fffffffu, raw[j].y & 0x7fffffffu),
                     max(raw[j].z & 0x7fffffffu, raw[j].w & 0x7fffffffu)));
    }
  }
  if constexpr (V == 8) m = of_two(m);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) top[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kColThreads / 32; ++i) m = max(m, top[i]);
  const uint32_t s = scale_code(m);
  const float f = inv_scale(s);
  if (tid == 0)
    sc[(static_cast<size_t>(e) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] =
        static_cast<uint8_t>(s);
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int k = k0 + j * RPP;
    if (n >= N || k >= K) continue;
    uint8_t* to = q + at + static_cast<size_t>(k) * N + n;
    if constexpr (V == 8) {
      const uint32_t inv = inv_pair(s, s), f4[4] = {inv, inv, inv, inv};
      *reinterpret_cast<uint2*>(to) = scaled_codes(raw[j], f4);
    } else {
      float v[V];
      unpack<T>(raw[j], v);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= f;
      st_codes(to, v);
    }
  }
}

// ---------------------------------------------------------------- and back
// [experts][rows][cols] codes with a scale for `per` (1 or 128) rows x 128
// columns, `pitch` of them to a line. A block takes 128 x 128, a thread 8
// codes of every 16th row, all loaded before the first is written. Bound by
// HBM: the same weights back in 57 us, 6.6 TB/s (83 with 8 codes a thread at a
// time), to fp32 120 us, 5.2 TB/s.
template <typename T>
__global__ void __launch_bounds__(kColThreads)
    fp8_back_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc, int rows,
                    int cols, int per, int pitch, T* __restrict__ out) {
  constexpr int PASS = 8;
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.y * 128 + threadIdx.x % 16 * 8, r0 = blockIdx.x * 128 + threadIdx.x / 16;
  if (c >= cols) return;
  const size_t e = blockIdx.z;
  const uint8_t* s0 = sc + e * up_div(rows, per) * pitch + blockIdx.y;
  uint2 w[PASS];
  uint8_t s[PASS];
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int r = min(r0 + j * 16, rows - 1);
    w[j] = __ldg(reinterpret_cast<const uint2*>(q + (e * rows + r) * cols + c));
    s[j] = __ldg(s0 + static_cast<size_t>(r / per) * pitch);
  }
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int r = r0 + j * 16;
    if (r >= rows) return;
    const float f = scale_value(s[j]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 two = code_values((i < 2 ? w[j].x : w[j].y) >> (i & 1) * 16);
      v[2 * i] = two.x * f;
      v[2 * i + 1] = two.y * f;
    }
    T* o = out + (e * rows + r) * cols + c;
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        p[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(p[0], p[1], p[2], p[3]);
    }
  }
}

// ---------------------------------------------------------------- products
// MODE 0: Y = rows . W[e], 1: dX = rows . W[e]^T, 2: dW[e] = columns^T . columns.
//
// Tiles of 128 rows x up to 256 columns on one CTA, or of 256 x 256 on a pair
// of CTAs (cta_group::2: each stages its own 128 rows and 128 of the columns,
// so a byte staged feeds twice the products); persistent. A stage of the ring
// holds 128 steps of the contraction, which is one block of scales: codes by
// TMA in boxes of 128 x 128 bytes (128-byte swizzle; a warp loads each side)
// as they lie in memory, k- or row-major as the mode has it (the tensor core
// takes 8-bit operands either way, so the one copy of W serves both
// products). A chunk of scales is 512 bytes, four for each of 128 rows, and a
// product names the one of the four it takes: those of four stages. A warp of
// its own writes the chunks, those of GROUP x 4 stages to a slot of a ring, and
// hands the slot over with an arrival that releases them: to the issuing thread
// in its CTA; a pair's odd CTA first, at cluster scope, to the even CTA's warp,
// which passes both on. That release takes about 1 us, so it is made once for
// eight stages, ahead of the products (for every four 363, 374 and 488 us for
// Y, dX and dW of 8192 cubed, for eight 315, 350 and 487; by the warp that loads
// the columns' side, in its ring, 522, 542 and 662). One thread copies the
// chunks to tensor memory (tcgen05.cp, in line with the products: a copy every
// stage took 323, 362 and 423 us, every four 319, 355 and 376, dW in one chain)
// and issues the products of all the columns x 32 steps
// (kind::mxf8f6f4) that read them. Three accumulators of 128 columns: tiles
// take the first two and the last two in turn, and the next tile starts once
// the middle one is drained, which is drained first. (Products of half the
// columns, a tile on any two accumulators and the next on the third, read the
// rows' side twice: 1 to 4 % slower.) Eight warps drain: into registers, which
// frees the accumulator, and then to out.
//
// Bound, of many rows: power. 8192 x 8192 x 8192 of random numbers takes 317 to
// 340 us for Y and 335 to 357 for dX, as the power state has it (3.2 to 3.5
// PFLOP/s), of zeros or ones 276 and 272; after seconds the cap leaves 1350 MHz
// and 2.9 PFLOP/s. dW, fp32 in chains, 464 to 500 us (2.2 to 2.4 PFLOP/s), of
// zeros 440: behind power the epilogue's traffic. Behind both a pair's
// stage: 32 KB into each SM, which at 64 bytes a clock take what its four
// products take, 512 clocks (with a quarter of the products, dW in one chain,
// 267, 232 and 263 us). Copies to L2 ahead of the ring: Y 16 % longer. 16384
// skewed rows of 32 experts, 7168 x 2048: 181 to 186 us for 481 GFLOP, nine
// rounds of tiles of which 6.7 are rows that exist (rows as the products'
// columns, 32 at a time, did away with the others: no faster, for the loads
// stay). dW of 16 x 5120 x 1536 from 16384 rows 123 us, 4.1 TB/s written beside
// its loads; of 64 x 1408 x 2048 from 8191 rows 143 us, 5.2 TB/s. Two rows of 8
// experts of 4096 x 11008: 22 us, 7 TB/s and 9 us of start and join. Y of 16 x
// 5120 x 1536 from 16384 rows ending in SiLU: bf16 85 -> 89 us, fp32 118 -> 146.
namespace f8 {
using namespace ptx;
constexpr int HN = 128, KS = 128;  // half a tile's columns, a stage's steps
constexpr int BOX = 128 * 128, CHUNK = 512;
// tensor memory columns: 3 x 128, then scales. A slot of scales is written
// again SLOTS uses later, of a stage or more each, so after products that a
// ring of fewer stages has seen the end of.
constexpr int SF_COL = 384, SF_SLOT = 12, SLOTS = 10;
// Scales in shared memory: a ring of their own, of GROUP chunks of four stages
constexpr int GROUP = 2, GROUP_STAGES = 4 * GROUP, SF_RING = 8 / GROUP;
constexpr int GROUP_BYTES = GROUP * 3 * CHUNK;
constexpr int TMEM_COLS = 512;
constexpr int EPI_THREADS = 256, THREADS = 128 + EPI_THREADS;

template <bool PAIR>
struct Cfg {
  static constexpr int BM = PAIR ? 256 : 128;
  static constexpr int B_BOXES = PAIR ? 1 : 2;
  static constexpr int OFF_B = BOX, STAGE = OFF_B + B_BOXES * BOX;
  static constexpr int STAGES = PAIR ? 6 : 4;  // (shared memory's most)
  static constexpr int OFF_SF = STAGES * STAGE;
  static constexpr int OFF_BAR = OFF_SF + SF_RING * GROUP_BYTES;
  static constexpr int OFF_SEG = OFF_BAR + (2 * STAGES + 6 + 3 * SF_RING) * 8 + 24;
  static constexpr int SMEM = OFF_SEG + 3 * (kMaxExperts + 1) * 4 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(SF_COL + SLOTS * SF_SLOT <= TMEM_COLS && SLOTS > STAGES, "tensor memory");
};

struct Params {
  const uint8_t *as, *bs;  // scales
  const int32_t* offsets;
  void* out;
  uint32_t* err;
  uint32_t* ctr;  // arrivals per tile of a split launch, zero between launches
  float* part;    // [CTA][2][kSplitRows][256]
  int E, R, K, N;
  int silu;
};

// kind::mxf8f6f4, E4M3 both sides, E8M0 scales, fp32 accumulator, K = 32; an
// operand whose rows are the contraction's steps is "transposed"; sf_byte:
// which of the four bytes, for both sides
__device__ __forceinline__ uint32_t sf_byte(uint32_t i) { return i << 4 | i << 29; }
constexpr uint32_t idesc(int m, int n, bool a_steps, bool b_steps) {
  return (a_steps ? 1u << 15 : 0u) | (b_steps ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 7) << 27);
}
// Operand descriptors: the low word holds the address (and, not used by
// operands of one 128-byte column, the distance of the next), the high one
// does not change (128-byte swizzle, groups of 8 rows 1024 bytes apart,
// version 1).
constexpr uint32_t AB_HI = (1024 >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t SF_HI = (128 >> 4) | 1u << 14;  // no swizzle, 8-row groups 128 bytes apart
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
  return (saddr & 0x3FFFFu) >> 4 | (BOX >> 4) << 16;
}
__device__ __forceinline__ uint32_t sf_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t sfa,
                                    uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, "
        "[%4], [%5], p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(AB_HI)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, "
        "[%4], [%5], p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(AB_HI)
        : "memory");
}
// 32 rows of 16 bytes, contiguous, to 4 columns of all four lane quarters
// (of a pair: in each CTA from its own shared memory).
template <bool PAIR>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t desc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], a;\n\t}\n" ::"r"(taddr),
        "r"(desc), "r"(SF_HI)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], a;\n\t}\n" ::"r"(taddr),
        "r"(desc), "r"(SF_HI)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR)
    tc_commit_pair_mc(bar, 0x3);
  else
    tc_commit(bar);
}
__device__ __forceinline__ void bar_epi() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(EPI_THREADS) : "memory");
}
__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// v += what this thread wrote at p before
__device__ __forceinline__ void add_sector(uint32_t (&v)[8], const float* p) {
  float o[8];
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3])
               : "l"(p)
               : "memory");
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
               : "l"(p + 4)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(o[i] + __uint_as_float(v[i]));
}

// Tile t of a weight gradient: expert by expert, its rows (of K) inside
template <int BM>
__device__ __forceinline__ Tile grad_tile(int t, int K, int N) {
  const int mt = up_div(K, BM), each = mt * up_div(N, kTileCols);
  Tile r;
  r.e = t / each;
  const int l = t - r.e * each, nb = l / mt;
  r.mt = 0;
  r.row0 = (l - nb * mt) * BM;
  r.rows = min(BM, K - r.row0);
  r.n0 = nb * kTileCols;
  r.n = min(kTileCols, N - r.n0);
  return r;
}
}  // namespace f8

template <int MODE, bool PAIR, typename TO>
__global__ void __launch_bounds__(f8::THREADS, 1)
    fp8_product_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmA32,
                       const __grid_constant__ CUtensorMap tmB, const f8::Params p) {
  using namespace f8;
  using C = Cfg<PAIR>;
  constexpr int STAGES = C::STAGES, BM = C::BM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // pair: the even CTA's
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;  // by a tile's parity
  uint64_t* tfree = tfull + 2;       // accumulators 0, 1 and 2; pair: the even CTA's
  uint64_t* drain = tfree + 3;
  uint64_t* sfull = drain + 1;  // of the scales' ring; pair: the even CTA's
  uint64_t* sodd = sfull + SF_RING;  // the odd CTA's are written (the even CTA's barriers)
  uint64_t* sempty = sodd + SF_RING;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + SF_RING);
  int* s_ok = reinterpret_cast<int*>(tmem_slot + 1);
  uint32_t* s_last = tmem_slot + 2;
  int* s_wide = reinterpret_cast<int*>(tmem_slot + 3);
  int* seg = reinterpret_cast<int*>(smem + C::OFF_SEG);
  int* base = seg + kMaxExperts + 1;
  int* tb = PAIR ? base + kMaxExperts + 1 : base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const int cta = PAIR ? blockIdx.x >> 1 : blockIdx.x, grid = PAIR ? gridDim.x >> 1 : gridDim.x;
  const int E = p.E, K = p.K, N = p.N;
  const int width = MODE == 1 ? K : N, len = MODE == 1 ? N : K;  // (len: of the rows' modes)

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&tfree[i], PAIR ? 16 : 8);
    mbar_init(drain, 1);
    for (int i = 0; i < SF_RING; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sodd[i], 1);
      mbar_init(&sempty[i], 1);
    }
    *s_wide = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, TMEM_COLS);
      tmem_relinquish();
    }
  }
  pdl_wait();
  pdl_trigger();
  const bool ok = load_segments(p.offsets, E, p.R, seg, base, s_ok, p.err);
  for (int e = tid; ok && e < E; e += THREADS)
    if (seg[e + 1] - seg[e] > kSplitRows) *s_wide = 1;
  if (MODE != 2 && PAIR && warp == 0) {
    // tiles of 256 rows before each expert
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane, n = e < E ? (base[e + 1] - base[e] + 1) / 2 : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (e < E) tb[e] = run + inc - n;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) tb[E] = run;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int kst = up_div(len, KS);
  const int tiles = !ok         ? 0
                    : MODE == 2 ? E * up_div(K, BM) * up_div(N, kTileCols)
                                : tb[E] * up_div(width, kTileCols);
  auto tile = [&](int t) {
    if constexpr (MODE == 2)
      return grad_tile<BM>(t, K, N);
    else
      return tile_at<BM>(t, seg, base, tb, E, width);
  };
  // Few rows everywhere and fewer tiles than CTAs: the tiles' stages are one
  // sequence cut into equal ranges, and a tile's partial sums are joined by
  // the last CTA to arrive, in CTA order. Otherwise whole tiles in turn.
  const bool split = MODE != 2 && !PAIR && tiles < grid && *s_wide == 0;
  const Range rg(split ? tiles : 0, kst, grid);
  // Chains: the tensor core drops what is below its accumulator's last place,
  // always towards zero, which adds up over a long contraction: the norm of the
  // error, of the sum's, after 8, 32, 128 and 512 stages was 5.8e-8, 2.2e-7,
  // 1.2e-6 and 7.3e-6 for normal values, 1.9e-7, 1.4e-6, 9.7e-6 and 5.9e-5 for
  // values of one sign, and 8.7e-7, 2.8e-6, 1.1e-5 and 3.9e-5 where rows and
  // blocks differ by powers of two up to 2^18 (plain fp32 sums of the same: at
  // most 1.4e-7, 1.1e-7 and 7.1e-7). Where fp32 is stored (bf16's own rounding
  // is 2^-9), the accumulator therefore starts anew after at most CHAIN stages,
  // and the epilogue adds the chains, rounded to nearest, one after the other
  // where they lie: Y and dX 2.3e-7, 1.4e-6 and 2.8e-6, dW 1.5e-7, 5.0e-7 and
  // 1.3e-6 at any of these lengths; rounding over more chains adds at most half
  // a step for each. Longer for Y and dX, whose products the epilogue's traffic
  // slows more: of 8192 cubed 331, 327 and 350 us in one chain, 371, 369 and 460
  // us so, with 16 for all 467, 456 and 445. (By reductions instead of reading
  // back: 458, 454, 542; with the sums kept in 128 registers a thread, which
  // the other warps give up: 359, 360, 438, but 183 us for ragged dW in one
  // chain, here 140. All with scales in the stages' ring, on one box.)
  constexpr int CHAIN = sizeof(TO) == 2 ? 0 : MODE == 2 ? 16 : 32;
  auto chains = [&](auto& f, int t, int p0, int p1) {
    const int n = CHAIN ? max(1, up_div(p1 - p0, max(CHAIN, 1))) : 1, each = up_div(p1 - p0, n);
    for (int i = 0, k0 = p0; i < n; ++i, k0 += each)
      if (!f(t, k0, min(k0 + each, p1), p0, p1)) return false;
    return true;
  };
  // Walk this CTA's pieces: f(tile, first stage, end stage, the piece's first
  // and end)
  auto walk = [&](auto f) {
    if (split) {
      const int end = rg.start(cta + 1);
      for (int i = rg.start(cta); i < end;) {
        const int t = i / kst, k0 = i - t * kst, k1 = min(kst, k0 + end - i);
        if (!chains(f, t, k0, k1)) return;
        i += k1 - k0;
      }
    } else {
      for (int t = cta; t < tiles; t += grid) {
        int k1 = kst;
        if constexpr (MODE == 2) {
          const int e = tile(t).e;
          k1 = base[e + 1] - base[e];
        }
        if (!chains(f, t, 0, k1)) return;
      }
    }
  };

  if (warp == 0 || warp == 2) {
    // the first loads the A side, the other the scales and the B side (the
    // whole warp, converged: elect_one says why)
    const bool a_side = warp == 0;
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmA32);
      prefetch_tmap(&tmB);
    }
    __syncwarp();
    int s = 0, used = 0;
    uint32_t ph = 0;
    bool dead = false;
    const uint32_t base0 = smem_u32(smem);
    const uint32_t bar0 = PAIR ? mapa_shared(smem_u32(full), 0) : 0;
    auto load2 = [&](uint8_t* dst, const CUtensorMap* m, int c0, int c1) {
      if constexpr (PAIR)
        tma_load_2d_pair(dst, m, bar0 + s * 8, c0, c1);
      else
        tma_load_2d(dst, m, &full[s], c0, c1);
    };
    auto load3 = [&](uint8_t* dst, const CUtensorMap* m, int c0, int c1, int c2) {
      if constexpr (PAIR)
        tma_load_3d_pair(dst, m, bar0 + s * 8, c0, c1, c2);
      else
        tma_load_3d(dst, m, &full[s], c0, c1, c2);
    };
    // the next stage, once it is free
    auto take = [&] {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, kWaitLimitNs))) {
        dead = true;
        return false;
      }
      return true;
    };
    auto next = [&] {
      if (++s == STAGES) {
        s = 0;
        ph ^= 1u;
      }
    };
    // CTA r's rows come in one box of 128 or, few, of 32, its columns in
    // boxes of 128; rows that are not loaded feed only sums that are not stored
    auto a_bytes = [](const Tile& tl, int r) {
      const int left = tl.rows - r * 128;
      return left <= 0 ? 0 : (MODE != 2 && left <= 32 ? BOX / 4 : BOX);
    };
    auto b_boxes = [](const Tile& tl) { return !PAIR && tl.n > 128 ? 2 : 1; };
    if (a_side) {
      walk([&](int t, int k0, int k1, int, int) {
        const Tile tl = tile(t);
        const int na = a_bytes(tl, rank), both = a_bytes(tl, 0) + (PAIR ? a_bytes(tl, 1) : 0);
        const uint32_t expect = both + (PAIR ? 2 : b_boxes(tl)) * BOX;
        const CUtensorMap* ma = na == BOX ? &tmA : &tmA32;
        const int row0 = tl.row0 + rank * 128;
        const int first = MODE == 2 ? base[tl.e] * 128 : 0;
        for (int kb = k0; kb < k1; ++kb) {
          if (!take()) return false;
          if (used < STAGES) ++used;
          if (elect_one()) {
            uint8_t* st = smem + s * C::STAGE;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], expect);
            if (na > 0) {
              if constexpr (MODE == 2)
                load2(st, &tmA, row0, first + kb * KS);
              else
                load2(st, ma, kb * KS, row0);
            }
          }
          __syncwarp();
          next();
        }
        return true;
      });
      // the latest use of each stage has landed before this CTA may exit (a
      // pair: the even CTA's barrier counts both, and both exit together)
      for (int j = 0; rank == 0 && j < used; ++j) {
        if (s == 0) {
          s = STAGES;
          ph ^= 1u;
        }
        --s;
        if (!mbar_wait(&full[s], ph, kWaitLimitNs)) {
          dead = true;
          break;
        }
      }
    } else {
      walk([&](int t, int k0, int k1, int, int) {
        const Tile tl = tile(t);
        const int first = MODE == 2 ? base[tl.e] : 0;
        const int nb = b_boxes(tl), col0 = tl.n0 + rank * 128;
        for (int kb = k0; kb < k1; ++kb) {
          if (!take()) return false;
          if (elect_one()) {
            uint8_t* dst = smem + s * C::STAGE + C::OFF_B;
#pragma unroll
            for (int b = 0; b < C::B_BOXES; ++b)
              if (b < nb) {
                if constexpr (MODE == 2)
                  load2(dst + b * BOX, &tmB, col0 + b * 128, (first + kb) * KS);
                else if constexpr (MODE == 1)
                  load3(dst + b * BOX, &tmB, kb * KS, col0 + b * 128, tl.e);
                else
                  load3(dst + b * BOX, &tmB, col0 + b * 128, kb * KS, tl.e);
              }
          }
          __syncwarp();
          next();
        }
        return true;
      });
    }
    if (dead && lane == 0) atomicOr(p.err, kErrTimeout);
  } else if (warp == 3) {
    // four stages' scales, as chunks: row i's four bytes at (i % 32) 16 + (i
    // / 32) 4. Loaded a group ahead.
    int sl = 0;
    uint32_t ph = 0;
    bool dead = false;
    const uint32_t sf0 = smem_u32(smem + C::OFF_SF) + lane * 16;
    const uint32_t odd0 = PAIR ? mapa_shared(smem_u32(sodd), 0) : 0;
    const int pitch = up_div(kst, 4) * 4, nbk = up_div(K, 128), nbn = up_div(N, 128);
    constexpr uint32_t ONE = 0x7f7f7f7fu;
    walk([&](int t, int k0, int k1, int, int) {
      const Tile tl = tile(t);
      const int rows = min(128, tl.rows - static_cast<int>(rank) * 128);
      const int first = MODE == 2 ? base[tl.e] : 0;
      struct Quad {
        uint32_t w[MODE == 2 ? 12 : 5];
      } quad[GROUP];
      auto load = [&](int q) {
        Quad r;
        if constexpr (MODE == 2) {
          // a word is rows lane + 32 i of one block: of A's and of the two of columns
          const int m = tl.row0 / 128 + rank, n = tl.n0 / 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kb = first + min(q * 4 + i, k1 - 1);
            const uint32_t* a = reinterpret_cast<const uint32_t*>(p.as) +
                                (static_cast<size_t>(kb) * nbk + m) * 32 + lane;
            const uint32_t* b = reinterpret_cast<const uint32_t*>(p.bs) +
                                (static_cast<size_t>(kb) * nbn + n) * 32 + lane;
            r.w[i] = m < nbk ? __ldg(a) : ONE;
            r.w[4 + i] = __ldg(b);
            r.w[8 + i] = n + 1 < nbn ? __ldg(b + 32) : ONE;
          }
        } else {
          // rows lane + 32 i, four blocks each; lanes 0..7: a block of the
          // two blocks of columns each
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = tl.row0 + static_cast<int>(rank) * 128 + min(lane + 32 * i, rows - 1);
            r.w[i] = rows > 0 ? __ldg(reinterpret_cast<const uint32_t*>(
                                    p.as + static_cast<size_t>(row) * pitch + q * 4))
                              : ONE;
          }
          const int nb = min(tl.n0 / 128 + (lane & 1), up_div(width, 128) - 1);
          const int kb = min(q * 4 + (lane >> 1 & 3), kst - 1);
          const int at = MODE == 1 ? nb * nbn + kb : kb * nbn + nb;
          r.w[4] = __ldg(p.bs + static_cast<size_t>(tl.e) * nbk * nbn + at);
        }
        return r;
      };
      // the four bytes of each of four words, by byte
      auto turn = [](const uint32_t* t) {
        const uint32_t a = __byte_perm(t[0], t[1], 0x5140), b = __byte_perm(t[2], t[3], 0x5140);
        const uint32_t c = __byte_perm(t[0], t[1], 0x7362), d = __byte_perm(t[2], t[3], 0x7362);
        return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632),
                          __byte_perm(c, d, 0x5410), __byte_perm(c, d, 0x7632));
      };
      // the chunks of the group that stage g is in, from g on
      auto some = [&](int g, int i) {
        const int k = (g & ~(GROUP_STAGES - 1)) + i * 4;
        return k + 3 >= g && k < k1;
      };
      auto fetch = [&](int g) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
          if (some(g, i)) quad[i] = load((g / GROUP_STAGES) * GROUP + i);
      };
      if (k0 < k1) fetch(k0);
      for (int g = k0; g < k1;) {
        const int after = (g | (GROUP_STAGES - 1)) + 1;
        const bool in_time = mbar_wait(&sempty[sl], ph ^ 1u, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, in_time)) {
          dead = true;
          return false;
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          if (!some(g, i)) continue;
          uint4 a, b0, b1;
          if constexpr (MODE == 2) {
            a = turn(quad[i].w);
            b0 = turn(quad[i].w + 4);
            b1 = turn(quad[i].w + 8);
          } else {
            a = make_uint4(quad[i].w[0], quad[i].w[1], quad[i].w[2], quad[i].w[3]);
            uint32_t s[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
              s[j & 1] |= __shfl_sync(0xffffffffu, quad[i].w[4], j) << (j >> 1) * 8;
            b0 = make_uint4(s[0], s[0], s[0], s[0]);
            b1 = make_uint4(s[1], s[1], s[1], s[1]);
          }
          const uint32_t sf = sf0 + sl * GROUP_BYTES + i * 3 * CHUNK;
          st_shared(sf, a);
          st_shared(sf + CHUNK, b0);
          st_shared(sf + 2 * CHUNK, b1);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (rank != 0) {
          if (lane == 0) mbar_arrive_remote(odd0 + sl * 8);
        } else {
          if constexpr (PAIR)
            if (!__all_sync(0xffffffffu, mbar_wait_spin_cluster(&sodd[sl], ph, kWaitLimitNs))) {
              dead = true;
              return false;
            }
          if (lane == 0) mbar_arrive(&sfull[sl]);
        }
        __syncwarp();
        if (after < k1) fetch(after);  // (behind the release, which would wait for it)
        g = after;
        if (++sl == SF_RING) {
          sl = 0;
          ph ^= 1u;
        }
      }
      return true;
    });
    if (dead && lane == 0) atomicOr(p.err, kErrTimeout);
  } else if (warp == 1) {
    // (one lane issues: elect_one says how)
    if (rank == 0) {
      int s = 0;
      uint32_t ph = 0, tiles_done = 0;
      bool dead = false;
      constexpr bool A_STEPS = MODE == 2, B_STEPS = MODE != 1;
      constexpr uint32_t id_all = idesc(BM, kTileCols, A_STEPS, B_STEPS),
                         id_half = idesc(BM, HN, A_STEPS, B_STEPS);
      // 32 steps on: 32 rows of 128 bytes, or 32 bytes of a row
      constexpr uint32_t A_ON = A_STEPS ? 4096 >> 4 : 32 >> 4, B_ON = B_STEPS ? 4096 >> 4 : 32 >> 4;
      const uint32_t base0 = smem_u32(smem);
      const uint32_t ad0 = desc_lo(base0), bd0 = desc_lo(base0 + C::OFF_B),
                     sa0 = sf_lo(base0 + C::OFF_SF);
      int slot = SLOTS - 1, sl = 0;
      uint32_t sph = 0;
      // a stage's products of `steps` x 32 (inlined with a constant for whole ones)
      auto products = [&](int kb, int steps, uint32_t id, uint32_t d, uint32_t more) {
        const uint32_t off = static_cast<uint32_t>(s) * (C::STAGE / 16);
        const uint32_t sf = tmem_base + SF_COL + slot * SF_SLOT;
        const uint32_t idk = id | sf_byte(kb & 3);
#pragma unroll
        for (int kk = 0; kk < steps; ++kk)
          mma<PAIR>(d, ad0 + off + kk * A_ON, bd0 + off + kk * B_ON, idk, sf, sf + 4,
                    kk > 0 ? 1u : more);
      };
      if (elect_one()) walk([&](int t, int k0, int k1, int, int) {
        if (k0 == k1) return true;
        // the middle accumulator, free of the tile before, and this tile's
        // other one, free of the tile before that
        const uint32_t odd = tiles_done & 1, use = tiles_done >> 1 & 1;
        ++tiles_done;
        if (!mbar_wait_spin_cluster(&tfree[odd * 2], use ^ 1u, kWaitLimitNs) ||
            !mbar_wait_spin_cluster(&tfree[1], odd ^ 1u, kWaitLimitNs)) {
          dead = true;
          return false;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + odd * HN;
        const uint32_t id = !PAIR && tile(t).n <= HN ? id_half : id_all;
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait_spin(&full[s], ph, kWaitLimitNs)) {
            dead = true;
            break;
          }
          tc_fence_after();
          if (kb == k0 || (kb & 3) == 0) {
            // four stages' scales, to the next slot
            if (kb == k0 || kb % GROUP_STAGES == 0) {
              if (!mbar_wait_spin(&sfull[sl], sph, kWaitLimitNs)) {
                dead = true;
                break;
              }
              tc_fence_after();
            }
            if (++slot == SLOTS) slot = 0;
            const uint32_t off = (sl * GROUP + (kb >> 2) % GROUP) * (3 * CHUNK / 16);
#pragma unroll
            for (int c = 0; c < 3; ++c)
              cp_scales<PAIR>(tmem_base + SF_COL + slot * SF_SLOT + c * 4,
                              sa0 + off + c * (CHUNK / 16));
            const int after = (kb | 3) + 1;
            if (after >= k1 || after % GROUP_STAGES == 0) {
              commit<PAIR>(&sempty[sl]);
              if (++sl == SF_RING) {
                sl = 0;
                sph ^= 1u;
              }
            }
          }
          const uint32_t more = kb > k0 ? 1u : 0u;
          if (MODE == 2 || kb < len / KS)
            products(kb, 4, id, d, more);
          else
            products(kb, (len - kb * KS) / 32, id, d, more);
          commit<PAIR>(&empty[s]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        commit<PAIR>(&tfull[odd]);
        return !dead;
      });
      dead = __any_sync(0xffffffffu, dead);
      if (elect_one()) {
        if constexpr (PAIR)
          tc_commit_pair_mc(drain, 0x1);
        else
          tc_commit(drain);
      }
      __syncwarp();
      if ((!mbar_wait(drain, 0, kWaitLimitNs) || dead) && lane == 0) atomicOr(p.err, kErrTimeout);
    }
  } else if (warp >= 4) {
    // two warps to a quarter of the rows, 64 of an accumulator's columns each
    const int w = warp & 3, half = (warp - 4) >> 2;
    uint32_t tiles_done = 0;
    bool dead = false;
    TO* out = static_cast<TO*>(p.out);
    const uint32_t leader_tfree = PAIR ? mapa_shared(smem_u32(tfree), 0) : 0;
    auto finish = [&](float v) { return MODE == 0 && p.silu ? silu_of<TO>(v) : v; };
    const bool sectors = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;  // (rows are multiples of 128)
    walk([&](int t, int k0, int k1, int p0, int p1) {
      const Tile tl = tile(t);
      const bool whole = MODE == 2 || (p0 == 0 && p1 == kst);
      const bool more = k0 > p0, last_chain = k1 == p1;
      // rows of this warp's 32 lanes
      const int r0 = static_cast<int>(rank) * 128 + w * 32, rows = min(32, tl.rows - r0);
      const size_t out_row = (MODE == 2 ? static_cast<size_t>(tl.e) * K : 0) + tl.row0 + r0;
      const int first = split ? rg.owner(t * kst) : 0;
      // a CTA's part of the tile its range starts in comes first, of the one
      // it ends in second
      auto slice = [&](int c) {
        return p.part + static_cast<size_t>(c * 2 + (c > first ? 0 : 1)) * kSplitRows * kTileCols;
      };
      if (MODE == 2 && k0 == k1) {
        // an expert without rows
        for (int i = lane; i < rows * 32; i += 32) {
          const int col = (i >> 4 & 1) * HN + half * 64 + (i & 15) * 4;
          if (col < tl.n)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) +
                                       (out_row + (i >> 5)) * width + tl.n0 + col) =
                float4{0.f, 0.f, 0.f, 0.f};
        }
        return true;
      }
      const uint32_t odd = tiles_done & 1;
      // after a wait that ran out the loops go on, so that the eight warps
      // still meet at every barrier
      if (!dead && !mbar_wait(&tfull[odd], tiles_done >> 1 & 1, kWaitLimitNs)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      tc_fence_after();
      ++tiles_done;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        // the middle accumulator first: an even tile's second half
        const int j = i ^ static_cast<int>(odd) ^ 1;
        const int col = j * HN + half * 64;
        const bool some = rows > 0 && col < tl.n;
        uint32_t r[2][32];
        if (some) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(w * 32) << 16) + (odd + j) * HN +
                                   half * 64 + i * 32,
                               r[i]);
          tmem_ld_wait();
        }
        // free before the stores: the next tile waits for the middle one.
        // (What was read is in registers, so there is nothing to release: as
        // releases at cluster scope the two arrivals took a third of a weight
        // gradient's time, 200 us where it then took 139.)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_remote_relaxed(leader_tfree + (odd + j) * 8);
          else
            mbar_arrive(&tfree[odd + j]);
        }
        if (some && whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (CHAIN == 0)
              put_rows32(out, sectors, out_row, rows, width, tl.n0 + col + i * 32, r[i], finish);
            else
              put_rows32_by(out, out_row, rows, width, tl.n0 + col + i * 32, r[i],
                            [](float v) { return v; }, [&](TO* to, uint32_t (&v)[8]) {
                              if (more) add_sector(v, to);
                              if (MODE == 0 && last_chain && p.silu) {
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                  v[c] = __float_as_uint(finish(__uint_as_float(v[c])));
                              }
                              st_sector(sectors, to, v);
                            });
          }
        } else if (some && lane < rows) {
          // (at most kSplitRows rows: the first quarter's)
          uint32_t* o = reinterpret_cast<uint32_t*>(slice(cta) + lane * kTileCols + col);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              uint32_t v[8] = {r[i][c],     r[i][c + 1], r[i][c + 2], r[i][c + 3],
                               r[i][c + 4], r[i][c + 5], r[i][c + 6], r[i][c + 7]};
              if (CHAIN != 0 && more) add_sector(v, reinterpret_cast<float*>(o + i * 32 + c));
              st_sector(true, o + i * 32 + c, v);
            }
        }
      }
      if (!whole && last_chain) {
        const int last_cta = rg.owner((t + 1) * kst - 1);
        __threadfence();
        bar_epi();
        if (tid == 128) {
          const bool last = atomicAdd(p.ctr + t, 1u) == static_cast<uint32_t>(last_cta - first);
          if (last) p.ctr[t] = 0;
          *s_last = last ? 1u : 0u;
        }
        bar_epi();
        if (*s_last != 0) {
          __threadfence();
          const int quads = tl.n / 4;
          for (int i = tid - 128; i < tl.rows * quads; i += EPI_THREADS) {
            const int row = i / quads, col = (i - row * quads) * 4;
            float4 v = {0.f, 0.f, 0.f, 0.f};
            for (int cb = first; cb <= last_cta; cb += 8) {
              float4 o[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                o[j] = cb + j <= last_cta
                           ? __ldcg(reinterpret_cast<const float4*>(slice(cb + j) +
                                                                    row * kTileCols + col))
                           : float4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                v.x += o[j].x;
                v.y += o[j].y;
                v.z += o[j].z;
                v.w += o[j].w;
              }
            }
            TO* o = out + static_cast<size_t>(tl.row0 + row) * width + tl.n0 + col;
            o[0] = static_cast<TO>(finish(v.x));
            o[1] = static_cast<TO>(finish(v.y));
            o[2] = static_cast<TO>(finish(v.z));
            o[3] = static_cast<TO>(finish(v.w));
          }
        }
      }
      return true;
    });
    if (dead && lane == 0) atomicOr(p.err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else
      tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Rows per expert, on average, from which pairs of CTAs work on Y and dX (dW:
// always). One CTA and pairs, Y, us: at 128 rows each 40 and 46 (64 experts of
// 2048 x 1408), 67 and 71 (8 of 4096 x 11008), 79 and 95 (32 of 7168 x 2048); at
// 448 85 and 78, 146 and 125, 178 and 161; skewed 84 and 83, 147 and 132, 176 and
// 172. Between, tiles of 256 rows decide: at 256 each 55 and 50, 83 and 75, 110
// and 105; at 384 67 and 74, 105 and 120, 147 and 147; skewed at 320 69 and 69,
// 111 and 107, 139 and 163.
constexpr int kPairRows = 448;

template <int MODE, bool PAIR, typename TO>
cudaError_t launch_product(const CUtensorMap& mA, const CUtensorMap& mA32, const CUtensorMap& mB,
                           const f8::Params& p, int grid, cudaStream_t s) {
  using C = f8::Cfg<PAIR>;
  auto* kernel = fp8_product_kernel<MODE, PAIR, TO>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(PAIR ? grid / 2 * 2 : grid);
  lc.blockDim = dim3(f8::THREADS);
  lc.dynamicSmemBytes = C::SMEM;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, mA, mA32, mB, p);
}

template <typename T, int ACT>
cudaError_t launch_rows(const void* x, const int32_t* src, int x_rows, const float* weight,
                        const void* z, const int32_t* offsets, int E, int R, int C, uint8_t* q,
                        uint8_t* sc, uint8_t* cq, uint8_t* csc, uint32_t* err, int num_sms,
                        cudaStream_t s) {
  const T *xt = static_cast<const T*>(x), *zt = static_cast<const T*>(z);
  auto grid = [](long long items, long long most) {
    return dim3(static_cast<unsigned>(items < most ? items : most));
  };
  if (cq == nullptr) {
    const long long groups = static_cast<long long>(R) * up_div(C, sizeof(T) == 4 ? 512 : 1024);
    auto go = [&](auto kernel) {
      return launch_pdl(kernel, grid((groups + 7) / 8, static_cast<long long>(num_sms) * kRowBlocks),
                        dim3(256), 0, s, xt, src, x_rows, weight, zt, offsets, E, R, C, q, sc, err);
    };
    if constexpr (sizeof(T) == 2 && ACT == MOE_ACT_NONE)
      if (weight == nullptr) return go(fp8_rows_kernel<T, ACT, true>);
    return go(fp8_rows_kernel<T, ACT, false>);
  }
  const long long tiles = static_cast<long long>(row_tiles(R, E)) * up_div(C, 128);
  const ColOut o{q, sc, cq, csc};
  auto go = [&](auto kernel, int smem, auto... args) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int each = smem <= 64 * 1024 ? 3 : smem <= 96 * 1024 ? 2 : 1;  // blocks on an SM
    return launch_pdl(kernel, grid(tiles, static_cast<long long>(num_sms) * each),
                      dim3(kColThreads), smem, s, xt, src, x_rows, args..., offsets, E, R, C, o,
                      err);
  };
  if constexpr (sizeof(T) == 2 && ACT == MOE_ACT_NONE)
    if (weight == nullptr) {
      constexpr int SMEM = ColRing<T, 1, 2>::SMEM;
      return q == nullptr ? go(fp8_columns_bf16_kernel<false>, SMEM)
                          : go(fp8_columns_bf16_kernel<true>, SMEM);
    }
  constexpr int SMEM = ColRing<T, ACT == MOE_ACT_SILU_GRAD ? 2 : 1, 3>::SMEM;
  return q == nullptr ? go(fp8_columns_kernel<T, ACT, false>, SMEM, weight, zt)
                      : go(fp8_columns_kernel<T, ACT, true>, SMEM, weight, zt);
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
                        int per, int pitch, void* out, cudaStream_t s) {
  return launch_pdl(fp8_back_kernel<T>, dim3(up_div(rows, 128), up_div(cols, 128), experts),
                    dim3(kColThreads), 0, s, q, sc, rows, cols, per, pitch, static_cast<T*>(out));
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
  const dim3 grid(up_div(N, 128), up_div(K, 128), E), block(kColThreads);
  return dtype == 0 ? launch_pdl(fp8_weights_kernel<float>, grid, block, 0, s,
                                 static_cast<const float*>(W), K, N, q, sc)
                    : launch_pdl(fp8_weights_kernel<__nv_bfloat16>, grid, block, 0, s,
                                 static_cast<const __nv_bfloat16*>(W), K, N, q, sc);
}

cudaError_t launch_fp8_back(int dtype, const uint8_t* q, const uint8_t* sc, int experts, int rows,
                            int cols, int per, int pitch, void* out, cudaStream_t s) {
  return dtype == 0 ? launch_back<float>(q, sc, experts, rows, cols, per, pitch, out, s)
                    : launch_back<__nv_bfloat16>(q, sc, experts, rows, cols, per, pitch, out, s);
}

cudaError_t launch_fp8_product(int mode, const uint8_t* a, const uint8_t* as, const uint8_t* b,
                               const uint8_t* bs, const int32_t* offsets, int E, int R, int K,
                               int N, int out_f32, int silu, void* out, uint32_t* err,
                               uint32_t* ctr, float* part, int num_sms, cudaStream_t s) {
  CUtensorMap mA, mA32, mB;
  const uint64_t cr = row_tiles(R, E) * 128;
  const uint64_t len = mode == 1 ? N : K;
  if (mode == 2 ? !make_map_2d_bytes(&mA, a, cr, K, 128) || !make_map_2d_bytes(&mB, b, cr, N, 128)
                : !make_map_2d_bytes(&mA, a, R, len, 128) ||
                      !make_map_2d_bytes(&mA32, a, R, len, 32) ||
                      !make_map_3d_bytes(&mB, b, E, K, N))
    return cudaErrorInvalidValue;
  if (mode == 2) mA32 = mA;
  const f8::Params p{as, bs, offsets, out, err, ctr, part, E, R, K, N, silu};
  const int grid = num_sms < kProductCtas ? num_sms : kProductCtas;
  if (mode == 2) return launch_product<2, true, float>(mA, mA32, mB, p, grid, s);
  const bool pair = R >= kPairRows * E;
  auto go = [&](auto kernel) { return kernel(mA, mA32, mB, p, grid, s); };
  if (mode == 1)
    return pair ? (out_f32 ? go(launch_product<1, true, float>)
                           : go(launch_product<1, true, __nv_bfloat16>))
                : (out_f32 ? go(launch_product<1, false, float>)
                           : go(launch_product<1, false, __nv_bfloat16>));
  return pair ? (out_f32 ? go(launch_product<0, true, float>)
                         : go(launch_product<0, true, __nv_bfloat16>))
              : (out_f32 ? go(launch_product<0, false, float>)
                         : go(launch_product<0, false, __nv_bfloat16>));
}

}  // namespace moe
