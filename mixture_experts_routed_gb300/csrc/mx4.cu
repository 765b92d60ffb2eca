// mx4.cu - microscaled 4-bit floating point for the expert products: the
// quantisation of rows and of expert weights, and the expert-grouped product
// of the two on the tensor cores (tcgen05.mma kind::mxf4 with block scales).
//
// Format (OCP Microscaling, MXFP4): blocks of 32 values along the
// contraction share a power-of-two scale 2^(s - 127), s one byte (E8M0);
// each value is E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives):
//   s - 127 = max(floor(log2 amax) - 2, -127)   (s = 127 for a zero block,
//   255, which stands for NaN, for a block with an infinity or NaN)
//   q = E2M1(v / 2^(s - 127)), to nearest even, saturating at +-6
// Scaling by a power of two is exact, so the form is a function of the input
// bits alone.
//
//   Y[r][n] = sum_k a[r][k] w[e][n][k]      r a row of expert e's segment
//
// Codes: two to a byte, the even k in the low half: rows [R][K / 2], weights
// [E][N][K / 2] (transposed, so that k is innermost on both sides, which the
// 4-bit products want). Scales: for the tensor core, in chunks of 128 rows x
// 4 blocks (128 values of k), 512 bytes: row i, block j at (i % 32) 16 +
// (i / 32) 4 + j; weights [E][ceil(N / 128)][ceil(K / 128)] chunks, rows
// [row tile][ceil(K / 128)] chunks, the row tiles being each expert's
// segment cut into tiles of 128 rows, one expert after the other, so that a
// product's tile finds its scales in one piece wherever its segment starts.
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "grouped.cuh"
#include "ptx.cuh"
#include "range.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int CHUNK = 512;  // bytes of scales of 128 rows x 128 values

__device__ __forceinline__ uint32_t scale_code(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  if (amax_bits == 0u) return 127u;
  // floor(log2): the exponent field, or for a subnormal the leading bit's
  const int e = amax_bits >= 0x00800000u ? static_cast<int>(amax_bits >> 23) - 127
                                         : -118 - __clz(amax_bits);
  return static_cast<uint32_t>(max(e - 2, -127) + 127);
}
// 1 / scale = 2^(127 - s): exact for s in 0..252
__device__ __forceinline__ float inv_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (254u - s) << 23);
}
// the scale 2^(s - 127) (s = 0: 2^-127, subnormal)
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (s == 0u ? 0x00400000u : s << 23));
}

// 8 scaled values to 8 codes, v[0] lowest
__device__ __forceinline__ uint32_t pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The value of code j of the eight in w: its bits as the top of a number
// (sign; exponent and mantissa at 24..22, so 2^-126 times the value, the code
// .5 a subnormal) and then scaled; four instructions where the conversion
// instruction runs at a fraction of the rate.
__device__ __forceinline__ float code_value(uint32_t w, int j) {
  const uint32_t t = w << (28 - 4 * j);
  return __uint_as_float((t & 0x80000000u) | ((t >> 6) & 0x01c00000u)) * 0x1p126f;
}

// first byte of row r's scales of 128-value group 0 (groups CHUNK apart)
__device__ __forceinline__ size_t row_scale_at(int r, const int* seg, const int* base, int E,
                                               int kc) {
  const int e = last_at_most(seg, E - 1, r);  // (empty segments share their start)
  const int i = r - seg[e];
  return static_cast<size_t>(base[e] + (i >> 7)) * kc * CHUNK + (i & 31) * 16 +
         ((i & 127) >> 5) * 4;
}

// ---------------------------------------------------------------- rows
// A warp quantises groups of four spans (256 bf16 or 128 fp32 values each) of
// a row: a lane loads 16 bytes of a span, a block's 4 (8) lanes agree on its
// amax, and a lane stores 4 (2) bytes of codes. The groups of all rows are
// shared out evenly, each warp's one after the other, and a group is loaded
// while the one before it is quantised. Bound by HBM: the row is read once.
// 16384 rows of 7168 bf16 values: 51.6 us, 5.7 TB/s (55.2 with whole rows to a
// warp: 9728 warps took one row or two; 60.6 with neighbouring groups to
// neighbouring warps). kRowBlocks: those of 256 threads an SM holds at once (2,
// 3, 4, 6: 57.6, 52.0, 51.6, 54.8 us).
constexpr int kRowBlocks = 4;

template <typename T>
__global__ void __launch_bounds__(256)
    mx4_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ src, int x_rows,
                    const int32_t* __restrict__ offsets, int E, int R, int K,
                    uint8_t* __restrict__ q, uint8_t* __restrict__ sc, uint32_t* err) {
  constexpr int V = 16 / sizeof(T), LPB = 32 / V, SPAN = 32 * V, F = 4;
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  pdl_wait();
  pdl_trigger();
  if (!load_segments(offsets, E, R, seg, base, &ok, err)) return;
  const int lane = threadIdx.x & 31;
  const int kc = up_div(K, 128), groups = up_div(K, F * SPAN);
  // (at most 2^24 rows of 128 groups)
  const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
  const uint32_t total = static_cast<uint32_t>(seg[E] - seg[0]) * groups;
  const uint32_t share = total / warps, more = total - share * warps;
  const uint32_t g0 = share * warp + min(warp, more);
  int left = share + (warp < more ? 1 : 0);
  if (left == 0) return;
  int r = seg[0] + static_cast<int>(g0 / groups), g = static_cast<int>(g0 % groups);
  const T* row;
  bool in;
  auto find = [&](int r) {
    const int xr = src != nullptr ? __ldg(src + r) : r;
    in = xr >= 0 && xr < x_rows;
    if (!in && lane == 0) atomicOr(err, kErrBadIndex);
    row = x + static_cast<size_t>(in ? xr : 0) * K;
  };
  uint4 raw[F];
  auto load = [&](int kb) {
#pragma unroll
    for (int f = 0; f < F; ++f)
      raw[f] = in && kb + f * SPAN < K ? ld_once(row + kb + f * SPAN) : uint4{0, 0, 0, 0};
  };
  find(r);
  load(g * F * SPAN + lane * V);
  size_t at = row_scale_at(r, seg, base, E, kc);
  while (true) {
    uint8_t* qr = q + static_cast<size_t>(r) * (K / 2);
    uint8_t* sr = sc + at;
    const int kb = g * F * SPAN + lane * V;
    uint4 now[F];
#pragma unroll
    for (int f = 0; f < F; ++f) now[f] = raw[f];
    if (--left > 0) {
      if (++g == groups) {
        g = 0;
        find(++r);
        at = row_scale_at(r, seg, base, E, kc);
      }
      load(g * F * SPAN + lane * V);
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int k = kb + f * SPAN;
      const uint32_t w[4] = {now[f].x, now[f].y, now[f].z, now[f].w};
      // |v| orders as its bits do, infinities and NaN above every number
      uint32_t m;
      if constexpr (V == 8) {
        m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                     __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = max(m << 16, m & 0xffff0000u);
      } else {
        m = max(max(w[0] & 0x7fffffffu, w[1] & 0x7fffffffu),
                max(w[2] & 0x7fffffffu, w[3] & 0x7fffffffu));
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      const uint32_t s = scale_code(m);
      const float inv = inv_scale(s);
      float v[8] = {};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (V == 8)
          v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16) * inv;
        else
          v[j] = __uint_as_float(w[j]) * inv;
      }
      const uint32_t codes = pack8(v);
      // the four blocks of a 128-value group, as one word from its first lane
      uint32_t word = s | __shfl_down_sync(0xffffffffu, s, LPB) << 8;
      word |= __shfl_down_sync(0xffffffffu, word, 2 * LPB) << 16;
      if (k < K) {
        if constexpr (V == 8)
          *reinterpret_cast<uint32_t*>(qr + k / 2) = codes;
        else
          *reinterpret_cast<uint16_t*>(qr + k / 2) = static_cast<uint16_t>(codes);
        if (lane % (4 * LPB) == 0)
          *reinterpret_cast<uint32_t*>(sr + static_cast<size_t>(k >> 7) * CHUNK) = word;
      }
    }
    if (left == 0) return;
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
    mx4_rows_back_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc,
                         const int32_t* __restrict__ offsets, int E, int R, int K,
                         T* __restrict__ out) {
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  pdl_wait();
  pdl_trigger();
  if (!load_segments(offsets, E, R, seg, base, &ok, nullptr)) return;
  const int kc = up_div(K, 128), words = K / 8;
  const long long total = static_cast<long long>(seg[E] - seg[0]) * words;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * 256) {
    const int r = seg[0] + static_cast<int>(i / words), k = static_cast<int>(i % words) * 8;
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(q + static_cast<size_t>(r) * (K / 2) + k / 2));
    const float s = scale_value(__ldg(sc + row_scale_at(r, seg, base, E, kc) +
                                      static_cast<size_t>(k >> 7) * CHUNK + ((k >> 5) & 3)));
    T* o = out + static_cast<size_t>(r) * K + k;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = code_value(c, j) * s;
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------- weights
// W [E][K][N] -> codes [E][N][K / 2]: a block takes 256 (fp32: 128) values of
// k x 64 of n through shared memory; a thread quantises two blocks of 32 of
// one n, so that the rows of W and the runs of codes (32 bytes) are read and
// written in whole sectors. Bound by HBM: 16 x 1536 x 5120 bf16 values to 4
// bits in 59 us, 5.4 TB/s.
template <typename T>
constexpr int kWeightK = 512 / sizeof(T);
template <typename T>
constexpr int kWeightThreads = kWeightK<T>;  // 64 n x (k / 64)

// byte of the scale of column n, block k / 32 of expert e
__device__ __forceinline__ size_t weight_scale_at(int e, int n, int k, int K, int N) {
  return ((static_cast<size_t>(e) * up_div(N, 128) + (n >> 7)) * up_div(K, 128) + (k >> 7)) *
             CHUNK +
         (n & 31) * 16 + ((n & 127) >> 5) * 4 + ((k >> 5) & 3);
}

template <typename T>
__global__ void __launch_bounds__(kWeightThreads<T>)
    mx4_weights_kernel(const T* __restrict__ W, int K, int N, uint8_t* __restrict__ q,
                       uint8_t* __restrict__ sc) {
  constexpr int KT = kWeightK<T>, TH = kWeightThreads<T>, V = 16 / sizeof(T), PER = 64 / V;
  __shared__ __align__(16) T tile[KT][64];
  pdl_wait();
  pdl_trigger();
  const int n0 = blockIdx.x * 64, k0 = blockIdx.y * KT, e = blockIdx.z;
  const T* We = W + static_cast<size_t>(e) * K * N;
#pragma unroll
  for (int j = 0; j < KT * PER / TH; ++j) {
    const int i = threadIdx.x + j * TH, k = i / PER, c = (i % PER) * V;
    if (k0 + k < K)
      ptx::cp_async16(ptx::smem_u32(&tile[k][c]), We + static_cast<size_t>(k0 + k) * N + n0 + c);
  }
  ptx::cp_async_commit();
  ptx::cp_async_wait<0>();
  __syncthreads();
  const int n = threadIdx.x & 63, kt = (threadIdx.x >> 6) * 64;
  if (k0 + kt >= K) return;  // (K is a multiple of 64)
  uint32_t s2[2];
  uint4 w4[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = static_cast<float>(tile[kt + h * 32 + j][n]);
      m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    s2[h] = scale_code(m);
    const float inv = inv_scale(s2[h]);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = v[8 * j + i] * inv;
      w[j] = pack8(u);
    }
    w4[h] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  uint4* o = reinterpret_cast<uint4*>(q + (static_cast<size_t>(e) * N + n0 + n) * (K / 2) +
                                      (k0 + kt) / 2);
  o[0] = w4[0];
  o[1] = w4[1];
  *reinterpret_cast<uint16_t*>(sc + weight_scale_at(e, n0 + n, k0 + kt, K, N)) =
      static_cast<uint16_t>(s2[0] | s2[1] << 8);
}

// And back: a thread takes one block of 32 of two neighbouring n, so that it
// writes both values of a k at once. 69 us for the same weights, 252 MB
// written, which is what filling that memory takes (66).
template <typename T>
__global__ void __launch_bounds__(kWeightThreads<T>)
    mx4_weights_back_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc, int K,
                            int N, T* __restrict__ W) {
  constexpr int KT = kWeightK<T>, TH = kWeightThreads<T>, V = 16 / sizeof(T), PER = 64 / V;
  __shared__ __align__(16) T tile[KT][64];
  pdl_wait();
  pdl_trigger();
  const int n0 = blockIdx.x * 64, k0 = blockIdx.y * KT, e = blockIdx.z;
  const int n = (threadIdx.x & 31) * 2, kt = (threadIdx.x >> 5) * 32;
  if (k0 + kt < K) {
    const uint8_t* c = q + (static_cast<size_t>(e) * N + n0 + n) * (K / 2) + (k0 + kt) / 2;
    const uint4 a4 = __ldg(reinterpret_cast<const uint4*>(c));
    const uint4 b4 = __ldg(reinterpret_cast<const uint4*>(c + K / 2));
    const size_t at = weight_scale_at(e, n0 + n, k0 + kt, K, N);
    const float sa = scale_value(__ldg(sc + at)), sb = scale_value(__ldg(sc + at + 16));
    const uint32_t wa[4] = {a4.x, a4.y, a4.z, a4.w}, wb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float fa = code_value(wa[j >> 3], j & 7) * sa, fb = code_value(wb[j >> 3], j & 7) * sb;
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2*>(&tile[kt + j][n]) = make_float2(fa, fb);
      } else {
        *reinterpret_cast<__nv_bfloat162*>(&tile[kt + j][n]) = __floats2bfloat162_rn(fa, fb);
      }
    }
  }
  __syncthreads();
  T* We = W + static_cast<size_t>(e) * K * N;
#pragma unroll
  for (int j = 0; j < KT * PER / TH; ++j) {
    const int i = threadIdx.x + j * TH, k = i / PER, c0 = (i % PER) * V;
    if (k0 + k < K)
      *reinterpret_cast<uint4*>(We + static_cast<size_t>(k0 + k) * N + n0 + c0) =
          *reinterpret_cast<const uint4*>(&tile[k][c0]);
  }
}

// ---------------------------------------------------------------- product
// Tiles of 128 rows of one expert x up to 256 columns on one CTA, or of 256
// rows x 256 columns on a pair of CTAs (cta_group::2: each stages its own 128
// rows and half of the columns, so a byte staged feeds twice the products);
// persistent. A stage of the TMA ring holds 256 values of k: the rows' and
// the weights' codes (128-byte rows, 128-byte swizzle, both k-major; a warp
// loads each) and their scale chunks (of a pair's columns: all of them, on
// both sides). One thread copies a stage's scales to tensor memory
// (tcgen05.cp, the 512 bytes of a chunk to 4 columns of each of the four lane
// quarters) and issues the products of 128 columns x K 64 that read them; the
// scales have a ring of columns of their own, one stage shorter than the
// data's (tensor memory's most), so a stage's copy never meets a product still
// reading. Three accumulators of 128 columns: a tile takes two, and the next
// tile starts once one of them is drained, with the first half's products of
// its first stages. Eight warps drain: into registers, which frees the
// accumulator, and then to out.
//
// Bound: a product takes the tensor core 64 clocks whatever its columns' split
// (one of 256 columns: 128), so a pair's stage 514, 9.5 PFLOP/s in all. Dense
// 8192 x 8192 x 8192 in bf16: 148 us, 7.4 PFLOP/s (171 with the accumulators
// freed after the stores by four warps that wrote a sector of each row at a
// time, one loading warp and five stages: of a stage's 790 clocks 100 went to
// accumulators not yet drained and 150 to the issuing loop). 16384 skewed rows
// of 32 experts, 7168 x 2048 to fp32: 109 us (116), where 445 MB move and 632
// tiles over 76 pairs leave the last of nine waves two thirds empty.
namespace mx {
constexpr int BN = kTileCols, HN = 128, KS = 256;  // a tile's columns, an accumulator's, a stage's k
constexpr int B_BOX = 64 * 128;             // a box of 64 columns
constexpr int A_BYTES = 128 * 128;
constexpr int SF_COL = 384, SF_STAGE = 24;  // tensor memory columns: 3 x 128, then scales
constexpr int TMEM_COLS = 512, ACCS = 3;
constexpr int EPI_THREADS = 256, THREADS = 128 + EPI_THREADS;

template <bool PAIR>
struct Cfg {
  static constexpr int BM = PAIR ? 256 : 128;
  static constexpr int B_BYTES = (PAIR ? 128 : 256) * 128;
  static constexpr int OFF_B = A_BYTES, OFF_SFA = OFF_B + B_BYTES, OFF_SFB = OFF_SFA + 2 * CHUNK;
  static constexpr int STAGE = OFF_SFB + 4 * CHUNK;
  static constexpr int STAGES = PAIR ? 6 : 4;  // (shared memory's most)
  static constexpr int SLOTS = STAGES < 5 ? STAGES : 5;  // of scales (tensor memory's most)
  static constexpr int OFF_BAR = STAGES * STAGE;
  static constexpr int OFF_SEG = OFF_BAR + (2 * STAGES + 2 * ACCS + 1) * 8 + 24;
  static constexpr int SMEM = OFF_SEG + 3 * (kMaxExperts + 1) * 4 + 1024;
  static_assert(STAGE % 1024 == 0 && SMEM <= 227 * 1024, "shared memory");
  static_assert(SF_COL + SLOTS * SF_STAGE <= TMEM_COLS && STAGES - SLOTS <= 1, "tensor memory");
};

struct Params {
  const int32_t* offsets;
  void* out;
  uint32_t* err;
  uint32_t* ctr;  // arrivals per tile of a split launch, zero between launches
  float* part;    // [CTA][2][kSplitRows][256]
  int E, R, K, N;
  int silu;
};

// kind::mxf4, E2M1 both sides, E8M0 scales, fp32 accumulator, both K-major,
// K = 64; sf: which half of a scale column's four bytes
__device__ __forceinline__ uint32_t idesc_mxf4(int m, int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 7) << 27) | (sf << 29);
}
// Operand descriptors: the low word holds the address, the high one does not
// change (128-byte swizzle, 8-row groups 1024 bytes apart, version 1).
constexpr uint32_t AB_HI = (1024 >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t SF_HI = (128 >> 4) | 1u << 14;  // no swizzle, 8-row groups 128 bytes apart
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }

template <bool PAIR>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, "
        "[%4], [%5], p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(AB_HI)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, "
        "[%4], [%5], p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(AB_HI)
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

}  // namespace mx

// TO: the output type
template <bool PAIR, typename TO>
__global__ void __launch_bounds__(mx::THREADS, 1)
    mx4_product_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmA32,
                       const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmSA,
                       const __grid_constant__ CUtensorMap tmSB, const mx::Params p) {
  using namespace mx;
  using C = Cfg<PAIR>;
  constexpr int STAGES = C::STAGES, BM = C::BM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // pair: the even CTA's
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + ACCS;  // pair: the even CTA's
  uint64_t* drain = tempty + ACCS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
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

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], PAIR ? 16 : 8);
    }
    mbar_init(drain, 1);
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
  if (PAIR && warp == 0) {
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
  const int kst = up_div(K, KS), kc = up_div(K, 128);
  const int tiles = ok ? tb[E] * up_div(N, BN) : 0;
  // Few rows everywhere and fewer tiles than CTAs: the tiles' stages are one
  // sequence cut into equal ranges, and a tile's partial sums are joined by
  // the last CTA to arrive, in CTA order. Otherwise whole tiles in turn.
  const bool split = !PAIR && tiles < grid && *s_wide == 0;
  const Range rg(split ? tiles : 0, kst, grid);
  // Walk this CTA's pieces: f(tile, first stage, end stage)
  auto walk = [&](auto f) {
    if (split) {
      const int end = rg.start(cta + 1);
      for (int i = rg.start(cta); i < end;) {
        const int t = i / kst, k0 = i - t * kst, k1 = min(kst, k0 + end - i);
        if (!f(t, k0, k1)) return;
        i += k1 - k0;
      }
    } else {
      for (int t = cta; t < tiles; t += grid)
        if (!f(t, 0, kst)) return;
    }
  };

  if (warp == 0 || warp == 2) {
    // the first loads the rows, the other the weights (the whole warp,
    // converged: elect_one says why)
    const bool a_side = warp == 0;
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmA32);
      prefetch_tmap(&tmB);
      prefetch_tmap(&tmSA);
      prefetch_tmap(&tmSB);
    }
    __syncwarp();
    int s = 0, used = 0;
    uint32_t ph = 0;
    bool dead = false;
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
    walk([&](int t, int k0, int k1) {
      const Tile tl = tile_at<BM>(t, seg, base, tb, E, N);
      const int nt = up_div(N, HN);
      // CTA r's rows come in one box of 128 or, few, of 32, and its columns
      // in boxes of 64; what is not loaded feeds only sums that are not stored
      auto a_bytes = [&](int r) {
        const int left = tl.rows - r * 128;
        return left <= 0 ? 0 : (left <= 32 ? A_BYTES / 4 : A_BYTES);
      };
      auto b_boxes = [&](int r) {
        if (!PAIR) return tl.n / 64;
        const int left = tl.n - r * 64;
        return (left > 0) + (left > HN);
      };
      auto bytes = [&](int r) {
        const int na = a_bytes(r);
        return na + b_boxes(r) * B_BOX + (na > 0 ? 2 * CHUNK : 0) + 4 * CHUNK;
      };
      const int na = a_bytes(rank), nb = b_boxes(rank);
      const uint32_t expect = PAIR ? bytes(0) + bytes(1) : bytes(0);
      const CUtensorMap* ma = na == A_BYTES ? &tmA : &tmA32;
      const int mt = tl.mt + rank, row0 = tl.row0 + rank * 128;
      const int col0 = tl.e * N + tl.n0 + (PAIR ? static_cast<int>(rank) * 64 : 0);
      const int sbt = tl.e * nt + tl.n0 / HN;
      for (int kb = k0; kb < k1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, kWaitLimitNs))) {
          dead = true;
          return false;
        }
        if (used < STAGES) ++used;
        if (elect_one()) {
          uint8_t* st = smem + s * C::STAGE;
          if (a_side) {
            if (rank == 0) mbar_arrive_expect_tx(&full[s], expect);
            if (na > 0) {
              load2(st, ma, kb * 128, row0);
              load3(st + C::OFF_SFA, &tmSA, 0, kb * 2, mt);
            }
          } else {
#pragma unroll
            for (int b = 0; b < (PAIR ? 2 : 4); ++b)
              if (b < nb)
                load2(st + C::OFF_B + b * B_BOX, &tmB, kb * 128, col0 + b * (PAIR ? HN : 64));
            load3(st + C::OFF_SFB, &tmSB, 0, kb * 2, sbt);
          }
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      return true;
    });
    // the latest use of each stage has landed before this CTA may exit (a
    // pair: the even CTA's barrier counts both, and both exit together)
    for (int j = 0; a_side && rank == 0 && j < used; ++j) {
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
    if (dead && lane == 0) atomicOr(p.err, kErrTimeout);
  } else if (warp == 1) {
    // (one lane issues: elect_one says how)
    if (rank == 0) {
      int s = 0, acc = 0, slot = 0;
      uint32_t ph = 0, aph = 0;
      bool dead = false;
      constexpr int LEAD = C::SLOTS - 1;
      const uint32_t base0 = smem_u32(smem);
      const uint32_t ad0 = desc_lo(base0), bd0 = desc_lo(base0 + C::OFF_B),
                     sa0 = desc_lo(base0 + C::OFF_SFA), sb0 = desc_lo(base0 + C::OFF_SFB);
      constexpr int B_HALF = (PAIR ? 1 : 2) * B_BOX;
      const uint32_t id0 = idesc_mxf4(BM, HN, 0), id2 = idesc_mxf4(BM, HN, 2);
      // the stage, and the slot its scales go to, whose last products were
      // SLOTS steps ago, are there
      auto take = [&] {
        const bool last = s + 1 == STAGES;
        if (mbar_wait_spin(&full[s], ph, kWaitLimitNs) &&
            (C::SLOTS == STAGES ||
             mbar_wait_spin(&empty[last ? 0 : s + 1], last ? ph : ph ^ 1u, kWaitLimitNs))) {
          tc_fence_after();
          return true;
        }
        return false;
      };
      auto next = [&] {
        if (++slot == C::SLOTS) slot = 0;
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      };
      // a stage's scales, and its products for the halves j0..j1 of the
      // columns (inlined with constants for whole stages)
      auto scales = [&](int chunks, int nj) {
        const uint32_t off = static_cast<uint32_t>(s) * (C::STAGE / 16);
        const uint32_t sf = tmem_base + SF_COL + slot * SF_STAGE;
#pragma unroll
        for (int c = 0; c < chunks; ++c) {
          cp_scales<PAIR>(sf + c * 4, sa0 + off + c * (CHUNK / 16));
#pragma unroll
          for (int j = 0; j < nj; ++j)
            cp_scales<PAIR>(sf + 8 + c * 8 + j * 4,
                            sb0 + off + (2 * j + c) * (CHUNK / 16));
        }
      };
      auto products = [&](int steps, int j0, int j1, uint32_t d0, uint32_t d1, uint32_t more) {
        const uint32_t off = static_cast<uint32_t>(s) * (C::STAGE / 16);
        const uint32_t sf = tmem_base + SF_COL + slot * SF_STAGE;
#pragma unroll
        for (int kk = 0; kk < steps; ++kk)
#pragma unroll
          for (int j = j0; j < j1; ++j)
            mma_mxf4<PAIR>(j == 0 ? d0 : d1, ad0 + off + kk * 2,
                           bd0 + off + j * (B_HALF / 16) + kk * 2, (kk & 1) ? id2 : id0,
                           sf + (kk >> 1) * 4, sf + 8 + (kk >> 1) * 8 + j * 4,
                           kk > 0 ? 1u : more);
      };
      if (elect_one()) walk([&](int t, int k0, int k1) {
        const int n = tile_at<BM>(t, seg, base, tb, E, N).n;
        const int nj = n > HN ? 2 : 1;
        const int acc1 = acc + 1 == ACCS ? 0 : acc + 1;
        const uint32_t aph1 = acc + 1 == ACCS ? aph ^ 1u : aph;
        if (!mbar_wait_spin_cluster(&tempty[acc], aph ^ 1u, kWaitLimitNs)) {
          dead = true;
          return false;
        }
        tc_fence_after();
        const uint32_t d0 = tmem_base + acc * HN, d1 = tmem_base + acc1 * HN;
        const int whole = nj == 2 ? K / KS : 0;  // stages with nothing left out
        int kb = k0;
        if (nj == 2) {
          // until the second accumulator is drained too: the first half's
          // products of a few stages, and after that the second's
          const int s0 = s, slot0 = slot, most = min(min(k1, whole), k0 + LEAD);
          const uint32_t ph0 = ph;
          while (kb < most && !mbar_test_wait_cluster(&tempty[acc1], aph1 ^ 1u)) {
            if (!take()) {
              dead = true;
              return false;
            }
            scales(2, 2);
            products(4, 0, 1, d0, d1, kb > k0 ? 1u : 0u);
            next();
            ++kb;
          }
          if (!mbar_wait_spin_cluster(&tempty[acc1], aph1 ^ 1u, kWaitLimitNs)) {
            dead = true;
            return false;
          }
          tc_fence_after();
          s = s0;
          ph = ph0;
          slot = slot0;
          for (int i = k0; i < kb; ++i) {
            products(4, 1, 2, d0, d1, i > k0 ? 1u : 0u);
            commit<PAIR>(&empty[s]);
            next();
          }
        }
        for (; kb < k1; ++kb) {
          if (!take()) {
            dead = true;
            break;
          }
          const uint32_t more = kb > k0 ? 1u : 0u;
          if (kb < whole) {
            scales(2, 2);
            products(4, 0, 2, d0, d1, more);
          } else {
            scales(K - kb * KS > 128 ? 2 : 1, nj);
            products(min(4, K / 64 - kb * 4), 0, nj, d0, d1, more);
          }
          commit<PAIR>(&empty[s]);
          next();
        }
        for (int j = 0; j < nj; ++j) {
          commit<PAIR>(&tfull[acc]);
          if (++acc == ACCS) {
            acc = 0;
            aph ^= 1u;
          }
        }
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
    int acc = 0;
    uint32_t aph = 0;
    bool dead = false;
    TO* out = static_cast<TO*>(p.out);
    const uint32_t leader_tempty = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0;
    auto finish = [&](float v) { return p.silu ? silu_of<TO>(v) : v; };
    const bool sectors = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;  // (rows are multiples of 128)
    auto put32 = [&](size_t row0, int rows, int col, const uint32_t (&r)[32]) {
      put_rows32(out, sectors, row0, rows, N, col, r, finish);
    };
    walk([&](int t, int k0, int k1) {
      const Tile tl = tile_at<BM>(t, seg, base, tb, E, N);
      const bool whole = k0 == 0 && k1 == kst;
      // rows of this warp's 32 lanes
      const int r0 = static_cast<int>(rank) * 128 + w * 32, rows = min(32, tl.rows - r0);
      const int first = split ? rg.owner(t * kst) : 0;
      // a CTA's part of the tile its range starts in comes first, of the one
      // it ends in second
      auto slice = [&](int c) {
        return p.part + static_cast<size_t>(c * 2 + (c > first ? 0 : 1)) * kSplitRows * BN;
      };
      for (int h = 0; h < tl.n; h += HN) {
        // after a wait that ran out the loops go on, so that the eight warps
        // still meet at every barrier
        if (!dead && !mbar_wait(&tfull[acc], aph, kWaitLimitNs)) dead = true;
        dead = __any_sync(0xffffffffu, dead);
        tc_fence_after();
        const int col = h + half * 64;
        const bool some = rows > 0 && col < tl.n;
        uint32_t r[2][32];
        if (some) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(w * 32) << 16) + acc * HN +
                                   half * 64 + i * 32,
                               r[i]);
          tmem_ld_wait();
        }
        // free before the stores: the next tile waits for this one's first half
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_remote(leader_tempty + acc * 8);
          else
            mbar_arrive(&tempty[acc]);
        }
        if (some && whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            put32(static_cast<size_t>(tl.row0 + r0), rows, tl.n0 + col + i * 32, r[i]);
        } else if (some && lane < rows) {
          // (at most kSplitRows rows: the first quarter's)
          uint32_t* o = reinterpret_cast<uint32_t*>(slice(cta) + lane * BN + col);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              const uint32_t v[8] = {r[i][j],     r[i][j + 1], r[i][j + 2], r[i][j + 3],
                                     r[i][j + 4], r[i][j + 5], r[i][j + 6], r[i][j + 7]};
              st_sector(true, o + i * 32 + j, v);
            }
        }
        if (++acc == ACCS) {
          acc = 0;
          aph ^= 1u;
        }
      }
      if (!whole) {
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
                           ? __ldcg(reinterpret_cast<const float4*>(slice(cb + j) + row * BN + col))
                           : float4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                v.x += o[j].x;
                v.y += o[j].y;
                v.z += o[j].z;
                v.w += o[j].w;
              }
            }
            TO* o = out + static_cast<size_t>(tl.row0 + row) * N + tl.n0 + col;
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

template <bool PAIR, typename TO>
cudaError_t launch_product(const CUtensorMap& mA, const CUtensorMap& mA32, const CUtensorMap& mB, const CUtensorMap& mSA,
                           const CUtensorMap& mSB, const mx::Params& p, int grid, cudaStream_t s) {
  using C = mx::Cfg<PAIR>;
  auto* kernel = mx4_product_kernel<PAIR, TO>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(PAIR ? grid / 2 * 2 : grid);
  lc.blockDim = dim3(mx::THREADS);
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
  return cudaLaunchKernelEx(&lc, kernel, mA, mA32, mB, mSA, mSB, p);
}

int blocks_for(long long items, int per_block, int most) {
  const long long b = (items + per_block - 1) / per_block;
  return static_cast<int>(b < 1 ? 1 : (b < most ? b : most));
}

}  // namespace

cudaError_t launch_mx4_rows(int dtype, const void* x, const int32_t* src, int x_rows,
                            const int32_t* offsets, int E, int R, int K, uint8_t* q, uint8_t* sc,
                            uint32_t* err, int num_sms, cudaStream_t s) {
  const long long groups = static_cast<long long>(R) * up_div(K, dtype == 0 ? 512 : 1024);
  const dim3 grid(blocks_for(groups, 8, num_sms * kRowBlocks));
  return dtype == 0
             ? launch_pdl(mx4_rows_kernel<float>, grid, dim3(256), 0, s,
                          static_cast<const float*>(x), src, x_rows, offsets, E, R, K, q, sc, err)
             : launch_pdl(mx4_rows_kernel<__nv_bfloat16>, grid, dim3(256), 0, s,
                          static_cast<const __nv_bfloat16*>(x), src, x_rows, offsets, E, R, K, q,
                          sc, err);
}

cudaError_t launch_mx4_rows_back(int dtype, const uint8_t* q, const uint8_t* sc,
                                 const int32_t* offsets, int E, int R, int K, void* out,
                                 int num_sms, cudaStream_t s) {
  const dim3 grid(blocks_for(static_cast<long long>(R) * (K / 8), 256, num_sms * 8));
  return dtype == 0 ? launch_pdl(mx4_rows_back_kernel<float>, grid, dim3(256), 0, s, q, sc, offsets,
                                 E, R, K, static_cast<float*>(out))
                    : launch_pdl(mx4_rows_back_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, q, sc,
                                 offsets, E, R, K, static_cast<__nv_bfloat16*>(out));
}

cudaError_t launch_mx4_weights(int dtype, const void* W, int E, int K, int N, uint8_t* q,
                               uint8_t* sc, cudaStream_t s) {
  const dim3 grid(N / 64, up_div(K, dtype == 0 ? kWeightK<float> : kWeightK<__nv_bfloat16>), E);
  return dtype == 0 ? launch_pdl(mx4_weights_kernel<float>, grid, dim3(kWeightThreads<float>), 0, s,
                                 static_cast<const float*>(W), K, N, q, sc)
                    : launch_pdl(mx4_weights_kernel<__nv_bfloat16>, grid, dim3(kWeightThreads<__nv_bfloat16>), 0, s,
                                 static_cast<const __nv_bfloat16*>(W), K, N, q, sc);
}

cudaError_t launch_mx4_weights_back(int dtype, const uint8_t* q, const uint8_t* sc, int E, int K,
                                    int N, void* W, cudaStream_t s) {
  const dim3 grid(N / 64, up_div(K, dtype == 0 ? kWeightK<float> : kWeightK<__nv_bfloat16>), E);
  return dtype == 0 ? launch_pdl(mx4_weights_back_kernel<float>, grid, dim3(kWeightThreads<float>), 0, s, q, sc, K, N,
                                 static_cast<float*>(W))
                    : launch_pdl(mx4_weights_back_kernel<__nv_bfloat16>, grid, dim3(kWeightThreads<__nv_bfloat16>), 0, s, q, sc,
                                 K, N, static_cast<__nv_bfloat16*>(W));
}

cudaError_t launch_mx4_product(const uint8_t* aq, const uint8_t* as, const uint8_t* wq,
                               const uint8_t* wsc, const int32_t* offsets, int E, int R, int K,
                               int N, int out_f32, int silu, void* out, uint32_t* err,
                               uint32_t* ctr, float* part, int num_sms, cudaStream_t s) {
  CUtensorMap mA, mA32, mB, mSA, mSB;
  const uint64_t kc = up_div(K, 128);
  if (!make_map_2d_bytes(&mA, aq, R, K / 2, 128) || !make_map_2d_bytes(&mA32, aq, R, K / 2, 32) ||
      !make_map_2d_bytes(&mB, wq, static_cast<uint64_t>(E) * N, K / 2, 64) ||
      !make_map_3d_chunks(&mSA, as, row_tiles(R, E), kc, 1) ||
      !make_map_3d_chunks(&mSB, wsc, static_cast<uint64_t>(E) * up_div(N, 128), kc, 2))
    return cudaErrorInvalidValue;
  const mx::Params p{offsets, out, err, ctr, part, E, R, K, N, silu};
  const int grid = num_sms < kProductCtas ? num_sms : kProductCtas;
  const bool pair = R >= kMx4PairRows * E;
  if (pair)
    return out_f32 ? launch_product<true, float>(mA, mA32, mB, mSA, mSB, p, grid, s)
                   : launch_product<true, __nv_bfloat16>(mA, mA32, mB, mSA, mSB, p, grid, s);
  return out_f32 ? launch_product<false, float>(mA, mA32, mB, mSA, mSB, p, grid, s)
                 : launch_product<false, __nv_bfloat16>(mA, mA32, mB, mSA, mSB, p, grid, s);
}

}  // namespace moe
