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
#include "ptx.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int CHUNK = 512;  // bytes of scales of 128 rows x 128 values

__host__ __device__ constexpr int up_div(int a, int b) { return (a + b - 1) / b; }

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
__device__ __forceinline__ float code_value(uint32_t c) {
  // magnitudes 0, .5 and (1 + m / 2) 2^(e - 1)
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e == 0 ? 0.5f * m : __uint_as_float(((e + 126u) << 23) | (m << 22));
  return c & 8u ? -v : v;
}

// The segments' row tiles: seg[e] = offsets[e], base[e] = row tiles before
// expert e. Every thread of the block takes part; false (and the error
// flagged) when the offsets leave [0, R] or fall.
__device__ bool load_segments(const int32_t* __restrict__ offsets, int E, int R, int* seg,
                              int* base, int* ok, uint32_t* err) {
  const int tid = threadIdx.x;
  if (tid == 0) *ok = 1;
  for (int e = tid; e <= E; e += blockDim.x) seg[e] = __ldg(offsets + e);
  __syncthreads();
  for (int e = tid; e <= E; e += blockDim.x)
    if (seg[e] < 0 || seg[e] > R || (e > 0 && seg[e] < seg[e - 1])) *ok = 0;
  __syncthreads();
  if (tid < 32) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + tid;
      int n = *ok && e < E ? up_div(seg[e + 1] - seg[e], 128) : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= o) inc += v;
      }
      if (e < E) base[e] = run + inc - n;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (tid == 0) base[E] = run;
  }
  __syncthreads();
  if (!*ok && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && err != nullptr)
    atomicOr(err, kErrBadIndex);
  return *ok != 0;
}
// the last i of v[0..n] with v[i] <= x (v rising, v[0] <= x)
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
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
// A warp quantises 256 (bf16) or 128 (fp32) consecutive values of a row: a
// lane loads 16 bytes, a block's 4 (8) lanes agree on its amax, and a lane
// stores 4 (2) bytes of codes. Bound by HBM: the row is read once.
template <typename T>
__global__ void __launch_bounds__(256)
    mx4_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ src, int x_rows,
                    const int32_t* __restrict__ offsets, int E, int R, int K,
                    uint8_t* __restrict__ q, uint8_t* __restrict__ sc, uint32_t* err) {
  constexpr int V = 16 / sizeof(T), LPB = 32 / V, SPAN = 32 * V;
  __shared__ int seg[kMaxExperts + 1], base[kMaxExperts + 1], ok;
  pdl_wait();
  pdl_trigger();
  if (!load_segments(offsets, E, R, seg, base, &ok, err)) return;
  const int lane = threadIdx.x & 31;
  const int kc = up_div(K, 128), spans = up_div(K, SPAN);
  const long long total = static_cast<long long>(seg[E] - seg[0]) * spans;
  const long long step = static_cast<long long>(gridDim.x) * 8;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total;
       i += step) {
    const int r = seg[0] + static_cast<int>(i / spans), k = static_cast<int>(i % spans) * SPAN + lane * V;
    int xr = src != nullptr ? __ldg(src + r) : r;
    const bool in = xr >= 0 && xr < x_rows;
    if (!in && lane == 0) atomicOr(err, kErrBadIndex);
    uint4 raw = {0, 0, 0, 0};
    if (in && k < K)
      raw = __ldg(reinterpret_cast<const uint4*>(x + static_cast<size_t>(xr) * K + k));
    float v[8] = {};
    if constexpr (V == 4) {
      v[0] = __uint_as_float(raw.x);
      v[1] = __uint_as_float(raw.y);
      v[2] = __uint_as_float(raw.z);
      v[3] = __uint_as_float(raw.w);
    } else {
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
    // |v| orders as its bits do, infinities and NaN above every number
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LPB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t s = scale_code(m);
    const float inv = inv_scale(s);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= inv;
    const uint32_t codes = pack8(v);
    uint8_t* qr = q + static_cast<size_t>(r) * (K / 2) + k / 2;
    if (k < K) {
      if constexpr (V == 8)
        *reinterpret_cast<uint32_t*>(qr) = codes;
      else
        *reinterpret_cast<uint16_t*>(qr) = static_cast<uint16_t>(codes);
    }
    // the four blocks of a 128-value group, as one word from its first lane
    uint32_t word = s;
#pragma unroll
    for (int j = 1; j < 4; ++j)
      word |= __shfl_down_sync(0xffffffffu, s, j * LPB) << (8 * j);
    if (lane % (4 * LPB) == 0 && k < K)
      *reinterpret_cast<uint32_t*>(sc + row_scale_at(r, seg, base, E, kc) +
                                   static_cast<size_t>(k >> 7) * CHUNK) = word;
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
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = static_cast<T>(code_value((c >> (4 * j)) & 15u) * s);
  }
}

// ---------------------------------------------------------------- weights
// W [E][K][N] -> codes [E][N][K / 2]: a block takes 256 (fp32: 128) values of
// k x 64 of n through shared memory, so that both the rows of W and the runs
// of codes are read and written in whole sectors; a thread quantises one
// block of 32.
template <typename T>
constexpr int kWeightK = 512 / sizeof(T);
template <typename T>
constexpr int kWeightThreads = kWeightK<T> / 32 * 64;

template <typename T>
__global__ void __launch_bounds__(kWeightThreads<T>)
    mx4_weights_kernel(const T* __restrict__ W, int K, int N, uint8_t* __restrict__ q,
                       uint8_t* __restrict__ sc) {
  __shared__ __align__(16) T tile[kWeightK<T>][64];
  pdl_wait();
  pdl_trigger();
  const int n0 = blockIdx.x * 64, k0 = blockIdx.y * kWeightK<T>, e = blockIdx.z;
  const T* We = W + static_cast<size_t>(e) * K * N;
  constexpr int V = 16 / sizeof(T), PER = 64 / V;
  for (int i = threadIdx.x; i < kWeightK<T> * PER; i += kWeightThreads<T>) {
    const int k = i / PER, c = (i % PER) * V;
    if (k0 + k < K)
      *reinterpret_cast<uint4*>(&tile[k][c]) =
          __ldg(reinterpret_cast<const uint4*>(We + static_cast<size_t>(k0 + k) * N + n0 + c));
  }
  __syncthreads();
  const int n = threadIdx.x & 63, kb = threadIdx.x >> 6;
  if (k0 + kb * 32 >= K) return;
  float v[32];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = static_cast<float>(tile[kb * 32 + j][n]);
    m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  const uint32_t s = scale_code(m);
  const float inv = inv_scale(s);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[8 * j + i] * inv;
    w[j] = pack8(u);
  }
  const size_t row = static_cast<size_t>(e) * N + n0 + n;
  *reinterpret_cast<uint4*>(q + row * (K / 2) + (k0 + kb * 32) / 2) =
      make_uint4(w[0], w[1], w[2], w[3]);
  const int kc = up_div(K, 128), nt = up_div(N, 128), ni = n0 + n;
  sc[((static_cast<size_t>(e) * nt + (ni >> 7)) * kc + ((k0 + kb * 32) >> 7)) * CHUNK +
     (ni & 31) * 16 + ((ni & 127) >> 5) * 4 + (kb & 3)] = static_cast<uint8_t>(s);
}

template <typename T>
__global__ void __launch_bounds__(kWeightThreads<T>)
    mx4_weights_back_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc, int K,
                            int N, T* __restrict__ W) {
  __shared__ __align__(16) T tile[kWeightK<T>][64];
  pdl_wait();
  pdl_trigger();
  const int n0 = blockIdx.x * 64, k0 = blockIdx.y * kWeightK<T>, e = blockIdx.z;
  const int n = threadIdx.x & 63, kb = threadIdx.x >> 6;
  if (k0 + kb * 32 < K) {
    const size_t row = static_cast<size_t>(e) * N + n0 + n;
    const int kc = up_div(K, 128), nt = up_div(N, 128), ni = n0 + n;
    const float s = scale_value(__ldg(
        sc + ((static_cast<size_t>(e) * nt + (ni >> 7)) * kc + ((k0 + kb * 32) >> 7)) * CHUNK +
        (ni & 31) * 16 + ((ni & 127) >> 5) * 4 + (kb & 3)));
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(q + row * (K / 2) + (k0 + kb * 32) / 2));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 32; ++j)
      tile[kb * 32 + j][n] = static_cast<T>(code_value((w[j >> 3] >> (4 * (j & 7))) & 15u) * s);
  }
  __syncthreads();
  T* We = W + static_cast<size_t>(e) * K * N;
  constexpr int V = 16 / sizeof(T), PER = 64 / V;
  for (int i = threadIdx.x; i < kWeightK<T> * PER; i += kWeightThreads<T>) {
    const int k = i / PER, c0 = (i % PER) * V;
    if (k0 + k < K)
      *reinterpret_cast<uint4*>(We + static_cast<size_t>(k0 + k) * N + n0 + c0) =
          *reinterpret_cast<const uint4*>(&tile[k][c0]);
  }
}

// ---------------------------------------------------------------- product
// Tiles of 128 rows of one expert x up to 256 columns, one CTA each,
// persistent. A stage of the TMA ring holds 256 values of k: the rows' and
// the weights' codes (128-byte rows, 128-byte swizzle, both k-major) and
// their scale chunks. One thread copies a stage's scales to tensor memory
// (tcgen05.cp, the 512 bytes of a chunk to 4 columns of each of the four
// lane quarters) and issues the M128 N256 K64 products that read them; the
// scales have columns of their own per stage, so a stage's copy never meets
// a product still reading.
namespace mx {
constexpr int BM = 128, BN = 256, KS = 256;  // a stage's rows, columns, values of k
constexpr int A_BYTES = BM * 128, B_BOX = 64 * 128, B_BYTES = BN / 64 * B_BOX;
constexpr int SFA_BYTES = 2 * CHUNK, SFB_BYTES = 4 * CHUNK;
constexpr int OFF_B = A_BYTES, OFF_SFA = OFF_B + B_BYTES, OFF_SFB = OFF_SFA + SFA_BYTES;
constexpr int STAGE = OFF_SFB + SFB_BYTES;
constexpr int STAGES = 4;
constexpr int OFF_STG = STAGES * STAGE;  // 4 KB an epilogue warp
constexpr int OFF_BAR = OFF_STG + 4 * 4096;
constexpr int OFF_SEG = OFF_BAR + (2 * STAGES + 3) * 8 + 24;
constexpr int SMEM = OFF_SEG + 2 * (kMaxExperts + 1) * 4 + 1024;
constexpr int TMEM_COLS = 512, SF_COL = 256, SF_STAGE = 24;
constexpr int THREADS = 256;
static_assert(STAGE % 1024 == 0 && OFF_BAR % 8 == 0 && SMEM <= 227 * 1024, "shared memory");

struct Params {
  const uint8_t* as;
  const uint8_t* ws;
  const int32_t* offsets;
  void* out;
  uint32_t* err;
  uint32_t* ctr;  // arrivals per tile of a split launch, zero between launches
  float* part;    // [CTA][2][kMx4SplitRows][256]
  int E, R, K, N;
  int silu;
};

// kind::mxf4, E2M1 both sides, E8M0 scales, fp32 accumulator, both K-major,
// M = 128, K = 64; sf: which half of a scale column's four bytes
__device__ __forceinline__ uint32_t idesc_mxf4(int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (1u << 27) | (sf << 29);
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 32 rows of 16 bytes, contiguous, to 4 columns of all four lane quarters
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t saddr) {
  // no swizzle; 8-row groups 128 bytes apart; descriptor version 1
  const uint64_t desc = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
                        (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void bar_epi() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

struct Tile {
  int e, row0, rows, mt, n0, n;
};
// Tile t: expert by expert, column blocks outside, row tiles inside, so that
// the CTAs at work side by side share a column block's weights.
__device__ __forceinline__ Tile tile_at(int t, const int* seg, const int* base, int E, int N) {
  const int nt = up_div(N, BN);
  Tile r;
  r.e = last_at_most(base, E - 1, t / nt);
  const int l = t - base[r.e] * nt, m = base[r.e + 1] - base[r.e];
  const int nb = l / m, mt = l - nb * m;
  r.mt = base[r.e] + mt;
  r.row0 = seg[r.e] + mt * BM;
  r.rows = min(BM, seg[r.e + 1] - r.row0);
  r.n0 = nb * BN;
  r.n = min(BN, N - r.n0);
  return r;
}
}  // namespace mx

__device__ __forceinline__ float mx_silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// TO: the output type
template <typename TO>
__global__ void __launch_bounds__(mx::THREADS, 1)
    mx4_product_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const mx::Params p) {
  using namespace mx;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* s_ok = reinterpret_cast<int*>(tmem_slot + 1);
  uint32_t* s_last = tmem_slot + 2;
  int* s_wide = reinterpret_cast<int*>(tmem_slot + 3);
  int* seg = reinterpret_cast<int*>(smem + OFF_SEG);
  int* base = seg + kMaxExperts + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int E = p.E, K = p.K, N = p.N;

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 4);
    mbar_init(drain, 1);
    *s_wide = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const bool ok = load_segments(p.offsets, E, p.R, seg, base, s_ok, p.err);
  for (int e = tid; ok && e < E; e += THREADS)
    if (seg[e + 1] - seg[e] > kMx4SplitRows) *s_wide = 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int kst = up_div(K, KS), kc = up_div(K, 128);
  const int tiles = ok ? base[E] * up_div(N, BN) : 0;
  // Few rows everywhere and fewer tiles than CTAs: the tiles' stages are one
  // sequence cut into equal ranges, and a tile's partial sums are joined by
  // the last CTA to arrive, in CTA order. Otherwise whole tiles in turn.
  const bool split = tiles < grid && *s_wide == 0;
  const int total = split ? tiles * kst : 0, G = min(grid, total);
  auto start = [&](int c) {
    return c >= G ? total : static_cast<int>(static_cast<long long>(total) * c / G);
  };
  // Walk this CTA's pieces: f(tile, first stage, end stage)
  auto walk = [&](auto f) {
    if (split) {
      const int end = start(cta + 1);
      for (int i = start(cta); i < end;) {
        const int t = i / kst, k0 = i - t * kst, k1 = min(kst, k0 + end - i);
        if (!f(t, k0, k1)) return;
        i += k1 - k0;
      }
    } else {
      for (int t = cta; t < tiles; t += grid)
        if (!f(t, 0, kst)) return;
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      int s = 0, used = 0;
      uint32_t ph = 0;
      bool dead = false;
      walk([&](int t, int k0, int k1) {
        const Tile tl = tile_at(t, seg, base, E, N);
        const int nb = tl.n / 64, nj = up_div(tl.n, 128), nt = up_div(N, 128);
        const uint8_t* as = p.as + static_cast<size_t>(tl.mt) * kc * CHUNK;
        const uint8_t* ws = p.ws + (static_cast<size_t>(tl.e) * nt + tl.n0 / 128) * kc * CHUNK;
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1u, kWaitLimitNs)) {
            dead = true;
            return false;
          }
          if (used < STAGES) ++used;
          uint8_t* st = smem + s * STAGE;
          const uint32_t sf = static_cast<uint32_t>(min(2, kc - 2 * kb)) * CHUNK;
          mbar_arrive_expect_tx(&full[s], A_BYTES + nb * B_BOX + (1 + nj) * sf);
          tma_load_2d(st, &tmA, &full[s], kb * 128, tl.row0);
          for (int b = 0; b < nb; ++b)
            tma_load_2d(st + OFF_B + b * B_BOX, &tmB, &full[s], kb * 128,
                        tl.e * N + tl.n0 + b * 64);
          bulk_load(st + OFF_SFA, as + static_cast<size_t>(kb) * 2 * CHUNK, sf, &full[s]);
          for (int j = 0; j < nj; ++j)
            bulk_load(st + OFF_SFB + j * 2 * CHUNK,
                      ws + (static_cast<size_t>(j) * kc + kb * 2) * CHUNK, sf, &full[s]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        return true;
      });
      // the latest use of each stage has landed before this CTA may exit
      for (int j = 0; j < used; ++j) {
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
      if (dead) atomicOr(p.err, kErrTimeout);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, aph = 0;
      bool dead = false;
      walk([&](int t, int k0, int k1) {
        const Tile tl = tile_at(t, seg, base, E, N);
        const int nj = up_div(tl.n, 128);
        if (!mbar_wait(tempty, aph ^ 1u, kWaitLimitNs)) {
          dead = true;
          return false;
        }
        tc_fence_after();
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait_spin(&full[s], ph, kWaitLimitNs)) {
            dead = true;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + s * STAGE), b = a + OFF_B;
          const uint32_t sf = tmem_base + SF_COL + s * SF_STAGE;
          const int chunks = min(2, kc - 2 * kb), steps = min(4, (K - kb * KS) / 64);
          for (int c = 0; c < chunks; ++c) {
            cp_scales(sf + c * 4, a + OFF_SFA + c * CHUNK);
            for (int j = 0; j < nj; ++j)
              cp_scales(sf + 8 + c * 8 + j * 4, a + OFF_SFB + (2 * j + c) * CHUNK);
          }
          for (int kk = 0; kk < steps; ++kk)
            mma_mxf4(tmem_base, make_sdesc_sw128(a + kk * 32, 16, 1024),
                     make_sdesc_sw128(b + kk * 32, 16, 1024), idesc_mxf4(tl.n, (kk & 1) * 2),
                     sf + (kk >> 1) * 4, sf + 8 + (kk >> 1) * 8, (kb > k0 || kk > 0) ? 1u : 0u);
          tc_commit(&empty[s]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        tc_commit(tfull);
        aph ^= 1u;
        return !dead;
      });
      tc_commit(drain);
      if (!mbar_wait(drain, 0, kWaitLimitNs) || dead) atomicOr(p.err, kErrTimeout);
    }
  } else if (warp >= 4) {
    const int w = warp & 3;
    uint8_t* stg = smem + OFF_STG + w * 4096;
    uint32_t aph = 0;
    bool dead = false;
    TO* out = static_cast<TO*>(p.out);
    auto put = [&](size_t row, int col, float4 v) {
      if (p.silu) v = make_float4(mx_silu(v.x), mx_silu(v.y), mx_silu(v.z), mx_silu(v.w));
      TO* o = out + row * N + col;
      if constexpr (sizeof(TO) == 4) {
        *reinterpret_cast<float4*>(o) = v;
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                  *reinterpret_cast<const uint32_t*>(&hi));
      }
    };
    walk([&](int t, int k0, int k1) {
      const Tile tl = tile_at(t, seg, base, E, N);
      const bool whole = k0 == 0 && k1 == kst;
      const int a = t * kst;
      auto slice = [&](int c) {
        return p.part + (static_cast<size_t>(c) * 2 + (start(c) > a ? 0 : 1)) * kMx4SplitRows * BN;
      };
      // after a wait that ran out the loops go on, so that the four warps
      // still meet at every barrier
      if (!dead && !mbar_wait(tfull, aph, kWaitLimitNs)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      aph ^= 1u;
      tc_fence_after();
      for (int c0 = 0; c0 < tl.n; c0 += 32) {
        if (w * 32 < tl.rows) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(w * 32) << 16) + c0, r);
          tmem_ld_wait();
          // 32 x 32 through shared memory, 16-byte pieces swizzled by row
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = j * 4 + (lane >> 3), c4 = lane & 7;
            const float4 v =
                *reinterpret_cast<const float4*>(stg + row * 128 + ((c4 ^ (row & 7)) * 16));
            if (w * 32 + row < tl.rows) {
              if (whole)
                put(tl.row0 + w * 32 + row, tl.n0 + c0 + c4 * 4, v);
              else  // (at most kMx4SplitRows rows: warp 0's)
                __stcg(reinterpret_cast<float4*>(slice(cta) + row * BN + c0 + c4 * 4), v);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);
      if (!whole) {
        const int c0 = static_cast<int>((static_cast<long long>(a + 1) * G - 1) / total);
        const int c1 = static_cast<int>((static_cast<long long>(a + kst) * G - 1) / total);
        __threadfence();
        bar_epi();
        if (tid == 128) {
          const bool last = atomicAdd(p.ctr + t, 1u) == static_cast<uint32_t>(c1 - c0);
          if (last) p.ctr[t] = 0;
          *s_last = last ? 1u : 0u;
        }
        bar_epi();
        if (*s_last != 0) {
          __threadfence();
          const int quads = tl.n / 4;
          for (int i = tid - 128; i < tl.rows * quads; i += 128) {
            const int row = i / quads, col = (i - row * quads) * 4;
            float4 v = {0.f, 0.f, 0.f, 0.f};
            for (int c = c0; c <= c1; ++c) {
              const float4 o = __ldcg(reinterpret_cast<const float4*>(slice(c) + row * BN + col));
              v.x += o.x;
              v.y += o.y;
              v.z += o.z;
              v.w += o.w;
            }
            put(tl.row0 + row, tl.n0 + col, v);
          }
        }
      }
      return true;
    });
    if (dead && lane == 0) atomicOr(p.err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

int blocks_for(long long items, int per_block, int most) {
  const long long b = (items + per_block - 1) / per_block;
  return static_cast<int>(b < 1 ? 1 : (b < most ? b : most));
}

}  // namespace

size_t mx4_row_tiles(int R, int E) { return static_cast<size_t>(R / 128) + (R < E ? R : E); }

cudaError_t launch_mx4_rows(int dtype, const void* x, const int32_t* src, int x_rows,
                            const int32_t* offsets, int E, int R, int K, uint8_t* q, uint8_t* sc,
                            uint32_t* err, int num_sms, cudaStream_t s) {
  const int span = dtype == 0 ? 128 : 256;
  const dim3 grid(blocks_for(static_cast<long long>(R) * up_div(K, span), 8, num_sms * 8));
  return dtype == 0 ? launch_pdl(mx4_rows_kernel<float>, grid, dim3(256), 0, s,
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
  using namespace mx;
  CUtensorMap mA, mB;
  if (!make_map_2d_bytes(&mA, aq, R, K / 2, 128) ||
      !make_map_2d_bytes(&mB, wq, static_cast<uint64_t>(E) * N, K / 2, 64))
    return cudaErrorInvalidValue;
  const Params p{as, wsc, offsets, out, err, ctr, part, E, R, K, N, silu};
  const int grid = num_sms < kMx4MaxCtas ? num_sms : kMx4MaxCtas;
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(THREADS), SMEM, s, mA, mB, p);
  };
  return out_f32 ? go(mx4_product_kernel<float>) : go(mx4_product_kernel<__nv_bfloat16>);
}

}  // namespace moe
