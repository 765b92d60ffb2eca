// grouped.cuh - what the expert-grouped products in 4 and 8 bits share: the
// segments' row tiles, a product's tiles over them, SiLU and the way a tile's
// rows leave the registers.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {
namespace {

__host__ __device__ constexpr int up_div(int a, int b) { return (a + b - 1) / b; }

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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
constexpr int kTileCols = 256;  // a product tile's columns

struct Tile {
  int e, row0, rows, mt, n0, n;
};
// Tile t: expert by expert, column blocks outside, row tiles inside, so that
// the CTAs at work side by side share a column block's weights. tb: tiles of
// BM rows before each expert; base: tiles of 128 rows (scale chunks).
template <int BM>
__device__ __forceinline__ Tile tile_at(int t, const int* seg, const int* base, const int* tb,
                                        int E, int N) {
  const int nt = up_div(N, kTileCols);
  Tile r;
  r.e = last_at_most(tb, E - 1, t / nt);
  const int l = t - tb[r.e] * nt, m = tb[r.e + 1] - tb[r.e];
  const int nb = l / m, mt = l - nb * m;
  r.mt = base[r.e] + mt * (BM / 128);
  r.row0 = seg[r.e] + mt * BM;
  r.rows = min(BM, seg[r.e + 1] - r.row0);
  r.n0 = nb * kTileCols;
  r.n = min(kTileCols, N - r.n0);
  return r;
}

// 32 bytes: one store where they are 32-byte aligned, else two of 16
__device__ __forceinline__ void st_sector(bool whole, void* p, const uint32_t (&v)[8]) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
// SiLU of an fp32 sum. Where fp32 is stored: with t = exp(-|z|) (2 units of the
// last place), z / (1 + t), or z t / (1 + t) below 0, so that nothing overflows;
// the denominator is in [1, 2], its approximate reciprocal y needs no special
// cases, and one correction of q = n y by its residual (P. Markstein, IBM J.
// Res. Dev. 34(1), 1990) leaves the quotient's own rounding: 7 half steps in
// all (2047 rows of 64 experts of 2048 x 1408 30.3 us, with a plain division 53.5).
// Where bf16 is stored: approximate exponential and quotient, whose error (some
// 60 half steps of fp32) is a thousandth of the rounding that follows; below
// z = -87.3 they give 0 for at most 1.1e-36.
template <typename TO>
__device__ __forceinline__ float silu_of(float z) {
  if constexpr (sizeof(TO) == 4) {
    const float t = expf(-fabsf(z)), d = 1.f + t, n = z < 0.f ? z * t : z;
    const float y = __fdividef(1.f, d), q = n * y;
    return isinf(q) ? q : fmaf(fmaf(-q, d, n), y, q);
  }
  return __fdividef(z, 1.f + __expf(-z));
}

// 32 columns of up to 32 rows, a row to a lane, through `finish` to out [..][N]:
// neighbouring lanes exchange 32-byte pieces first, so that a store
// instruction writes contiguous runs of 128 bytes (fp32; bf16: 64), not a
// sector of each row. store(address, piece) writes one.
template <typename TO, typename F, typename S>
__device__ __forceinline__ void put_rows32_by(TO* out, size_t row0, int rows, int N, int col,
                                              const uint32_t (&r)[32], F finish, S store) {
  constexpr int PER = 32 / sizeof(TO), NC = 32 / PER;  // a piece's columns, a row's pieces
  const int lane = threadIdx.x & 31;
  uint32_t v[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(TO) == 4) {
        v[c][i] = __float_as_uint(finish(__uint_as_float(r[c * PER + i])));
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(finish(__uint_as_float(r[c * PER + 2 * i])),
                                                       finish(__uint_as_float(r[c * PER + 2 * i + 1])));
        v[c][i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  // a transposition within groups of NC lanes: v[i] is then piece `lane % NC`
  // of the group's row i
#pragma unroll
  for (int m = 1; m < NC; m <<= 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (c & m) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool up = lane & m;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[c][i] : v[c | m][i], m);
        v[c][i] = up ? got : v[c][i];
        v[c | m][i] = up ? v[c | m][i] : got;
      }
    }
  }
  const int g = lane & ~(NC - 1);
  TO* o = out + (row0 + g) * N + col + (lane - g) * PER;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (g + i < rows) store(o + static_cast<size_t>(i) * N, v[i]);
}
// sectors: out is 32-byte aligned (rows are multiples of 128 bytes)
template <typename TO, typename F>
__device__ __forceinline__ void put_rows32(TO* out, bool sectors, size_t row0, int rows, int N,
                                           int col, const uint32_t (&r)[32], F finish) {
  put_rows32_by(out, row0, rows, N, col, r, finish,
                [&](TO* p, const uint32_t (&v)[8]) { st_sector(sectors, p, v); });
}

}  // namespace
}  // namespace moe
