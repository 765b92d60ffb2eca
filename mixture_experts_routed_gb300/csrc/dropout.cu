// dropout.cu - dropout of a block's branch before the residual sum, its mask
// drawn by element from a counter-based generator and never stored.
//
//   out = residual + keep x / (1 - p')      dx = keep dout / (1 - p')
//
// Element i takes 16 bits of Philox 4x32 with ten rounds (J. Salmon, M.
// Moraes, R. Dror, D. Shaw, Parallel random numbers: as easy as 1, 2, 3, SC
// 2011): counter (i / 8 low, i / 8 high, site, step), key the 64-bit seed,
// word (i % 8) / 2 of the four, the low half for an even i. It is kept where
// those bits are at least thr = round(65536 p), so p' = thr / 65536 exactly.
#include <cstdint>

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {
namespace {

// ten rounds; the key grows by fixed steps
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint32_t h0 = __umulhi(c.x, 0xD2511F53u), l0 = c.x * 0xD2511F53u;
    const uint32_t h1 = __umulhi(c.z, 0xCD9E8D57u), l1 = c.z * 0xCD9E8D57u;
    c = make_uint4(h1 ^ c.y ^ k0, l1, h0 ^ c.w ^ k1, l0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// 16 bytes that are read once and may be written by this call (in place)
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// A thread takes kGroups groups of 8 elements, 256 groups apart; their loads
// are under way while the draws are computed. A product and a select for
// each element, the sum in one rounding with the product (fma).
// Bound by HBM: 16384 x 5120 bf16 with a residual 72.5 us, 6.9 TB/s, without
// 50.5, 6.6 TB/s (16 bits an element: a generator call for 8 of them, some 70
// instructions, a third of what the SMs issue meanwhile).
constexpr int kThreads = 256, kGroups = 2;

template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(const T* x, const T* residual, const int64_t* __restrict__ state, uint32_t site,
                   uint32_t thr, float scale, long long groups, T* out) {
  constexpr int PIECES = 8 * sizeof(T) / 16;
  pdl_wait();
  pdl_trigger();
  const uint64_t seed = static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(state)));
  const uint32_t step =
      static_cast<uint32_t>(__ldg(reinterpret_cast<const long long*>(state) + 1));
  const long long g0 = static_cast<long long>(blockIdx.x) * (kThreads * kGroups) + threadIdx.x;
  uint4 xv[kGroups][PIECES], rv[kGroups][RES ? PIECES : 1];
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    const long long g = g0 + j * kThreads;
    if (g >= groups) continue;
#pragma unroll
    for (int h = 0; h < PIECES; ++h) {
      xv[j][h] = ld_stream(x + g * 8 + h * (8 / PIECES));
      if constexpr (RES) rv[j][h] = ld_stream(residual + g * 8 + h * (8 / PIECES));
    }
  }
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    const long long g = g0 + j * kThreads;
    if (g >= groups) continue;
    const uint4 d = philox(make_uint4(static_cast<uint32_t>(g), static_cast<uint32_t>(g >> 32),
                                      site, step),
                           static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
    const uint32_t draw[4] = {d.x, d.y, d.z, d.w};
    // (a dropped infinity or NaN is 0: selected, not multiplied)
    auto one = [&](int i, float v, float r) {
      const uint32_t u = i & 1 ? draw[i / 2] >> 16 : draw[i / 2] & 0xffffu;
      const bool keep = u >= thr;
      if constexpr (RES) return keep ? fmaf(v, scale, r) : r;
      return keep ? v * scale : 0.f;
    };
#pragma unroll
    for (int h = 0; h < PIECES; ++h) {
      const uint32_t a[4] = {xv[j][h].x, xv[j][h].y, xv[j][h].z, xv[j][h].w};
      uint32_t b[4] = {}, o[4];
      if constexpr (RES) {
        b[0] = rv[j][h].x;
        b[1] = rv[j][h].y;
        b[2] = rv[j][h].z;
        b[3] = rv[j][h].w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          o[i] = __float_as_uint(one(h * 4 + i, __uint_as_float(a[i]), __uint_as_float(b[i])));
        } else {
          const __nv_bfloat162 p = __floats2bfloat162_rn(
              one(2 * i, __uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16)),
              one(2 * i + 1, __uint_as_float(a[i] & 0xffff0000u),
                  __uint_as_float(b[i] & 0xffff0000u)));
          o[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      *reinterpret_cast<uint4*>(out + g * 8 + h * (8 / PIECES)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <typename T>
cudaError_t launch(const void* x, const void* residual, const int64_t* state, uint32_t site,
                   uint32_t thr, float scale, long long groups, void* out, cudaStream_t s) {
  const long long blocks = (groups + kThreads * kGroups - 1) / (kThreads * kGroups);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  return residual != nullptr
             ? launch_pdl(dropout_kernel<T, true>, grid, block, 0, s, static_cast<const T*>(x),
                          static_cast<const T*>(residual), state, site, thr, scale, groups,
                          static_cast<T*>(out))
             : launch_pdl(dropout_kernel<T, false>, grid, block, 0, s, static_cast<const T*>(x),
                          static_cast<const T*>(nullptr), state, site, thr, scale, groups,
                          static_cast<T*>(out));
}

}  // namespace

cudaError_t launch_dropout(int dtype, const void* x, const void* residual, const int64_t* state,
                           uint32_t site, uint32_t thr, long long n, void* out, cudaStream_t s) {
  const float scale = 65536.f / static_cast<float>(65536u - thr);
  return dtype == 0 ? launch<float>(x, residual, state, site, thr, scale, n / 8, out, s)
                    : launch<__nv_bfloat16>(x, residual, state, site, thr, scale, n / 8, out, s);
}

}  // namespace moe
