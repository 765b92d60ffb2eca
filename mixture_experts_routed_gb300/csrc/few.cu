// few.cu - the whole routed layer for a few tokens (T <= 32: a decode step)
// in one kernel: gate and router (DeepSeek-V4 EP article, sections 2.1 and
// 3.2), W1, SiLU, W2 of the chosen experts and the weighted sum.
//
//   L = x W_g + b        top-k and weights as moe_route
//   h[t, e] = SiLU(x[t] W1[e])          (t routed to e)
//   out[t] = sum over the chosen e of w[t, e] (h[t, e] W2[e])
//
// Bound: each chosen expert's weights cross HBM once (4 d f bytes); the
// products are thin. So the grid is one CTA per SM and every CTA streams an
// equal, contiguous share of the weight tiles through a deep TMA ring, from
// the first W1 tile to the last W2 tile without draining.
//
// Products: the weights are the M operand of tcgen05.mma, 128 output
// features x 64 contraction rows a tile, read MN-major straight from their
// row-major storage; the tokens are the N operand. Every token multiplies
// every chosen expert (N = 16..64 costs the tensor core nothing here) and
// the epilogue keeps the routed ones, so nothing is permuted or packed. For
// W2 the tokens' h rows are carried as bf16 hi + lo, side by side in N
// (h to 2^-17 relative, so out is rounded once).
//
// Work split: the tiles of a phase, k innermost, are one sequence of steps
// (64 contraction rows x 128 features), cut into equal ranges, one per CTA.
// A feature block whose steps fall to several CTAs is joined from their fp32
// partial sums by the last of them to arrive, in CTA order: no atomics on
// values, so the result is bitwise reproducible on one GPU model. In phase 1
// a block is one expert's 128 features of h; in phase 2 it is 128 features
// of out with every expert's steps one after the other, the routing weights
// applied as each expert's accumulator is read.
//
// The CTAs wait on one another (gate sums -> router -> h), so the launch is
// cooperative: all of them are resident. While a CTA waits for h its ring
// already holds its first W2 tiles. Every wait is bounded: a wait on other
// CTAs that runs out sets kErrTimeout and goes on (with what is in memory:
// in bounds, wrong values); one on this CTA's own copies or products sets it
// and ends the role.
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "tmap.cuh"
#include "topk.cuh"

namespace moe {
namespace {

using namespace ptx;

namespace fw {
constexpr int THREADS = 256;
constexpr int BM = 128, BK = 64;            // features, contraction rows of a step
constexpr int BOX_BYTES = BK * 64 * 2;      // [64 k][64 features] bf16
constexpr int A_BYTES = 2 * BOX_BYTES;
constexpr int GATE_E = 64;                  // experts of a gate CTA
constexpr int GATE_ROWS = 64;               // x rows staged at a time
constexpr int MAX_CHUNKS = 64;              // partial sums of a logit
constexpr int TMEM_COLS = 128;              // two accumulators of 64 columns
constexpr int MAX_ROWS = kFewMaxTokens * kMaxFanout;

template <int TP>
struct Cfg {
  static constexpr int N1 = TP < 16 ? 16 : TP;  // x rows of phase 1's products
  static constexpr int N2 = 2 * TP;             // h rows (hi, lo) of phase 2's
  static constexpr int B_BYTES = (N1 > N2 ? N1 : N2) * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 200 * 1024 / STAGE;
  static constexpr int OFF_BAR = STAGES * STAGE;
  static constexpr int OFF_TAB = OFF_BAR + (2 * STAGES + 5) * 8;
  static constexpr int SMEM = OFF_TAB + 256 * 4 + 256 * 2 + MAX_ROWS * 2 + MAX_ROWS * 4 + 64 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(GATE_ROWS * TP * 4 + 4 * TP * GATE_E * 4 + kMaxExperts * 4 <= OFF_BAR, "scratch");
};

struct Params {
  const __nv_bfloat16* x;
  const __nv_bfloat16* Wg;
  const float* bias;
  RouterSpec rs;
  int T, d, E, f, k;
  int gate_groups, gate_chunks, gate_len;  // expert groups x chunks of gate_len rows
  int32_t* idx;
  float* w;
  float* gpart;      // [chunks][T][E]
  uint32_t* tiles;   // arrivals: [slots][f blocks], then [d blocks]
  int ntiles;
  __nv_bfloat16* h;  // [slots][2 TP][f]
  float* part;       // [phase][CTA][2][TP][128]
  __nv_bfloat16* out;
  uint32_t* err;
  uint32_t* sync;    // four counters, 8 words apart, zero between launches
};
constexpr int SYNC_GATE = 0, SYNC_ROUTE = 8, SYNC_H = 16, SYNC_EXIT = 24;

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t o;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;"
               : "=r"(o)
               : "l"(p), "r"(v)
               : "memory");
  return o;
}
__device__ __forceinline__ bool wait_count(const uint32_t* p, uint32_t target, uint64_t limit_ns) {
  if (ld_acquire(p) >= target) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (ld_acquire(p) >= target) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ void bar_epi() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// The steps of one phase (`units` accumulators of `len` steps) and each
// CTA's range of them.
struct Range {
  int len;
  long long total;
  int G;
  __device__ Range(int units, int len_, int grid) : len(len_) {
    total = static_cast<long long>(units) * len;
    G = total < grid ? static_cast<int>(total) : grid;  // every range holds a step
  }
  __device__ long long start(int c) const { return c >= G ? total : total * c / G; }
  // the CTA whose range holds step i
  __device__ int owner(long long i) const { return static_cast<int>(((i + 1) * G - 1) / total); }
};
}  // namespace fw

template <int TP>
__global__ void __launch_bounds__(fw::THREADS, 1)
    few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW1,
               const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmH,
               const fw::Params p) {
  using namespace fw;
  using C = Cfg<TP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* smask = reinterpret_cast<uint32_t*>(smem + C::OFF_TAB);  // slot -> its tokens
  float* rw = reinterpret_cast<float*>(smask + kMaxExperts);         // [T][k] weights
  int16_t* ridx = reinterpret_cast<int16_t*>(rw + MAX_ROWS);         // [T][k] experts, -1: none
  int16_t* sexp = ridx + MAX_ROWS;                                   // slot -> expert
  uint32_t* misc = reinterpret_cast<uint32_t*>(sexp + kMaxExperts);
  uint32_t* tmem_slot = misc;
  int* s_nslots = reinterpret_cast<int*>(misc + 1);
  uint32_t* s_last = misc + 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int T = p.T, d = p.d, E = p.E, f = p.f, k = p.k;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }

  // ---------------------------------------------------------------- gate sums
  for (int i = cta * THREADS + tid; i < p.ntiles; i += grid * THREADS) p.tiles[i] = 0;
  {
    float* xs = reinterpret_cast<float*>(smem);  // [GATE_ROWS][TP]
    float* red = xs + GATE_ROWS * TP;            // [4][TP][GATE_E]
    const int chunk = cta / p.gate_groups, e0 = (cta % p.gate_groups) * GATE_E;
    if (chunk < p.gate_chunks) {
      const int r0 = chunk * p.gate_len, r1 = min(d, r0 + p.gate_len);
      const int e = e0 + (tid & 63), rg = tid >> 6;
      float acc[TP];
#pragma unroll
      for (int t = 0; t < TP; ++t) acc[t] = 0.f;
      for (int rb = r0; rb < r1; rb += GATE_ROWS) {
        const int n = min(GATE_ROWS, r1 - rb);
        __syncthreads();
        for (int i = tid; i < GATE_ROWS * TP; i += THREADS) {
          const int t = i / GATE_ROWS, r = i % GATE_ROWS;
          xs[r * TP + t] =
              t < T && r < n ? __bfloat162float(p.x[static_cast<size_t>(t) * d + rb + r]) : 0.f;
        }
        // this thread's weights: rows rg, rg + 4, ...
        float wv[GATE_ROWS / 4];
#pragma unroll
        for (int j = 0; j < GATE_ROWS / 4; ++j) {
          const int r = rg + 4 * j;
          wv[j] = e < E && r < n
                      ? __bfloat162float(p.Wg[static_cast<size_t>(rb + r) * E + e])
                      : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < GATE_ROWS / 4; ++j) {
          const float4* xr = reinterpret_cast<const float4*>(xs + (rg + 4 * j) * TP);
#pragma unroll
          for (int t = 0; t < TP; t += 4) {
            const float4 v = xr[t / 4];
            acc[t] = fmaf(v.x, wv[j], acc[t]);
            acc[t + 1] = fmaf(v.y, wv[j], acc[t + 1]);
            acc[t + 2] = fmaf(v.z, wv[j], acc[t + 2]);
            acc[t + 3] = fmaf(v.w, wv[j], acc[t + 3]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TP; ++t) red[(rg * TP + t) * GATE_E + (tid & 63)] = acc[t];
      __syncthreads();
      for (int i = tid; i < T * GATE_E; i += THREADS) {
        const int t = i / GATE_E, c = i % GATE_E;
        if (e0 + c < E) {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < 4; ++g) s += red[(g * TP + t) * GATE_E + c];
          p.gpart[(static_cast<size_t>(chunk) * T + t) * E + e0 + c] = s;
        }
      }
    }
  }
  __threadfence();
  __syncthreads();
  bool lost = false;  // thread 0: a wait on other CTAs ran out
  if (tid == 0) add_acq_rel(p.sync + SYNC_GATE, 1);

  // ---------------------------------------------------------------- router
  for (int t = cta; t < T; t += grid) {
    float* logits = reinterpret_cast<float*>(smem);  // [kMaxExperts]
    if (tid == 0 && !lost) lost = !wait_count(p.sync + SYNC_GATE, grid, kWaitLimitNs);
    __syncthreads();
    if (tid < E) {
      // the chunks' sums, compensated
      float s = p.bias != nullptr ? __ldg(p.bias + tid) : 0.f, comp = 0.f;
      const float* g = p.gpart + static_cast<size_t>(t) * E + tid;
#pragma unroll 16
      for (int c = 0; c < p.gate_chunks; ++c) {
        const float yv = __fsub_rn(__ldcg(g + static_cast<size_t>(c) * T * E), comp);
        const float sum = __fadd_rn(s, yv);
        comp = __fsub_rn(__fsub_rn(sum, s), yv);
        s = sum;
      }
      logits[tid] = s;
    }
    __syncthreads();
    if (warp == 0) {
      float v[8];
      int id[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        id[j] = lane + 32 * j;
        v[j] = id[j] < E ? logits[id[j]] : -INFINITY;
      }
      if (p.rs.mode == topk::kRouterSoft) {
        topk::warp_soft_weigh<8>(v, id, E, p.rs, t, p.idx, p.w);
      } else {
        if (p.rs.mode == topk::kRouterGroup) topk::warp_group_limit<8>(v, id, E, p.rs);
        topk::warp_select_and_weigh<8>(v, id, p.rs, t, p.idx, p.w);
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) add_acq_rel(p.sync + SYNC_ROUTE, 1);
    }
    __syncthreads();
  }
  if (tid == 0 && !lost) lost = !wait_count(p.sync + SYNC_ROUTE, T, kWaitLimitNs);
  for (int e = tid; e < kMaxExperts; e += THREADS) smask[e] = 0;
  __syncthreads();

  // ---------------------------------------------------------------- slots
  // the chosen experts in id order, and each one's tokens as a bit mask
  for (int i = tid; i < T * k; i += THREADS) {
    const int e = __ldcg(p.idx + i);
    const bool ok = e >= 0 && e < E;
    ridx[i] = static_cast<int16_t>(ok ? e : -1);
    rw[i] = ok ? __ldcg(p.w + i) : 0.f;
    if (ok)
      atomicOr(&smask[e], 1u << (i / k));
    else
      atomicOr(p.err, kErrBadIndex);
  }
  __syncthreads();
  if (warp == 0) {
    // in place: slot <= expert, and a round's masks are read before it writes
    int n = 0;
    for (int j = 0; j < kMaxExperts / 32; ++j) {
      const uint32_t m = smask[j * 32 + lane];
      const uint32_t have = __ballot_sync(0xffffffffu, m != 0);
      const int at = n + __popc(have & ((1u << lane) - 1));
      __syncwarp();
      if (m != 0) {
        smask[at] = m;
        sexp[at] = static_cast<int16_t>(j * 32 + lane);
      }
      n += __popc(have);
      __syncwarp();
    }
    if (lane == 0) *s_nslots = n;
  }
  // the ring's memory held the gate's scratch: order that before the copies
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int nslots = *s_nslots;
  const int FB = (f + BM - 1) / BM, DB = (d + BM - 1) / BM;
  const Range r1(nslots * FB, d / BK, grid), r2(DB * nslots, f / BK, grid);

  if (nslots == 0) {
    for (size_t i = static_cast<size_t>(cta) * THREADS + tid; i < static_cast<size_t>(T) * d;
         i += static_cast<size_t>(grid) * THREADS)
      p.out[i] = __float2bfloat16(0.f);
  } else if (warp == 0) {
    // -------------------------------------------------------------- TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmX);
      prefetch_tmap(&tmW1);
      prefetch_tmap(&tmW2);
      prefetch_tmap(&tmH);
      int s = 0;
      uint32_t ph = 0;
      int used = 0;  // stages filled at least once
      bool dead = false;
      // the weight boxes of a step: expert e's rows [k0, k0 + 64), features [c0, c0 + 128)
      auto load_a = [&](const CUtensorMap* m, int row, int c0, int cols, uint32_t b_bytes) {
        const int nb = min(2, (cols - c0) / 64);
        mbar_arrive_expect_tx(&full[s], nb * BOX_BYTES + b_bytes);
        uint8_t* st = smem + s * C::STAGE;
        for (int b = 0; b < nb; ++b) tma_load_2d(st + b * BOX_BYTES, m, &full[s], c0 + b * 64, row);
      };
      auto next = [&]() {
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1u;
        }
      };
      auto claim = [&]() {
        if (!mbar_wait(&empty[s], ph ^ 1u, kWaitLimitNs)) {
          dead = true;
          return false;
        }
        if (used < C::STAGES) ++used;
        return true;
      };
      {
        const long long end = r1.start(cta + 1);
        for (long long i = r1.start(cta); i < end && !dead;) {
          const int u = static_cast<int>(i / r1.len), k0 = static_cast<int>(i - static_cast<long long>(u) * r1.len);
          const int n = static_cast<int>(min(static_cast<long long>(r1.len - k0), end - i));
          const int slot = u / FB, c0 = (u - slot * FB) * BM, row = sexp[slot] * d;
          for (int j = k0; j < k0 + n; ++j) {
            if (!claim()) break;
            load_a(&tmW1, row + j * BK, c0, f, C::N1 * 128);
            tma_load_2d(smem + s * C::STAGE + A_BYTES, &tmX, &full[s], j * BK, 0);
            next();
          }
          i += n;
        }
      }
      if (!dead) {
        // the first W2 tiles go out before h is known to be there; their h
        // rows follow once every h tile has been counted
        const long long first = r2.start(cta), end = r2.start(cta + 1);
        auto w2_step = [&](long long i, bool a, bool b) {
          const int u = static_cast<int>(i / r2.len), j = static_cast<int>(i - static_cast<long long>(u) * r2.len);
          const int db = u / nslots, slot = u - db * nslots;
          if (a) load_a(&tmW2, sexp[slot] * f + j * BK, db * BM, d, C::N2 * 128);
          if (b)
            tma_load_2d(smem + s * C::STAGE + A_BYTES, &tmH, &full[s], j * BK, slot * C::N2);
        };
        const int s0 = s;
        const uint32_t ph0 = ph;
        long long ahead = first;
        for (; ahead < end && ahead < first + C::STAGES; ++ahead) {
          if (!claim()) break;
          w2_step(ahead, true, false);
          next();
        }
        if (!lost) lost = !wait_count(p.sync + SYNC_H, nslots * FB, kWaitLimitNs);
        asm volatile("fence.proxy.async;" ::: "memory");
        const int s1 = s;
        const uint32_t ph1 = ph;
        s = s0;
        ph = ph0;
        for (long long i = first; i < ahead; ++i) {
          w2_step(i, false, true);
          next();
        }
        s = s1;
        ph = ph1;
        for (long long i = ahead; i < end && !dead;) {
          const int u = static_cast<int>(i / r2.len), k0 = static_cast<int>(i - static_cast<long long>(u) * r2.len);
          const int n = static_cast<int>(min(static_cast<long long>(r2.len - k0), end - i));
          const int db = u / nslots, slot = u - db * nslots;
          const int row = sexp[slot] * f;
          for (int j = k0; j < k0 + n; ++j) {
            if (!claim()) break;
            load_a(&tmW2, row + j * BK, db * BM, d, C::N2 * 128);
            tma_load_2d(smem + s * C::STAGE + A_BYTES, &tmH, &full[s], j * BK, slot * C::N2);
            next();
          }
          i += n;
        }
      }
      // no copy may still be on its way into this CTA when it exits: the
      // latest use of each stage has landed (its phase is the one before s, ph)
      for (int j = 0; j < used; ++j) {
        if (s == 0) {
          s = C::STAGES;
          ph ^= 1u;
        }
        --s;
        if (!mbar_wait(&full[s], ph, kWaitLimitNs)) {
          dead = true;
          break;
        }
      }
      if (dead || lost) atomicOr(p.err, kErrTimeout);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issue
    if (lane == 0) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool dead = false;
      auto phase = [&](const Range& r, uint32_t idesc) {
        const long long end = r.start(cta + 1);
        for (long long i = r.start(cta); i < end && !dead;) {
          const int k0 = static_cast<int>(i % r.len);
          const int n = static_cast<int>(min(static_cast<long long>(r.len - k0), end - i));
          if (!mbar_wait(&tempty[acc], aph ^ 1u, kWaitLimitNs)) {
            dead = true;
            break;
          }
          tc_fence_after();
          const uint32_t dt = tmem_base + acc * 64;
          for (int j = 0; j < n; ++j) {
            if (!mbar_wait_spin(&full[s], ph, kWaitLimitNs)) {
              dead = true;
              break;
            }
            tc_fence_after();
            const uint32_t a = smem_u32(smem + s * C::STAGE), b = a + A_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              tc_mma_f16(dt, make_sdesc_sw128(a + kk * 2048, BOX_BYTES, 1024),
                         make_sdesc_sw128(b + kk * 32, 16, 1024), idesc, (j | kk) != 0 ? 1u : 0u);
            tc_commit(&empty[s]);
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
          tc_commit(&tfull[acc]);
          if (++acc == 2) {
            acc = 0;
            aph ^= 1u;
          }
          i += n;
        }
      };
      phase(r1, make_idesc_bf16_f32(BM, C::N1, true, false));
      if (!dead) phase(r2, make_idesc_bf16_f32(BM, C::N2, true, false));
      // nothing this thread issued may still run when tensor memory is freed
      tc_commit(drain);
      if (!mbar_wait(drain, 0, kWaitLimitNs) || dead) atomicOr(p.err, kErrTimeout);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int col = (warp & 3) * 32 + lane;  // feature of the block = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int acc = 0;
    uint32_t aph = 0;
    bool dead = false;
    // the accumulator's first TP columns, or its hi + lo columns (parts = 2)
    auto take = [&](float (&v)[TP], int parts) {
      // after a wait that ran out the loops go on, so that the four warps
      // still meet at every barrier
      if (!dead && !mbar_wait(&tfull[acc], aph, kWaitLimitNs)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      tc_fence_after();
      uint32_t r[32];
      const uint32_t at = tmem_base + lane_base + acc * 64;
      tmem_ld_32x32b_x32(at, r);
      tmem_ld_wait();
#pragma unroll
      for (int t = 0; t < TP; ++t) v[t] = __uint_as_float(r[t]);
      if (parts == 2) {
        if constexpr (TP == 32) {
          tmem_ld_32x32b_x32(at + 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < TP; ++t) v[t] += __uint_as_float(r[t]);
        } else {
#pragma unroll
          for (int t = 0; t < TP; ++t) v[t] += __uint_as_float(r[TP + t]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    };
    // Joins block `blk` of range r (steps [a, b)) that this CTA holds a part
    // v of: true for the last CTA to arrive, with the sum in v.
    float* part = p.part;
    auto join = [&](const Range& r, long long a, long long b, uint32_t* ctr, uint32_t mask,
                    float (&v)[TP]) {
      auto slice = [&](int c) {
        return part + (static_cast<size_t>(c) * 2 + (r.start(c) > a ? 0 : 1)) * TP * BM + col;
      };
      float* mine = slice(cta);
#pragma unroll
      for (int t = 0; t < TP; ++t)
        if ((mask >> t) & 1u) __stcg(mine + t * BM, v[t]);
      const int c0 = r.owner(a), c1 = r.owner(b - 1);
      __threadfence();
      bar_epi();
      if (tid == 128) *s_last = add_acq_rel(ctr, 1) == static_cast<uint32_t>(c1 - c0) ? 1u : 0u;
      bar_epi();
      const bool last = *s_last != 0;
      if (last) {
        __threadfence();
#pragma unroll
        for (int t = 0; t < TP; ++t) v[t] = 0.f;
        for (int c = c0; c <= c1; ++c) {
          const float* o = slice(c);
#pragma unroll
          for (int t = 0; t < TP; ++t)
            if ((mask >> t) & 1u) v[t] += __ldcg(o + t * BM);
        }
      }
      return last;
    };
    {
      const long long end = r1.start(cta + 1);
      for (long long i = r1.start(cta); i < end;) {
        const int u = static_cast<int>(i / r1.len);
        const long long a = static_cast<long long>(u) * r1.len, b = a + r1.len;
        const long long stop = min(b, end);
        const int slot = u / FB, fb = u - slot * FB;
        const uint32_t mask = smask[slot];
        float v[TP];
        take(v, 1);
        if ((i == a && stop == b) || join(r1, a, b, p.tiles + u, mask, v)) {
          const int c = fb * BM + col;
          if (c < f) {
            __nv_bfloat16* hr = p.h + static_cast<size_t>(slot) * C::N2 * f + c;
#pragma unroll
            for (int t = 0; t < TP; ++t)
              if ((mask >> t) & 1u) {
                const float z = v[t], hv = z / (1.f + expf(-z));
                const __nv_bfloat16 hi = __float2bfloat16_rn(hv);
                hr[static_cast<size_t>(t) * f] = hi;
                hr[static_cast<size_t>(TP + t) * f] =
                    __float2bfloat16_rn(hv - __bfloat162float(hi));
              }
          }
          // h is read by other CTAs' TMA copies
          __threadfence();
          asm volatile("fence.proxy.async;" ::: "memory");
          bar_epi();
          if (tid == 128) add_acq_rel(p.sync + SYNC_H, 1);
        }
        i = stop;
      }
    }
    part += static_cast<size_t>(grid) * 2 * TP * BM;
    {
      const long long end = r2.start(cta + 1), blk = static_cast<long long>(nslots) * r2.len;
      for (long long i = r2.start(cta); i < end;) {
        const int db = static_cast<int>(i / blk);
        const long long a = db * blk, b = a + blk, begin = i, stop = min(b, end);
        float o[TP];
#pragma unroll
        for (int t = 0; t < TP; ++t) o[t] = 0.f;
        while (i < stop) {
          const int u = static_cast<int>(i / r2.len);
          const int slot = u - db * nslots, e = sexp[slot];
          // lane t holds token t's weight for this expert
          float wt = 0.f;
          if (lane < T)
            for (int j = 0; j < k; ++j)
              if (ridx[lane * k + j] == e) wt = rw[lane * k + j];
          const uint32_t mask = smask[slot];
          float v[TP];
          take(v, 2);
#pragma unroll
          for (int t = 0; t < TP; ++t) {
            const float w = __shfl_sync(0xffffffffu, wt, t);
            if ((mask >> t) & 1u) o[t] = fmaf(w, v[t], o[t]);
          }
          i = min(static_cast<long long>(u + 1) * r2.len, stop);
        }
        const uint32_t all = T == 32 ? 0xffffffffu : (1u << T) - 1u;
        if ((begin == a && stop == b) || join(r2, a, b, p.tiles + nslots * FB + db, all, o)) {
          const int c = db * BM + col;
          if (c < d) {
#pragma unroll
            for (int t = 0; t < TP; ++t)
              if (t < T) p.out[static_cast<size_t>(t) * d + c] = __float2bfloat16_rn(o[t]);
          }
        }
      }
    }
    if (dead && lane == 0) atomicOr(p.err, kErrTimeout);
  }

  // ---------------------------------------------------------------- exit
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
  if (tid == 0) {
    if (lost) atomicOr(p.err, kErrTimeout);
    // the last CTA out leaves the counters zero for the next launch
    if (add_acq_rel(p.sync + SYNC_EXIT, 1) == static_cast<uint32_t>(grid) - 1) {
      p.sync[SYNC_GATE] = 0;
      p.sync[SYNC_ROUTE] = 0;
      p.sync[SYNC_H] = 0;
      p.sync[SYNC_EXIT] = 0;
    }
  }
}

template <int TP>
cudaError_t launch_tp(const CUtensorMap& mX, const CUtensorMap& mW1, const CUtensorMap& mW2,
                      const CUtensorMap& mH, const fw::Params& p, int grid, cudaStream_t s) {
  using C = fw::Cfg<TP>;
  cudaError_t e = cudaFuncSetAttribute(few_kernel<TP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(fw::THREADS);
  lc.dynamicSmemBytes = C::SMEM;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait on one another
  attr[0].val.cooperative = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, few_kernel<TP>, mX, mW1, mW2, mH, p);
}

int padded_tokens(int T) { return T <= 8 ? 8 : (T <= 16 ? 16 : 32); }

}  // namespace

FewLayout few_layout(int T, int d, int E, int k, int f) {
  FewLayout L;
  const size_t TP = padded_tokens(T), R = static_cast<size_t>(T) * k;
  const size_t slots = R < static_cast<size_t>(E) ? R : E;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.idx = take(R * 4);
  L.w = take(R * 4);
  L.gpart = take(static_cast<size_t>(fw::MAX_CHUNKS) * T * E * 4);
  L.ntiles = slots * ceil_div(f, fw::BM) + ceil_div(d, fw::BM);
  L.tiles = take(L.ntiles * 4);
  L.h_rows = slots * 2 * TP;
  L.h = take(L.h_rows * f * 2);
  L.part = take(static_cast<size_t>(2) * kFewMaxCtas * 2 * TP * fw::BM * 4);
  L.total = o;
  return L;
}

cudaError_t launch_few(const void* x, const void* Wg, const float* bias, const void* W1,
                       const void* W2, int T, int d, int E, int f, RouterSpec rs, void* out,
                       void* ws, int num_sms, cudaStream_t s) {
  const FewLayout L = few_layout(T, d, E, rs.k, f);
  const int grid = num_sms < kFewMaxCtas ? num_sms : kFewMaxCtas;
  const int TP = padded_tokens(T);
  char* base = static_cast<char*>(ws);
  fw::Params p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.Wg = static_cast<const __nv_bfloat16*>(Wg);
  p.bias = bias;
  p.rs = rs;
  p.T = T;
  p.d = d;
  p.E = E;
  p.f = f;
  p.k = rs.k;
  p.gate_groups = ceil_div(E, fw::GATE_E);
  // chunks of the contraction: at least 32 rows each, at most one per CTA of
  // an expert group
  int chunks = grid / p.gate_groups;
  if (chunks > fw::MAX_CHUNKS) chunks = fw::MAX_CHUNKS;
  if (chunks > d / 32) chunks = d / 32;
  if (chunks < 1) return cudaErrorInvalidConfiguration;  // fewer SMs than expert groups
  p.gate_len = ceil_div(d, chunks);
  p.gate_chunks = ceil_div(d, p.gate_len);
  p.idx = reinterpret_cast<int32_t*>(base + L.idx);
  p.w = reinterpret_cast<float*>(base + L.w);
  p.gpart = reinterpret_cast<float*>(base + L.gpart);
  p.tiles = reinterpret_cast<uint32_t*>(base + L.tiles);
  p.ntiles = static_cast<int>(L.ntiles);
  p.h = reinterpret_cast<__nv_bfloat16*>(base + L.h);
  p.part = reinterpret_cast<float*>(base + L.part);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = reinterpret_cast<uint32_t*>(base);
  p.sync = reinterpret_cast<uint32_t*>(base + kFewSyncOffset);
  CUtensorMap mX, mW1, mW2, mH;
  const uint64_t Eu = static_cast<uint64_t>(E);
  if (!make_map_2d(&mX, x, T, d, 64, TP < 16 ? 16 : TP) ||
      !make_map_2d(&mW1, W1, Eu * d, f, 64, fw::BK) ||
      !make_map_2d(&mW2, W2, Eu * f, d, 64, fw::BK) ||
      !make_map_2d(&mH, p.h, L.h_rows, f, 64, 2 * TP))
    return cudaErrorInvalidValue;
  switch (TP) {
    case 8: return launch_tp<8>(mX, mW1, mW2, mH, p, grid, s);
    case 16: return launch_tp<16>(mX, mW1, mW2, mH, p, grid, s);
    default: return launch_tp<32>(mX, mW1, mW2, mH, p, grid, s);
  }
}

}  // namespace moe
