// few.cu - the whole routed layer for a few tokens (T <= 32: a decode step)
// in one kernel: gate and router (DeepSeek-V4 EP article, sections 2.1 and
// 3.2), W1, SiLU, W2 of the chosen experts and the weighted sum.
//
//   L = x W_g + b        top-k and weights as moe_route
//   h[t, e] = SiLU(x[t] W1[e])          (t routed to e)
//   out[t] = sum over the chosen e of w[t, e] (h[t, e] W2[e])
//
// Bound: each chosen expert's weights cross HBM once (4 d f bytes); the
// products are thin. So the grid is one CTA per SM and every CTA streams its
// share of the weight tiles through a deep TMA ring, from the first W1 tile
// to the last W2 tile without draining.
//
// Products: the weights are the M operand of tcgen05.mma, 128 output
// features x 128 contraction rows a step, read MN-major straight from their
// row-major storage; the tokens are the N operand. Every token multiplies
// every chosen expert (N = 16..64 costs the tensor core nothing here) and
// the epilogue keeps the routed ones, so nothing is permuted or packed. For
// W2 the tokens' h rows are carried as bf16 hi + lo, side by side in N
// (h to 2^-17 relative, so out is rounded once).
//
// Work split: a feature block (phase 1: one expert's 128 features of h; phase
// 2: 128 features of out, every expert's steps one after the other) is a run
// of steps of 128 contraction rows, cut into equal chunks where there are
// fewer blocks than the SMs want units of work. CTAs take units in order from
// a counter, one ahead: SMs differ by a tenth in the bandwidth they get, and
// equal shares left them waiting for the slowest (one token through 8 of 256
// experts: 89.8 us so, 85.5 now; 8 tokens: 416 and 400). A cut block's fp32
// partial sums are joined by the last CTA to arrive, in chunk order, whoever
// computed them: no atomics on values, so the result is bitwise reproducible.
// In phase 2 the routing weights are applied as each expert's accumulator is
// read.
//
// Measured: 7 tokens, 8 experts of 4096 x 11008, two chosen: 179 us with the
// weights out of L2, 7.0 TB/s (163 over and over); one token, 256 experts of
// 7168 x 2048, eight chosen: 87 us, 5.4 TB/s; two of 64 experts of
// 2048 x 1408: 18.6 us, where the chain gate -> router -> W1 -> W2 and its
// four hand-overs between CTAs bound it, not the 3.4 us of bytes.
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
constexpr int BM = 128, BK = 128;           // features, contraction rows of a step
constexpr int BOX_BYTES = 64 * 64 * 2;      // [64 k][64 features] bf16
constexpr int A_BYTES = 4 * BOX_BYTES;      // [k half][feature half]
constexpr int GATE_E = 64;                  // experts of a gate CTA
constexpr int GATE_ROWS = 256;              // contraction rows staged at a time
constexpr int MAX_LOADS = 32;               // partial sums of a logit a thread adds up
constexpr int ACCS = 4, TMEM_COLS = 256;    // accumulators of 64 columns
constexpr int QUEUE = 8;                    // units on their way through a CTA
// Units a CTA is to take in a phase: more even out the SMs better, but each
// costs a partial sum and its arrival, about 1 us of the epilogue (one token
// and 256 experts, eight chosen: 2, 3, 5, 10 units 89.5, 85.5, 86.1, 96.9 us);
// and the fewest steps to a unit of a cut block (1: 21.1 us for 18.7 at one
// token and two experts of 2048 x 1408).
constexpr int UNITS = 3, UNIT_STEPS = 2;
constexpr int MAX_ROWS = kFewMaxTokens * kMaxFanout;

// TP: the tokens a launch is compiled for
template <int TP>
struct Cfg {
  static constexpr int N1 = TP < 16 ? 16 : TP;  // columns of phase 1's products: x rows
  static constexpr int HR = 2 * TP;             // h rows of an expert: hi, lo
  static constexpr int N2 = HR < 16 ? 16 : HR;  // columns of phase 2's (past HR: unused)
  // gate: experts a thread takes, lanes to a row of W_g, rows side by side
  static constexpr int VE = TP <= 8 ? 8 : 64 / TP;
  static constexpr int LPR = GATE_E / VE, RG = THREADS / LPR;
  static constexpr int CB = 32 / TP;            // partial sums joined at a time
  static constexpr int B_HALF = (N1 > N2 ? N1 : N2) * 128;  // 64 k of every column
  static constexpr int B_BYTES = 2 * B_HALF;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 219 * 1024 / STAGE;
  static constexpr int OFF_BAR = STAGES * STAGE;
  static_assert(STAGES < QUEUE, "a stage may wait for h in each of as many units");
  static constexpr int OFF_TAB = OFF_BAR + (2 * STAGES + 2 * ACCS + 2 * QUEUE + 1) * 8;
  static constexpr int SMEM = OFF_TAB + 256 * 4 + 256 * 2 + MAX_ROWS * 4 + MAX_ROWS * 4 + 64 +
                              QUEUE * 4 + QUEUE * 12 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(GATE_ROWS * TP * 4 + RG * TP * GATE_E * 4 + GATE_ROWS * GATE_E * 2 <= OFF_BAR,
                "scratch");
};

struct Params {
  const __nv_bfloat16* x;
  const __nv_bfloat16* Wg;
  const float* bias;
  RouterSpec rs;
  int T, d, E, f, k;
  int gate_groups, gate_chunks, gate_len;  // expert groups x chunks of gate_len rows
  int gate_vec;                            // W_g rows can be read a vector at a time
  int32_t* idx;
  float* w;
  float* gpart;      // [chunks][T][E]
  uint32_t* tiles;   // arrivals: [slots][f blocks], then [d blocks]
  int ntiles;
  __nv_bfloat16* h;  // [slots][2 TP][f]
  float* part;       // [phase][unit][TP][128]
  __nv_bfloat16* out;
  uint32_t* err;
  uint32_t* sync;    // five counters, zero between launches
};
constexpr int SYNC_GATE = 0, SYNC_CLAIM = 4, SYNC_ROUTE = 8, SYNC_H = 16, SYNC_EXIT = 24;

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
__device__ __forceinline__ void add_release(uint32_t* p, uint32_t v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
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
// Threads side by side that add up E logits.
__host__ __device__ constexpr int expert_lanes(int E) {
  return E <= 32 ? 32 : (E <= 64 ? 64 : (E <= 128 ? 128 : 256));
}

// One warp: token t's choice from its logits row (NJ logits a lane), ranked
// and weighted as topk::warp_select_and_weigh does it, in a loop: this code
// runs once a launch, and unrolled its instructions arrive more slowly than
// they run (4 us at 8 rounds). The argmax of a round is one reduction of
// order-preserving integer keys and one of the ids that have the best key.
template <int NJ>
__device__ __forceinline__ void choose(const float* row, int E, const RouterSpec& rs, int t,
                                       int32_t* idx, float* w) {
  constexpr uint32_t ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  float v[NJ];
  int id[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    id[j] = lane + 32 * j;
    v[j] = id[j] < E ? row[id[j]] : -INFINITY;
  }
  if (rs.mode == topk::kRouterGroup) topk::warp_group_limit<NJ>(v, id, E, rs);
  uint32_t key[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    // -0 as +0; a NaN, like the padding, is never chosen (key 0)
    const uint32_t b = __float_as_uint(v[j] + 0.f);
    key[j] = id[j] >= E || isnan(v[j]) ? 0u : (b & 0x80000000u ? ~b : b | 0x80000000u);
  }
  const int rounds = topk::rounds_of(rs);
  float mine = -INFINITY, m = 0.f;  // lane s: round s's logit
  int mine_id = 0x7fffffff;
#pragma unroll 1
  for (int s = 0; s < rounds; ++s) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) best = max(best, key[j]);
    best = __reduce_max_sync(ALL, best);
    int bi = 0x7fffffff;
#pragma unroll
    for (int j = NJ - 1; j >= 0; --j) bi = best != 0 && key[j] == best ? id[j] : bi;
    bi = __reduce_min_sync(ALL, bi);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (id[j] == bi) key[j] = 0;
    const float bv = best == 0 ? -INFINITY
                               : __uint_as_float(best & 0x80000000u ? best & 0x7fffffffu : ~best);
    if (s == 0) m = bv;
    if (lane == s) {
      mine = bv;
      mine_id = bi;
    }
  }
  const float ex = lane < rounds ? expf(mine - m) : 0.f;
  float den = 0.f;
#pragma unroll 1
  for (int s = 0; s < rounds; ++s) den += __shfl_sync(ALL, ex, s);
  if (lane < rs.k) {
    idx[t * rs.k + lane] = mine_id;
    w[t * rs.k + lane] = ex / den;
  }
}
// Soft gating (E <= 16): every expert, weighted.
__device__ __forceinline__ void weigh_all(const float* row, int E, const RouterSpec& rs, int t,
                                          int32_t* idx, float* w) {
  const int lane = threadIdx.x & 31;
  const int id[1] = {lane};
  const float v[1] = {lane < E ? row[lane] : -INFINITY};
  topk::warp_soft_weigh<1>(v, id, E, rs, t, idx, w);
}
// A phase's units: blocks of `len` steps in `chunks` chunks of `per`; unit v
// is chunk v / blocks of block v % blocks, so that the CTAs at work side by
// side read whole rows of the weights between them (the other way round they
// read one column of them: 222 us for 165 at 7 tokens and 8 wide experts).
struct Cut {
  int blocks, len, per, chunks, units;
  __device__ Cut(int blocks_, int len_, int want) : blocks(blocks_), len(len_) {
    if (len == 0) {  // no token has an expert
      per = chunks = units = 0;
      return;
    }
    per = max(UNIT_STEPS, (blocks * len + want - 1) / want);
    chunks = per >= len ? 1 : (len + per - 1) / per;
    per = (len + chunks - 1) / chunks;
    chunks = (len + per - 1) / per;
    units = blocks * chunks;
  }
};
__device__ __forceinline__ void bar_epi() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
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
  uint64_t* tempty = tfull + ACCS;
  uint64_t* qfull = tempty + ACCS;
  uint64_t* qempty = qfull + QUEUE;
  uint64_t* drain = qempty + QUEUE;
  uint32_t* smask = reinterpret_cast<uint32_t*>(smem + C::OFF_TAB);  // slot -> its tokens
  float* rw = reinterpret_cast<float*>(smask + kMaxExperts);         // [T][k] weights
  int32_t* ridx = reinterpret_cast<int32_t*>(rw + MAX_ROWS);         // [T][k] experts, -1: none
  int16_t* sexp = reinterpret_cast<int16_t*>(ridx + MAX_ROWS);       // slot -> expert
  uint32_t* misc = reinterpret_cast<uint32_t*>(sexp + kMaxExperts);
  uint32_t* tmem_slot = misc;
  int* s_nslots = reinterpret_cast<int*>(misc + 1);
  uint32_t* s_last = misc + 2;
  volatile int* queue = reinterpret_cast<volatile int*>(misc + 16);   // unit numbers, -1: no more
  int* pending = reinterpret_cast<int*>(misc + 16 + QUEUE);           // steps that wait for h
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int T = p.T, d = p.d, E = p.E, f = p.f, k = p.k;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    for (int i = 0; i < QUEUE; ++i) {
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], 5);  // the MMA warp, four epilogue warps
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
    float* red = xs + GATE_ROWS * TP;            // [RG][TP][GATE_E]
    __nv_bfloat16* wg = reinterpret_cast<__nv_bfloat16*>(red + C::RG * TP * GATE_E);
    const int chunk = cta / p.gate_groups, e0 = (cta % p.gate_groups) * GATE_E;
    if (chunk < p.gate_chunks) {
      const int r0 = chunk * p.gate_len, r1 = min(d, r0 + p.gate_len);
      const int ec = tid % C::LPR * C::VE, rg = tid / C::LPR;
      float acc[TP][C::VE];
#pragma unroll
      for (int t = 0; t < TP; ++t)
#pragma unroll
        for (int i = 0; i < C::VE; ++i) acc[t][i] = 0.f;
      for (int rb = r0; rb < r1; rb += GATE_ROWS) {
        const int n = min(GATE_ROWS, r1 - rb);  // a multiple of 8
        __syncthreads();
        // the weights of all rows in flight at once
        const __nv_bfloat16* g = p.Wg + static_cast<size_t>(rb) * E + e0;
        if (p.gate_vec != 0) {
#pragma unroll 4
          for (int i = tid; i < n * (GATE_E / 8); i += THREADS) {
            const int r = i / (GATE_E / 8), c = i % (GATE_E / 8) * 8;
            if (e0 + c < E) cp_async16(smem_u32(wg + r * GATE_E + c), g + r * E + c);
          }
        } else {
#pragma unroll 4
          for (int i = tid; i < n * GATE_E; i += THREADS) {
            const int r = i / GATE_E, c = i % GATE_E;
            if (e0 + c < E) wg[i] = g[r * E + c];
          }
        }
        cp_async_commit();
        for (int i = tid; i < T * (GATE_ROWS / 8); i += THREADS) {
          const int t = i / (GATE_ROWS / 8), r = i % (GATE_ROWS / 8) * 8;
          if (r >= n) continue;
          const uint4 v =
              __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * d + rb + r));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            xs[(r + 2 * q) * TP + t] = __uint_as_float(w[q] << 16);
            xs[(r + 2 * q + 1) * TP + t] = __uint_as_float(w[q] & 0xffff0000u);
          }
        }
        cp_async_wait<0>();
        __syncthreads();
        // (tokens past T and experts past E: sums of stale values, not stored)
#pragma unroll 1
        for (int r = rg; r < n; r += C::RG) {
          float xv[TP];
          if constexpr (TP >= 4) {
#pragma unroll
            for (int t = 0; t < TP; t += 4) {
              const float4 v = *reinterpret_cast<const float4*>(xs + r * TP + t);
              xv[t] = v.x;
              xv[t + 1] = v.y;
              xv[t + 2] = v.z;
              xv[t + 3] = v.w;
            }
          } else {
            xv[0] = xs[r];
          }
          const uint32_t* wr = reinterpret_cast<const uint32_t*>(wg + r * GATE_E + ec);
#pragma unroll
          for (int i = 0; i < C::VE; i += 2) {
            const uint32_t w2 = wr[i / 2];
            const float lo = __uint_as_float(w2 << 16), hi = __uint_as_float(w2 & 0xffff0000u);
#pragma unroll
            for (int t = 0; t < TP; ++t) {
              acc[t][i] = fmaf(xv[t], lo, acc[t][i]);
              acc[t][i + 1] = fmaf(xv[t], hi, acc[t][i + 1]);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TP; ++t)
        if (t < T)
#pragma unroll
          for (int i = 0; i < C::VE; ++i) red[(rg * TP + t) * GATE_E + ec + i] = acc[t][i];
      __syncthreads();
      for (int i = tid; i < T * GATE_E; i += THREADS) {
        const int t = i / GATE_E, c = i % GATE_E;
        if (e0 + c < E) {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < C::RG; ++g) s += red[(g * TP + t) * GATE_E + c];
          p.gpart[(static_cast<size_t>(chunk) * T + t) * E + e0 + c] = s;
        }
      }
    }
  }
  // (a release after a barrier covers what the barrier's other threads wrote)
  __syncthreads();
  bool lost = false;  // thread 0: a wait on other CTAs ran out
  if (tid == 0) add_release(p.sync + SYNC_GATE, 1);

  // ---------------------------------------------------------------- router
  // One token: every CTA adds up its sums (at most 32 KB) and routes it
  // itself, which saves a trip through L2 (about 1 us). Several: CTA t routes
  // token t and the others wait (7 tokens routed by every CTA took 10 us,
  // shared out 4.6).
  const bool local = T == 1;
  if (local || cta < T) {
    float* logits = reinterpret_cast<float*>(smem);  // [E]
    float* sums = logits + kMaxExperts;              // [THREADS]
    if (tid == 0) lost = !wait_count(p.sync + SYNC_GATE, grid, kWaitLimitNs);
    __syncthreads();
    // a logit's sums are shared by 256 / EP threads
    const int EP = expert_lanes(E), parts = THREADS / EP;
    const int e = tid % EP, part = tid / EP;
    const int t = cta < T ? cta : 0;
    // all loads in flight, then a tree
    float v[MAX_LOADS];
    const float* g = p.gpart + (static_cast<size_t>(part) * T + t) * E + e;
    const int n = e < E ? p.gate_chunks - part : 0, step = parts * T * E;
#pragma unroll
    for (int j = 0; j < MAX_LOADS; ++j) v[j] = j * parts < n ? __ldcg(g + j * step) : 0.f;
#pragma unroll
    for (int w = MAX_LOADS / 2; w > 0; w >>= 1)
#pragma unroll
      for (int j = 0; j < w; ++j) v[j] += v[j + w];
    sums[tid] = v[0] + (part == 0 && e < E && p.bias != nullptr ? __ldg(p.bias + e) : 0.f);
    __syncthreads();
    if (part == 0 && e < E) {
      float s = sums[tid];
      for (int q = 1; q < parts; ++q) s += sums[tid + q * EP];
      logits[e] = s;
    }
    __syncthreads();
    if (warp == 0) {
      int32_t* oi = local ? ridx : p.idx;
      float* ow = local ? rw : p.w;
      if (p.rs.mode == topk::kRouterSoft)
        weigh_all(logits, E, p.rs, t, oi, ow);
      else if (E <= 64)
        choose<2>(logits, E, p.rs, t, oi, ow);
      else
        choose<8>(logits, E, p.rs, t, oi, ow);
      if (!local) {
        __syncwarp();
        if (lane == 0) add_release(p.sync + SYNC_ROUTE, 1);
      }
    }
  }
  if (!local) {
    if (tid == 0 && !lost) lost = !wait_count(p.sync + SYNC_ROUTE, T, kWaitLimitNs);
  }
  for (int e = tid; e < kMaxExperts; e += THREADS) smask[e] = 0;
  __syncthreads();

  // ---------------------------------------------------------------- slots
  // the chosen experts in id order, and each one's tokens as a bit mask
  for (int i = tid; i < T * k; i += THREADS) {
    const int e = local ? ridx[i] : __ldcg(p.idx + i);
    const float w = local ? rw[i] : __ldcg(p.w + i);
    const bool ok = e >= 0 && e < E;
    ridx[i] = ok ? e : -1;
    rw[i] = ok ? w : 0.f;
    if (ok)
      atomicOr(&smask[e], 1u << (i / k));
    else
      atomicOr(p.err, kErrBadIndex);
  }
  __syncthreads();
  if (warp == 0) {
    // in place: slot <= expert, and a round's masks are read before it writes
    int n = 0;
    for (int j = 0; j < (E + 31) / 32; ++j) {
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
  // (fewer than 2 want units of a cut phase: cut blocks are fewer than want)
  const int len2 = (f + BK - 1) / BK, want = grid * UNITS;
  const Cut c1(nslots * FB, (d + BK - 1) / BK, want), c2(DB, nslots * len2, want);

  if (nslots == 0) {
    for (size_t i = static_cast<size_t>(cta) * THREADS + tid; i < static_cast<size_t>(T) * d;
         i += static_cast<size_t>(grid) * THREADS)
      p.out[i] = __float2bfloat16(0.f);
  } else if (warp == 0) {
    // -------------------------------------------------------------- TMA producer
    // (the whole warp, converged: elect_one says why)
    if (lane == 0) {
      prefetch_tmap(&tmX);
      prefetch_tmap(&tmW1);
      prefetch_tmap(&tmW2);
      prefetch_tmap(&tmH);
    }
    __syncwarp();
    int s = 0;
    uint32_t ph = 0;
    int used = 0;  // stages filled at least once
    bool dead = false;
    // a step's loads: weight rows [row, row + 64 nk) x features [c0, c0 + 64
    // nb), and as much of k from column k on of box rows at b_row of the
    // tokens' side (b_bytes a 64-wide box); nk = 1 in a last half step
    auto load_a = [&](const CUtensorMap* m, int row, int c0, int nk, int nb, uint32_t b_bytes) {
      uint8_t* st = smem + s * C::STAGE;
      mbar_arrive_expect_tx(&full[s], nk * (nb * BOX_BYTES + b_bytes));
      for (int h = 0; h < nk; ++h)
        for (int b = 0; b < nb; ++b)
          tma_load_2d(st + (2 * h + b) * BOX_BYTES, m, &full[s], c0 + b * 64, row + h * 64);
    };
    auto load_b = [&](const CUtensorMap* m, int k, int nk, int b_row) {
      for (int h = 0; h < nk; ++h)
        tma_load_2d(smem + s * C::STAGE + A_BYTES + h * C::B_HALF, m, &full[s], k + h * 64, b_row);
    };
    auto next = [&]() {
      if (++s == C::STAGES) {
        s = 0;
        ph ^= 1u;
      }
    };
    auto claim = [&]() {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, kWaitLimitNs))) {
        dead = true;
        return false;
      }
      if (used < C::STAGES) ++used;
      return true;
    };
    // hand unit v (-1: the end) to the other roles
    int qi = 0;
    uint32_t qph = 0;
    auto push = [&](int v) {
      if (!__all_sync(0xffffffffu, mbar_wait(&qempty[qi], qph ^ 1u, kWaitLimitNs))) dead = true;
      if (lane == 0) {
        queue[qi] = v;
        mbar_arrive(&qfull[qi]);
      }
      __syncwarp();
      if (++qi == QUEUE) {
        qi = 0;
        qph ^= 1u;
      }
    };
    // Before h is known to be there, W2 tiles go out without their h rows, as
    // many as the ring holds; those follow once every h tile has been counted.
    bool ready = false;
    int npend = 0;
    auto h_ready = [&]() {
      if (lane == 0 && !lost) lost = !wait_count(p.sync + SYNC_H, nslots * FB, kWaitLimitNs);
      __syncwarp();
      asm volatile("fence.proxy.async.global;" ::: "memory");
      ready = true;
      if (dead) return;
      s -= npend;
      if (s < 0) s += C::STAGES;
      for (int i = 0; i < npend; ++i) {
        if (elect_one()) load_b(&tmH, pending[3 * i], pending[3 * i + 1], pending[3 * i + 2]);
        __syncwarp();
        if (++s == C::STAGES) s = 0;  // (the phase is already the next stage's)
      }
    };
    int v = cta;
    while (v < c1.units + c2.units && !dead) {
      push(v);
      // the next one, on its way while this one is loaded
      int v_next = 0;
      if (lane == 0) v_next = grid + static_cast<int>(atomicAdd(p.sync + SYNC_CLAIM, 1u));
      if (v < c1.units) {
        const int j1 = v / c1.blocks, u = v - j1 * c1.blocks, k0 = j1 * c1.per;
        const int slot = u / FB, c0 = (u - slot * FB) * BM, row = sexp[slot] * d;
        const int nb = min(2, (f - c0) / 64), k1 = min(c1.len, k0 + c1.per);
        for (int j = k0; j < k1; ++j) {
          if (!claim()) break;
          const int nk = min(2, d / 64 - 2 * j);
          if (elect_one()) {
            load_a(&tmW1, row + j * BK, c0, nk, nb, C::N1 * 128);
            load_b(&tmX, j * BK, nk, 0);
          }
          __syncwarp();
          next();
        }
      } else {
        const int w = v - c1.units, j2 = w / c2.blocks, db = w - j2 * c2.blocks, i0 = j2 * c2.per;
        const int i1 = min(c2.len, i0 + c2.per), nb = min(2, (d - db * BM) / 64);
        int slot = i0 / len2, j = i0 - slot * len2;
        for (int i = i0; i < i1; ++i) {
          if (!ready && npend == C::STAGES) h_ready();
          if (!claim()) break;
          const int nk = min(2, f / 64 - 2 * j);
          if (elect_one()) {
            load_a(&tmW2, sexp[slot] * f + j * BK, db * BM, nk, nb, C::HR * 128);
            if (ready) {
              load_b(&tmH, j * BK, nk, slot * C::HR);
            } else {
              pending[3 * npend] = j * BK;
              pending[3 * npend + 1] = nk;
              pending[3 * npend + 2] = slot * C::HR;
            }
          }
          __syncwarp();
          if (!ready) ++npend;
          next();
          if (++j == len2) {
            j = 0;
            ++slot;
          }
        }
      }
      v = __shfl_sync(0xffffffffu, v_next, 0);
    }
    if (!ready && npend > 0) h_ready();
    push(-1);
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
    if (lane == 0 && (dead || lost)) atomicOr(p.err, kErrTimeout);
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issue
    // (the whole warp, converged: elect_one says why)
    int s = 0, acc = 0;
    uint32_t ph = 0, aph = 0;
    bool dead = false;
    const uint64_t ad0 = make_sdesc_sw128(smem_u32(smem), BOX_BYTES, 1024),
                   bd0 = make_sdesc_sw128(smem_u32(smem) + A_BYTES, 16, 1024);
    // n steps into the next accumulator, the first at step k0 of k64 half steps
    auto run = [&](int k0, int n, int k64, uint32_t idesc) {
      if (!__all_sync(0xffffffffu, mbar_wait(&tempty[acc], aph ^ 1u, kWaitLimitNs))) {
        dead = true;
        return;
      }
      tc_fence_after();
      const uint32_t dt = tmem_base + acc * 64;
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait_spin(&full[s], ph, kWaitLimitNs))) {
          dead = true;
          break;
        }
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(s) * (C::STAGE / 16);
        const uint32_t more = j > 0 ? 1u : 0u;
        const bool both = k64 - 2 * (k0 + j) >= 2;  // both k halves
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16(dt, ad0 + off + kk * (2048 / 16), bd0 + off + kk * 2, idesc,
                       kk > 0 ? 1u : more);
          if (both) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16(dt, ad0 + off + (2 * BOX_BYTES + kk * 2048) / 16,
                         bd0 + off + C::B_HALF / 16 + kk * 2, idesc, 1u);
          }
          tc_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (elect_one()) tc_commit(&tfull[acc]);
      __syncwarp();
      if (++acc == ACCS) {
        acc = 0;
        aph ^= 1u;
      }
    };
    int qi = 0;
    uint32_t qph = 0;
    while (!dead) {
      if (!__all_sync(0xffffffffu, mbar_wait(&qfull[qi], qph, kWaitLimitNs))) {
        dead = true;
        break;
      }
      const int v = queue[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&qempty[qi]);
      if (++qi == QUEUE) {
        qi = 0;
        qph ^= 1u;
      }
      if (v < 0) break;
      if (v < c1.units) {
        const int k0 = v / c1.blocks * c1.per;
        run(k0, min(c1.per, c1.len - k0), d / 64, make_idesc_bf16_f32(BM, C::N1, true, false));
      } else {
        const int i0 = (v - c1.units) / c2.blocks * c2.per, i1 = min(c2.len, i0 + c2.per);
        for (int i = i0; i < i1 && !dead;) {
          const int j = i % len2, n = min(len2 - j, i1 - i);
          run(j, n, f / 64, make_idesc_bf16_f32(BM, C::N2, true, false));
          i += n;
        }
      }
    }
    // nothing this thread issued may still run when tensor memory is freed
    if (elect_one()) tc_commit(drain);
    __syncwarp();
    if ((!mbar_wait(drain, 0, kWaitLimitNs) || dead) && lane == 0) atomicOr(p.err, kErrTimeout);
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
      if (++acc == ACCS) {
        acc = 0;
        aph ^= 1u;
      }
    };
    // Joins a block of `chunks` chunks, of which v is chunk j's sum; parts: the
    // first one's. True for the last CTA to arrive, with the block's sum in v.
    auto join = [&](float* parts, int chunks, int j, uint32_t* ctr, uint32_t mask,
                    float (&v)[TP]) {
      float* mine = parts + static_cast<size_t>(j) * TP * BM + col;
#pragma unroll
      for (int t = 0; t < TP; ++t)
        if ((mask >> t) & 1u) __stcg(mine + t * BM, v[t]);
      bar_epi();
      if (tid == 128) *s_last = add_acq_rel(ctr, 1) == static_cast<uint32_t>(chunks) - 1 ? 1u : 0u;
      bar_epi();
      const bool last = *s_last != 0;
      if (last) {
#pragma unroll
        for (int t = 0; t < TP; ++t) v[t] = 0.f;
        for (int cb = 0; cb < chunks; cb += C::CB) {
          float o[C::CB][TP];
          const float* from = parts + static_cast<size_t>(cb) * TP * BM + col;
#pragma unroll
          for (int q = 0; q < C::CB; ++q)
#pragma unroll
            for (int t = 0; t < TP; ++t)
              o[q][t] = cb + q < chunks && ((mask >> t) & 1u) ? __ldcg(from + (q * TP + t) * BM)
                                                              : 0.f;
#pragma unroll
          for (int q = 0; q < C::CB; ++q)
#pragma unroll
            for (int t = 0; t < TP; ++t) v[t] += o[q][t];
        }
      }
      return last;
    };
    int qi = 0;
    uint32_t qph = 0;
    while (true) {
      // (four warps meet at barriers below: a wait that runs out ends none of
      // them before the others, the queue being one for all)
      if (!mbar_wait(&qfull[qi], qph, kWaitLimitNs)) dead = true;
      const int unit = ptx::bar_and(2, 128, !dead) ? queue[qi] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&qempty[qi]);
      if (++qi == QUEUE) {
        qi = 0;
        qph ^= 1u;
      }
      if (unit < 0) break;
      if (unit < c1.units) {
        const int j = unit / c1.blocks, u = unit - j * c1.blocks;
        const int slot = u / FB, fb = u - slot * FB;
        const uint32_t mask = smask[slot];
        float v[TP];
        take(v, 1);
        if (c1.chunks == 1 ||
            join(p.part + static_cast<size_t>(u) * c1.chunks * TP * BM, c1.chunks, j, p.tiles + u,
                 mask, v)) {
          const int c = fb * BM + col;
          if (c < f) {
            __nv_bfloat16* hr = p.h + static_cast<size_t>(slot) * C::HR * f + c;
#pragma unroll
            for (int t = 0; t < TP; ++t)
              if ((mask >> t) & 1u) {
                const float z = v[t], hv = z / (1.f + expf(-z));
                // (past bf16's range hi is cut off, and of an infinity lo is 0)
                __nv_bfloat16 hi = __float2bfloat16_rn(hv);
                if (__hisinf(hi)) hi = __float2bfloat16_rz(hv);
                hr[static_cast<size_t>(t) * f] = hi;
                hr[static_cast<size_t>(TP + t) * f] =
                    __float2bfloat16_rn(isinf(hv) ? 0.f : hv - __bfloat162float(hi));
              }
          }
          // h is read by other CTAs' TMA copies
          asm volatile("fence.proxy.async.global;" ::: "memory");
          bar_epi();
          if (tid == 128) add_release(p.sync + SYNC_H, 1);
        }
      } else {
        const int w = unit - c1.units, j = w / c2.blocks, db = w - j * c2.blocks;
        const int i0 = j * c2.per, i1 = min(c2.len, i0 + c2.per);
        float o[TP];
#pragma unroll
        for (int t = 0; t < TP; ++t) o[t] = 0.f;
        for (int i = i0; i < i1;) {
          const int slot = i / len2, e = sexp[slot];
          // lane t holds token t's weight for this expert
          float wt = 0.f;
          if (lane < T)
            for (int q = 0; q < k; ++q)
              if (ridx[lane * k + q] == e) wt = rw[lane * k + q];
          const uint32_t mask = smask[slot];
          float v[TP];
          take(v, 2);
#pragma unroll
          for (int t = 0; t < TP; ++t) {
            const float wv = __shfl_sync(0xffffffffu, wt, t);
            if ((mask >> t) & 1u) o[t] = fmaf(wv, v[t], o[t]);
          }
          i = min((slot + 1) * len2, i1);
        }
        const uint32_t all = T >= 32 ? 0xffffffffu : (1u << T) - 1u;
        float* parts = p.part + (static_cast<size_t>(2) * want + static_cast<size_t>(db) * c2.chunks) *
                                    TP * BM;
        if (c2.chunks == 1 || join(parts, c2.chunks, j, p.tiles + nslots * FB + db, all, o)) {
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
      p.sync[SYNC_CLAIM] = 0;
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

// Chunks of the gate's contraction, at most: what the threads that share a
// logit add up, and one per CTA.
int max_chunks(int E) {
  const int n = fw::MAX_LOADS * (fw::THREADS / fw::expert_lanes(E));
  return n < kFewMaxCtas ? n : kFewMaxCtas;
}

int padded_tokens(int T) { return T <= 1 ? 1 : (T <= 8 ? 8 : (T <= 16 ? 16 : 32)); }

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
  L.gpart = take(static_cast<size_t>(max_chunks(E)) * T * E * 4);
  L.ntiles = slots * ceil_div(f, fw::BM) + ceil_div(d, fw::BM);
  L.tiles = take(L.ntiles * 4);
  L.h_rows = slots * 2 * TP;
  L.h = take(L.h_rows * f * 2);
  // two phases of fewer than 2 x CTAs x units partial sums
  L.part = take(static_cast<size_t>(4) * kFewMaxCtas * fw::UNITS * TP * fw::BM * 4);
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
  // chunks of the contraction: at least 32 rows each (a multiple of 8), at
  // most one per CTA of an expert group, and every token's router on a CTA
  int chunks = grid / p.gate_groups;
  const int most = max_chunks(E);
  if (chunks > most) chunks = most;
  if (chunks > d / 32) chunks = d / 32;
  if (chunks < 1 || grid < T) return cudaErrorInvalidConfiguration;
  p.gate_len = ceil_div(ceil_div(d, chunks), 8) * 8;
  p.gate_chunks = ceil_div(d, p.gate_len);
  p.gate_vec = E % 8 == 0 && reinterpret_cast<uintptr_t>(Wg) % 16 == 0 ? 1 : 0;
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
      !make_map_2d(&mW1, W1, Eu * d, f, 64, 64) ||
      !make_map_2d(&mW2, W2, Eu * f, d, 64, 64) ||
      !make_map_2d(&mH, p.h, L.h_rows, f, 64, 2 * TP))
    return cudaErrorInvalidValue;
  switch (TP) {
    case 1: return launch_tp<1>(mX, mW1, mW2, mH, p, grid, s);
    case 8: return launch_tp<8>(mX, mW1, mW2, mH, p, grid, s);
    case 16: return launch_tp<16>(mX, mW1, mW2, mH, p, grid, s);
    default: return launch_tp<32>(mX, mW1, mW2, mH, p, grid, s);
  }
}

}  // namespace moe
