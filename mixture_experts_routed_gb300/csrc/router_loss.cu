// router_loss.cu - the router's balance loss, by sequence or over the batch,
// its z loss and the experts' counts, and the gradient of the logits.
//
// Over the tokens t of sequence s that count (n_s of them; c_se chose e):
//   p_t = softmax(L_t)   f_se = E c_se / (k n_s)   P_se = sum_t p_te / n_s
//   balance = 1/S' sum_s sum_e f_se P_se          S' sequences with n_s > 0
//   z       = 1/N sum_t lse_t^2                   N = sum_s n_s
//   loss    = a balance + b z
//   dL_te   = a / (S' n_s) p_te (f_se - sum_j p_tj f_sj) + 2 b / N lse_t p_te
// (the counts are constants to the gradient). Bound by latency: two launches
// of a few dependent loads, sums and a hand-over each. 256 tokens of 8 experts
// 7.1 us, 8192 of 64 in 17 sequences 10.8, 16384 of 256 (17 MB) 14.8; the
// gradients 1.6, 3.8 and 7.6 us, the last at 4.4 TB/s.
#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kJoinWarps = 32;

// Tokens are cut into chunks of `len` of one sequence. Chunk j of sequence s
// has the slot offsets[s] / len + s + j, which no other chunk has (a sequence
// begins at most one slot behind the one before it, plus its own chunks).
struct Seqs {
  const int32_t* offsets;  // null: one sequence of all T
  int T, S, len;
  __device__ int at(int s) const { return offsets != nullptr ? __ldg(offsets + s) : (s ? T : 0); }
  __device__ int slot(int s) const { return at(s) / len + s; }
  // the last s whose value is at most x, 0 if none
  template <typename F>
  __device__ int last(int x, F value) const {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (value(mid) <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
  // sequence s begins and ends within [0, T], in this order
  __device__ bool good(int s) const {
    const int a = at(s), b = at(s + 1);
    return a >= 0 && a <= b && b <= T;
  }
};

// what a token's row is to its lanes: values at lane + 32 j, NJ of them
template <int NJ>
struct Row {
  float v[NJ];
  __device__ void load(const float* p, int E, int lane) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] = lane + 32 * j < E ? __ldg(p + lane + 32 * j) : -INFINITY;
  }
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// hi + lo += v without loss (D. Knuth, The Art of Computer Programming 2,
// 4.2.2); both are read together where hi is finite
__device__ __forceinline__ void add_exact(float& hi, float& lo, float v) {
  const float s = hi + v, b = s - hi;
  lo += (hi - (s - b)) + (v - b);
  hi = s;
}
__device__ __forceinline__ float both(float hi, float lo) { return isfinite(hi) ? hi + lo : hi; }

// A block sums one chunk, a token to a warp at a time, the next two's logits
// loaded meanwhile. A lane's sums of kRun pairs of tokens are plain; those of
// the runs are added without loss, so that a batch of 2^26 tokens, 18000 to a
// lane, rounds no more often than one of 10^5 (plain sums of equal tokens were
// off by 1.6e-4 there). RUNS: the chunks are longer than a run, from 456 x 8 x
// 32 tokens (1048576 x 256: 349 -> 356 us); without, the loop has none of it
// (with, 16384 x 256 took 15.2 us for 14.8).
constexpr int kRun = 16;

template <int NJ, bool RUNS>
__global__ void __launch_bounds__(kWarps * 32)
    router_loss_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                       const Seqs q, const uint8_t* __restrict__ mask, int E, int k,
                       float* __restrict__ lse, float* __restrict__ psum, int32_t* __restrict__ cnt,
                       float2* __restrict__ tail, uint32_t* __restrict__ bad, uint32_t* err) {
  // the runs' sums, and what they lost
  __shared__ float ps[kWarps][NJ * 32], pl[RUNS ? kWarps : 1][RUNS ? NJ * 32 : 1];
  __shared__ int cs[NJ * 32];
  __shared__ float zs[kWarps];
  __shared__ int ns[kWarps];
  pdl_wait();
  pdl_trigger();
  // (a sequence a block is checked for all; each block's own, before it reads)
  if (threadIdx.x == 0 && static_cast<int>(blockIdx.x) < q.S && !q.good(blockIdx.x)) {
    *bad = 1;
    atomicOr(err, kErrBadIndex);
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = q.last(blockIdx.x, [&](int i) { return q.slot(i); });
  if (!q.good(s)) return;
  const int t0 = q.at(s) + (static_cast<int>(blockIdx.x) - q.slot(s)) * q.len;
  const int t1 = min(t0 + q.len, q.at(s + 1));
  if (t0 >= t1 || t0 < q.at(s)) return;
  for (int e = tid; e < E; e += kWarps * 32) cs[e] = 0;
  __syncthreads();
  Row<NJ> sum;
#pragma unroll
  for (int j = 0; j < NJ; ++j) sum.v[j] = 0.f;
  float zsum = 0.f;
  int n = 0;
  struct Token {
    Row<NJ> L;
    int e;    // this lane's choice
    bool on;  // (a masked token's row is not read)
  } ahead[2];
  auto load = [&](Token& k0, int t) {
    k0.on = t < t1 && (mask == nullptr || __ldg(mask + t) != 0);
    if (!k0.on) return;
    k0.L.load(logits + static_cast<size_t>(t) * E, E, lane);
    if (lane < k) k0.e = __ldg(idx + static_cast<size_t>(t) * k + lane);
  };
  auto add = [&](Token& k0, int t) {
    if (!k0.on) {
      if (t < t1 && lane == 0) lse[t] = 0.f;
      return;
    }
    if (lane < k) {
      if (k0.e >= 0 && k0.e < E)
        atomicAdd(&cs[k0.e], 1);
      else
        atomicOr(err, kErrBadIndex);
    }
    Row<NJ>& L = k0.L;
    float top = L.v[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) top = fmaxf(top, L.v[j]);
    top = warp_max(top);
    float den = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      L.v[j] = lane + 32 * j < E ? expf(L.v[j] - top) : 0.f;
      den += L.v[j];
    }
    den = warp_sum(den);
    const float inv = 1.f / den, l = top + logf(den);
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum.v[j] = fmaf(L.v[j], inv, sum.v[j]);
    zsum = fmaf(l, l, zsum);
    ++n;
    if (lane == 0) lse[t] = l;
  };
  load(ahead[0], t0 + warp);
  load(ahead[1], t0 + warp + kWarps);
  float zhi = 0.f, zlo = 0.f;
  if constexpr (RUNS) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) ps[warp][lane + 32 * j] = pl[warp][lane + 32 * j] = 0.f;
  }
  auto end_run = [&] {
    if constexpr (RUNS) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        add_exact(ps[warp][lane + 32 * j], pl[warp][lane + 32 * j], sum.v[j]);
        sum.v[j] = 0.f;
      }
      add_exact(zhi, zlo, zsum);
      zsum = 0.f;
    }
  };
  int left = kRun;
  for (int t = t0 + warp; t < t1; t += 2 * kWarps) {
    if (RUNS && left-- == 0) {
      left = kRun - 1;
      end_run();
    }
    Token now[2] = {ahead[0], ahead[1]};
    load(ahead[0], t + 2 * kWarps);
    load(ahead[1], t + 3 * kWarps);
    add(now[0], t);
    add(now[1], t + kWarps);
  }
  if constexpr (RUNS) {
    end_run();
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      ps[warp][lane + 32 * j] = both(ps[warp][lane + 32 * j], pl[warp][lane + 32 * j]);
    zsum = both(zhi, zlo);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) ps[warp][lane + 32 * j] = sum.v[j];
  }
  if (lane == 0) {
    zs[warp] = zsum;
    ns[warp] = n;
  }
  __syncthreads();
  const size_t at = static_cast<size_t>(blockIdx.x) * E;
  for (int i = tid; i < E; i += kWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += ps[w][i];
    psum[at + i] = v;
    cnt[at + i] = cs[i];
  }
  if (tid == 0) {
    float v = 0.f;
    int m = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      v += zs[w];
      m += ns[w];
    }
    tail[blockIdx.x] = make_float2(v, __int_as_float(m));
  }
}

// A block joins the chunks of one sequence for 32 experts, every 32nd to a
// warp, in order, and then over the warps; the last block to be done adds up the
// sequences, in order.
__global__ void __launch_bounds__(kJoinWarps * 32)
    router_loss_join_kernel(const Seqs q, int E, int k, float balance, float zcoef,
                            const float* __restrict__ psum, const int32_t* __restrict__ cnt,
                            const float2* __restrict__ tail, float* term, uint32_t* bad, uint32_t* done,
                            float* __restrict__ loss, int32_t* __restrict__ counts,
                            int32_t* tokens) {
  // (a warp writes a row and reads a column)
  __shared__ float ps[kJoinWarps][33], zs[kJoinWarps], vs[32];
  __shared__ int cs[kJoinWarps][33], ns[kJoinWarps];
  __shared__ int last;
  pdl_wait();
  pdl_trigger();
  const bool fine = __ldcg(bad) == 0;  // (else nothing is written)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = ceil_div(E, 32);
  const int s = blockIdx.x / parts, part = blockIdx.x - s * parts, e = part * 32 + lane;
  const int first = fine ? q.slot(s) : 0,
            chunks = fine ? ceil_div(q.at(s + 1) - q.at(s), q.len) : 0;
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
  // (eight chunks' loads under way at a time)
  for (int j = warp; j < chunks; j += kJoinWarps * 8) {
    float pv[8];
    int cv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool some = e < E && j + i * kJoinWarps < chunks;
      const size_t at = static_cast<size_t>(first + j + i * kJoinWarps) * E + e;
      pv[i] = some ? __ldcg(psum + at) : 0.f;
      cv[i] = some ? __ldcg(cnt + at) : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p += pv[i];
      c += cv[i];
    }
  }
  for (int j = tid; j < chunks; j += kJoinWarps * 32) {
    const float2 v = __ldcg(tail + first + j);
    z += v.x;
    n += __float_as_int(v.y);
  }
  ps[warp][lane] = p;
  cs[warp][lane] = c;
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    zs[warp] = z;
    ns[warp] = n;
  }
  __syncthreads();
  // warp w: expert part * 32 + w
  n = __reduce_add_sync(0xffffffffu, ns[lane]);
  p = warp_sum(ps[lane][warp]);
  c = __reduce_add_sync(0xffffffffu, cs[lane][warp]);
  if (lane == 0) {
    const int mine = part * 32 + warp;
    const float tokens_f = static_cast<float>(n);
    if (mine < E && fine) counts[static_cast<size_t>(s) * E + mine] = c;
    // f P = E c / (k n) p / n
    vs[warp] = n > 0 && mine < E ? static_cast<float>(E) * static_cast<float>(c) /
                                       (static_cast<float>(k) * tokens_f) * (p / tokens_f)
                                 : 0.f;
  }
  __syncthreads();
  if (warp == 0) {
    const float v = warp_sum(vs[lane]);
    z = warp_sum(zs[lane]);
    if (lane == 0) {
      term[2 * blockIdx.x] = v;
      term[2 * blockIdx.x + 1] = part == 0 ? z : 0.f;
      if (part == 0 && fine) tokens[s] = n;
      __threadfence();
      last = atomicAdd(done, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  if (!fine) {
    if (tid == 0) *bad = *done = 0;
    return;
  }
  __threadfence();
  // (a thread's part is long where sequences are many: 2^13 blocks)
  float bal = 0.f, zz = 0.f, blo = 0.f, zlo = 0.f;
  int used = 0, all = 0;
  for (int i = tid; i < static_cast<int>(gridDim.x); i += kJoinWarps * 32) {
    add_exact(bal, blo, __ldcg(term + 2 * i));
    add_exact(zz, zlo, __ldcg(term + 2 * i + 1));
  }
  bal = both(bal, blo);
  zz = both(zz, zlo);
  for (int i = tid; i < q.S; i += kJoinWarps * 32) {
    const int m = __ldcg(tokens + i);
    used += m > 0;
    all += m;
  }
  bal = warp_sum(bal);
  zz = warp_sum(zz);
  used = __reduce_add_sync(0xffffffffu, used);
  all = __reduce_add_sync(0xffffffffu, all);
  if (lane == 0) {
    vs[warp] = bal;
    zs[warp] = zz;
    cs[warp][0] = used;
    ns[warp] = all;
  }
  __syncthreads();
  if (warp != 0) return;
  bal = warp_sum(vs[lane]);
  zz = warp_sum(zs[lane]);
  used = __reduce_add_sync(0xffffffffu, cs[lane][0]);
  all = __reduce_add_sync(0xffffffffu, ns[lane]);
  if (lane != 0) return;
  if (used > 0) bal /= static_cast<float>(used);
  if (all > 0) zz /= static_cast<float>(all);
  loss[0] = fmaf(balance, bal, zcoef * zz);
  loss[1] = bal;
  loss[2] = zz;
  tokens[q.S] = used;
  tokens[q.S + 1] = all;
  *done = 0;
}

// A token to a warp.
template <int NJ>
__global__ void __launch_bounds__(kWarps * 32)
    router_loss_bwd_kernel(const float* __restrict__ logits, const Seqs q,
                           const uint8_t* __restrict__ mask, int E, int k, float balance,
                           float zcoef, const int32_t* __restrict__ counts,
                           const int32_t* __restrict__ tokens, const float* __restrict__ lse,
                           const float* __restrict__ dloss, float* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= q.T) return;
  float* out = dlogits + static_cast<size_t>(t) * E;
  const int s = q.last(t, [&](int i) { return q.at(i); });
  const int n = __ldg(tokens + s), used = __ldg(tokens + q.S), all = __ldg(tokens + q.S + 1);
  const bool on = t >= q.at(s) && t < q.at(s + 1) && n > 0 && used > 0 && all > 0 &&
                  (mask == nullptr || __ldg(mask + t) != 0);
  if (!on) {
    for (int e = lane; e < E; e += 32) out[e] = 0.f;
    return;
  }
  const float g = dloss != nullptr ? __ldg(dloss) : 1.f, l = __ldg(lse + t);
  const float fs = static_cast<float>(E) / (static_cast<float>(k) * static_cast<float>(n));
  Row<NJ> L;
  L.load(logits + static_cast<size_t>(t) * E, E, lane);
  float f[NJ], den, dot;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 32 * j;
    f[j] = e < E ? fs * static_cast<float>(__ldg(counts + static_cast<size_t>(s) * E + e)) : 0.f;
  }
  // p = exp(L - shift) over its own sum, whatever the shift: exp(L - lse) alone would be off by half
  // a step of |lse|, which is many of p's where logits share an offset. The lse is at hand before a
  // maximum is (16384 x 256: 7.9 us with one); past some 2^24 its half step is too wide for a shift.
  auto weigh = [&](float shift) {
    den = dot = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      L.v[j] = lane + 32 * j < E ? expf(L.v[j] - shift) : 0.f;
      den += L.v[j];
      dot = fmaf(L.v[j], f[j], dot);
    }
    den = warp_sum(den);
    dot = warp_sum(dot);
  };
  weigh(l);
  if (!(den > 0.25f && den < 4.f)) {
    L.load(logits + static_cast<size_t>(t) * E, E, lane);
    float top = L.v[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) top = fmaxf(top, L.v[j]);
    weigh(warp_max(top));
  }
  const float inv = 1.f / den;
  dot *= inv;
  const float cb = g * balance / (static_cast<float>(used) * static_cast<float>(n));
  const float cz = g * 2.f * zcoef / static_cast<float>(all) * l;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 32 * j;
    if (e < E) out[e] = L.v[j] * inv * fmaf(cb, f[j] - dot, cz);
  }
}

// f with the number of experts a lane takes: 1, 2, 4 or 8
template <typename F>
cudaError_t by_experts(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>());
  if (E <= 64) return f(std::integral_constant<int, 2>());
  return E <= 128 ? f(std::integral_constant<int, 4>()) : f(std::integral_constant<int, 8>());
}

// Chunks of a warp's token or more, about three blocks to an SM.
int chunk_len(int T) {
  const int len = ceil_div(ceil_div(T, 456), kWarps) * kWarps;
  return len < kWarps ? kWarps : len;
}
int slots_of(int T, int S) { return T / chunk_len(T) + S; }

struct Layout {
  size_t bad, done, psum, cnt, tail, term, total;
};
Layout layout(int T, int E, int S) {
  Layout L;
  const size_t slots = slots_of(T, S);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  take(4);  // the error word, and two of the kernels'
  L.bad = 64;
  L.done = 128;
  L.psum = take(slots * E * 4);
  L.cnt = take(slots * E * 4);
  L.tail = take(slots * 8);
  L.term = take(static_cast<size_t>(S) * ceil_div(E, 32) * 8);
  L.total = o;
  return L;
}

}  // namespace

size_t router_loss_ws(int T, int E, int S) { return layout(T, E, S).total; }

cudaError_t launch_router_loss(const float* logits, const int32_t* idx, const int32_t* offsets,
                               const uint8_t* mask, int T, int E, int k, int S, float balance,
                               float z, float* loss, int32_t* counts, int32_t* tokens, float* lse,
                               void* ws, cudaStream_t s) {
  const Layout L = layout(T, E, S);
  char* w = static_cast<char*>(ws);
  const Seqs q{offsets, T, S, chunk_len(T)};
  float* psum = reinterpret_cast<float*>(w + L.psum);
  int32_t* cnt = reinterpret_cast<int32_t*>(w + L.cnt);
  float2* tail = reinterpret_cast<float2*>(w + L.tail);
  const cudaError_t e = by_experts(E, [&](auto nj) {
    constexpr int NJ = decltype(nj)::value;
    auto go = [&](auto kernel) {
      return launch_pdl(kernel, dim3(slots_of(T, S)), dim3(kWarps * 32), 0, s, logits, idx, q, mask,
                        E, k, lse, psum, cnt, tail, reinterpret_cast<uint32_t*>(w + L.bad),
                        reinterpret_cast<uint32_t*>(w));
    };
    return q.len > 2 * kRun * kWarps ? go(router_loss_kernel<NJ, true>)
                                     : go(router_loss_kernel<NJ, false>);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(router_loss_join_kernel, dim3(S * ceil_div(E, 32)), dim3(kJoinWarps * 32), 0, s, q,
                    E, k, balance, z, static_cast<const float*>(psum),
                    static_cast<const int32_t*>(cnt), static_cast<const float2*>(tail),
                    reinterpret_cast<float*>(w + L.term), reinterpret_cast<uint32_t*>(w + L.bad),
                    reinterpret_cast<uint32_t*>(w + L.done), loss, counts, tokens);
}

cudaError_t launch_router_loss_bwd(const float* logits, const int32_t* offsets, const uint8_t* mask,
                                   int T, int E, int k, int S, float balance, float z,
                                   const int32_t* counts, const int32_t* tokens, const float* lse,
                                   const float* dloss, float* dlogits, cudaStream_t s) {
  const Seqs q{offsets, T, S, chunk_len(T)};
  return by_experts(E, [&](auto nj) {
    return launch_pdl(router_loss_bwd_kernel<decltype(nj)::value>, dim3(ceil_div(T, kWarps)),
                      dim3(kWarps * 32), 0, s, logits, q, mask, E, k, balance, z, counts, tokens,
                      lse, dloss, dlogits);
  });
}

}  // namespace moe
