// range.cuh - a sequence of equal steps cut into one contiguous range per
// CTA, for kernels that stream a fixed amount of data with every SM and join
// the blocks that a cut falls into.
#pragma once

namespace moe {

// `units` accumulators of `len` steps, fewer than 2^28 in all, and each CTA's
// range of them: start(c) = floor(total c / G).
struct Range {
  int len, total, G, q, r;
  __device__ Range(int units, int len_, int grid) : len(len_) {
    total = units * len;
    G = total < grid ? total : grid;  // every range holds a step
    q = G > 0 ? total / G : 0;
    r = total - q * G;
  }
  __device__ int start(int c) const { return c >= G ? total : q * c + r * c / G; }
  // the CTA whose range holds step i: an estimate, put right
  __device__ int owner(int i) const {
    int c = static_cast<int>((static_cast<float>(i) + 1.f) * static_cast<float>(G) /
                             static_cast<float>(total));
    c = c < G ? c : G - 1;
    while (c > 0 && start(c) > i) --c;
    while (c + 1 < G && start(c + 1) <= i) ++c;
    return c;
  }
};

}  // namespace moe
