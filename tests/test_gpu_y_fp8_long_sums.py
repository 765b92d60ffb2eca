"""fp32 sums of the 8-bit products over long contractions: no worse than those of one chain of 32
stages of 128 steps, whatever the length.

The limit: an accumulator that drops what is below its last place loses half a step of 2^-23 on
average with each addition, always towards zero. A step is 0.72 of 2^-23 of the value it belongs to on
average (between a half and all of it, evenly in its logarithm), and the partial sums that lose it
are 2/3 of the last one (they grow with the root of their length). A chain of 32 stages is 128
additions of 32 steps: 128 x 0.72 x 2/3 = 61 half steps of its sum. The chains of a sum lose the same
share of theirs each, and adding up to 16 of them, rounded to nearest, is off by less than three half
steps (16 errors of either sign, each a third of half a step of at most the whole): 64 in all.
In one chain the loss grows with the length, to 16 times that for 512 stages."""
import pytest
import torch

from block_plain import U32
from train_plain import F64, decode
from test_gpu_u_fp8 import check_products, problem, run_product

pytestmark = pytest.mark.gpu
LIMIT = 64 * U32


def check_norms(p, transposed, out):
    r, lo = p["dy" if transposed else "x"], p["first"]
    a = decode(r.q, r.scale[:, :-(-r.C // 128)].contiguous(), 1, 128)
    for e, n in enumerate(p["counts"]):
        w = decode(p["wq"][e], p["wsc"][e], 128, 128)
        y = a[lo:lo + n] @ (w.t() if transposed else w)
        err = float((out[lo:lo + n].to(F64) - y).norm() / y.norm())
        assert err <= LIMIT, (e, err / U32)
        lo += n


# one CTA to a tile and pairs; more than 32 rows, so that a tile's contraction is not cut, 128,
# 256 and 512 stages long, and a ragged end
@pytest.mark.parametrize("counts,length", [([130], 65536), ([40, 200], 32768), ([500], 65536),
                                           ([470, 460], 16384 + 64)])
@pytest.mark.parametrize("transposed", [False, True])
def test_long_contractions(cuda_ok, counts, length, transposed):
    K, N = (64, length) if transposed else (length, 64)
    p = problem(counts, K, N, seed=length + len(counts))
    out = run_product(p, transposed)
    check_products(p, transposed, out)
    check_norms(p, transposed, out)


# few rows: ranges of the contraction, of several chains each, joined from the workspace
@pytest.mark.parametrize("transposed", [False, True])
def test_cut_contractions_of_several_chains(cuda_ok, transposed):
    K, N = (8192, 65536) if transposed else (65536, 8192)
    p = problem([5], K, N, seed=5)
    out = run_product(p, transposed)
    check_products(p, transposed, out)
    check_norms(p, transposed, out)
