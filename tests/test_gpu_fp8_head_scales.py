"""bf16 queries over FP8 caches: what one head of a group holds does not reach the
others.  Queries become fp16 under a power of two, each head under its own: beside
a head that holds an infinity or a NaN, or is 2^40 times larger, the rest of its
group is as exact as alone.

Tolerances as in test_gpu_sparse.py (2^-11 + 2^-14 of sum_j p_j |v_j|, and half a
step of the output).  The head of 2^40 has logits of up to 32 * 2^40 in magnitude,
off by at most 2^-12 * 2^40 (2^-12 for logits below 32): its largest is further than
2^30 above the next for these inputs, so that its softmax is one token's."""
import math

import numpy as np
import pytest
import torch

import oracle.sparse as S
from test_gpu_fp4 import f64, pa  # noqa: F401  (pa is the fixture)
from test_gpu_sparse import Batch, chosen, pool, sparse

pytestmark = pytest.mark.gpu
KS, VS = 0.5, 0.25


def batch(seed, lens, H, G, d, bs):
    b = Batch(seed, lens, H, G, d, bs, "bf16", "fp8", mean=0.0)
    vc, vvals = pool(b.rng, b.rng.standard_normal((b.NB, H, bs, d)), "fp8", "bf16", bs, d)
    return b, vc, vvals


def heads_beside(b, G, odd):
    """Makes one head of every group odd; the other heads' numbers."""
    Hq = b.H * G
    at = [h * G + h % G for h in range(b.H)]
    b.q[:, at] *= odd
    return [h for h in range(Hq) if h not in at], at


def compare(b, vvals, out, tables, lens, scale, heads):
    ref, mag = S.attend(b.q.double().numpy(), b.kvals * KS, vvals * VS, tables, lens, scale)
    got, ref, mag = f64(out)[:, heads], ref[:, heads], mag[:, heads]
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= mag * (2.0 ** -11 + 2.0 ** -14) + np.abs(ref) * 2.0 ** -8 + 2.0 ** -126).all()


def gaps(b, tables, lens, scale, heads, G):
    """Between the largest and the second largest logit of a row and head; infinity where there is one."""
    for r in range(len(lens)):
        for h in heads:
            n = int(lens[r, h // G])
            if n > 1:
                ids = tables[r, h // G, : -(-n // b.bs)]
                K = b.kvals[ids, h // G].reshape(-1, b.d)[:n] * KS
                z = np.sort(K @ b.q[r, h].double().numpy() * scale)
                yield z[-1] - z[-2]


@pytest.mark.parametrize("odd", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d,bs,H,G", [(128, 16, 2, 4), (64, 32, 3, 7), (128, 32, 1, 8), (64, 16, 2, 2)])
def test_sparse_decode_beside_a_head_that_is_not_finite(pa, odd, d, bs, H, G):  # noqa: F811
    b, vc, vvals = batch(5, [300, 40, 1, 700], H, G, d, bs)
    tables, lens = chosen(b, b.rng, 4, 12)
    others, _ = heads_beside(b, G, odd)
    scale = 1 / math.sqrt(d)
    out = sparse(pa, b, vc, tables, lens, scale, KS, VS)
    b.q[~torch.isfinite(b.q)] = 0
    compare(b, vvals, out, tables, lens, scale, others)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("d,bs,H,G", [(128, 16, 2, 4), (64, 32, 3, 7), (128, 32, 1, 8), (64, 16, 2, 2)])
def test_sparse_decode_of_heads_of_other_magnitudes(pa, d, bs, H, G):  # noqa: F811
    b, vc, vvals = batch(6, [300, 40, 1, 700], H, G, d, bs)
    tables, lens = chosen(b, b.rng, 4, 12)
    for r in range(4):  # (a block twice in a table would give the largest logit twice)
        for h in range(H):
            n = -(-int(lens[r, h]) // bs)
            tables[r, h, :n] = b.rng.permutation(b.NB)[:n]
    others, large = heads_beside(b, G, 2.0 ** 40)
    scale = 1 / math.sqrt(d)
    assert min(gaps(b, tables, lens, scale, large, G)) > 2.0 ** 30
    out = sparse(pa, b, vc, tables, lens, scale, KS, VS)
    compare(b, vvals, out, tables, lens, scale, others + large)
    assert pa.pa_device_errors() == 0
