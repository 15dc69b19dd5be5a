"""FP4 attention where logits are far from the ordinary: cache scales at the ends
of their range, queries of zeros, of very large and of very small numbers.

Keys are constant rows here (one E2M1 value in every dimension, scale 1), so a
logit is (the query's sum) x value x k_scale x scale, and what decides is
arithmetic that is exact: a query's sum and its products with the seven values
have few bits.  Logits that differ lie either far apart (the larger takes all)
or within the softmax's reach; equal keys tie exactly.  The tolerance is that of
test_gpu_fp4.py: P in fp16, and the rest in fp32.
"""
import numpy as np
import pytest
import torch

import oracle.fp4 as F
from test_gpu_fp4 import Batch, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu

# (sequences, KV heads, group, tokens of a chunk (0: decode), partition size)
PATHS = {
    "decode, clusters": (3, 2, 4, 0, 0),
    "decode, one CTA a row": (330, 2, 3, 0, 0),
    "decode, joined by the last CTA": (3, 2, 8, 0, 48),
    "decode, joined by the reduction": (3, 2, 4, 0, 16),
    "prefill, 12 rows": (3, 2, 4, 3, 0),
    "prefill, 24 rows, one CTA each": (330, 2, 2, 12, 0),
    "prefill, 64-row tiles": (160, 2, 4, 12, 0),
    "prefill, two tiles in clusters": (3, 2, 4, 80, 0),
    "prefill, two tiles": (80, 2, 4, 50, 0),
}


def constant_keys(path, seed, d, bs, dtype, ks, rows):
    """A batch whose keys are constant rows and whose query rows are constants
    out of ``rows``, in turn."""
    n, H, G, q, ps = PATHS[path]
    rng = np.random.default_rng(seed)
    lens = rng.integers(max(q, 1), q + 120, n)
    lens[0], lens[-1] = q + 600, max(q, 1)
    b = Batch(seed, lens, H, G, d, bs, dtype, ks=ks, vs=0.5,
              q_lens=[q] * n if q else None)
    codes, scales = F.views(b.kc, bs, d)
    pick = rng.integers(1, 8, codes.shape[:3]).astype(np.uint8)
    codes[...] = (pick * 17)[..., None]
    scales[...] = np.where(scales == 0x7F, 0x7F, 0x38)
    at = np.resize(rows, b.q.shape[0] * b.q.shape[1]).reshape(*b.q.shape[:2])
    b.q = torch.from_numpy(np.repeat(at[..., None], d, axis=2)).to(b.q.dtype)
    return b, ps


def run(pa, b, ps):
    out = b.decode(pa, ps) if b.start is None else b.prefill(pa)
    b.check(out)
    assert pa.pa_device_errors() == 0
    return out


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("ks", [2.0 ** -20, 2.0 ** -40, 2.0 ** -100])
@pytest.mark.parametrize("d,bs,dtype", [(128, 16, "fp16"), (64, 32, "bf16")])
def test_small_scales_with_rows_of_zeros(pa, path, ks, d, bs, dtype):  # noqa: F811
    b, ps = constant_keys(path, 81, d, bs, dtype, ks, [1.0, -1.0, 0.0, -3.0, 0.5])
    run(pa, b, ps)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("ks", [2.0 ** -27, 2.0 ** -100, 2.0 ** 90])
def test_tiny_bf16_queries_at_the_ends_of_the_scales(pa, path, ks):  # noqa: F811
    b, ps = constant_keys(path, 83, 128, 16, "bf16", ks, [2.0 ** -110, 0.0, -2.0 ** -126, 1.0])
    run(pa, b, ps)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("ks", [2.0 ** 100, 2.0 ** 60, 2.0 ** 28, 2.0 ** 10])
@pytest.mark.parametrize("d,bs,dtype", [(128, 16, "fp16"), (64, 32, "bf16")])
def test_large_scales(pa, path, ks, d, bs, dtype):  # noqa: F811
    """Positive and negative logits up to 2^112, rows of zeros (uniform), and
    rows of ordinary queries, side by side."""
    b, ps = constant_keys(path, 81, d, bs, dtype, ks, [1.0, -1.0, 0.0, -3.0, 0.5])
    run(pa, b, ps)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("rows", [[1e30, -1e30, 1.0, 0.0], [-1e30], [2.0 ** -110, 0.0, -2.0 ** -120],
                                  [2.0 ** 20, -2.0 ** 20, 1e10]])
@pytest.mark.parametrize("d,bs", [(128, 32), (64, 16)])
def test_bf16_queries_of_any_magnitude(pa, path, rows, d, bs):  # noqa: F811
    b, ps = constant_keys(path, 82, d, bs, "bf16", 1.0, rows)
    run(pa, b, ps)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("d,bs,dtype", [(128, 16, "fp16"), (64, 16, "bf16")])
def test_a_softmax_on_top_of_a_large_common_logit(pa, path, sign, d, bs, dtype):  # noqa: F811
    """Half of the dimensions add the same 32,000 or so to every logit, 16 others
    what tells the keys apart: their sums are exact in fp32 (multiples of 0.5
    below 2^18), so the differences must come out as if the common part were not."""
    b, ps = constant_keys(path, 84, d, bs, dtype, 1.0, [1.0])
    rng = np.random.default_rng(85)
    codes, scales = F.views(b.kc, bs, d)
    codes[..., : d // 4] = 0x77 if sign > 0 else 0xFF              # 6 or -6 in the first half
    codes[..., d // 4:] = rng.integers(0, 256, codes[..., d // 4:].shape)
    q = np.zeros(d)
    q[: d // 2] = 512 if d == 128 else 1024
    q[d // 2: d // 2 + 16] = 1
    b.q[...] = torch.from_numpy(q).to(b.q.dtype)
    run(pa, b, ps)


@pytest.mark.parametrize("path", [p for p in PATHS if p.startswith("decode")])
@pytest.mark.parametrize("scale", [-0.125, 0.0, -1e-30])
def test_decode_takes_scales_of_any_sign(pa, path, scale):  # noqa: F811
    for dtype in ("fp16", "bf16"):
        b, ps = constant_keys(path, 86, 64, 16, dtype, 1.0, [1.0, -2.0, 0.0])
        b.scale = scale
        run(pa, b, ps)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("vs", [2.0 ** 100, 2.0 ** -100])
@pytest.mark.parametrize("ks", [2.0 ** 100, 2.0 ** 40, 1.0])
def test_v_scales_at_the_ends_of_their_range(pa, path, vs, ks):  # noqa: F811
    """bf16 holds the outputs; they are compared after the (exact) product with 1 / vs."""
    b, ps = constant_keys(path, 87, 128, 16, "bf16", ks, [1.0, -1.0, 0.0, -3.0])
    b.vs = vs
    out = b.decode(pa, ps) if b.start is None else b.prefill(pa)
    b.vs = 1.0
    b.check(out.double() / vs)
    assert pa.pa_device_errors() == 0
