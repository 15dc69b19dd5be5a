"""bf16 queries over FP8 caches in the dense decode call: what one head of a group
holds does not reach the others (test_gpu_fp8_head_scales.py has the reasons and the
tolerances)."""
import math

import numpy as np
import pytest
import torch

from test_gpu_fp4 import dev, pa  # noqa: F401  (pa is the fixture)
from test_gpu_fp8_head_scales import KS, VS, batch, compare, gaps, heads_beside

pytestmark = pytest.mark.gpu


def dense(pa, b, vc, scale, part):  # noqa: F811
    out, most = torch.full_like(b.q, 7.0, device="cuda"), int(b.lens.max())
    pa.pa_decode_fp8(out, b.q.cuda(), b.kc, vc, dev(b.tables), dev(b.lens), scale, KS, VS, most, part)
    return out, np.repeat(b.tables[:, None], b.H, 1), np.repeat(b.lens[:, None], b.H, 1)


@pytest.mark.parametrize("part", [0, 128])
@pytest.mark.parametrize("odd", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d,bs,H,G", [(128, 16, 2, 4), (64, 32, 3, 7), (128, 32, 1, 8), (64, 16, 2, 2)])
def test_decode_beside_a_head_that_is_not_finite(pa, odd, d, bs, H, G, part):  # noqa: F811
    b, vc, vvals = batch(7, [300, 40, 1, 700], H, G, d, bs)
    others, _ = heads_beside(b, G, odd)
    out, tables, lens = dense(pa, b, vc, 1 / math.sqrt(d), part)
    b.q[~torch.isfinite(b.q)] = 0
    compare(b, vvals, out, tables, lens, 1 / math.sqrt(d), others)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("part", [0, 128])
@pytest.mark.parametrize("d,bs,H,G", [(128, 16, 2, 4), (64, 32, 3, 7), (128, 32, 1, 8), (64, 16, 2, 2)])
def test_decode_of_heads_of_other_magnitudes(pa, d, bs, H, G, part):  # noqa: F811
    b, vc, vvals = batch(8, [300, 40, 1, 700], H, G, d, bs)
    others, large = heads_beside(b, G, 2.0 ** 40)
    scale = 1 / math.sqrt(d)
    out, tables, lens = dense(pa, b, vc, scale, part)
    assert min(gaps(b, tables, lens, scale, large, G)) > 2.0 ** 30
    compare(b, vvals, out, tables, lens, scale, others + large)
    assert pa.pa_device_errors() == 0
