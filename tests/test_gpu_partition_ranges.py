"""Split-context decode with a max_context_len that bounds nothing (2^31 - 1): the
partitions past a table's end lie around 2^31 tokens, and contexts that fit one
partition must come out as ever.

Against 64 bits, with the tolerance of test_gpu_fp4.py, which covers the 16-bit
and FP8 caches too: P has at least 11 bits there, the sums are fp32 alike.
"""
import numpy as np
import pytest
import torch

import oracle.fp4 as F
from test_gpu_fp4 import Batch, dev, f64, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu
ANY = 2 ** 31 - 1
SIZES = [0, 2 ** 20, 2 ** 30, 2 ** 31 - 16]


@pytest.mark.parametrize("ps", SIZES)
@pytest.mark.parametrize("d,bs,dtype", [(128, 16, "fp16"), (64, 32, "bf16")])
def test_fp4(pa, ps, d, bs, dtype):  # noqa: F811
    b = Batch(91, [700, 0, 1, 333], 1, 4, d, bs, dtype)
    out = b.decode(pa, ps, maxctx=ANY)
    b.check(out)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("ps", SIZES)
@pytest.mark.parametrize("kv", ["fp16", "bf16", "fp8"])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32)])
def test_16_bit_and_fp8(pa, ps, kv, d, bs):  # noqa: F811
    rng = np.random.default_rng(92)
    t = torch.bfloat16 if kv == "bf16" else torch.float16
    lens, NB = np.array([700, 0, 1, 333], np.int32), 80
    per = -(-lens // bs)
    tables = np.full((4, int(per.max())), -1, np.int32)
    ids = rng.permutation(NB)
    for i, n in enumerate(per):
        tables[i, :n] = ids[per[:i].sum():per[:i].sum() + n]
    kv_type = torch.float8_e4m3fn if kv == "fp8" else t
    kc, vc = (torch.from_numpy(rng.standard_normal((NB, 1, bs, d))).to(kv_type) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((4, 4, d))).to(t)
    k, v = (x.double().numpy() for x in (kc, vc))
    ref = F.decode(f64(q), k, v, tables, lens, d ** -0.5)
    A = F.decode(f64(q), k, np.abs(v), tables, lens, d ** -0.5)
    out = torch.full_like(q, float("nan"), device="cuda")
    if kv == "fp8":
        pa.pa_decode_fp8(out, q.cuda(), kc.view(torch.uint8).cuda(), vc.view(torch.uint8).cuda(),
                         dev(tables), dev(lens), d ** -0.5, 1.0, 1.0, ANY, ps)
    else:
        pa.pa_decode(out, q.cuda(), kc.cuda(), vc.cuda(), dev(tables), dev(lens), d ** -0.5, ANY, ps)
    tol = torch.finfo(t).eps / 2 * np.abs(ref) * (1 + 2 ** -8) + A * (2 ** -11 + 2 ** -12) + 2.0 ** -24
    ok = np.abs(f64(out) - ref) <= tol
    assert ok.all()
    assert pa.pa_device_errors() == 0
