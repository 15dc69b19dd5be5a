"""How many bits of P the sparse decode keeps, 16-bit and FP8 caches: outputs that are
small beside A = sum_j p_j |v_j|, because the values cancel, show the error of P
that an output's own rounding hides otherwise.

Queries and keys have one element each, on a grid of four bits, and logits are
their product: exact.  In units of A, p_j is off by 2^-21 (the logit in base 2, below
48 for the tokens that count for nothing and 9 for the others, and the exponential's
2^-22), in two 16-bit parts by 2^-18 at most (bf16, two roundings of 8 bits), the
sums of at most 10 products of 16 tokens each by 2^-18, row sums, rescaling and
joins by 2^-19: 2^-16 for all of it.  P in one part, of 11 bits even, is off by more:
the test makes sure of that for its inputs."""
import numpy as np
import pytest
import torch

import oracle
import oracle.sparse as S
from test_gpu_fp4 import TYPES, dev, f64, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu
KEYS = [0.0, -0.25, -0.5, -0.75, -1.5, -3.0, -4.5, -6.0]  # the last four give values to cancel what is left
FAR = -30.0


def stored(x, kv, dtype):
    """(cache, its values in 64 bits)"""
    if kv == "fp8":
        codes = oracle.e4m3_from_f32(x.astype(np.float32))
        return dev(codes), oracle.e4m3_to_f64(codes).reshape(x.shape)
    t = torch.from_numpy(x).to(TYPES[dtype])
    return t.cuda(), t.double().numpy()


def problem(rng, R, H, bs, d, n, kv, dtype):
    """A pool whose blocks each row and head has for itself, with n tokens."""
    per = -(-n // bs)
    tables = rng.permutation(R * H * per).reshape(R, H, per).astype(np.int32)
    k, v = np.zeros((R * H * per, H, bs, d)), np.zeros((R * H * per, H, bs, d))
    for r in range(R):
        for h in range(H):
            at = rng.permutation(n)[: len(KEYS)]
            z = np.full(n, FAR)
            z[at] = KEYS
            x = rng.uniform(0.5, 1.0, (n, d)) * rng.choice([-1.0, 1.0], (n, d))
            p = np.exp(z)
            left = np.zeros(d)
            for i, j in enumerate(at):
                if i >= 4:
                    x[j] = stored(-left / p[j], kv, dtype)[1]
                left += p[j] * stored(x[j], kv, dtype)[1]
            for j in range(n):
                k[tables[r, h, j // bs], h, j % bs, (7 * h) % d] = z[j]
                v[tables[r, h, j // bs], h, j % bs] = x[j]
    return tables, np.full((R, H), n, np.int32), stored(k, kv, dtype), stored(v, kv, dtype)


@pytest.mark.parametrize("kv", ["16", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bs,d,H,G,R,n", [(16, 64, 2, 1, 3, 20), (32, 128, 1, 8, 2, 150), (16, 128, 2, 3, 1, 150)])
def test_cancelling_values(pa, kv, dtype, bs, d, H, G, R, n):  # noqa: F811
    rng = np.random.default_rng(n + d)
    tables, lens, (kc, kvals), (vc, vvals) = problem(rng, R, H, bs, d, n, kv, dtype)
    q = torch.zeros(R, H * G, d, dtype=TYPES[dtype])
    for h in range(H):
        q[:, h * G:(h + 1) * G, (7 * h) % d] = 1.0
    ref, mag = S.attend(q.double().numpy(), kvals, vvals, tables, lens, 1.0)
    tol = mag * 2.0 ** -16 + np.abs(ref) * torch.finfo(TYPES[dtype]).eps / 2 + 2.0 ** -25
    # P in one part of 11 bits would not do
    one = np.zeros_like(ref)
    for r in range(R):
        for h in range(H * G):
            ids = tables[r, h // G]
            K, V = (x[ids, h // G].reshape(-1, d)[:n] for x in (kvals, vvals))
            p = np.exp(K @ q[r, h].double().numpy())
            one[r, h] = p.astype(np.float16).astype(np.float64) @ V / p.sum()
    assert (np.abs(one - ref) > tol).mean() > 0.5
    out = torch.full_like(q, 7.0, device="cuda")
    pair = () if kv == "16" else (1.0, 1.0)
    getattr(pa, "pa_decode_sparse" + ("" if kv == "16" else "_fp8"))(out, q.cuda(), kc, vc, dev(tables), dev(lens), 1.0, *pair)
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), float((err / tol).max())
    assert pa.pa_device_errors() == 0
