"""FP8 prefill and shared-prefix decode with query rows of zeros and of tiny
numbers over caches of a small scale: a row's softmax scale is carried with the
power of two that its queries were scaled by, and the product may fall below the
smallest normal number.  Such rows attend (nearly) uniformly.

Tolerance: the probabilities are near 1 / n, P in fp16 is off by 2^-11 of each
and the row sum is of the unrounded ones, so 2^-11 of sum_j p_j |v_j|; the fp32
sums are below 2^-12 of it; the output is rounded by half a bf16 step, 2^-8.
"""
import numpy as np
import pytest
import torch

from test_gpu_fp4 import dev, f64, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu
ROWS = [0.0, 2.0 ** -110, -2.0 ** -126, 1.0, 0.0]


def pool(seed, lens, H, bs, d, vs):
    rng = np.random.default_rng(seed)
    per = -(-np.asarray(lens) // bs)
    NB = int(per.sum()) + 1
    ids = rng.permutation(NB)
    tables = np.full((len(lens), int(per.max())), -1, np.int32)
    at = 0
    for i, n in enumerate(per):
        tables[i, :n] = ids[at:at + n]
        at += n
    kc, vc = (torch.from_numpy(rng.standard_normal((NB, H, bs, d))).to(torch.float8_e4m3fn)
              for _ in range(2))
    return rng, tables, kc, vc, kc.double().numpy(), vc.double().numpy() * vs


def queries(n, Hq, d, dtype=torch.bfloat16):
    at = np.resize(ROWS, n * Hq).reshape(n, Hq, 1)
    return torch.from_numpy(np.broadcast_to(at, (n, Hq, d)).copy()).to(dtype)


def attend(q, k, v, G, scale):
    """q [Hq, d] over k, v [H, n, d]: the output and sum_j p_j |v_j|."""
    out, A = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(q.shape[0]):
        z = k[h // G] @ q[h] * scale
        p = np.exp(z - z.max())
        p /= p.sum()
        out[h], A[h] = p @ v[h // G], p @ np.abs(v[h // G])
    return out, A


def check(got, ref, A):
    got = f64(got)
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2 ** -8) + A * (2.0 ** -11 + 2.0 ** -12) + 2.0 ** -24
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("q_len,G,d,bs", [(3, 4, 128, 16), (40, 2, 64, 32), (70, 4, 128, 32),
                                          (150, 2, 64, 16)])
@pytest.mark.parametrize("ks,dtype", [(2.0 ** -27, torch.bfloat16), (2.0 ** -60, torch.bfloat16),
                                      (2.0 ** -120, torch.bfloat16), (2.0 ** -148, torch.bfloat16),
                                      (2.0 ** -148, torch.float16)])
def test_prefill_fp8(pa, q_len, G, d, bs, ks, dtype):  # noqa: F811
    H, lens = 2, [q_len + 83, q_len]
    _, tables, kc, vc, k, v = pool(1, lens, H, bs, d, 0.5)
    q = queries(2 * q_len, H * G, d, dtype)
    out = torch.full_like(q, float("nan"), device="cuda")
    scale = 1 / np.sqrt(d)
    pa.pa_prefill_fp8(out, q.cuda(), dev(np.array([0, q_len, 2 * q_len], np.int32)),
                      kc.view(torch.uint8).cuda(), vc.view(torch.uint8).cuda(), dev(tables),
                      dev(np.array(lens, np.int32)), scale, ks, 0.5, q_len)
    ref, A = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(lens):
        K, V = (x[tables[i, :-(-n // bs)]].transpose(1, 0, 2, 3).reshape(H, -1, d) for x in (k, v))
        for t in range(q_len):
            m = n - q_len + t + 1
            r = i * q_len + t
            ref[r], A[r] = attend(f64(q[r]), K[:, :m], V[:, :m], G, scale * ks)
    check(out, ref, A)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("ks", [2.0 ** -27, 2.0 ** -120])
def test_shared_prefix_fp8(pa, ks):  # noqa: F811
    H, G, d, bs, shared, ps = 2, 4, 128, 16, 200, 64
    lens = np.array([260, 233, 300], np.int32)
    _, tables, kc, vc, k, v = pool(2, lens, H, bs, d, 0.5)
    tables[1:, :shared // bs] = tables[0, :shared // bs]
    q = queries(3, H * G, d)
    out = torch.full_like(q, float("nan"), device="cuda")
    scale = 1 / np.sqrt(d)
    pa.pa_decode_shared_prefix_fp8(
        out, q.cuda(), kc.view(torch.uint8).cuda(), vc.view(torch.uint8).cuda(), dev(tables),
        dev(lens), dev(np.array([0, 3], np.int32)), dev(np.full(3, shared // bs * bs, np.int32)), 3,
        scale, ks, 0.5, 300, ps)
    ref, A = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(lens):
        K, V = (x[tables[i, :-(-n // bs)]].transpose(1, 0, 2, 3).reshape(H, -1, d)[:, :n]
                for x in (k, v))
        ref[i], A[i] = attend(f64(q[i]), K, V, G, scale * ks)
    check(out, ref, A)
    assert pa.pa_device_errors() == 0
