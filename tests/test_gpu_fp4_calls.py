"""FP4 calls as a caller may make them: bounds that are loose, rows and table
entries behind the batch, blocks that sequences share, captured graphs that share
a workspace, arguments that are no tensors."""
import numpy as np
import pytest
import torch

import oracle.fp4 as F
from test_gpu_fp4 import Batch, dev, f64, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu


def prefill(pa, b, most, extra=0):  # noqa: F811
    """b's prefill with a bound of ``most`` and ``extra`` rows behind the last
    sequence, which must stay as they were."""
    q = torch.cat([b.q, torch.full((extra, *b.q.shape[1:]), float("nan"), dtype=b.q.dtype)])
    out = torch.full_like(q, 7.0, device="cuda")
    kc, vc, bt, cl = b.gpu()
    pa.pa_prefill_fp4(out, q.cuda(), dev(b.start), kc, vc, bt, cl, b.scale, b.ks, b.vs, most)
    n = b.q.shape[0]
    assert (out[n:] == 7).all()
    b.check(out[:n])
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("most", [3, 6, 7, 16, 17, 100, 5000, 2 ** 22])
@pytest.mark.parametrize("n", [3, 160])
def test_prefill_under_a_loose_bound_with_rows_behind_the_batch(pa, most, n):  # noqa: F811
    """max_q_len alone picks the kernel; every kernel takes shorter chunks, empty ones among them."""
    rng = np.random.default_rng(n)
    q_lens = rng.integers(0, 4, n)
    q_lens[0] = q_lens[-1] = 0
    q_lens[1] = 3
    lens = q_lens + rng.integers(0, 80, n)
    lens[0], lens[1] = 0, 700
    b = Batch(1, lens, 2, 4, 128, 16, "bf16", ks=0.5, q_lens=q_lens)
    prefill(pa, b, most, extra=5)


@pytest.mark.parametrize("beyond", [-1, -2 ** 31, 2 ** 31 - 1])
def test_table_entries_past_the_contexts_are_not_looked_at(pa, beyond):  # noqa: F811
    for q_lens in (None, [5, 5, 5], [60, 60, 60]):
        b = Batch(2, [200, 61, 130], 2, 4, 128, 16, "fp16", q_lens=q_lens)
        b.tables = np.concatenate([b.tables, np.zeros((3, 60), np.int32)], 1)
        used = -(-b.lens // b.bs)
        for i, n in enumerate(used):
            b.tables[i, n:] = beyond
        if q_lens is None:
            for ps in (0, 32, 64):
                b.check(b.decode(pa, ps))
        else:
            b.check(b.prefill(pa))
        assert pa.pa_device_errors() == 0


def test_blocks_shared_by_sequences_and_within_one(pa):  # noqa: F811
    for q_lens in (None, [4, 4, 4], [70, 70, 70]):
        b = Batch(3, [256, 256, 256], 2, 4, 64, 16, "fp16", q_lens=q_lens)
        b.tables[1] = b.tables[0]
        b.tables[2, 1:16:2] = b.tables[2, 0:16:2]
        if q_lens is None:
            for ps in (0, 16, 48):
                b.check(b.decode(pa, ps))
        else:
            b.check(b.prefill(pa))
    assert pa.pa_device_errors() == 0


def test_two_captured_graphs_share_a_workspace(pa):  # noqa: F811
    """Replayed in turn on one stream, with new queries in place each time."""
    a = Batch(4, [900, 1500, 3], 2, 4, 128, 16, "fp16")
    b = Batch(5, [700, 20], 1, 8, 64, 32, "bf16")
    ws = pa.new_decode_workspace(3, 8, 128, 1500, 16)
    runs = []
    for x, ps in ((a, 64), (b, 128), (a, 16)):
        kc, vc, bt, cl = x.gpu()
        q, out = x.q.cuda(), torch.zeros_like(x.q, device="cuda")

        def call(x=x, ps=ps, q=q, out=out, kc=kc, vc=vc, bt=bt, cl=cl):
            pa.pa_decode_fp4(out, q, kc, vc, bt, cl, x.scale, x.ks, x.vs, int(x.lens.max()), ps, ws)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((x, q, out, g))
    rng = np.random.default_rng(6)
    for _ in range(2):
        for x, q, out, g in runs:
            x.q = torch.from_numpy(rng.standard_normal(x.q.shape)).to(x.q.dtype)
            q.copy_(x.q)
            out.zero_()
            g.replay()
            x.check(out)
    assert pa.pa_device_errors() == 0
    assert not ws[:pa.DECODE_COUNTER_BYTES].any()


def test_one_tensor_as_key_and_value(pa):  # noqa: F811
    d, bs, H = 128, 16, 2
    x = torch.from_numpy(np.random.default_rng(7).standard_normal((20, H, d))).half()
    want = [np.zeros((2, H, bs * d * 9 // 16), np.uint8) for _ in range(2)]
    slots = np.arange(3, 23)
    F.reshape_and_cache(x.float().numpy(), x.float().numpy(), *want, slots, bs, 1.0, 0.5)
    kc, vc = pa.new_fp4_cache(2, H, bs, d), pa.new_fp4_cache(2, H, bs, d)
    xd = x.cuda()
    pa.pa_reshape_and_cache_fp4(xd, xd, kc, vc, dev(slots), 1.0, 0.5)
    assert np.array_equal(kc.cpu().numpy(), want[0]) and np.array_equal(vc.cpu().numpy(), want[1])
    back = [torch.zeros_like(xd) for _ in range(2)]
    pa.pa_gather_cache_fp4(*back, kc, vc, dev(slots), 1.0, 0.5)
    for got, c, g in zip(back, want, (1.0, 0.5)):
        v = F.values(c, bs, d, g)[slots // bs, :, slots % bs]
        assert np.array_equal(f64(got), v)


def test_what_is_no_tensor_is_named(pa):  # noqa: F811
    """A missing or foreign argument is a ValueError that names what is wanted."""
    kc = pa.new_fp4_cache(4, 2, 16, 64)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda")
    bt = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    cl = torch.ones(3, dtype=torch.int32, device="cuda")
    sm = torch.zeros(3, dtype=torch.int64, device="cuda")
    qs = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    for bad in (None, 3, np.zeros((3, 2, 64), np.float16)):
        for f in (pa.pa_reshape_and_cache_fp4, pa.pa_gather_cache_fp4):
            args = [k, k, kc, kc, sm]
            for i in range(5):
                with pytest.raises(ValueError):
                    f(*args[:i], bad, *args[i + 1:])
        for f, args, tail in ((pa.pa_decode_fp4, [q, q, kc, kc, bt, cl], (0.1, 1.0, 1.0, 10)),
                              (pa.pa_prefill_fp4, [q, q, qs, kc, kc, bt, cl], (0.1, 1.0, 1.0, 1))):
            for i in range(len(args)):
                with pytest.raises(ValueError):
                    f(*args[:i], bad, *args[i + 1:], *tail)
    assert pa.pa_device_errors() == 0
