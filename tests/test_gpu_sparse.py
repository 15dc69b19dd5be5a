"""GPU parity of key bounds, block selection and sparse decode with the 64-bit
reference in ``oracle/sparse.py``.

Bounds, scales, tables and lengths are exact: integers, powers of two, and scores
of two fp32 roundings that the reference makes, too.

Attention, per output element, with A = sum_j p_j |v_j| of the reference: the
logits are sums of at most 128 products in fp32 (off by at most 128 * 2^-24 of
sum |q k| scale < 32 for these inputs: 2^-12 in units of a logit, and 2^-11 A where
every logit is off by that in the worst direction for numerator and
denominator), P in 16 bits or more (FP4: 2^-11 of each p_j), the running sums
2^-14 A and the output eps / 2 of its value."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.fp4 as F
import oracle.sparse as S
from test_gpu_fp4 import TYPES, dev, f64, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu
END = {"16": "", "fp8": "_fp8", "fp4": "_fp4"}


def pool(rng, x, kv, dtype, bs, d, g=1.0):
    """x [NB, H, bs, d] as a cache: (device tensor, the values without the cache's scale in 64 bits)."""
    if kv == "16":
        t = torch.from_numpy(x).to(TYPES[dtype])
        return t.cuda(), t.double().numpy()
    if kv == "fp8":
        codes = oracle.e4m3_from_f32((x / g).astype(np.float32))
        return dev(codes), oracle.e4m3_to_f64(codes).reshape(x.shape)
    codes, scales = F.quantise(x.astype(np.float32), g)
    n = bs * d // 2
    raw = np.concatenate([codes.reshape(*x.shape[:2], n), scales.reshape(*x.shape[:2], -1)], 2)
    return dev(raw), F.values(raw, bs, d, 1.0)


class Batch:
    """Contexts in blocks scattered over a pool; q_lens: rows of each sequence (None: one, without query_start)."""

    def __init__(self, seed, lens, Hkv, G, d, bs, dtype, kv="16", q_lens=None, extra=3, mean=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.bs, self.d, self.kv, self.dtype = np.asarray(lens, np.int32), bs, d, kv, dtype
        per = -(-self.lens // bs)
        NB = int(per.sum()) + extra
        ids = rng.permutation(NB)
        self.tables = np.full((len(lens), max(1, int(per.max()))), -1, np.int32)
        for i, n in enumerate(per):
            self.tables[i, :n] = ids[per[:i].sum():per[:i].sum() + n]
        x = rng.standard_normal((NB, Hkv, bs, d)) + mean * rng.standard_normal((1, Hkv, 1, d))
        self.kc, self.kvals = pool(rng, x, kv, dtype, bs, d)
        self.H, self.NB = Hkv, NB
        self.q_lens = None if q_lens is None else np.asarray(q_lens, np.int32)
        rows = len(lens) if q_lens is None else int(np.sum(q_lens))
        self.q = torch.from_numpy(rng.standard_normal((rows, Hkv * G, d))).to(TYPES[dtype])
        if q_lens is None:
            self.seqs, self.seen, self.start = np.arange(rows), self.lens.copy(), None
        else:
            self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
            self.seqs = np.repeat(np.arange(len(lens)), q_lens)
            self.seen = np.array([n - q + t + 1 for n, q in zip(lens, q_lens) for t in range(q)], np.int32)
        self.bounds, self.scales = np.zeros((NB, Hkv, 2, d), np.int8), np.zeros((NB, Hkv), np.float32)

    def all_bounds(self):
        S.update_bounds(self.bounds, self.scales, self.kvals, self.tables, self.lens, self.lens)

    def rows_args(self):
        return (None, 1) if self.start is None else (dev(self.start), max(1, int(self.q_lens.max())))

    def select(self, pa, keep, sink, recent, q=None, most=None, rows=None):  # noqa: F811
        q = self.q.cuda() if q is None else q
        R = q.shape[0]
        t = torch.full((R, self.H, keep), 77, dtype=torch.int32, device="cuda")
        n = torch.full((R, self.H), 77, dtype=torch.int32, device="cuda")
        pa.pa_select_blocks(t, n, q, dev(self.bounds), dev(self.scales), dev(self.tables), dev(self.lens),
                            self.bs, int(self.lens.max()) if most is None else most, sink, recent,
                            *self.rows_args())
        return t.cpu().numpy(), n.cpu().numpy()

    def want(self, keep, sink, recent, q=None):
        q = self.q if q is None else q
        return S.select(q.double().numpy(), self.bounds, self.scales, self.tables, self.seqs, self.seen,
                        self.bs, keep, sink, recent)


# ----------------------------------------------------------------------- bounds

@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
@pytest.mark.parametrize("d,bs,dtype,H", [(64, 16, "fp16", 1), (128, 16, "bf16", 3), (64, 32, "bf16", 8),
                                          (128, 32, "fp16", 2)])
@pytest.mark.parametrize("q_lens", [None, [1, 0, 5, 16, 1, 33, 100, 0], [16, 17, 5, 16, 1, 1, 99, 0]])
def test_bounds(pa, kv, d, bs, dtype, H, q_lens):  # noqa: F811
    lens = [16, 17, 5, 32, 1, 33, 100, 0]
    b = Batch(1, lens, H, 1, d, bs, dtype, kv, q_lens)
    q = [min(1, n) for n in lens] if q_lens is None else q_lens
    want, scales = np.full_like(b.bounds, 9), np.full_like(b.scales, 9)
    S.update_bounds(want, scales, b.kvals, b.tables, b.lens, q)
    got, gs = torch.full(want.shape, 9, dtype=torch.int8, device="cuda"), dev(np.full_like(scales, 9))
    getattr(pa, "pa_update_key_bounds" + END[kv])(got, gs, b.kc, dev(b.tables), dev(b.lens), *b.rows_args())
    assert np.array_equal(gs.cpu().numpy(), scales)
    assert np.array_equal(got.cpu().numpy(), want)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_bounds_of_odd_values(pa, dtype, d):  # noqa: F811
    """Infinities, NaN, zeros, the borders of the powers of two, the smallest and
    largest numbers of the type; and NaN in rows past the context."""
    info = torch.finfo(TYPES[dtype])
    tops = [0.0, -0.0, 127.0, -127.0, 127.5, 128.0, -254.0, 255.0, info.max, -info.max, info.smallest_normal,
            info.smallest_normal / 4, -info.smallest_normal, math.inf, -math.inf, math.nan, 1.0, 0.9921875, 1 / 128]
    n, bs = len(tops), 16
    x = np.zeros((n, 2, bs, d))
    rng = np.random.default_rng(2)
    for i, a in enumerate(tops):
        if np.isfinite(a) and a:
            x[i] = rng.uniform(-1, 1, (2, bs, d)) * a / 2
        x[i, :, i % 5, (7 * i) % d] = a
    x[:, :, 5:] = math.nan
    t = torch.from_numpy(x).to(TYPES[dtype])
    b, s = np.zeros((n, 2, 2, d), np.int8), np.zeros((n, 2), np.float32)
    tables, lens = np.arange(n, dtype=np.int32)[:, None], np.full(n, 5, np.int32)
    S.update_bounds(b, s, t.double().numpy(), tables, lens, [1] * n)
    gb, gs = pa.new_key_bounds(n, 2, d)
    pa.pa_update_key_bounds(gb, gs, t.cuda(), dev(tables), dev(lens))
    assert np.array_equal(gs.cpu().numpy(), s) and np.array_equal(gb.cpu().numpy(), b)
    assert np.isinf(s[13:16]).all() and (s[:2] == 0).all()


@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32)])
def test_bounds_of_tiny_keys_beside_large_ones(pa, d, bs):  # noqa: F811
    """Whatever is above zero has a bound above zero: keys whose quotient by the scale is below every fp32 number."""
    x = np.zeros((3, 2, bs, d))
    tiny = 2.0 ** np.arange(-133, -60)  # from bf16's smallest number on
    rng = np.random.default_rng(77)
    x[...] = rng.choice(tiny, x.shape) * rng.choice([-1.0, 0.0, 1.0], x.shape)
    x[:, :, :, 5] = np.abs(x[:, :, :, 5]) + tiny[0]
    x[:, :, :, 6] = -np.abs(x[:, :, :, 6]) - tiny[0]
    x[0, :, 3, 9], x[1, :, 0, 9], x[2, :, bs - 1, 9] = 2.0 ** 127, -2.0 ** 120, 1.9 * 2.0 ** 126
    t = torch.from_numpy(x).bfloat16()
    tables, lens = np.arange(3, dtype=np.int32)[:, None], np.full(3, bs, np.int32)
    b, s = np.zeros((3, 2, 2, d), np.int8), np.zeros((3, 2), np.float32)
    S.update_bounds(b, s, t.double().numpy(), tables, lens, [bs] * 3)
    gb, gs = pa.new_key_bounds(3, 2, d)
    pa.pa_update_key_bounds(gb, gs, t.cuda(), dev(tables), dev(lens))
    assert np.array_equal(gs.cpu().numpy(), s) and np.array_equal(gb.cpu().numpy(), b)
    assert (b[:, :, :, 5] == [1, 0]).all() and (b[:, :, :, 6] == [0, -1]).all()


@pytest.mark.parametrize("kv", ["fp8", "fp4"])
def test_bounds_of_nan_codes(pa, kv):  # noqa: F811
    """A NaN among a block's tokens gives the infinite scale; past the context it does not count."""
    b = Batch(50, [20, 20, 20], 2, 1, 64, 16, "fp16", kv)
    x = b.rng.standard_normal((b.NB, 2, 16, 64))
    x[b.tables[0, 1], 0, 3, 40] = math.nan   # token 19 of sequence 0: the newest
    x[b.tables[1, 1], 1, 4:, :] = math.nan   # past sequence 1's context
    b.kc, b.kvals = pool(b.rng, x, kv, "fp16", 16, 64)
    want, s = np.zeros_like(b.bounds), np.zeros_like(b.scales)
    S.update_bounds(want, s, b.kvals, b.tables, b.lens, [1, 1, 1])
    gb, gs = pa.new_key_bounds(b.NB, 2, 64)
    getattr(pa, "pa_update_key_bounds" + END[kv])(gb, gs, b.kc, dev(b.tables), dev(b.lens))
    assert np.array_equal(gb.cpu().numpy(), want) and np.array_equal(gs.cpu().numpy(), s)
    assert np.isinf(s[b.tables[0, 1], 0]) and np.isfinite(s[b.tables[1, 1]]).all()


def test_bounds_of_bad_lengths_and_blocks(pa):  # noqa: F811
    b = Batch(3, [40, 20, 33, 7], 2, 1, 64, 16, "fp16", q_lens=[3, 3, 3, 3])
    want, s = np.zeros_like(b.bounds), np.zeros_like(b.scales)
    S.update_bounds(want, s, b.kvals, b.tables, b.lens, [3, 0, 0, 3])
    for lens, start, flag in (
            ([40, -1, 2, 7], b.start, pa.DEVERR_BAD_LEN), ([40, 2, 1 << 20, 7], b.start, pa.DEVERR_BAD_LEN)):
        gb, gs = pa.new_key_bounds(b.NB, 2, 64)
        pa.pa_update_key_bounds(gb, gs, b.kc, dev(b.tables), dev(np.array(lens, np.int32)), dev(start), 3)
        assert pa.pa_device_errors() == flag
        assert np.array_equal(gb.cpu().numpy(), want) and np.array_equal(gs.cpu().numpy(), s)
    tables = b.tables.copy()
    tables[1, 1], tables[2, 2] = -1, b.NB
    gb, gs = pa.new_key_bounds(b.NB, 2, 64)
    pa.pa_update_key_bounds(gb, gs, b.kc, dev(tables), dev(b.lens), dev(b.start), 3)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_BLOCK
    want, s = np.zeros_like(b.bounds), np.zeros_like(b.scales)
    S.update_bounds(want, s, b.kvals, tables, b.lens, [3, 3, 3, 3])
    assert np.array_equal(gb.cpu().numpy(), want) and np.array_equal(gs.cpu().numpy(), s)


# -------------------------------------------------------------------- selection

@pytest.mark.parametrize("d,bs,dtype,H,G", [(64, 16, "fp16", 4, 1), (128, 16, "bf16", 2, 4),
                                            (128, 32, "fp16", 1, 8), (64, 32, "bf16", 3, 7)])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 0, 1), (6, 1, 2), (6, 6, 0), (6, 2, 4), (33, 4, 8),
                                              (200, 1, 1)])
def test_select(pa, d, bs, dtype, H, G, keep, sink, recent):  # noqa: F811
    b = Batch(keep + d, [0, 1, bs, bs + 1, 6 * bs, 6 * bs + 1, 7 * bs, 1500, 3001, 40 * bs - 1], H, G, d, bs, dtype)
    b.all_bounds()
    t, n = b.select(pa, keep, sink, recent)
    wt, wn = b.want(keep, sink, recent)
    assert np.array_equal(t, wt) and np.array_equal(n, wn)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("keep,sink,recent", [(3, 1, 1), (8, 0, 0), (20, 2, 2)])
@pytest.mark.parametrize("G,dtype", [(1, "bf16"), (4, "fp16")])
def test_select_for_chunks(pa, keep, sink, recent, G, dtype):  # noqa: F811
    """Several rows a sequence, none among them; each sees the tokens up to its own."""
    q_lens = [1, 5, 0, 8, 37, 2]
    b = Batch(4, [700, 5, 0, 16 * 25 + 3, 37, 2000], 2, G, 128, 16, dtype, q_lens=q_lens)
    b.all_bounds()
    t, n = b.select(pa, keep, sink, recent)
    wt, wn = b.want(keep, sink, recent)
    assert np.array_equal(t, wt) and np.array_equal(n, wn)
    # rows behind the last sequence, under a bound that is loose
    q = torch.cat([b.q, b.q[:3]]).cuda()
    b.q_lens[4] = 41
    t, n = b.select(pa, keep, sink, recent, q=q, most=1 << 18)
    assert np.array_equal(t[:-3], wt) and np.array_equal(n[:-3], wn)
    assert (t[-3:] == 77).all() and (n[-3:] == 77).all()
    b.q_lens[4] = 2 ** 31 - 1  # a bound far above what any context holds
    t, n = b.select(pa, keep, sink, recent, q=q)
    assert np.array_equal(t[:-3], wt) and np.array_equal(n[:-3], wn)
    assert pa.pa_device_errors() == 0


def test_no_rows(pa):  # noqa: F811
    """Sequences without new tokens alone, and no sequences."""
    b = Batch(42, [40, 0], 2, 2, 64, 16, "fp16", q_lens=[0, 0])
    b.all_bounds()
    for most in (0, 5, np.int64(5)):
        b.q_lens[0] = most
        t, n = b.select(pa, 2, 1, 1)
        assert t.shape == (0, 2, 2) and n.shape == (0, 2)
        pa.pa_update_key_bounds(*pa.new_key_bounds(b.NB, 2, 64), b.kc, dev(b.tables), dev(b.lens), dev(b.start), most)
    none = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda")
    t = torch.zeros(0, 2, 2, dtype=torch.int32, device="cuda")
    assert pa.pa_decode_sparse(none, none, b.kc, b.kc, t, t[..., 0], 0.1) is none
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(t, t[..., 0], none, dev(b.bounds), dev(b.scales), t[:, 0], lens, 16, 40)
    pa.pa_update_key_bounds(dev(b.bounds), dev(b.scales), b.kc, t[:, 0], lens)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("lens,keep", [([70000, 16, 33333], 128), ([16 * 9000], 1000), ([131072], 2), ([20001] * 3, 77)])
@pytest.mark.parametrize("bs,d", [(16, 128), (32, 64)])
def test_select_of_long_contexts(pa, lens, keep, bs, d):  # noqa: F811
    b = Batch(5, lens, 1, 4, d, bs, "bf16")
    b.bounds = b.rng.integers(-127, 128, b.bounds.shape).astype(np.int8)
    b.scales = np.exp2(b.rng.integers(-9, -3, b.scales.shape)).astype(np.float32)
    t, n = b.select(pa, keep, 1, 1)
    wt, wn = b.want(keep, 1, 1)
    assert np.array_equal(t, wt) and np.array_equal(n, wn)


@pytest.mark.parametrize("lens,q_lens,keep", [
    ([20000, 70, 30017], [5, 3, 4], 128), ([40000, 33, 17000, 0], [9, 1, 0, 0], 70), ([66000], [2], 500),
    ([16 * 1100 + 2] * 3, [4, 3, 8], 1100), ([70001] * 2, [1, 7], 9)])
@pytest.mark.parametrize("bs,d,G,dtype", [(16, 128, 4, "bf16"), (32, 64, 1, "fp16")])
def test_select_for_drafts_of_long_contexts(pa, lens, q_lens, keep, bs, d, G, dtype):  # noqa: F811
    b = Batch(23, lens, 2, G, d, bs, dtype, "16", q_lens)
    b.all_bounds()
    got, n = b.select(pa, keep, 1, 4)
    want, wn = b.want(keep, 1, 4)
    assert np.array_equal(got, want) and np.array_equal(n, wn)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("seqs,q", [(3, 3), (3, 7), (40, 3), (40, 7), (160, 4)])
@pytest.mark.parametrize("longest,bs", [(16 * 400 + 3, 16), (16 * 513, 16), (16 * 1024 - 9, 16), (32 * 700 + 1, 32)])
def test_select_for_drafts_of_many_and_few_sequences(pa, seqs, q, longest, bs):  # noqa: F811
    lens = [longest, longest - 1000] + [70 + 11 * i % 300 for i in range(seqs - 2)]
    b = Batch(29, lens, 2, 2, 64, bs, "bf16", "16", [1 + (i + q) % q for i in range(1, seqs)] + [q])
    b.all_bounds()
    got, n = b.select(pa, 9, 1, 2)
    want, wn = b.want(9, 1, 2)
    assert np.array_equal(got, want) and np.array_equal(n, wn)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("n,keep", [(3000, 600), (2000, 700), (8192, 128), (8192, 500), (5000, 90), (1500, 1499)])
@pytest.mark.parametrize("d", [64, 128])
def test_select_where_large_scores_are_neighbours(pa, n, keep, d):  # noqa: F811
    """Runs of blocks with nearly the same large scores, among many that are small or
    negative, and more blocks wanted than there are runs."""
    b = Batch(41, [16 * 3] * 3, 2, 2, d, 16, "bf16", extra=n)
    b.bounds = b.rng.integers(-20, 21, b.bounds.shape).astype(np.int8)
    b.bounds[:, :, 1] = np.minimum(b.bounds[:, :, 0], b.bounds[:, :, 1])
    b.scales[:] = 2.0 ** -4
    b.tables = np.stack([b.rng.permutation(b.NB)[:n] for _ in range(3)]).astype(np.int32)
    b.lens = b.seen = np.full(3, 16 * n - 5, np.int32)
    for r in range(3):
        for at in (0, n // 3, n - 300 if n > 1800 else n // 2):
            b.bounds[b.tables[r, at:at + 250], :, 0] = np.clip(
                b.bounds[b.tables[r, at:at + 250], :, 0].astype(int) + 100, -127, 127)
    for sink, recent in ((0, 0), (3, 5)):
        t, m = b.select(pa, keep, sink, recent)
        wt, wm = b.want(keep, sink, recent)
        assert np.array_equal(t, wt) and np.array_equal(m, wm)


@pytest.mark.parametrize("blocks,keep", [(49152, 300), (49151, 49000), (700, 699), (257, 8)])
def test_select_among_few_different_scores(pa, blocks, keep):  # noqa: F811
    """Blocks of one pool of 5 over and over: ties go to the first ones; up to the most candidates."""
    b = Batch(6, [16 * 5] * 2, 2, 2, 64, 16, "fp16", extra=0)
    b.all_bounds()
    b.tables = b.rng.integers(0, 5, (2, blocks)).astype(np.int32)
    b.lens = np.array([16 * blocks - 3, 16 * blocks // 2], np.int32)
    b.seen = b.lens.copy()
    for sink, recent in ((0, 0), (2, 1)):
        t, n = b.select(pa, keep, sink, recent)
        at = b.q.double().numpy()
        for r in range(2):
            m = -(-int(b.lens[r]) // 16)
            for h in range(2):
                s = S.scores(at[r].reshape(2, 2, 64)[h], b.bounds[:, h], b.scales[:, h])[b.tables[r, :m]].astype(np.float64)
                s[:sink] = s[m - recent:] = math.inf
                got = np.sort(np.lexsort((np.arange(m), -s))[:keep])
                assert np.array_equal(t[r, h, : len(got)], b.tables[r, got])
                assert (t[r, h, len(got):] == -1).all()
                assert n[r, h] == len(got) * 16 - (m * 16 - b.lens[r] if got[-1] == m - 1 else 0)


@pytest.mark.parametrize("lens", [[16 * 60] * 4, [16 * 1500] * 4])
@pytest.mark.parametrize("d", [64, 128])
def test_select_with_the_largest_sums(pa, lens, d):  # noqa: F811
    """Codes and weights at the ends of their ranges: 8 heads that add up to the
    largest weights, weights with full low bytes, codes of 127 and -127, with
    scores that differ by one."""
    b = Batch(40, [16 * 3] * 4, 1, 8, d, 16, "fp16", extra=80)
    b.bounds[:] = np.where(b.rng.random(b.bounds.shape) < 0.9, 127, -127)
    b.bounds[: b.NB // 2, :, 1] = -127
    b.bounds[:, :, :, 0] = b.rng.integers(-127, 128, b.bounds[:, :, :, 0].shape)
    b.scales[:] = 1
    blocks = -(-lens[0] // 16)
    b.tables = np.stack([b.rng.permutation(b.NB)[np.arange(blocks) % b.NB] for _ in lens]).astype(np.int32)
    b.lens = b.seen = np.asarray(lens, np.int32)
    q = np.zeros((4, 8, d))
    q[0] = 4095                             # weights of 32760
    q[1] = np.where(np.arange(d) % 2, 255, -1)  # low bytes of 255, high ones of -1
    q[1, 0, 3] = 4095
    q[2], q[2, :4], q[2, 0] = -4095, 4095, 1
    q[3] = b.rng.integers(-4095, 4096, (8, d))
    b.q = torch.from_numpy(q).to(torch.float16)
    for keep in (1, 7, 40):
        t, n = b.select(pa, keep, 0, 0)
        wt, wn = b.want(keep, 0, 0)
        assert np.array_equal(t, wt) and np.array_equal(n, wn)


def test_select_with_odd_scores(pa):  # noqa: F811
    """Blocks of infinite scale first (in order), zeros, scores of both signs, queries that are zero or not finite."""
    b = Batch(7, [16 * 60] * 6, 2, 4, 128, 16, "fp16", mean=0.0)
    b.all_bounds()
    b.bounds[:, :, 1] = b.rng.integers(-127, 0, b.bounds[:, :, 1].shape)
    b.bounds[:, :, 0] = b.rng.integers(-127, 60, b.bounds[:, :, 1].shape)
    odd = b.rng.random(b.scales.shape) < 0.1
    b.bounds[odd] = 0
    b.scales[odd] = math.inf
    b.scales[b.rng.random(b.scales.shape) < 0.1] = 0
    big = b.rng.random(b.scales.shape) < 0.05
    b.scales[big] = 2.0 ** 120
    b.q[1] = 0
    b.q[2, 3, 5], b.q[3, 1, 0], b.q[4, 7, 127] = math.nan, math.inf, -math.inf
    b.q[5] *= 2.0 ** -14
    for keep, sink, recent in ((5, 0, 0), (12, 1, 1), (40, 0, 3)):
        t, n = b.select(pa, keep, sink, recent)
        wt, wn = b.want(keep, sink, recent)
        assert np.array_equal(t, wt) and np.array_equal(n, wn)


@pytest.mark.parametrize("lens", [[16 * 60, 16 * 200], [16 * 1500]])
def test_select_with_scales_of_zero(pa, lens):  # noqa: F811
    b = Batch(19, lens, 2, 2, 64, 16, "fp16")
    b.all_bounds()
    b.scales[:] = 0  # scores 0 and -0 are equal: the first blocks
    got, n = b.select(pa, 9, 1, 1)
    want, wn = b.want(9, 1, 1)
    assert np.array_equal(want[..., :8], np.broadcast_to(b.tables[:, None, :8], want[..., :8].shape))
    assert np.array_equal(got, want) and np.array_equal(n, wn)
    assert pa.pa_device_errors() == 0


def test_select_of_bad_lengths_and_blocks(pa):  # noqa: F811
    b = Batch(8, [200, 300, 150], 2, 2, 64, 16, "bf16")
    b.all_bounds()
    wt, wn = b.want(4, 1, 1)
    for bad in (-1, 16 * b.tables.shape[1] + 1, 301):
        good = b.lens.copy()
        b.lens[0] = bad
        t, n = b.select(pa, 4, 1, 1, most=300)
        assert pa.pa_device_errors() == pa.DEVERR_BAD_LEN
        assert np.array_equal(t[1:], wt[1:]) and np.array_equal(n[1:], wn[1:])
        assert (t[0] == -1).all() and (n[0] == 0).all()
        b.lens = good
    b.tables[1, 3], b.tables[1, 18] = b.NB, -5  # among the others, and the last (forced) one
    t, n = b.select(pa, 4, 1, 1)
    wt, wn = b.want(4, 1, 1)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_BLOCK
    assert np.array_equal(t, wt) and np.array_equal(n, wn) and (t[1, :, 3] == -5).all()
    # chunks: rows of a bad sequence stay as they were
    b = Batch(9, [200, 300, 150], 2, 2, 64, 16, "bf16", q_lens=[2, 3, 2])
    b.all_bounds()
    wt, wn = b.want(4, 1, 1)
    b.lens[1] = 2
    t, n = b.select(pa, 4, 1, 1)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_LEN
    assert (t[2:5] == 77).all() and (n[2:5] == 77).all()
    assert np.array_equal(t[[0, 1, 5, 6]], wt[[0, 1, 5, 6]]) and np.array_equal(n[[0, 1, 5, 6]], wn[[0, 1, 5, 6]])


# ----------------------------------------------------------------------- sparse

def sparse(pa, b, vc, tables, lens, scale, ks, vs, q=None, **kw):  # noqa: F811
    q = b.q.cuda() if q is None else q
    out = torch.full_like(q, 7.0)
    scales = () if b.kv == "16" else (ks, vs)
    return getattr(pa, "pa_decode_sparse" + END[b.kv])(out, q, b.kc, vc, dev(tables), dev(lens), scale, *scales, **kw)


def check(b, out, vvals, tables, lens, scale, ks, vs, rows=slice(None)):
    ref, mag = S.attend(b.q.double().numpy()[rows], b.kvals * ks, vvals * vs, tables[rows], lens[rows], scale)
    got = f64(out)[rows]
    eps = torch.finfo(TYPES[b.dtype]).eps / 2
    own = 2.0 ** -11 if b.kv == "fp4" else 0.0
    tiny = float(torch.finfo(TYPES[b.dtype]).smallest_normal) * 2 * eps
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= mag * (2.0 ** -11 + 2.0 ** -14 + own) + np.abs(ref) * eps + tiny).all()


def chosen(b, rng, R, keep, most=None):
    """Random tables of valid blocks, and lengths up to all of their tokens, zero among them."""
    tables = rng.integers(0, b.NB, (R, b.H, keep)).astype(np.int32)
    lens = rng.integers(0, keep * b.bs + 1, (R, b.H)).astype(np.int32)
    lens[rng.random((R, b.H)) < 0.1] = 0
    lens[0] = keep * b.bs
    for r in range(R):
        for h in range(b.H):
            tables[r, h, -(-int(lens[r, h]) // b.bs):] = -1
    return tables, lens


@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
@pytest.mark.parametrize("d,bs,dtype,H,G", [(64, 16, "fp16", 4, 1), (128, 16, "bf16", 2, 4),
                                            (128, 32, "fp16", 1, 8), (64, 32, "bf16", 3, 7)])
@pytest.mark.parametrize("R,keep", [(1, 1), (5, 3), (3, 40), (1, 300), (40, 9)])
def test_sparse_decode(pa, kv, d, bs, dtype, H, G, R, keep):  # noqa: F811
    b = Batch(R + keep, [900, 70] + [1] * (R - 1), H, G, d, bs, dtype, kv, q_lens=[R, 0] + [0] * (R - 1), mean=0.0)
    x = b.rng.standard_normal((b.NB, H, bs, d))
    vc, vvals = pool(b.rng, x, kv, dtype, bs, d)
    ks, vs = (1.0, 1.0) if kv == "16" else (0.7, 0.25)
    tables, lens = chosen(b, b.rng, R, keep)
    out = sparse(pa, b, vc, tables, lens, 1 / math.sqrt(d), ks, vs)
    check(b, out, vvals, tables, lens, 1 / math.sqrt(d), ks, vs)
    assert (f64(out).reshape(R, H, G, d)[lens == 0] == 0).all()
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
def test_sparse_decode_leaves_other_tokens_alone(pa, kv):  # noqa: F811
    """NaN in blocks that no table names, and in the rows past a length."""
    d, bs, H = 128, 16, 2
    b = Batch(11, [600], H, 4, d, bs, "fp16", kv, q_lens=[4], mean=0.0)
    x = [b.rng.standard_normal((b.NB, H, bs, d)) for _ in range(2)]
    tables = b.rng.permutation(b.NB)[: 4 * H * 3].reshape(4, H, 3).astype(np.int32)
    lens = b.rng.integers(33, 48, (4, H)).astype(np.int32)
    for y in x:
        keep = np.zeros(y.shape[:3], bool)
        for r in range(4):
            for h in range(H):
                for j in range(3):
                    keep[tables[r, h, j], h, : lens[r, h] - j * bs] = True
        y[~keep] = np.nan
    b.kc, b.kvals = pool(b.rng, x[0], kv, "fp16", bs, d)
    vc, vvals = pool(b.rng, x[1], kv, "fp16", bs, d)
    out = sparse(pa, b, vc, tables, lens, 0.1, 1.0, 1.0)
    check(b, out, vvals, tables, lens, 0.1, 1.0, 1.0)


@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
def test_sparse_decode_of_bad_lengths_and_blocks(pa, kv):  # noqa: F811
    d, bs, H = 64, 16, 3
    b = Batch(12, [300], H, 2, d, bs, "bf16", kv, q_lens=[4], mean=0.0)
    vc, vvals = pool(b.rng, b.rng.standard_normal((b.NB, H, bs, d)), kv, "bf16", bs, d)
    tables = b.rng.integers(0, b.NB, (4, H, 5)).astype(np.int32)
    lens = np.full((4, H), 70, np.int32)
    lens[1, 2], lens[2, 1] = -1, 81
    out = sparse(pa, b, vc, tables, lens, 0.1, 1.0, 1.0)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_LEN
    ok = np.clip(lens, 0, 80)
    ok[2, 1] = ok[1, 2] = 0
    check(b, out, vvals, tables, ok, 0.1, 1.0, 1.0)
    # a bad block: its tokens are left out
    lens[:] = 70
    wrong = tables.copy()
    wrong[0, 1, 2], wrong[3, 0, 0] = b.NB, -7
    out = sparse(pa, b, vc, wrong, lens, 0.1, 1.0, 1.0)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_BLOCK
    ref = tables.copy()
    less = lens.copy()
    ref[0, 1] = [*tables[0, 1, :2], *tables[0, 1, 3:], 0]
    ref[3, 0] = [*tables[3, 0, 1:], 0]
    less[0, 1] = less[3, 0] = 70 - 16
    check(b, out, vvals, ref, less, 0.1, 1.0, 1.0)


# -------------------------------------------------------------- a run of them all

class Step:
    """A decode step on the device: append, bounds, select, sparse; new tokens in place."""

    def __init__(self, pa, seed, lens, H, G, d, bs, dtype, kv, keep, sink, recent):  # noqa: F811
        b = self.b = Batch(seed, [n + 8 for n in lens], H, G, d, bs, dtype, kv)  # room for 8 tokens more
        b.lens = np.asarray(lens, np.int32)
        self.pa, self.keep, self.sink, self.recent = pa, keep, sink, recent
        self.ks, self.vs = (1.0, 1.0) if kv == "16" else (0.5, 0.25)
        self.vc, self.vvals = pool(b.rng, b.rng.standard_normal((b.NB, H, bs, d)), kv, dtype, bs, d)
        b.all_bounds()
        self.gb, self.gs = dev(b.bounds), dev(b.scales)
        self.table = pa.new_rope_table(int(max(lens)) + 8, d)
        R = len(lens)
        self.new = torch.zeros(R, H * G + 2 * H, d, dtype=TYPES[dtype], device="cuda")
        self.q, self.k, self.v = self.new.split([H * G, H, H], 1)
        self.qr, self.out = (torch.zeros(R, H * G, d, dtype=TYPES[dtype], device="cuda") for _ in range(2))
        self.picked = torch.zeros(R, H, keep, dtype=torch.int32, device="cuda")
        self.plens = torch.zeros(R, H, dtype=torch.int32, device="cuda")
        self.bt = dev(b.tables)
        self.cl = dev(b.lens)
        self.most = int(max(lens)) + 8
        self.slots = torch.zeros(R, dtype=torch.int64, device="cuda")
        self.pos = torch.zeros(R, dtype=torch.int64, device="cuda")

    def draw(self):
        """The next token's rows."""
        b = self.b
        b.lens = b.lens + 1
        self.host = torch.from_numpy(b.rng.standard_normal(tuple(self.new.shape))).to(self.new.dtype)
        self.new.copy_(self.host)
        self.cl.copy_(torch.from_numpy(b.lens))
        self.pos.copy_(torch.from_numpy(b.lens.astype(np.int64) - 1))
        at = b.tables[np.arange(len(b.lens)), (b.lens - 1) // b.bs].astype(np.int64)
        self.hslots = at * b.bs + (b.lens - 1) % b.bs
        self.slots.copy_(torch.from_numpy(self.hslots))

    def call(self):
        pa, b, end = self.pa, self.b, END[self.b.kv]
        pair = () if b.kv == "16" else (self.ks, self.vs)
        getattr(pa, "pa_rope_and_cache" + end)(self.qr, self.q, self.k, self.v, b.kc, self.vc, self.slots, self.pos,
                                               self.table, *pair)
        getattr(pa, "pa_update_key_bounds" + end)(self.gb, self.gs, b.kc, self.bt, self.cl)
        pa.pa_select_blocks(self.picked, self.plens, self.qr, self.gb, self.gs, self.bt, self.cl, b.bs, self.most,
                            self.sink, self.recent)
        getattr(pa, "pa_decode_sparse" + end)(self.out, self.qr, b.kc, self.vc, self.picked, self.plens,
                                              1 / math.sqrt(b.d), *pair)

    def check(self):
        b = self.b
        G = self.q.shape[1]
        q, k, v = self.host[:, :G], self.host[:, G:G + b.H], self.host[:, G + b.H:]
        turned = [torch.from_numpy(S.rotate(x.float().numpy(), b.lens - 1, self.table.cpu().numpy(), False)).to(x.dtype)
                  for x in (q, k)]
        assert np.array_equal(f64(self.qr), turned[0].double().numpy())
        for vals, x, g in ((b.kvals, turned[1], self.ks), (self.vvals, v, self.vs)):
            row = np.zeros((len(b.lens), b.H, 1, b.d))
            row[:, :, 0] = x.double().numpy()
            if b.kv == "16":
                new = row[:, :, 0]
            elif b.kv == "fp8":
                new = oracle.e4m3_to_f64(oracle.e4m3_from_f32(row[:, :, 0].astype(np.float32) / np.float32(g))).reshape(
                    row[:, :, 0].shape)
            else:
                codes, sc = F.quantise(row[:, :, 0].astype(np.float32), g)
                e = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], b.d)
                new = F.E2M1[e] * np.repeat(F.E4M3[sc], 16, -1)
            vals[self.hslots // b.bs, :, self.hslots % b.bs] = new
        S.update_bounds(b.bounds, b.scales, b.kvals, b.tables, b.lens, [1] * len(b.lens))
        assert np.array_equal(self.gb.cpu().numpy(), b.bounds) and np.array_equal(self.gs.cpu().numpy(), b.scales)
        t, n = S.select(f64(self.qr), b.bounds, b.scales, b.tables, np.arange(len(b.lens)), b.lens, b.bs, self.keep,
                        self.sink, self.recent)
        assert np.array_equal(self.picked.cpu().numpy(), t) and np.array_equal(self.plens.cpu().numpy(), n)
        ref, mag = S.attend(f64(self.qr), b.kvals * self.ks, self.vvals * self.vs, t, n, 1 / math.sqrt(b.d))
        got, eps = f64(self.out), torch.finfo(TYPES[b.dtype]).eps / 2
        # (keys have a mean of their own: sum |q k| scale is below 128 here, four times the bound above)
        assert (np.abs(got - ref) <= mag * (2.0 ** -9 + 2.0 ** -11) + np.abs(ref) * eps + 2.0 ** -24).all()
        assert self.pa.pa_device_errors() == 0


STEPS = [("16", "fp16", 128, 16, 8), ("16", "bf16", 64, 32, 3), ("fp8", "bf16", 128, 16, 8), ("fp8", "fp16", 64, 16, 5),
         ("fp4", "fp16", 128, 32, 4), ("fp4", "bf16", 64, 16, 8)]


@pytest.mark.parametrize("kv,dtype,d,bs,keep", STEPS)
def test_steps_in_a_row(pa, kv, dtype, d, bs, keep):  # noqa: F811
    s = Step(pa, 20, [900, 2 * bs - 6, 17, 1, 333], 2, 4, d, bs, dtype, kv, keep, 1, 1)
    for _ in range(4):
        s.draw()
        s.call()
        s.check()


def test_captured_steps_of_two_batches(pa):  # noqa: F811
    """Two graphs replayed in turn, each with new tokens in place, on one stream."""
    steps = [Step(pa, 21, [700, 40, 3], 2, 4, 128, 16, "bf16", "16", 6, 1, 2),
             Step(pa, 22, [500, 90], 1, 8, 64, 16, "fp16", "fp8", 5, 0, 1)]
    graphs = []
    for s in steps:
        s.draw()
        s.call()
        torch.cuda.synchronize()
        s.check()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.call()
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(steps, graphs):
            s.draw()
            s.out.zero_()
            g.replay()
            s.check()


@pytest.mark.parametrize("longest", [9000, 70000])
def test_long_steps_on_two_streams_and_captured(pa, longest):  # noqa: F811
    """The selection in clusters: two batches at once, then each replayed."""
    steps = [Step(pa, 27 + i, [longest - 700 * i, 60, 4300], 2, 4, 128, 16, "bf16", kv, 12, 2, 3)
             for i, kv in enumerate(("16", "fp8"))]
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.draw()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.call()
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        s.check()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.call()
    for _ in range(2):
        for s, g in zip(steps, graphs):
            s.draw()
            s.out.zero_()
            g.replay()
            s.check()


def test_steps_on_two_streams_at_once(pa):  # noqa: F811
    steps = [Step(pa, 23 + i, [1200 + 100 * i, 60, 8], 2, 4, 128, 16, "fp16", "16", 7, 1, 1) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.draw()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.call()
    torch.cuda.synchronize()
    for s in steps:
        s.check()


@pytest.mark.parametrize("kv,dtype,d,bs,keep", STEPS)
def test_drafted_rows_through_all_calls(pa, kv, dtype, d, bs, keep):  # noqa: F811
    """Several new tokens a sequence, none for one: rotated and written, their blocks
    bounded, blocks chosen for each row by the tokens up to it, and attended to."""
    H, G, q_lens = 2, 4, [5, 1, 0, 3]
    lens = [700, 2 * bs + 1, 90, 3]
    b = Batch(24, lens, H, G, d, bs, dtype, kv, q_lens)
    ks, vs = (1.0, 1.0) if kv == "16" else (0.5, 0.25)
    pair = () if kv == "16" else (ks, vs)
    vc, _ = pool(b.rng, b.rng.standard_normal((b.NB, H, bs, d)), kv, dtype, bs, d)
    b.all_bounds()
    gb, gs = dev(b.bounds), dev(b.scales)
    new = torch.from_numpy(b.rng.standard_normal((9, (G + 2) * H, d))).to(TYPES[dtype]).cuda()
    q, k, v = new.split([G * H, H, H], 1)
    pos = (b.seen - 1).astype(np.int64)
    slots = b.tables[b.seqs, pos // bs].astype(np.int64) * bs + pos % bs
    table = pa.new_rope_table(700, d)
    getattr(pa, "pa_rope_and_cache" + END[kv])(q, q, k, v, b.kc, vc, dev(slots), dev(pos), table, *pair)
    bt, cl, start = dev(b.tables), dev(b.lens), dev(b.start)
    getattr(pa, "pa_update_key_bounds" + END[kv])(gb, gs, b.kc, bt, cl, start, 5)
    query = q.contiguous()
    t = torch.zeros(9, H, keep, dtype=torch.int32, device="cuda")
    n = torch.zeros(9, H, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(t, n, query, gb, gs, bt, cl, bs, 700, 1, 1, start, 5)
    out = torch.zeros_like(query)
    getattr(pa, "pa_decode_sparse" + END[kv])(out, query, b.kc, vc, t, n, 1 / math.sqrt(d), *pair)
    assert pa.pa_device_errors() == 0

    def values(cache):
        if kv == "16":
            return f64(cache)
        if kv == "fp8":
            return oracle.e4m3_to_f64(cache.cpu().numpy()).reshape(b.NB, H, bs, d)
        return F.values(cache.cpu().numpy(), bs, d, 1.0)

    b.kvals, vvals = values(b.kc), values(vc)  # (what append writes: test_gpu_rope.py)
    S.update_bounds(b.bounds, b.scales, b.kvals, b.tables, b.lens, q_lens)
    assert np.array_equal(gb.cpu().numpy(), b.bounds) and np.array_equal(gs.cpu().numpy(), b.scales)
    wt, wn = S.select(f64(query), b.bounds, b.scales, b.tables, b.seqs, b.seen, bs, keep, 1, 1)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(n.cpu().numpy(), wn)
    ref, mag = S.attend(f64(query), b.kvals * ks, vvals * vs, wt, wn, 1 / math.sqrt(d))
    eps = torch.finfo(TYPES[dtype]).eps / 2
    # (keys have a mean of their own: as in Step.check)
    assert (np.abs(f64(out) - ref) <= mag * (2.0 ** -9 + 2.0 ** -11) + np.abs(ref) * eps + 2.0 ** -24).all()


def test_bounds_move_with_blocks(pa):  # noqa: F811
    """A fork: blocks, bounds and scales copied within their pools, and a sequence that goes on in the copy."""
    b = Batch(25, [100, 100], 4, 2, 64, 16, "fp16", extra=0)
    b.all_bounds()
    gb, gs = dev(b.bounds), dev(b.scales)
    pairs = np.stack([b.tables[0], b.tables[1]], 1).astype(np.int64)
    for pool_ in (b.kc, gb, gs):
        pa.pa_swap_blocks(pool_, pool_, dev(pairs))
    b.kvals[b.tables[1]] = b.kvals[b.tables[0]]
    b.bounds[b.tables[1]], b.scales[b.tables[1]] = b.bounds[b.tables[0]], b.scales[b.tables[0]]
    assert np.array_equal(gb.cpu().numpy(), b.bounds) and np.array_equal(gs.cpu().numpy(), b.scales)
    b.lens[:] = 97, 100  # the first sequence gives up three tokens
    S.update_bounds(b.bounds, b.scales, b.kvals, b.tables, b.lens, [1, 1])
    pa.pa_update_key_bounds(gb, gs, b.kc, dev(b.tables), dev(b.lens))
    assert np.array_equal(gb.cpu().numpy(), b.bounds) and np.array_equal(gs.cpu().numpy(), b.scales)


def test_all_blocks_kept_is_dense_decode(pa):  # noqa: F811
    """Where every block is kept, the dense call of the same cache agrees within both calls' rounding."""
    for kv in ("16", "fp8", "fp4"):
        b = Batch(30, [1, 77, 640, 0, 2000], 2, 4, 128, 16, "fp16", kv, mean=0.0)
        vc, vvals = pool(b.rng, b.rng.standard_normal((b.NB, 2, 16, 128)), kv, "fp16", 16, 128)
        b.all_bounds()
        t, n = b.select(pa, 125, 1, 1)
        assert np.array_equal(n, np.repeat(b.lens[:, None], 2, 1))
        out = sparse(pa, b, vc, t, n, 0.09, 1.0, 1.0)
        check(b, out, vvals, t, n, 0.09, 1.0, 1.0)
        dense = torch.empty_like(out)
        pair = () if kv == "16" else (1.0, 1.0)
        getattr(pa, "pa_decode" + END[kv])(dense, b.q.cuda(), b.kc, vc, dev(b.tables), dev(b.lens), 0.09, *pair, 2000)
        check(b, dense, vvals, t, n, 0.09, 1.0, 1.0)


@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
def test_native_binding_takes_what_fits(pa, kv):  # noqa: F811
    """Not by way of the checks in Python."""
    kind, native = list(END).index(kv), pa._native()
    b = Batch(33, [40, 33], 2, 2, 64, 16, "bf16", kv)
    gb, gs = pa.new_key_bounds(b.NB, 2, 64)
    q = b.q.cuda()
    both = torch.cat([q, q], 1)
    slots, pos, table = dev(np.array([3, 20])), dev(np.array([0, 1])), pa.new_rope_table(4, 64)
    vc = b.kc.clone()
    assert native.rope(kind, q, both[:, :4], both[:, 4:6], both[:, 6:], b.kc, vc, slots, pos, table, 1, 0.5, False, None) == 0
    bt, cl = dev(b.tables), dev(b.lens)
    start = dev(np.array([0, 40, 73], np.int32))
    assert native.key_bounds(kind, gb, gs, b.kc, bt, cl, None, 1, None) == 0
    assert native.key_bounds(kind, gb, gs, b.kc, bt, cl, start, 40, torch.cuda.current_stream()) == 0
    t = torch.zeros(2, 2, 2, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    assert native.select(t, n, q, gb, gs, bt, cl, 16, 40, 1, 1, None, 1, None) == 0
    assert native.select(t, n, q, gb, gs, bt, cl, 16, 40, 2, 1, None, 1, None) == 1  # the call's own refusal
    out = torch.zeros_like(q)
    assert native.sparse(kind, out, q, b.kc, vc, t, n, 0.1, 1.0, 1, torch.cuda.current_stream().cuda_stream) == 0
    assert pa.pa_device_errors() == 0


def test_arguments_of_other_kinds(pa):  # noqa: F811
    """numpy numbers, a stream's handle, a stream object, single heads of any stride, one row of any
    stride: what the native binding leaves to the checks in Python."""
    b = Batch(32, [40, 33], 1, 2, 64, 16, "fp16", mean=0.0)
    vc, vvals = pool(b.rng, b.rng.standard_normal((b.NB, 1, 16, 64)), "16", "fp16", 16, 64)
    b.all_bounds()
    gb, gs = pa.new_key_bounds(b.NB, 1, 64)
    st = torch.cuda.Stream()
    handle = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    one = dev(np.array([0, 40, 73], np.int32))
    pa.pa_update_key_bounds(gb, gs, b.kc, dev(b.tables), dev(b.lens), one, np.int64(40), stream=st)
    st.synchronize()
    assert np.array_equal(gb.cpu().numpy(), b.bounds)
    t = torch.zeros(2, 1, 2, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(t, n, b.q.cuda(), gb, gs, dev(b.tables), dev(b.lens), np.int32(16), np.int64(40), np.int64(1),
                        stream=handle)
    wt, wn = b.want(2, 1, 1)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(n.cpu().numpy(), wn)
    out = torch.zeros_like(b.q, device="cuda")
    pa.pa_decode_sparse(out, b.q.cuda(), b.kc, vc, t, n, np.float32(0.1))
    check(b, out, vvals, wt, wn, float(np.float32(0.1)), 1.0, 1.0)
    # K of one head in rows whose heads are 200 apart; one token in a row of any length
    wide = torch.from_numpy(b.rng.standard_normal((3, 2, 200))).half().cuda()
    k = wide[:, :1, :64]
    q = torch.from_numpy(b.rng.standard_normal((3, 2, 64))).half().cuda()
    table = pa.new_rope_table(5, 64)
    slots, pos = dev(np.array([0, 1, 2])), dev(np.array([4, 0, 3]))
    res = torch.zeros_like(q)
    pa.pa_rope_and_cache(res, q, k, k, b.kc, vc, slots, pos, table)
    want = S.rotate(k.cpu().float().numpy(), [4, 0, 3], table.cpu().numpy(), False)
    assert np.array_equal(f64(b.kc[0, :, :3].transpose(0, 1)), torch.from_numpy(want).half().double().numpy())
    assert torch.equal(vc[0, 0, :3], k[:, 0])
    pa.pa_rope_and_cache(res[:1], q[:1], wide[:1, 1:, 3:67].clone(), k[:1], b.kc, vc, slots[:1], pos[:1], table)
    want = S.rotate(wide[:1, 1:, 3:67].cpu().float().numpy(), [4], table.cpu().numpy(), False)
    assert np.array_equal(f64(b.kc[0, :, :1].transpose(0, 1)), torch.from_numpy(want).half().double().numpy())
    assert pa.pa_device_errors() == 0


def test_offsets_past_32_bits(pa):  # noqa: F811
    """The last blocks of a pool of more than 2^31 elements a cache, through all calls."""
    H, bs, d, NB = 8, 32, 128, (1 << 31) // (8 * 32 * 128) + 9
    kc, vc = (torch.empty(NB, H, bs, d, dtype=torch.float16, device="cuda") for _ in range(2))
    gb, gs = pa.new_key_bounds(NB, H, d)
    rng = np.random.default_rng(60)
    ids = np.array([NB - 1, 0, NB - 2, 3, NB - 5, NB - 7], np.int32)
    n = 6 * bs - 7
    j = np.arange(n)
    slots = ids[j // bs].astype(np.int64) * bs + j % bs
    q, k, v = (torch.from_numpy(rng.standard_normal((n, h, d))).half() for h in (2 * H, H, H))
    table = pa.new_rope_table(n, d)
    out = torch.zeros_like(q, device="cuda")
    pa.pa_rope_and_cache(out, q.cuda(), k.cuda(), v.cuda(), kc, vc, dev(slots), dev(j.astype(np.int64)), table)
    tables, lens, start = ids[None], np.array([n], np.int32), np.array([0, n], np.int32)
    pa.pa_update_key_bounds(gb, gs, kc, dev(tables), dev(lens), dev(start), n)
    at = torch.from_numpy(ids.astype(np.int64)).cuda()
    keys, vals = f64(kc[at]), f64(vc[at])
    bounds, scales = np.zeros((6, H, 2, d), np.int8), np.zeros((6, H), np.float32)
    small = np.arange(6, dtype=np.int32)[None]
    S.update_bounds(bounds, scales, keys, small, lens, [n])
    assert np.array_equal(gb[at].cpu().numpy(), bounds) and np.array_equal(gs[at].cpu().numpy(), scales)
    last = out[-1:].contiguous()
    t = torch.zeros(1, H, 3, dtype=torch.int32, device="cuda")
    m = torch.zeros(1, H, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(t, m, last, gb, gs, dev(tables), dev(lens), bs, n)
    wt, wm = S.select(f64(last), bounds, scales, small, [0], [n], bs, 3, 1, 1)
    assert np.array_equal(t.cpu().numpy(), ids[wt]) and np.array_equal(m.cpu().numpy(), wm)
    o = torch.zeros_like(last)
    pa.pa_decode_sparse(o, last, kc, vc, t, m, 0.08)
    ref, mag = S.attend(f64(last), keys, vals, wt, wm, 0.08)
    assert (np.abs(f64(o) - ref) <= mag * (2.0 ** -11 + 2.0 ** -14) + np.abs(ref) * 2.0 ** -11 + 2.0 ** -24).all()
    assert pa.pa_device_errors() == 0


def test_refused_arguments(pa):  # noqa: F811
    b = Batch(31, [40, 50], 2, 2, 64, 16, "fp16")
    b.all_bounds()
    gb, gs, bt, cl, q = dev(b.bounds), dev(b.scales), dev(b.tables), dev(b.lens), b.q.cuda()
    t = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    qs = dev(np.array([0, 1, 2], np.int32))
    for args in ((gb.float(), gs, b.kc, bt, cl), (gb[:1], gs, b.kc, bt, cl), (gb, gs.double(), b.kc, bt, cl),
                 (gb, gs[:, :1], b.kc, bt, cl), (gb, gs, b.kc.float(), bt, cl), (gb, gs, b.kc[:, :1], bt, cl),
                 (gb, gs, b.kc, bt.long(), cl), (gb, gs, b.kc, bt[:1], cl), (gb, gs, b.kc, bt, cl.cpu()),
                 (gb, gs, b.kc, bt, cl, cl, 1), (gb, gs, b.kc, bt, cl, qs.long(), 1)):
        with pytest.raises(ValueError):
            pa.pa_update_key_bounds(*args)
    with pytest.raises(pa.PaError):
        pa.pa_update_key_bounds(gb, gs, b.kc, bt, cl, None, 2)
    good = [t, n, q, gb, gs, bt, cl]
    pa.pa_select_blocks(*good, 16, 50)
    for at, bad in ((0, t.long()), (0, t[:1]), (0, t[:, :1]), (1, n[:1]), (1, n.t()), (2, q[:1]), (2, q.float()),
                    (2, q.transpose(0, 1)), (3, gb.to(torch.uint8)), (3, gb[..., :32]), (4, gs[:1]), (5, bt[0]), (6, cl[:1])):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            pa.pa_select_blocks(*args, 16, 50)
    with pytest.raises(pa.PaError):
        pa.pa_select_blocks(*good, 24, 50)
    with pytest.raises(pa.PaError):
        pa.pa_select_blocks(*good, 16, 50, 2, 2)
    out = torch.empty_like(q)
    good = [out, q, b.kc, b.kc, t, n]
    pa.pa_decode_sparse(*good, 0.1)
    for at, bad in ((0, out[:1]), (0, out.bfloat16()), (1, q.cpu()), (2, b.kc.transpose(2, 3)), (2, b.kc.to(torch.uint8)),
                    (3, b.kc[:1]), (4, t[:1]), (4, t[0]), (4, t[..., ::2]), (5, n[:, :1]), (5, n.long())):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            pa.pa_decode_sparse(*args, 0.1)
    assert pa.pa_device_errors() == 0
