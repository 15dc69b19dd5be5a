"""GPU parity of the FP4 KV cache (write, read-back, decode, prefill) with the
64-bit reference in ``oracle/fp4.py``.

The write's codes and scales are compared byte for byte with the reference's,
and every byte of the pool that no token owns must stay as it was.  A read-back
element is the exact value rounded three times: s * g and the product with the
code in fp32 (2^-24 each), then to the 16-bit type (half a step, eps / 2).

Attention, per output element, with A = sum_j p_j |v_j| (the reference's
softmax over |V|): the values are exact in fp16, so what is rounded is P (fp16,
2^-11 of each p_j, hence 2^-11 A), the sums (at most d products of at most
scale |q| |k| each in fp32, the exponential, the running sums: below 2^-12 A
together for these inputs, d 128 * 2^-24 * a logit of at most 32 * 2) and the
output (eps / 2 of its value).
"""
import numpy as np
import pytest
import torch

import oracle.fp4 as F

pytestmark = pytest.mark.gpu
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
NAN_SCALE = 0x7F


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from pagedattention_kv_cache_attention_gb300 import build
    build.build()
    import pagedattention_kv_cache_attention_gb300 as pa
    pa._load()
    assert pa.pa_device_errors() == 0
    return pa


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


# -------------------------------------------------------------- write, read-back

def rows(rng, T, H, d, dtype):
    """16-bit rows whose groups have very different magnitudes, with zero groups."""
    mag = np.exp2(rng.integers(-12, 10, (T, H, d // 16))).repeat(16, axis=-1)
    x = rng.standard_normal((T, H, d)) * mag * (rng.random((T, H, d // 16)) > 0.05).repeat(16, -1)
    return torch.from_numpy(x).to(TYPES[dtype])


@pytest.mark.parametrize("T,H,d,bs,dtype,fused,ks,vs", [
    (1, 1, 64, 16, "fp16", False, 1.0, 1.0), (1, 8, 128, 32, "bf16", True, 0.5, 3.0),
    (37, 3, 64, 32, "bf16", True, 0.7, 1.0), (300, 8, 128, 16, "fp16", True, 1.0, 0.01),
    (17, 5, 128, 16, "bf16", False, 2.0 ** -90, 2.0 ** 90), (513, 2, 64, 16, "fp16", False, 1.3, 1.0),
    (2, 70, 128, 32, "fp16", False, 1.0, 1.0)])
def test_write_bytes_and_read_back(pa, T, H, d, bs, dtype, fused, ks, vs):
    rng = np.random.default_rng(T * 7 + H)
    NB = -(-T // bs) + 4
    k, v = rows(rng, T, H, d, dtype), rows(rng, T, H, d, dtype)
    slots = rng.permutation(NB * bs)[:T]
    slots[rng.random(T) < 0.1] = -1
    pool = [rng.integers(0, 256, (NB, H, bs * d * 9 // 16)).astype(np.uint8) for _ in range(2)]
    want = [p.copy() for p in pool]
    F.reshape_and_cache(k.float().numpy(), v.float().numpy(), *want, slots, bs, ks, vs)
    kc, vc = dev(pool[0]), dev(pool[1])
    if fused:
        both = torch.cat([torch.zeros(T, 2 * H, d, dtype=k.dtype), k, v], 1).cuda()
        kd, vd = both[:, 2 * H:3 * H], both[:, 3 * H:]
    else:
        kd, vd = k.cuda(), v.cuda()
    sm = dev(slots.astype(np.int64))
    pa.pa_reshape_and_cache_fp4(kd, vd, kc, vc, sm, ks, vs)
    assert np.array_equal(kc.cpu().numpy(), want[0])
    assert np.array_equal(vc.cpu().numpy(), want[1])
    # read back into rows with a margin on both sides, which stays as it was
    out = torch.full((T, 2 * H + 4, d), 7.0, dtype=k.dtype, device="cuda")
    pa.pa_gather_cache_fp4(out[:, 1:H + 1], out[:, H + 3:2 * H + 3], kc, vc, sm, ks, vs)
    eps = torch.finfo(k.dtype).eps / 2
    for lo, cache, g in ((1, want[0], ks), (H + 3, want[1], vs)):
        val = F.values(cache, bs, d, g)
        with np.errstate(invalid="ignore"):
            ref = val[np.maximum(slots, 0) // bs, :, np.maximum(slots, 0) % bs]
        got = f64(out[:, lo:lo + H])
        assert (got[slots < 0] == 7).all()
        got, ref = got[slots >= 0], ref[slots >= 0]
        big = float(torch.finfo(k.dtype).max)
        sub = float(torch.finfo(k.dtype).smallest_normal) * 2 * eps  # half a subnormal step
        fits = np.abs(ref) < big
        assert (np.abs(got - ref)[fits] <= (np.abs(ref) * (eps + 2 ** -22) + sub)[fits]).all()
        assert np.isinf(got[np.abs(ref) > big * (1 + eps)]).all()
    keep = torch.ones(2 * H + 4, dtype=torch.bool)
    keep[1:H + 1] = keep[H + 3:2 * H + 3] = False
    assert (out[:, keep] == 7).all()
    assert pa.pa_device_errors() == 0


def test_write_special_values(pa):
    """NaN, infinities, ties, signed zeros and groups whose scale rounds to zero."""
    d, bs = 64, 16
    x = np.zeros((6, 1, d), np.float32)
    x[0, 0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    x[0, 0, 16:24] = [-6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5]
    x[1, 0, 3], x[1, 0, 20] = np.nan, np.inf
    x[1, 0, 4], x[1, 0, 21] = 5.0, -1.0
    x[2, 0, 5], x[2, 0, 17] = 6 * 2.0 ** -10, 6.5 * 2.0 ** -10
    x[3, 0, :] = -0.0
    x[4, 0, :] = 60000.0
    x[5, 0, ::3] = np.linspace(-3, 3, 22)
    want = [np.zeros((1, 1, bs * d * 9 // 16), np.uint8) for _ in range(2)]
    t = torch.from_numpy(x).to(torch.float16)
    slots = np.arange(6)
    F.reshape_and_cache(t.float().numpy(), -t.float().numpy(), *want, slots, bs, 1.0, 1.0)
    kc = torch.zeros(1, 1, bs * d * 9 // 16, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    pa.pa_reshape_and_cache_fp4(t.cuda(), -t.cuda(), kc, vc, dev(slots))
    assert np.array_equal(kc.cpu().numpy(), want[0])
    assert np.array_equal(vc.cpu().numpy(), want[1])
    o, p = torch.zeros_like(t, device="cuda"), torch.zeros_like(t, device="cuda")
    pa.pa_gather_cache_fp4(o, p, kc, vc, dev(slots))
    assert torch.isnan(o[1, 0, :16]).all() and not torch.isnan(o[1, 0, 16:]).any()
    assert o[1, 0, 20] == 2688 and p[1, 0, 20] == -2688 and o[2, 0, 5] == 0


def test_slots_outside_the_pool_are_flagged_and_skipped(pa):
    d, bs, H, NB = 128, 16, 2, 3
    rng = np.random.default_rng(5)
    k = rows(rng, 4, H, d, "fp16")
    slots = np.array([NB * bs, 5, 1 << 40, NB * bs - 1])
    want = [np.zeros((NB, H, bs * d * 9 // 16), np.uint8) for _ in range(2)]
    F.reshape_and_cache(k.float().numpy(), k.float().numpy(), *want, np.where(slots < NB * bs, slots, -1),
                        bs, 1.0, 1.0)
    kc, vc = (torch.zeros(NB, H, bs * d * 9 // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    pa.pa_reshape_and_cache_fp4(k.cuda(), k.cuda(), kc, vc, dev(slots))
    assert pa.pa_device_errors() == pa.DEVERR_BAD_SLOT
    assert np.array_equal(kc.cpu().numpy(), want[0]) and np.array_equal(vc.cpu().numpy(), want[1])
    o = torch.full((4, H, d), 7.0, dtype=torch.float16, device="cuda")
    p = o.clone()
    pa.pa_gather_cache_fp4(o, p, kc, vc, dev(slots))
    assert pa.pa_device_errors() == pa.DEVERR_BAD_SLOT
    assert (o[[0, 2]] == 7).all() and (p[[0, 2]] == 7).all() and (o[[1, 3]] != 7).any()


def test_read_back_takes_a_slot_twice(pa):
    d, bs, H = 64, 32, 3
    rng = np.random.default_rng(6)
    kc, vc = (rng.integers(0, 256, (2, H, bs * d * 9 // 16)).astype(np.uint8) for _ in range(2))
    for c in (kc, vc):
        F.views(c, bs, d)[1][...] = 0x38
    slots = np.array([63, 0, 63, 63, 1])
    o = torch.zeros(5, H, d, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros_like(o)
    pa.pa_gather_cache_fp4(o, p, dev(kc), dev(vc), dev(slots))
    k = F.values(kc, bs, d, 1.0)
    assert np.array_equal(f64(o), k[slots // bs, :, slots % bs])


# ---------------------------------------------------------------------- attention

class Batch:
    """A pool of random codes and scales with NaN scales wherever no sequence's
    tokens are, block tables from a shuffled free list, N(0, 1) queries."""

    def __init__(self, seed, lens, H, G, d, bs, dtype, ks=1.0, vs=1.0, q_lens=None, spread=4,
                 slack=2):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        self.H, self.G, self.d, self.bs, self.dtype, self.ks, self.vs = H, G, d, bs, dtype, ks, vs
        per = -(-self.lens // bs)
        used = int(per.sum())
        self.NB = used + slack
        ids = rng.permutation(self.NB)[:used].astype(np.int32)
        self.tables = np.full((len(lens), max(1, int(per.max())) + 1), -1, np.int32)
        self.kc, self.vc = (rng.integers(0, 256, (self.NB, H, bs * d * 9 // 16)).astype(np.uint8)
                            for _ in range(2))
        for c in (self.kc, self.vc):
            s = F.views(c, bs, d)[1]
            s[...] = NAN_SCALE
        at = 0
        for i, n in enumerate(self.lens):
            self.tables[i, :per[i]] = ids[at:at + per[i]]
            at += per[i]
            for b in range(per[i]):
                m = min(bs, int(n) - b * bs)
                for c in (self.kc, self.vc):
                    s = F.views(c, bs, d)[1][self.tables[i, b], :, :m]
                    s[...] = rng.integers(0x2C, 0x2C + spread * 4, s.shape)
        self.scale = 1 / np.sqrt(d)
        self.q_lens = q_lens
        n_q = len(lens) if q_lens is None else int(np.sum(q_lens))
        self.start = None if q_lens is None else np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.q = torch.from_numpy(rng.standard_normal((n_q, H * G, d))).to(TYPES[dtype])

    def reference(self, absolute=False):
        k, v = F.values(self.kc, self.bs, self.d, self.ks), F.values(self.vc, self.bs, self.d, self.vs)
        v = np.abs(v) if absolute else v
        if self.start is None:
            return F.decode(f64(self.q), k, v, self.tables, self.lens, self.scale)
        return F.prefill(f64(self.q), self.start, k, v, self.tables, self.lens, self.scale)

    def gpu(self):
        return [dev(x) for x in (self.kc, self.vc, self.tables, self.lens)]

    def check(self, out, rows=None):
        ref, A, got = self.reference(), self.reference(True), f64(out)
        if rows is not None:
            ref, A, got = ref[rows], A[rows], got[rows]
        eps = torch.finfo(TYPES[self.dtype]).eps / 2
        tol = eps * np.abs(ref) * (1 + 2 ** -8) + A * (2 ** -11 + 2 ** -12) + 2.0 ** -24
        assert np.isfinite(got).all()
        bad = np.abs(got - ref) > tol
        assert not bad.any(), f"{int(bad.sum())} elements, worst {np.max(np.abs(got - ref) / tol):.3g} of the tolerance"

    def decode(self, pa, ps=0, ws=None, maxctx=None, stream=None, out=None):
        out = torch.full_like(self.q, float("nan"), device="cuda") if out is None else out
        kc, vc, bt, cl = self.gpu()
        pa.pa_decode_fp4(out, self.q.cuda(), kc, vc, bt, cl, self.scale, self.ks, self.vs,
                         maxctx or max(1, int(self.lens.max())), ps, ws, stream)
        torch.cuda.synchronize()
        return out

    def prefill(self, pa):
        out = torch.full_like(self.q, float("nan"), device="cuda")
        kc, vc, bt, cl = self.gpu()
        pa.pa_prefill_fp4(out, self.q.cuda(), dev(self.start), kc, vc, bt, cl, self.scale, self.ks,
                          self.vs, max(1, int(max(self.q_lens))))
        torch.cuda.synchronize()
        return out


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ps", [0, 16, 48, 64])
def test_decode_edge_lengths(pa, d, bs, dtype, ps):
    b = Batch(11, EDGES, 2, 4, d, bs, dtype)
    b.check(b.decode(pa, ps))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("G", range(1, 9))
def test_decode_groups(pa, G):
    b = Batch(20 + G, [100, 7, 333], 3, G, 128 if G % 2 else 64, 32 if G > 4 else 16,
              "bf16" if G in (2, 3, 7) else "fp16", ks=0.7, vs=0.03)
    for ps in (0, 128):
        b.check(b.decode(pa, ps))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("i", range(24))
def test_decode_random_shapes(pa, i):
    rng = np.random.default_rng(300 + i)
    lens = rng.integers(0, 3001, int(rng.integers(1, 6)))
    lens[0] = max(1, lens[0])
    b = Batch(400 + i, lens, int(rng.integers(1, 9)), int(rng.integers(1, 9)),
              int(rng.choice([64, 128])), int(rng.choice([16, 32])), str(rng.choice(["fp16", "bf16"])),
              ks=float(rng.choice([1.0, 0.3])), vs=float(rng.choice([1.0, 5.0])))
    ps = int(rng.choice([0, 16, 80, 256, 512, 1024]))
    b.check(b.decode(pa, ps))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("fp16", 32)])
def test_decode_long_context_through_the_reduce(pa, dtype, bs):
    """More partitions than one CTA joins (the reduce kernel's path)."""
    b = Batch(31, [20000, 0, 515, 8191], 1, 4, 128, bs, dtype)
    b.check(b.decode(pa, 512))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("G,d,bs,dtype", [(1, 128, 16, "fp16"), (4, 64, 32, "bf16"),
                                          (8, 128, 32, "fp16"), (5, 64, 16, "bf16")])
@pytest.mark.parametrize("long", [600, 1100, 4100])
def test_decode_empty_and_short_sequences_beside_a_long_one(pa, G, d, bs, dtype, long):
    """Unsplit: the work is split for the table's room, which most sequences do not fill."""
    b = Batch(40 + G, [long, 0, 1, 33, 64, 257], 2, G, d, bs, dtype, ks=2.0, vs=0.3)
    out = b.decode(pa, 0)
    b.check(out)
    assert (out[1] == 0).all()
    assert pa.pa_device_errors() == 0


def test_decode_workspace_reused_across_shapes(pa):
    a = Batch(33, [900, 1500, 3], 2, 4, 128, 16, "fp16")
    b = Batch(34, [700], 1, 8, 64, 32, "bf16")
    ws = pa.new_decode_workspace(3, 8, 128, 1500, 64)
    for _ in range(2):
        a.check(a.decode(pa, 64, ws))
        b.check(b.decode(pa, 128, ws))
    assert not ws[:pa.DECODE_COUNTER_BYTES].any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_keeps_the_mass_of_a_long_faint_tail(pa, dtype):
    """One key far above 40,000 others whose probabilities are near 2^-25 each:
    together they carry 2^-10 of the mass, with values 100 times the peak's, so
    a probability that is dropped below fp16's range shows."""
    n, d, bs = 40001, 64, 16
    b = Batch(35, [n], 1, 2, d, bs, dtype)
    kcodes, kscales = F.views(b.kc, bs, d)
    vcodes, vscales = F.views(b.vc, bs, d)
    kcodes[...] = 0
    kscales[...] = 0x38                      # every scale 1
    vcodes[...], vscales[...] = 0x77, 0x58   # value 6 * 16 = 96
    blk, row = b.tables[0, 1000], 5
    kcodes[blk, :, row] = 0x22               # 1.0 in every dimension
    vscales[blk, :, row] = 0x20              # 6 * 0.125
    q = np.full((1, 2, d), 25 * np.log(2) * np.sqrt(d) / d)
    b.q = torch.from_numpy(q).to(TYPES[dtype])
    b.check(b.decode(pa, 0))
    b.check(b.decode(pa, 4096))
    b.check(b.decode(pa, 512))


def same_with_nans(b, out):
    """out against the reference, NaN where the reference is and nowhere else."""
    with np.errstate(invalid="ignore"):
        ref, A, got = b.reference(), b.reference(True), f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    live = ~np.isnan(ref)
    eps = torch.finfo(TYPES[b.dtype]).eps / 2
    tol = eps * np.abs(ref) * (1 + 2 ** -8) + A * (2 ** -11 + 2 ** -12) + 2.0 ** -24
    assert (np.abs(got - ref)[live] <= tol[live]).all()
    return np.isnan(ref)


@pytest.mark.parametrize("ps", [0, 16, 64, 512])
@pytest.mark.parametrize("G,d,bs,dtype", [(4, 128, 16, "fp16"), (3, 64, 32, "bf16")])
def test_decode_nans_stay_where_they_belong(pa, ps, G, d, bs, dtype):
    """A NaN group of V, of K, and a NaN in one head's query."""
    b = Batch(37, [900, 1300, 40, 700], 2, G, d, bs, dtype)
    for i, j, cache in ((0, 899, b.vc), (1, 5, b.kc), (1, 1290, b.vc), (2, 17, b.vc)):
        F.views(cache, bs, d)[1][b.tables[i, j // bs], i % 2, j % bs, 1] = NAN_SCALE
    b.q[3, G - 1, 7] = float("nan")
    out = b.decode(pa, ps)
    nans = same_with_nans(b, out)
    assert nans.any() and not nans[0].all() and not nans[3, G].any()
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("G,q,d,n", [(4, 3, 128, 3), (4, 6, 64, 90), (4, 14, 128, 160), (3, 100, 128, 3),
                                     (8, 90, 64, 100)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_nan_queries_stay_in_their_rows(pa, G, q, d, n, dtype):
    b = Batch(38, np.full(n, 3 * q), 2, G, d, 16, dtype, q_lens=[q] * n)
    b.q[q // 2, G, 3] = float("nan")
    b.q[-1, 0, :] = float("nan")
    nans = same_with_nans(b, b.prefill(pa))
    assert nans.sum() == 2 * d
    assert pa.pa_device_errors() == 0


def test_decode_bad_block_and_bad_length(pa):
    b = Batch(36, [500, 900, 64], 2, 4, 128, 16, "fp16")
    good = b.tables.copy()
    b.tables[1, 7] = b.NB + 3
    out = b.decode(pa, 256)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_BLOCK
    assert torch.isfinite(out).all()
    b.tables = good
    b.check(out, rows=[0, 2])
    lens, b.lens = b.lens, b.lens.copy()
    b.lens[2] = 100000
    out = b.decode(pa, 0, maxctx=900)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_LEN
    assert (out[2] == 0).all()
    b.lens = lens
    b.check(out, rows=[0, 1])


PREFILL = [
    ([20, 37, 1, 64], [9, 9, 1, 9], 4, 1, 64, 16, "fp16"),
    ([30, 17], [30, 17], 2, 2, 64, 16, "bf16"),
    ([50, 3, 100], [1, 1, 1], 2, 4, 128, 32, "fp16"),
    ([600, 1500, 33], [300, 300, 33], 2, 4, 128, 16, "fp16"),
    ([200, 90], [77, 77], 2, 3, 128, 16, "bf16"),
    ([130, 1000, 31], [65, 65, 31], 2, 8, 128, 32, "fp16"),
    ([300, 64], [300, 64], 1, 8, 64, 32, "bf16"),
    ([100, 40], [100, 40], 3, 1, 128, 16, "fp16"),
    ([400, 900, 61], [140, 0, 61], 1, 5, 128, 32, "fp16"),
    ([260, 45, 700], [37, 37, 37], 1, 7, 128, 16, "bf16"),
    ([900, 300, 1700], [256, 256, 256], 1, 4, 64, 16, "fp16"),
    ([64, 128, 65, 127, 63], [64, 128, 65, 127, 63], 1, 2, 128, 16, "fp16"),
    ([15, 16, 17, 31, 32, 33], [15, 1, 2, 16, 32, 17], 1, 6, 64, 32, "bf16"),
]


@pytest.mark.parametrize("lens,q_lens,H,G,d,bs,dtype", PREFILL)
def test_prefill_cases(pa, lens, q_lens, H, G, d, bs, dtype):
    b = Batch(51, lens, H, G, d, bs, dtype, ks=0.7, vs=1.5, q_lens=q_lens)
    b.check(b.prefill(pa))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("i", range(24))
def test_prefill_random_shapes(pa, i):
    rng = np.random.default_rng(600 + i)
    lens = rng.integers(1, 1501, int(rng.integers(1, 5)))
    q_lens = np.minimum(lens, int(rng.choice([1, 2, 5, 16, 33, 64, 100, 257, 700])))
    b = Batch(700 + i, lens, int(rng.integers(1, 5)), int(rng.integers(1, 9)),
              int(rng.choice([64, 128])), int(rng.choice([16, 32])), str(rng.choice(["fp16", "bf16"])),
              ks=float(rng.choice([1.0, 0.3])), vs=float(rng.choice([1.0, 5.0])), q_lens=q_lens)
    b.check(b.prefill(pa))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 24, 25, 48, 63, 64, 65, 127, 128, 129, 255,
                                  256, 257, 300])
@pytest.mark.parametrize("G,d,bs,dtype", [(1, 128, 16, "fp16"), (8, 64, 32, "bf16"),
                                          (3, 128, 32, "bf16")])
def test_prefill_few_sequences_beside_a_long_one(pa, rows, G, d, bs, dtype):
    """The table has room for the longest context, so the keys of the short ones
    are fewer than the work is split for."""
    q = -(-rows // G)
    lens = [2600, q, q + 1, q + 40, q + 65]
    b = Batch(900 + rows, lens, 2, G, d, bs, dtype, ks=0.5, vs=2.0, q_lens=[q, q, q, max(1, q // 2), q])
    b.check(b.prefill(pa))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("n", [39, 64, 200, 256, 257])
@pytest.mark.parametrize("q,G,d,bs,dtype", [(0, 2, 64, 16, "fp16"), (3, 2, 64, 32, "bf16"),
                                            (6, 4, 64, 16, "fp16"), (13, 4, 64, 16, "bf16")])
@pytest.mark.parametrize("longest", [900, 1500])
def test_many_sequences_of_unequal_contexts(pa, n, q, G, d, bs, dtype, longest):
    """Every sequence is served once, in whichever order the kernels take them;
    q = 0: decode.  Zero and equal lengths among them."""
    rng = np.random.default_rng(n + q)
    lens = rng.integers(0, 90, n)
    lens[rng.integers(0, n, 5)] = rng.integers(500, longest, 5)
    lens[n // 2], lens[::7] = longest, 33
    if q == 0:
        b = Batch(57, lens, 8, G, d, bs, dtype)
        b.check(b.decode(pa, 0))
    else:
        b = Batch(58, lens, 8, G, d, bs, dtype, q_lens=np.minimum(lens, rng.integers(0, q + 1, n)))
        b.check(b.prefill(pa))
    assert pa.pa_device_errors() == 0


def test_prefill_more_sequences_than_multiprocessors(pa):
    rng = np.random.default_rng(77)
    lens = rng.integers(20, 400, 170)
    b = Batch(54, lens, 2, 2, 128, 16, "fp16", q_lens=[20] * 170)
    b.check(b.prefill(pa))
    assert pa.pa_device_errors() == 0


def test_prefill_keeps_the_mass_of_a_long_faint_tail(pa):
    n, d, bs = 9001, 64, 16
    b = Batch(52, [n], 1, 2, d, bs, "fp16", q_lens=[3])
    kcodes, kscales = F.views(b.kc, bs, d)
    vcodes, vscales = F.views(b.vc, bs, d)
    kcodes[...] = 0
    kscales[...] = 0x38
    vcodes[...], vscales[...] = 0x77, 0x58
    blk = b.tables[0, 100]
    kcodes[blk, :, 5] = 0x22
    vscales[blk, :, 5] = 0x20
    b.q = torch.from_numpy(np.full((3, 2, d), 25 * np.log(2) * np.sqrt(d) / d)).half()
    b.check(b.prefill(pa))


@pytest.mark.parametrize("G,q,d,bs,dtype,n", [
    (4, 2, 128, 16, "fp16", 3), (4, 5, 128, 32, "bf16", 3), (3, 7, 64, 16, "fp16", 3),
    (2, 12, 64, 32, "bf16", 80), (1, 24, 128, 16, "bf16", 170),
    (4, 12, 128, 16, "fp16", 160), (2, 30, 64, 32, "bf16", 160), (8, 8, 128, 32, "bf16", 155),
    (4, 20, 128, 16, "bf16", 3), (8, 70, 64, 16, "fp16", 3), (2, 150, 128, 32, "fp16", 2),
    (5, 60, 128, 16, "fp16", 100), (1, 300, 64, 32, "bf16", 80)])
def test_prefill_nan_reaches_only_the_rows_that_attend_to_it(pa, G, q, d, bs, dtype, n):
    """NaN groups of K and of V among the chunk's own tokens and before them:
    the rows before a NaN keep their values, a row that attends to a NaN of V is
    NaN in that group's dimensions alone, one that attends to a NaN of K in all."""
    rng = np.random.default_rng(G * 1000 + q)
    lens = rng.integers(q, q + 150, n)
    lens[0] = 700 + q
    b = Batch(56, lens, 2, G, d, bs, dtype, ks=0.5, vs=2.0, q_lens=[q] * n)
    vs, ks = F.views(b.vc, bs, d)[1], F.views(b.kc, bs, d)[1]
    for i in range(n):
        at = lens[i] - q + rng.integers(0, q, 2)           # two of the chunk's tokens
        for j, h, group in ((at[0], 0, rng.integers(d // 16)), (at[1], 0, rng.integers(d // 16))):
            vs[b.tables[i, j // bs], h, j % bs, group] = NAN_SCALE
        if i % 3 == 0 and lens[i] > q:                     # one before the chunk
            j = rng.integers(0, lens[i] - q)
            vs[b.tables[i, j // bs], 1, j % bs, rng.integers(d // 16)] = NAN_SCALE
        if i % 4 == 1:                                     # a K of the chunk
            j = lens[i] - 1 - rng.integers(0, q)
            ks[b.tables[i, j // bs], 1, j % bs, 0] = NAN_SCALE
    with np.errstate(invalid="ignore"):
        ref, A = b.reference(), b.reference(True)
    out = b.prefill(pa)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.isnan(ref).any() and not np.isnan(ref).all()
    eps = torch.finfo(TYPES[dtype]).eps / 2
    tol = eps * np.abs(ref) * (1 + 2 ** -8) + A * (2 ** -11 + 2 ** -12) + 2.0 ** -24
    live = ~np.isnan(ref)
    assert (np.abs(got - ref)[live] <= tol[live]).all()
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("q,d", [(300, 128), (20, 128), (200, 64), (10, 64)])
def test_prefill_bad_block_and_bad_length(pa, q, d):
    b = Batch(53, [700, 1400, 900], 2, 4, d, 16, "fp16", q_lens=[q, q, q])
    good = b.tables.copy()
    b.tables[1, 5] = b.NB + 7
    out = b.prefill(pa)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_BLOCK
    assert torch.isfinite(out).all()
    b.tables = good
    rows = np.r_[0:q, 2 * q:3 * q]
    b.check(out, rows=rows)
    lens, b.lens = b.lens, b.lens.copy()
    b.lens[1] = q - 1                         # fewer tokens than the chunk has
    out = b.prefill(pa)
    assert pa.pa_device_errors() == pa.DEVERR_BAD_LEN
    assert torch.isnan(out[q:2 * q]).all()    # skipped: left as it was
    b.lens = lens
    b.check(out, rows=rows)


# ------------------------------------------------------------------------ together

def test_pool_beyond_four_gigabytes(pa):
    """Byte offsets past 2^32: the last blocks of a 5 GB pool pair."""
    d, bs, H = 128, 16, 8
    NB = (5 << 30) // (H * bs * d * 9 // 16)
    kc = torch.empty(NB, H, bs * d * 9 // 16, dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    rng = np.random.default_rng(61)
    n = 50
    k, v = rows(rng, n, H, d, "fp16"), torch.from_numpy(rng.standard_normal((n, H, d))).half()
    k = torch.from_numpy(rng.standard_normal((n, H, d))).half()
    tables = np.array([[NB - 1, NB // 2, NB - 2, NB - 3]], np.int32)
    j = np.arange(n)
    slots = tables[0, j // bs].astype(np.int64) * bs + j % bs
    pa.pa_reshape_and_cache_fp4(k.cuda(), v.cuda(), kc, vc, dev(slots), 1.0, 1.0)
    ids = torch.from_numpy(tables[0].astype(np.int64)).cuda()
    small = [c[ids].cpu().numpy() for c in (kc, vc)]
    for c, x in zip(small, (k, v)):
        codes, scales = F.quantise(x.float().numpy(), 1.0)
        cv, sv = F.views(c, bs, d)
        got = cv.transpose(0, 2, 1, 3).reshape(-1, H, d // 2)[:n]
        assert np.array_equal(got, codes)
        assert np.array_equal(sv.transpose(0, 2, 1, 3).reshape(-1, H, d // 16)[:n], scales)
    o, p = torch.zeros(n, H, d, dtype=torch.float16, device="cuda"), torch.zeros(n, H, d, dtype=torch.float16, device="cuda")
    pa.pa_gather_cache_fp4(o, p, kc, vc, dev(slots))
    kv = F.values(small[0], bs, d, 1.0).transpose(0, 2, 1, 3).reshape(-1, H, d)[:n]
    assert np.array_equal(f64(o), kv)
    b = Batch(62, [n], H, 4, d, bs, "fp16", q_lens=[7])
    b.kc, b.vc, b.tables = small[0], small[1], np.arange(4, dtype=np.int32)[None]
    out = torch.zeros_like(b.q, device="cuda")
    args = (kc, vc, dev(tables), dev(b.lens), b.scale, 1.0, 1.0)
    pa.pa_prefill_fp4(out, b.q.cuda(), dev(b.start), *args, 7)
    b.check(out)
    b.q, b.start = b.q[:1], None
    out = torch.zeros_like(b.q, device="cuda")
    pa.pa_decode_fp4(out, b.q.cuda(), *args, n, 16)
    b.check(out)
    assert pa.pa_device_errors() == 0


def serve(pa, stream=None, graph=False):
    """A prompt is written and attended to in two chunks, then six tokens are
    decoded one by one; the caches are read back at the end.  Returns outputs
    and what they should be."""
    H, G, d, bs, lens = 2, 4, 128, 16, [70, 33]
    rng = np.random.default_rng(71)
    NB = 14
    tables = rng.permutation(NB)[:12].reshape(2, 6).astype(np.int32)
    kc, vc = pa.new_fp4_cache(NB, H, bs, d), pa.new_fp4_cache(NB, H, bs, d)
    hk, hv = kc.cpu().numpy(), vc.cpu().numpy()
    bt = dev(tables)
    ws = pa.new_decode_workspace(2, H * G, d, 96, 32)
    scale = 1 / np.sqrt(d)

    def slot(i, j):
        return int(tables[i, j // bs]) * bs + j % bs

    steps, want = [], []
    at = [0, 0]
    for chunk in ([40, 20], [30, 13], *[[1, 1]] * 6):
        n = [a + c for a, c in zip(at, chunk)]
        slots = np.array([slot(i, j) for i in range(2) for j in range(at[i], n[i])])
        T = len(slots)
        k, v = (torch.from_numpy(rng.standard_normal((T, H, d))).to(torch.bfloat16) for _ in range(2))
        q = torch.from_numpy(rng.standard_normal((T, H * G, d))).to(torch.bfloat16)
        start = np.array([0, chunk[0], T], np.int32)
        F.reshape_and_cache(k.float().numpy(), v.float().numpy(), hk, hv, slots, bs, 0.5, 1.0)
        kv, vv = F.values(hk, bs, d, 0.5), F.values(hv, bs, d, 1.0)
        a = (f64(q), start, kv)
        want.append((F.prefill(*a, vv, tables, n, scale), F.prefill(*a, np.abs(vv), tables, n, scale)))
        steps.append((k.cuda(), v.cuda(), q.cuda(), dev(slots), dev(start),
                      dev(np.array(n, np.int32)), torch.empty_like(q, device="cuda"), max(chunk)))
        at = n
    every = np.array([slot(i, j) for i in range(2) for j in range(at[i])])
    back = [torch.empty(len(every), H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots_all = dev(every)
    want_back = [F.values(c, bs, d, g)[every // bs, :, every % bs] for c, g in ((hk, 0.5), (hv, 1.0))]

    def run(s=None):
        for k, v, q, sm, start, cl, out, most in steps:
            pa.pa_reshape_and_cache_fp4(k, v, kc, vc, sm, 0.5, 1.0, stream=s)
            if most > 1:
                pa.pa_prefill_fp4(out, q, start, kc, vc, bt, cl, scale, 0.5, 1.0, most, stream=s)
            else:
                pa.pa_decode_fp4(out, q, kc, vc, bt, cl, scale, 0.5, 1.0, 96, 32, ws, stream=s)
        pa.pa_gather_cache_fp4(*back, kc, vc, slots_all, 0.5, 1.0, stream=s)

    def check():
        torch.cuda.synchronize()
        for (ref, A), st in zip(want, steps):
            tol = 2 ** -8 * np.abs(ref) * (1 + 2 ** -8) + A * (2 ** -11 + 2 ** -12) + 2.0 ** -24
            assert (np.abs(f64(st[6]) - ref) <= tol).all()
        for got, ref in zip(back, want_back):
            assert (np.abs(f64(got) - ref) <= np.abs(ref) * (2 ** -8 + 2 ** -22)).all()
        assert pa.pa_device_errors() == 0

    def clear():
        kc.zero_()
        vc.zero_()
        for st in steps:
            st[6].zero_()
        for x in back:
            x.zero_()
        torch.cuda.synchronize()

    return run, check, clear


def test_serving_steps_together(pa):
    run, check, clear = serve(pa)
    run()
    check()
    clear()
    run()
    check()


def test_serving_steps_on_another_stream(pa):
    run, check, clear = serve(pa)
    clear()
    run(torch.cuda.Stream())
    check()
    clear()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(s.cuda_stream)
    check()


def test_serving_steps_captured_and_replayed(pa):
    run, check, clear = serve(pa)
    run()  # the first launches set the kernels' attributes
    clear()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(2):
        clear()
        g.replay()
        check()


def test_calls_at_once_on_two_streams(pa):
    """Two batches, each on a stream and with a workspace of its own."""
    both = []
    for i, (lens, ps) in enumerate((([3000, 700, 5, 1900], 256), ([900] * 12, 64))):
        b = Batch(60 + i, lens, 2, 4, 128, 16, "fp16")
        p = Batch(62 + i, [400, 1300, 300], 2, 4, 128, 16, "bf16", q_lens=[200, 6, 300])
        dec, pre = b.gpu(), p.gpu()
        ws = pa.new_decode_workspace(len(lens), 8, 128, 3000, ps)
        outs = [torch.full_like(x.q, float("nan"), device="cuda") for x in (b, p)]
        both.append((b, p, dec, pre, ws, ps, outs, b.q.cuda(), p.q.cuda(), dev(p.start),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        for b, p, dec, pre, ws, ps, outs, q, pq, start, st in both:
            pa.pa_decode_fp4(outs[0], q, *dec, b.scale, 1.0, 1.0, 3000, ps, ws, st)
            pa.pa_prefill_fp4(outs[1], pq, start, *pre, p.scale, 1.0, 1.0, 300, st)
    torch.cuda.synchronize()
    for b, p, dec, pre, ws, ps, outs, *_ in both:
        b.check(outs[0])
        p.check(outs[1])
    assert pa.pa_device_errors() == 0


def test_decode_makes_its_own_workspace_on_the_calls_stream(pa):
    b = Batch(72, [3000, 100], 2, 4, 128, 16, "fp16")
    s = torch.cuda.Stream()
    out = torch.zeros_like(b.q, device="cuda")
    torch.cuda.synchronize()
    b.check(b.decode(pa, 256, stream=s, out=out))
    b.check(b.decode(pa, 256, stream=s.cuda_stream, out=out.zero_()))


def test_blocks_fork_and_swap(pa):
    """pa_swap_blocks moves FP4 blocks, within one pool (a copy-on-write fork)
    and to a pinned host pool and back."""
    b = Batch(73, [100, 40], 2, 2, 64, 16, "fp16", slack=4)
    kc, vc, bt, cl = b.gpu()
    free = sorted(set(range(b.NB)) - set(b.tables[b.tables >= 0].tolist()))
    moved = b.tables.copy()
    pairs = [(int(b.tables[0, 1]), free[0]), (int(b.tables[1, 2]), free[1])]
    moved[0, 1], moved[1, 2] = free[0], free[1]
    for c in (kc, vc):
        pa.pa_swap_blocks(c, c, dev(np.array(pairs, np.int64)))
    out = torch.zeros_like(b.q, device="cuda")
    pa.pa_decode_fp4(out, b.q.cuda(), kc, vc, dev(moved), cl, b.scale, b.ks, b.vs, 100)
    b.check(out)
    host = [torch.empty(b.NB, *c.shape[1:], dtype=torch.uint8).pin_memory() for c in (kc, vc)]
    ids = np.arange(b.NB, dtype=np.int64)
    there = dev(np.stack([ids, ids[::-1]], 1))
    back = dev(np.stack([ids[::-1], ids], 1))
    for c, h in zip((kc, vc), host):
        pa.pa_swap_blocks(c, h, there)
        c2 = c.clone()
        c.zero_()
        pa.pa_swap_blocks(h, c, back)
        assert torch.equal(c, c2)


def test_binding_refuses_what_does_not_fit(pa):
    kc = pa.new_fp4_cache(4, 2, 16, 64)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    bt = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    cl = torch.ones(3, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    sm = torch.zeros(3, dtype=torch.int64, device="cuda")
    ok = (q, q, kc, kc, bt, cl, 0.1, 1.0, 1.0, 10)

    def decode(i, x):
        return pa.pa_decode_fp4(*ok[:i], x, *ok[i + 1:])

    for i, x in ((0, q[:2]), (1, q.float()), (2, kc[:, :, ::2]), (2, kc.to(torch.int16)), (3, kc[:2]),
                 (4, bt[:2]), (4, bt.long()), (5, cl[:2])):
        with pytest.raises(ValueError):
            decode(i, x)
    for x in (-1.0, 0.0, float("nan")):
        with pytest.raises(pa.PaError):
            decode(7, x)
    with pytest.raises(pa.PaError):
        pa.pa_decode_fp4(*ok, 8)  # a partition size that is no multiple of 16
    with pytest.raises(ValueError):
        pa.pa_prefill_fp4(q, q, qs[:3], kc, kc, bt, cl, 0.1, 1.0, 1.0, 1)
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_fp4(k.transpose(0, 1), k.transpose(0, 1), kc, kc, sm)
    with pytest.raises(ValueError):
        pa.pa_gather_cache_fp4(k, k[:2], kc, kc, sm)
    with pytest.raises(ValueError):
        pa.pa_gather_cache_fp4(k, k, kc, kc, sm[:2])
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_fp4(k.float(), k.float(), kc, kc, sm)
    assert pa.pa_device_errors() == 0
