"""GPU parity of the rotated append (pa_rope_and_cache and its FP8 and FP4 forms).

Every step is an IEEE operation that the reference makes, too: the queries and
the caches are compared bit for bit, and every byte that no token owns must stay
as it was."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.fp4 as F
import oracle.sparse as S
from test_gpu_fp4 import TYPES, dev, pa  # noqa: F401  (pa is the fixture)

pytestmark = pytest.mark.gpu


def u16(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def table(rng, n, rotary):
    """Cosines and sines of a model, and in some rows any numbers."""
    freq = 10000.0 ** (-np.arange(rotary // 2) * 2 / rotary)
    a = rng.integers(0, 100000, n)[:, None] * freq
    t = np.concatenate([np.cos(a), np.sin(a)], 1)
    t[n // 2:] *= rng.standard_normal((n - n // 2, 1))
    return t.astype(np.float32)


class Case:
    def __init__(self, seed, T, Hq, Hkv, d, bs, dtype, kv, rotary, interleaved, ks=1.0, vs=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.kv, self.bs, self.d, self.ks, self.vs, self.interleaved = kv, bs, d, ks, vs, interleaved
        self.dtype, t = dtype, TYPES[dtype]
        self.q, self.k, self.v = (torch.from_numpy(rng.standard_normal((T, h, d)) * np.exp2(
            rng.integers(-6, 6, (T, h, 1)))).to(t) for h in (Hq, Hkv, Hkv))
        self.table = table(rng, 64, rotary)
        self.pos = rng.integers(0, 64, T)
        NB = -(-T // bs) + 2
        self.slots = rng.permutation(NB * bs)[:T]
        self.slots[rng.random(T) < 0.15] = -1
        if kv == "16":
            self.pool = [rng.integers(0, 2 ** 16, (NB, Hkv, bs, d)).astype(np.uint16) for _ in range(2)]
        else:
            size = (bs, d) if kv == "fp8" else (bs * d * 9 // 16,)
            self.pool = [rng.integers(0, 256, (NB, Hkv, *size)).astype(np.uint8) for _ in range(2)]

    def want(self):
        """Queries and caches, as bits."""
        ok = (self.slots >= 0) & (self.slots < self.pool[0].shape[0] * self.bs)
        ok &= (self.pos >= 0) & (self.pos < len(self.table))
        slots = np.where(ok, self.slots, -1)
        q, k = (torch.from_numpy(S.rotate(x.float().numpy(), self.pos, self.table, self.interleaved)).to(x.dtype)
                for x in (self.q, self.k))
        c = [p.copy() for p in self.pool]
        if self.kv == "16":
            oracle.reshape_and_cache(k, self.v, *c, torch.from_numpy(slots))
        elif self.kv == "fp8":
            oracle.reshape_and_cache_fp8(k, self.v, *c, torch.from_numpy(slots), self.dtype, self.ks, self.vs)
        else:
            F.reshape_and_cache(k.float().numpy(), self.v.float().numpy(), *c, slots, self.bs, self.ks, self.vs)
        return ok, u16(q), c

    def caches(self):
        if self.kv == "16":
            return [dev(p.view(np.int16)).view(TYPES[self.dtype]) for p in self.pool]
        return [dev(p) for p in self.pool]

    def call(self, pa, out, q, k, v, caches, **kw):  # noqa: F811
        scales = () if self.kv == "16" else (self.ks, self.vs)
        f = getattr(pa, "pa_rope_and_cache" + {"16": "", "fp8": "_fp8", "fp4": "_fp4"}[self.kv])
        return f(out, q, k, v, *caches, dev(self.slots.astype(np.int64)), dev(self.pos.astype(np.int64)),
                 dev(self.table), *scales, interleaved=self.interleaved, **kw)

    def check(self, out, caches, before=7.0):
        ok, q, c = self.want()
        got = u16(out)
        assert np.array_equal(got[ok], q[ok])
        assert (out[torch.from_numpy(~ok)] == before).all()
        for a, b in zip(caches, c):
            a = u16(a) if self.kv == "16" else a.cpu().numpy()
            assert np.array_equal(a, b)


SHAPES = [
    # T, Hq, Hkv, d, bs, dtype, rotary, interleaved
    (1, 1, 1, 64, 16, "fp16", 64, False), (3, 4, 4, 64, 16, "fp16", 64, True),
    (33, 32, 8, 128, 16, "bf16", 128, False), (20, 64, 8, 128, 32, "fp16", 128, True),
    (17, 5, 3, 128, 32, "bf16", 16, False), (40, 7, 7, 64, 32, "fp16", 48, False),
    (9, 3, 2, 128, 16, "bf16", 112, True), (65, 12, 1, 64, 16, "bf16", 32, True),
    (2, 100, 50, 128, 16, "fp16", 96, False), (300, 1, 1, 128, 16, "bf16", 80, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,bs,dtype,rotary,interleaved", SHAPES)
@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
@pytest.mark.parametrize("rows", ["packed", "fused"])
def test_append_bits(pa, T, Hq, Hkv, d, bs, dtype, rotary, interleaved, kv, rows):  # noqa: F811
    c = Case(T + Hq + rotary, T, Hq, Hkv, d, bs, dtype, kv, rotary, interleaved, 0.7, 0.25)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.full_like(q, 7.0)
    if rows == "fused":
        both = torch.cat([q, k, torch.zeros_like(k), v], 1)
        q, k, v = both[:, :Hq], both[:, Hq:Hq + Hkv], both[:, Hq + 2 * Hkv:]
        wide = torch.full((T, Hq + 2, d), 7.0, dtype=q.dtype, device="cuda")
        out = wide[:, 1:Hq + 1]
    caches = c.caches()
    assert c.call(pa, out, q, k, v, caches) is out
    c.check(out, caches)
    if rows == "fused":
        assert (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
def test_append_in_place(pa, kv):  # noqa: F811
    """query_out is query, a view of the fused rows: skipped rows keep their queries."""
    c = Case(5, 50, 16, 4, 128, 16, "fp16", kv, 128, False)
    both = torch.cat([c.q, c.k, c.v], 1).cuda()
    q, k, v = both[:, :16], both[:, 16:20], both[:, 20:]
    caches = c.caches()
    c.call(pa, q, q, k, v, caches)
    ok, want, _ = c.want()
    assert np.array_equal(u16(q)[ok], want[ok])
    assert np.array_equal(u16(q)[~ok], u16(c.q)[~ok])
    assert np.array_equal(u16(both[:, 16:]), u16(torch.cat([c.k, c.v], 1)))
    c.check(torch.where(torch.from_numpy(ok)[:, None, None].cuda(), q, 7.0), caches)


@pytest.mark.parametrize("kv", ["16", "fp8", "fp4"])
def test_slots_and_positions_outside_are_flagged_and_left_out(pa, kv):  # noqa: F811
    for what, flag in (("slot", "DEVERR_BAD_SLOT"), ("pos", "DEVERR_BAD_POS")):
        c = Case(6, 12, 8, 2, 64, 32, "bf16", kv, 64, True)
        c.slots = np.arange(12)
        total = c.pool[0].shape[0] * c.bs
        if what == "slot":
            c.slots[[2, 5]] = total, 1 << 40
        else:
            c.pos[[0, 3, 7]] = -1, len(c.table), 1 << 40
        out = torch.full_like(c.q, 7.0, device="cuda")
        caches = c.caches()
        c.call(pa, out, c.q.cuda(), c.k.cuda(), c.v.cuda(), caches)
        assert pa.pa_device_errors() == getattr(pa, flag)
        c.check(out, caches)
    # the position of a token without a slot is not looked at
    c.slots[:] = -1
    c.call(pa, out, c.q.cuda(), c.k.cuda(), c.v.cuda(), caches)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_infinities_and_nan_stay_in_their_pairs(pa, dtype):  # noqa: F811
    c = Case(7, 6, 2, 2, 64, 16, dtype, "16", 32, False)
    c.slots = np.arange(6)
    c.k[1, 0, 3], c.k[2, 1, 20], c.v[3, 0, 5], c.q[4, 1, 31] = math.nan, math.inf, math.nan, -math.inf
    out = torch.full_like(c.q, 7.0, device="cuda")
    caches = c.caches()
    c.call(pa, out, c.q.cuda(), c.k.cuda(), c.v.cuda(), caches)
    q, k = (S.rotate(x.float().numpy(), c.pos, c.table, False) for x in (c.q, c.k))
    for got, want in ((out, q), (caches[0][0, :, :6].transpose(0, 1), k)):
        got = got.float().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = np.isfinite(want)
        eps = torch.finfo(TYPES[dtype]).eps / 2  # one rounding to the type
        assert (np.abs(got[ok] - want[ok]) <= eps * np.abs(want[ok]) + 2.0 ** -25).all()
    assert np.isnan(k[1]).sum() == 2 and (~np.isfinite(k[2])).sum() == 2
    assert torch.isnan(caches[1]).sum() == torch.isnan(torch.from_numpy(c.pool[1].view(np.int16)).view(
        TYPES[dtype])[:, :, :]).sum() - torch.isnan(torch.from_numpy(c.pool[1].view(np.int16)).view(
            TYPES[dtype])[0, :, :6]).sum() + 1


def test_refused_arguments(pa):  # noqa: F811
    c = Case(8, 4, 4, 2, 64, 16, "fp16", "16", 64, False)
    q, k, v, (kc, vc) = c.q.cuda(), c.k.cuda(), c.v.cuda(), c.caches()
    out, sl, pos, tb = torch.empty_like(q), dev(c.slots.astype(np.int64)), dev(c.pos.astype(np.int64)), dev(c.table)
    good = [out, q, k, v, kc, vc, sl, pos, tb]
    pa.pa_rope_and_cache(*good)
    for at, bad in ((0, out[:3]), (0, out.float()), (1, q.cpu()), (1, q.transpose(0, 1)), (2, k[:, :1]),
                    (2, k.bfloat16()), (3, v[..., ::2]), (4, kc[:, :1]), (4, kc.to(torch.uint8)),
                    (5, vc.transpose(2, 3)), (6, sl.int()), (6, sl[:3]), (7, pos[1:]), (7, None),
                    (8, tb.double()), (8, tb[0]), (8, tb.t())):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            pa.pa_rope_and_cache(*args)
    with pytest.raises(pa.PaError):
        pa.pa_rope_and_cache(*good[:8], tb[:, :24].contiguous())
    odd = torch.zeros(4, 4 * 64 + 4, dtype=torch.float16, device="cuda")[:, :256].unflatten(1, (4, 64))
    with pytest.raises(pa.PaError):
        pa.pa_rope_and_cache(out, odd, *good[2:])
    assert pa.pa_device_errors() == 0


def test_no_tokens_and_another_stream(pa):  # noqa: F811
    c = Case(9, 64, 16, 8, 128, 16, "bf16", "fp8", 128, False)
    empty = torch.zeros(0, 16, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    caches = c.caches()
    pa.pa_rope_and_cache_fp8(empty, empty, empty[:, :8], empty[:, :8], *caches, none, none, dev(c.table), 1.0, 1.0)
    side = torch.cuda.Stream()
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    c.call(pa, out, q, k, v, caches, stream=side)
    side.synchronize()
    c.check(out, caches)
    assert pa.pa_device_errors() == 0
