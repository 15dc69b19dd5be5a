"""CPU checks of rotated append and sparse attention: the definitions in
``oracle/sparse.py`` against closed forms and invariants, and the refusals of
the C entry points and of the binding."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import oracle.sparse as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ definitions

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(interleaved):
    """In 64 bits of a table in 32: a pair's length stays, and the product of a
    rotated query and key depends on the distance of their positions alone."""
    rng = np.random.default_rng(0)
    r, d, n = 48, 64, 4000
    freq = 10000.0 ** (-np.arange(r // 2) * 2 / r)
    angle = np.arange(n)[:, None] * freq
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    q, k = rng.standard_normal((2, 1, 1, d)).astype(np.float32)

    def dot(p, s):
        return float((S.rotate(q, [p], table, interleaved).astype(np.float64)
                      * S.rotate(k, [s], table, interleaved)).sum())

    # every element is off by at most three roundings of fp32 and the table's two
    bound = 5 * 2.0 ** -24 * 4 * float(np.abs(q).sum() * np.abs(k).max())
    for p, s, by in ((5, 3, 100), (17, 900, 2000), (0, 0, 3999)):
        assert abs(dot(p, s) - dot(p + by if p + by < n else p, s + by if p + by < n else s)) <= bound
    x = S.rotate(q, [1234], table, interleaved).astype(np.float64)
    assert abs((x ** 2).sum() - (q.astype(np.float64) ** 2).sum()) <= bound
    assert np.array_equal(x[..., r:], q[..., r:])


def test_rotation_of_a_quarter_turn():
    table = np.array([[1, 1, 0, 0], [0, -1, 1, 0]], np.float32)  # cos, cos, sin, sin
    x = np.array([[[1, 2, 3, 4, 5]]], np.float32)
    assert S.rotate(x, [0], table, False).tolist() == x.tolist()
    assert S.rotate(x, [1], table, False).tolist() == [[[-3, -2, 1, -4, 5]]]
    assert S.rotate(x, [1], table, True).tolist() == [[[-2, 1, -3, -4, 5]]]


@pytest.mark.parametrize("mag", [1e-30, 1.0, 3e4])
def test_bounds_bound_every_key(mag):
    rng = np.random.default_rng(1)
    for _ in range(30):
        k = rng.standard_normal((int(rng.integers(1, 17)), 64)) * mag * np.exp2(rng.integers(-9, 3, 64))
        codes, g = S.bounds_of(k)
        assert (codes[0] * g >= k.max(0)).all() and (codes[1] * g <= k.min(0)).all()
        assert (codes[0] * g < k.max(0) + g).all() and (codes[1] * g > k.min(0) - g).all()
        assert math.frexp(g)[0] == 0.5 and np.abs(k).max() > 63.5 * g
        q = rng.standard_normal((4, 64))
        s = S.scores(q, codes[None], np.array([g]))[0] * 2.0 ** S.exponent(np.abs(q).max(), 4095)
        # the queries' rounding: half a unit of each, times a bound
        slack = 4 * 64 * 0.5 * 2.0 ** S.exponent(np.abs(q).max(), 4095) * 128 * g
        assert s >= (q @ k.T).sum(0).max() - slack


def test_bounds_of_odd_blocks():
    k = np.ones((3, 64))
    assert S.bounds_of(k * 0)[1] == 0 and not S.bounds_of(k * 0)[0].any()
    for odd in (math.inf, -math.inf, math.nan):
        k[1, 7] = odd
        codes, g = S.bounds_of(k)
        assert g == math.inf and not codes.any()
    codes, g = S.bounds_of(np.full((1, 64), 127.0))
    assert g == 1 and (codes == 127).all()
    assert S.bounds_of(np.full((1, 64), -127.5))[1] == 2


def test_choice_takes_ties_in_order_and_keeps_both_ends():
    s = np.array([5, 1, 7, 7, 7, 0, 7, -1, 2], np.float32)
    assert S.choose(s, 3, 0, 0) == [2, 3, 4]
    assert S.choose(s, 4, 1, 1) == [0, 2, 3, 8]
    assert S.choose(s, 9, 1, 1) == list(range(9))
    assert S.choose(s, 2, 0, 2) == [7, 8]
    assert S.choose(s, 1, 1, 0) == [0]


# ------------------------------------------------------------ the C entry points

@pytest.fixture(scope="module")
def pa():
    from pagedattention_kv_cache_attention_gb300 import build
    build.build()
    import pagedattention_kv_cache_attention_gb300 as pa
    pa._load()
    return pa


def prototypes():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pa.h")).read(), flags=re.S)
    return dict(re.findall(r"\b(pa_[a-z_0-9]+)\s*\(([^)]*)\)", text))


def test_bindings_have_the_headers_arguments(pa):
    """One letter for each parameter of the prototype, and of its type."""
    kinds = {"int32_t": "i", "int64_t": "l", "float": "f", "size_t": "z"}
    known = prototypes()
    for name, letters in pa._SPARSE_ARGS.items():
        want = ""
        for p in known[name].split(","):
            want += "P" if "*" in p else kinds[p.split()[-2]]
        assert letters == want, name


FAKE = 0x10000  # never dereferenced: every call below is refused by a host check
ROPE = dict(qo=FAKE, q=FAKE, k=FAKE, v=FAKE, qos=512, qs=512, ks=256, vs=256, kc=FAKE, vc=FAKE,
            slots=FAKE, pos=FAKE, table=FAKE, T=4, Hq=4, Hkv=2, d=128, rot=128, inter=0, bs=16, NB=64,
            most=100, dt=0)
BOUNDS = dict(b=FAKE, s=FAKE, kc=FAKE, bt=FAKE, mb=4, cl=FAKE, qs=None, B=2, mq=1, Hkv=2, d=128,
              bs=16, NB=64, dt=0)
SELECT = dict(t=FAKE, n=FAKE, q=FAKE, b=FAKE, s=FAKE, bt=FAKE, mb=4, cl=FAKE, qs=None, B=2, mq=1, Hq=4,
              Hkv=2, d=128, bs=16, NB=64, mc=64, keep=2, sink=1, recent=1, dt=0)
SPARSE = dict(o=FAKE, q=FAKE, kc=FAKE, vc=FAKE, t=FAKE, n=FAKE, R=2, keep=4, Hq=4, Hkv=2, d=128,
              bs=16, NB=64, scale=0.1, dt=0)


def status(pa, name, base, over, scales=None):
    args = dict(base)
    assert set(over) <= set(args) | {"ks_", "vs_"}
    args.update({k: v for k, v in over.items() if k in args})
    dt = args.pop("dt")
    vals = list(args.values())
    if "update" in name:
        tail = [] if name.endswith(("fp8", "fp4")) else [dt]
    elif scales is None:
        tail = [dt]
    else:
        tail = [dt, *scales] if "rope" in name else [*scales, dt]
    return pa._sparse_fn(name)(*vals, *tail, None)


@pytest.mark.parametrize("over,want", [
    (dict(T=0), 0), (dict(T=-1), 1), (dict(d=96), 2), (dict(bs=8), 2), (dict(rot=120), 2),
    (dict(rot=144), 2), (dict(rot=0), 1), (dict(rot=8), 2), (dict(inter=2), 1), (dict(Hq=0), 1),
    (dict(Hkv=0), 1), (dict(NB=0), 1), (dict(most=0), 1), (dict(dt=3), 1), (dict(qos=504), 1),
    (dict(qs=516), 1), (dict(ks=255), 1), (dict(vs=260), 1), (dict(pos=None), 1), (dict(table=None), 1),
    (dict(table=FAKE + 4), 1), (dict(q=FAKE + 2), 1), (dict(qo=None), 1), (dict(kc=FAKE + 8), 1),
    (dict(Hq=2 ** 21, qs=2 ** 28, qos=2 ** 28), 2), (dict(NB=2 ** 33), 2)])
@pytest.mark.parametrize("end", ["", "_fp8", "_fp4"])
def test_append_refusals(pa, over, want, end):
    assert status(pa, "pa_rope_and_cache" + end, ROPE, over, (1.0, 1.0) if end else None) == want


@pytest.mark.parametrize("end", ["", "_fp8", "_fp4"])
def test_append_in_place_has_one_stride(pa, end):
    assert status(pa, "pa_rope_and_cache" + end, ROPE, dict(qs=520), (1.0, 1.0) if end else None) == 1


@pytest.mark.parametrize("heads", [65536, 2 ** 20])
def test_append_of_more_heads_than_an_fp4_block_has_offsets_for(pa, heads):
    """The heads of an FP4 block lie 2,304 bytes apart at most, and offsets within it are 32-bit: 2^20 heads
    pass 2^31 bytes.  The limit is that of pa_reshape_and_cache_fp4."""
    over = dict(Hkv=heads, ks=heads * 128, vs=heads * 128)
    assert status(pa, "pa_rope_and_cache_fp4", ROPE, over, (1.0, 1.0)) == 2


@pytest.mark.parametrize("scales", [(0.0, 1.0), (1.0, -1.0), (math.nan, 1.0), (1.0, math.inf)])
@pytest.mark.parametrize("end", ["_fp8", "_fp4"])
def test_cache_scales_are_checked(pa, scales, end):
    assert status(pa, "pa_rope_and_cache" + end, ROPE, {}, scales) == 1
    assert status(pa, "pa_decode_sparse" + end, SPARSE, {}, scales) == 1


@pytest.mark.parametrize("over,want", [
    (dict(B=0), 0), (dict(mq=0), 0), (dict(B=-1), 1), (dict(mq=-1), 1), (dict(mq=2), 1),
    (dict(d=80), 2), (dict(bs=64), 2), (dict(b=None), 1), (dict(b=FAKE + 8), 1), (dict(s=None), 1),
    (dict(kc=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(mb=0), 1), (dict(NB=0), 1),
    (dict(B=65536), 2), (dict(NB=2 ** 31), 2)])
@pytest.mark.parametrize("end", ["", "_fp8", "_fp4"])
def test_bounds_refusals(pa, over, want, end):
    assert status(pa, "pa_update_key_bounds" + end, BOUNDS, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(B=0), 0), (dict(mq=0), 0), (dict(B=-1), 1), (dict(mq=2), 1), (dict(Hq=5), 1),
    (dict(Hq=18), 2), (dict(d=80), 2), (dict(bs=8), 2), (dict(keep=0), 1), (dict(sink=-1), 1),
    (dict(recent=-1), 1), (dict(sink=2, recent=1), 1), (dict(mc=-1), 1), (dict(dt=2), 1),
    (dict(t=None), 1), (dict(n=None), 1), (dict(q=FAKE + 4), 1), (dict(b=FAKE + 1), 1),
    (dict(mb=49153, mc=49153 * 16), 2), (dict(keep=2 ** 27), 2), (dict(B=65536), 2)])
def test_select_refusals(pa, over, want):
    assert status(pa, "pa_select_blocks", SELECT, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(R=0), 0), (dict(R=-1), 1), (dict(keep=0), 1), (dict(Hq=5), 1), (dict(Hq=18), 2),
    (dict(d=80), 2), (dict(bs=8), 2), (dict(scale=math.nan), 1), (dict(o=None), 1),
    (dict(t=None), 1), (dict(n=None), 1), (dict(q=FAKE + 8), 1), (dict(R=65536), 2),
    (dict(keep=2 ** 28), 2)])
@pytest.mark.parametrize("end", ["", "_fp8", "_fp4"])
def test_sparse_refusals(pa, over, want, end):
    assert status(pa, "pa_decode_sparse" + end, SPARSE, over, (1.0, 1.0) if end else None) == want


def test_what_is_no_cuda_tensor_is_named(pa):
    """Host tensors and foreign objects are ValueErrors before anything is launched."""
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    for bad in (x, None, 3):
        with pytest.raises(ValueError):
            pa.pa_rope_and_cache(bad, bad, x, x, x, x, i64, i64, x)
        with pytest.raises(ValueError):
            pa.pa_update_key_bounds(bad, x, x, i32, i32)
        with pytest.raises(ValueError):
            pa.pa_select_blocks(i32, i32, bad, x, x, i32, i32, 16, 10)
        with pytest.raises(ValueError):
            pa.pa_decode_sparse(x, bad, x, x, i32, i32, 0.1)


def test_native_binding_leaves_what_does_not_fit(pa):
    """-1 for a wrong number of arguments, for what is no tensor, and for host tensors."""
    native = pa._native()
    x, i32 = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    for f, n in ((native.rope, 14), (native.key_bounds, 9), (native.select, 14), (native.sparse, 11)):
        assert f() == -1 and f(1, 2, 3) == -1
        for bad in (None, 0, x, i32, "", 2 ** 70):
            assert f(*[bad] * n) == -1
            assert f(0, *[bad] * (n - 1)) == -1


def test_rope_table_holds_far_angles(pa):
    t = pa.new_rope_table(100001, 32, base=500000.0, device="cpu")
    assert t.shape == (100001, 32) and t.dtype == torch.float32
    for p, i in ((0, 0), (100000, 0), (99999, 7), (12345, 15)):
        a = p * 500000.0 ** (-2 * i / 32)
        assert abs(float(t[p, i]) - math.cos(a)) <= 2.0 ** -24 and abs(float(t[p, 16 + i]) - math.sin(a)) <= 2.0 ** -24
    with pytest.raises(ValueError):
        pa.new_rope_table(10, 31, device="cpu")
