"""FP4 KV cache on the CPU: the 64-bit reference against facts the format
fixes, and the refusals of the four entry points, made on the host before
anything reaches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.fp4 as F

NAN = float("nan")


def test_e2m1_and_e4m3_tables():
    assert F.E2M1[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert F.E2M1[8:].tolist() == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    lib = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(F.E4M3, lib, equal_nan=True)


def test_every_product_of_code_and_scale_is_exact_in_fp16():
    p = F.E2M1[None, :] * F.E4M3[:127, None]
    assert np.array_equal(p.astype(np.float16).astype(np.float64), p)
    assert np.abs(p).max() == 2688 and np.abs(p[p != 0]).min() == 2.0 ** -10


@pytest.mark.parametrize("x,code", [
    (0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499999, 1), (1.25, 2), (1.75, 4), (2.5, 4),
    (2.5000003, 5), (3.5, 6), (5.0, 6), (5.000001, 7), (6.0, 7), (6.4, 7)])
def test_codes_and_ties(x, code):
    """A group whose largest element is 6 has scale 1: codes are the nearest of x."""
    row = np.zeros(16, np.float32)
    row[0], row[1], row[2] = 6.0, x if x < 6 else 6.0, -(x if x < 6 else 6.0)
    c, s = F.quantise(row, 1.0)
    assert F.E4M3[s[0]] == 1.0
    assert (c[0] & 15, c[0] >> 4, c[1] & 15) == (7, code, code + 8)


def test_scale_clamps_zero_groups_nan_and_infinity():
    x = np.zeros((5, 16), np.float32)
    x[1, 3] = 6 * 2.0 ** -10          # half of the smallest scale: ties to 0
    x[2, 3] = 1e30                    # saturates: scale 448, code 6
    x[3, 2], x[3, 5] = NAN, 7.0
    x[4, 2], x[4, 5] = -np.inf, 1.0
    c, s = F.quantise(x, 1.0)
    assert s[:, 0].tolist() == [0, 0, 0x7E, 0x7F, 0x7E]
    assert not c[0].any() and not c[1].any() and not c[3].any()
    assert c[2, 1] >> 4 == 7 and c[4, 1] & 15 == 15 and c[4, 2] >> 4 == 0


def test_rounding_error_bound():
    """|x - read back| <= half the largest E2M1 gap (1) + what the scale's own
    rounding (2^-4) can cut off the largest element (6 / 16), in scale units."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((64, 128)) * np.exp2(rng.integers(-4, 6, (64, 1)))).astype(np.float32)
    for g in (1.0, 0.7):
        c, s = F.quantise(x, g)
        e = np.stack([F.E2M1[c & 15], F.E2M1[c >> 4]], -1).reshape(x.shape)
        z = np.repeat(F.E4M3[s], 16, axis=-1) * float(np.float32(g))
        assert (np.abs(e * z - x) <= 1.0 * z * (1 + 1e-6)).all()


def test_views_and_round_trip_through_slots():
    rng = np.random.default_rng(1)
    bs, d, H = 16, 64, 2
    kc, vc = np.zeros((3, H, bs * d * 9 // 16), np.uint8), np.zeros((3, H, bs * d * 9 // 16), np.uint8)
    key = F.E2M1[rng.integers(0, 16, (5, H, d))]
    key[..., ::16] = 6  # every group's scale is 1, so every value is stored as it is
    slots = np.array([33, 2, -1, 47, 16])
    F.reshape_and_cache(key, key * 2, kc, vc, slots, bs, 1.0, 2.0)
    k, v = F.values(kc, bs, d, 1.0), F.values(vc, bs, d, 2.0)
    for t, s in enumerate(slots):
        if s >= 0:
            assert np.array_equal(k[s // bs, :, s % bs], key[t])
            assert np.array_equal(v[s // bs, :, s % bs], key[t] * 2)
    # byte places of the layout, from its description
    assert kc[2, 1, (33 % bs) * (d // 2) + 5] == F.quantise(key[0, 1], 1.0)[0][5]
    assert kc[2, 1, bs * d // 2 + (33 % bs) * (d // 16) + 3] == 0x38
    k[[2, 0, 2, 1], :, [1, 2, 15, 0]] = 0
    assert not k.any()  # nothing else was written


def test_attention_against_torch():
    rng = np.random.default_rng(2)
    K, V = rng.standard_normal((2, 40, 64)), rng.standard_normal((2, 40, 64))
    q = rng.standard_normal((40, 6, 64))
    got = F.attend(q, K, V, 0.125, np.arange(1, 41))
    qt, kt, vt = (torch.from_numpy(x) for x in (q.transpose(1, 0, 2), K, V))
    ref = torch.nn.functional.scaled_dot_product_attention(
        qt, kt.repeat_interleave(3, 0), vt.repeat_interleave(3, 0), is_causal=True, scale=0.125)
    assert np.abs(got - ref.numpy().transpose(1, 0, 2)).max() < 1e-12


# ------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from pagedattention_kv_cache_attention_gb300 import build
    build.build()
    import pagedattention_kv_cache_attention_gb300 as pa
    return pa._load()


P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
FAKE, ODD = P(0x10000), P(0x10008)  # never dereferenced: the host checks come first
CALLS = {
    "pa_reshape_and_cache_fp4": (
        dict(k=FAKE, v=FAKE, kst=1024, vst=1024, kc=FAKE, vc=FAKE, sm=FAKE, T=4, H=8, d=128, bs=16,
             NB=64, dt=0, ks=1.0, vs=1.0, st=None),
        [P, P, i64, i64, P, P, P, i32, i32, i32, i32, i64, i32, f32, f32, P]),
    "pa_decode_fp4": (
        dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=64, cl=FAKE, B=4, Hq=32, Hkv=8, d=128,
             bs=16, NB=64, scale=0.088, ks=1.0, vs=1.0, maxctx=1000, ps=0, ws=None, wsb=0, dt=0,
             st=None),
        [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i64, f32, f32, f32, i32, i32, P,
         ctypes.c_size_t, i32, P]),
    "pa_prefill_fp4": (
        dict(out=FAKE, q=FAKE, qs=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=64, cl=FAKE, B=4, mq=64,
             Hq=32, Hkv=8, d=128, bs=16, NB=64, scale=0.088, ks=1.0, vs=1.0, dt=0, st=None),
        [P, P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i64, f32, f32, f32, i32, P]),
}
CALLS["pa_gather_cache_fp4"] = CALLS["pa_reshape_and_cache_fp4"]
COMMON = [(dict(ks=0.0), 1), (dict(vs=NAN), 1), (dict(ks=float("inf")), 1), (dict(vs=-1.0), 1),
          (dict(ks=2.0 ** -101), 1), (dict(vs=2.0 ** 101), 1), (dict(dt=2), 1), (dict(d=96), 2),
          (dict(d=32), 2), (dict(bs=64), 2), (dict(bs=8), 2), (dict(NB=0), 1),
          (dict(kc=None), 1), (dict(vc=ODD), 1)]
ROWS = COMMON + [(dict(T=0), 0), (dict(T=-1), 1), (dict(kst=512), 1), (dict(vst=1028), 1),
                 (dict(sm=None), 1), (dict(k=ODD), 1), (dict(H=0), 1), (dict(H=70000, kst=1 << 24,
                                                                              vst=1 << 24), 2)]
ATTN = COMMON + [(dict(B=0), 0), (dict(B=-1), 1), (dict(Hq=72), 2), (dict(Hq=30), 1),
                 (dict(scale=NAN), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(out=ODD), 1),
                 (dict(q=None), 1), (dict(mb=0), 1), (dict(B=70000), 2),
                 (dict(NB=1 << 24), 2)]  # rows of the pool beyond 31 bits
SETS = {"pa_reshape_and_cache_fp4": ROWS, "pa_gather_cache_fp4": ROWS,
        "pa_decode_fp4": ATTN + [(dict(ps=24), 1), (dict(ps=256), 1), (dict(maxctx=-1), 1),
                                 (dict(ps=256, ws=FAKE, wsb=1000), 1)],
        "pa_prefill_fp4": ATTN + [(dict(mq=0), 0), (dict(mq=-1), 1), (dict(qs=None), 1),
                                  (dict(scale=0.0), 1),
                                  # tiles of a chunk beyond the grid's second dimension
                                  (dict(mq=(1 << 22) + 1, mb=1 << 20), 2),
                                  (dict(mb=1 << 27), 2)]}


@pytest.mark.parametrize("name,over,status",
                         [(n, o, s) for n, cases in SETS.items() for o, s in cases])
def test_host_refusals(lib, name, over, status):
    args, types = CALLS[name]
    assert not set(over) - set(args)
    f = getattr(lib, name)
    f.argtypes, f.restype = types, i32
    assert f(*{**args, **over}.values()) == status


def test_binding_refusals():
    import pagedattention_kv_cache_attention_gb300 as pa
    c = torch.zeros(4, 2, 16 * 64 * 9 // 16, dtype=torch.uint8)
    assert pa.fp4_block_size(c, 64) == 16
    with pytest.raises(ValueError, match="FP4 cache"):
        pa.fp4_block_size(c[:, :, :-1], 64)
    with pytest.raises(ValueError, match="FP4 cache"):
        pa.fp4_block_size(torch.zeros(4, 2, 16, 36, dtype=torch.uint8), 64)
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    s = torch.zeros(3, dtype=torch.int64)
    for f in (pa.pa_reshape_and_cache_fp4, pa.pa_gather_cache_fp4):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f(k, k, c, c, s)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_decode_fp4(k, k, c, c, s, s, 0.1, 1.0, 1.0, 10)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_prefill_fp4(k, k, s, c, c, s, s, 0.1, 1.0, 1.0, 10)
