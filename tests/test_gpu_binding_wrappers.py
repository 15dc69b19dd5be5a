"""What torch.vmap and torch.func.grad hand to a function has no memory of its
own: every call of rotated append and sparse attention raises for it, whichever
argument it is, launches nothing and leaves the process as it was."""
import pytest
import torch

from test_gpu_fp4 import pa  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def calls(pa):  # noqa: F811
    """(function, arguments) of all ten entry points; each call is a good one."""
    def z(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    i32, u8 = torch.int32, torch.uint8
    bounds, scales = pa.new_key_bounds(3, 2, 64)
    cos_sin = pa.new_rope_table(5, 64)
    at = torch.arange(2, device="cuda")
    bt, cl = torch.tensor([[0, 1], [2, 1]], dtype=i32, device="cuda"), z(2, dtype=i32) + 3
    start = torch.arange(3, dtype=i32, device="cuda")
    t, n = z(2, 2, 1, dtype=i32), z(2, 2, dtype=i32)
    for end, pair in (("", ()), ("_fp8", (1.0, 1.0)), ("_fp4", (1.0, 1.0))):
        k, v = (z(3, 2, 576, dtype=u8) if end == "_fp4" else z(3, 2, 16, 64, dtype=u8 if end else torch.float16)
                for _ in range(2))
        yield "pa_rope_and_cache" + end, [z(2, 4, 64), z(2, 4, 64), z(2, 2, 64), z(2, 2, 64), k, v, at, at.clone(),
                                          cos_sin, *pair]
        yield "pa_update_key_bounds" + end, [bounds, scales, k, bt, cl, start, 1]
        yield "pa_decode_sparse" + end, [z(2, 4, 64), z(2, 4, 64), k, v, t, n, 0.1, *pair]
    yield "pa_select_blocks", [t, n, z(2, 4, 64), bounds, scales, bt, cl, 16, 32, 0, 1, start, 1]


def test_wrappers_are_refused_by_every_call(pa):  # noqa: F811
    tried = 0
    for name, args in calls(pa):
        f = getattr(pa, name)
        f(*args)
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            before = [x.clone() if isinstance(x, torch.Tensor) else x for x in args]

            def wrapped(x):
                with pytest.raises((RuntimeError, ValueError)):
                    f(*args[:i], x, *args[i + 1:])
                return x.float().sum()

            torch.vmap(wrapped)(torch.stack([a, a]))
            if a.is_floating_point():
                torch.func.grad(wrapped)(a)
            tried += 1
            torch.cuda.synchronize()
            for x, y in zip(args, before):
                if isinstance(x, torch.Tensor):
                    assert torch.equal(x, y), (name, i)
        f(*args)
    assert tried == 3 * (9 + 6 + 6) + 8
    assert pa.pa_device_errors() == 0
