"""The C++ part of the binding and tensors without memory of their own: the
wrappers that torch.vmap and torch.func.grad hand to the function they call have
no address.  Each native function answers -1 for those, and Python goes on.

Run on the CPU, on pa_bind.cpp with its two checks of the device taken out and
with a libpa.so whose calls do nothing but return 0 -- in a process of its own,
which an address asked for without the GIL would end."""
import os
import subprocess
import sys

import pytest

from pagedattention_kv_cache_attention_gb300 import build

CALLS = [n + end for n in ("pa_rope_and_cache", "pa_update_key_bounds", "pa_decode_sparse")
         for end in ("", "_fp8", "_fp4")] + ["pa_select_blocks"]
DEVICE_CHECKS = ("t.is_cuda() && ", "dev == at::detail::getCUDAHooks().getCurrentDevice()")

CHILD = """
import importlib.util, sys
import torch
spec = importlib.util.spec_from_file_location("pa_bind", sys.argv[1])
native = importlib.util.module_from_spec(spec)
spec.loader.exec_module(native)

def z(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)

i8, i32, i64, u8, f32 = torch.int8, torch.int32, torch.int64, torch.uint8, torch.float32
def calls():
    for kind in range(3):
        c = z(3, 2, 16, 64) if kind == 0 else z(3, 2, 16, 64, dtype=u8) if kind == 1 else z(3, 2, 576, dtype=u8)
        bounds, scales = z(3, 2, 2, 64, dtype=i8), z(3, 2, dtype=f32)
        q, kv, one = z(2, 4, 64), z(2, 2, 64), z(2, dtype=i64)
        t, n, bt, cl = z(2, 2, 1, dtype=i32), z(2, 2, dtype=i32), z(2, 2, dtype=i32), z(2, dtype=i32)
        start = z(3, dtype=i32)
        yield native.rope, [kind, q, q.clone(), kv, kv.clone(), c, c.clone(), one, one.clone(),
                            z(5, 64, dtype=f32), 1.0, 1.0, False, 0]
        yield native.key_bounds, [kind, bounds, scales, c, bt, cl, start, 1, 0]
        yield native.sparse, [kind, q, q.clone(), c, c.clone(), t, n, 0.1, 1.0, 1.0, 0]
    yield native.select, [t, n, q, bounds, scales, bt, cl, 16, 32, 0, 1, start, 1, 0]

tried = 0
for f, args in calls():
    assert f(*args) == 0, f
    for i, a in enumerate(args):
        if not isinstance(a, torch.Tensor):
            continue
        def wrapped(x):
            global tried
            tried += 1
            assert f(*args[:i], x, *args[i + 1:]) == -1, (f, i)
            return x.float().sum()
        torch.vmap(wrapped)(torch.stack([a, a]))
        if a.is_floating_point():
            torch.func.grad(wrapped)(a)
    assert f(*args) == 0, f
print("tried", tried)
"""


def test_addresses_are_asked_for_with_the_gil(tmp_path):
    text = open(os.path.join(build.CSRC, "pa_bind.cpp")).read()
    for check, with_ in zip(DEVICE_CHECKS, ("", "true")):
        assert text.count(check) == 1
        text = text.replace(check, with_)
    src, obj, lib = (str(tmp_path / n) for n in ("bind.cpp", "bind.o", "libpa.so"))
    open(src, "w").write(text)
    open(tmp_path / "none.c", "w").write("".join(f"int {n}() {{ return 0; }}\n" for n in CALLS))
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-std=gnu11", "-o", lib, str(tmp_path / "none.c")], check=True)
    build._compile_bind(src, obj)
    module = str(tmp_path / "pa_bind.so")
    build._link_bind(obj, str(tmp_path), module)
    r = subprocess.run([sys.executable, "-c", CHILD, module], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert int(r.stdout.split()[-1]) > 60, r.stdout
