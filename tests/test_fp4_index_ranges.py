"""Index arithmetic of the FP4 attention calls at the end of their ranges, on the
CPU: which tables the host accepts, and that no token index that the kernels form
for them leaves 32 bits.  A restatement of the decode kernel's look-ahead: a warp
numbers its tiles l = 0, 1, ...; it asks the table for windows of 32 of them, up
to two windows past its last tile."""
import pytest

from test_fp4_format import CALLS, i32, lib  # noqa: F401  (lib is the fixture)

ATTENTION = ("pa_decode_fp4", "pa_prefill_fp4")


def status(lib, name, **over):  # noqa: F811
    args, types = CALLS[name]
    f = getattr(lib, name)
    f.argtypes, f.restype = types, i32
    return f(*{**args, **over}.values())


def most_blocks(lib, name, bs):  # noqa: F811
    """The largest table that the host accepts (no sequences: nothing is launched)."""
    lo, hi = 1, 2 ** 31 - 1
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if status(lib, name, B=0, bs=bs, mb=mid) == 0:
            lo = mid
        else:
            hi = mid - 1
    return lo


@pytest.mark.parametrize("name", ATTENTION)
@pytest.mark.parametrize("bs", [16, 32])
def test_largest_table(lib, name, bs):  # noqa: F811
    most = most_blocks(lib, name, bs)
    assert most * bs == 2 ** 31 - 2 ** 17 - bs
    assert status(lib, name, bs=bs, mb=most + 1) == 2


def last_token_formed(ctx, bs, warps, wid):
    """The largest token index that warp ``wid`` of ``warps`` forms."""
    tiles = 32 // bs
    steps = -(-ctx // 32)
    mine = (steps - wid + warps - 1) // warps if steps > wid else 0
    last = 31                                  # the window read before the length arrives
    if mine * tiles > 32:
        last = 63
        base = 0
        for k in range(max(0, mine - 40), mine):   # fills move the window on
            base = max(base, k * tiles // 32 * 32)
        last = max(last, base + 63)
    k, t = divmod(last, tiles)
    return (wid + k * warps) * 32 + t * bs + bs - 1


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("warps", [1, 4, 8, 16, 32])  # a partition's, a CTA's, clusters'
def test_token_indexes_stay_within_32_bits(lib, bs, warps):  # noqa: F811
    most = most_blocks(lib, "pa_decode_fp4", bs) * bs
    for ctx in (most, most - 1, most - 31, most - 1000, most - 40000, most - 70000):
        for wid in {0, warps // 2, warps - 1}:
            assert ctx <= last_token_formed(ctx, bs, warps, wid) + 32 * warps
            assert last_token_formed(ctx, bs, warps, wid) < 2 ** 31
    # the room is needed: without it a cluster's look-ahead would pass 2^31
    if warps == 32:
        assert last_token_formed(2 ** 31 - 8192 - 64, bs, warps, 0) >= 2 ** 31


def test_prefill_windows_stay_within_32_bits(lib):  # noqa: F811
    """The widening warps ask for a window of 32 tiles of their share (32 keys) of
    64-key steps, from the step of their last tile on."""
    for bs in (16, 32):
        most = most_blocks(lib, "pa_prefill_fp4", bs) * bs
        tiles = 32 // bs
        steps = -(-most // 64)
        last = ((steps - 1) * tiles // 32 * 32 + 31) // tiles
        assert last * 64 + 64 < 2 ** 31


@pytest.mark.parametrize("name", ATTENTION)
@pytest.mark.parametrize("bs", [477218587, 954437175, 2 ** 31 - 1, 2 ** 30, 64, 17, 0, -16])
def test_any_other_block_size_is_refused(lib, name, bs):  # noqa: F811
    """The first two are block sizes that a 32-bit product with 9 wraps to a divisor of zero for."""
    assert status(lib, name, bs=bs) == 2


@pytest.mark.parametrize("name", ATTENTION)
@pytest.mark.parametrize("bs", [16, 32])
def test_largest_pool(lib, name, bs):  # noqa: F811
    for nb in (2 ** 31 // (8 * bs), 2 ** 31, 2 ** 59, 2 ** 60, 2 ** 63 - 1):
        assert status(lib, name, bs=bs, NB=nb, Hkv=8) == 2
