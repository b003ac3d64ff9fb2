"""The paged forward when a wait runs out (GPU).

Built with FA_PAGED_STOP, one warp of one CTA waits for an item on a barrier
that nothing arrives on, a millisecond long: to the kernel an arrival that got
lost.  Every other wait of that CTA then has to end too, the call has to
return with FA_ERR_DEVICE_TIMEOUT in the status word, and the next call has to
be as ever.  Nothing here faults, traps or hangs a GPU.
"""
import ctypes
import time

import pytest

from exact_io_aware_36_gb300 import build, fa
from tests.test_fwd_paged import state

pytestmark = pytest.mark.gpu

PRODUCER, MMA = 8, 9            # 0-3, 4-7: softmax of streams 0 and 1


@pytest.fixture(scope="module")
def lib():
    lib = fa.load(build.build_variant("pagedstop", ["FA_PAGED_STOP=1"], "fa_fwd_paged.cu"))
    lib.fa_selftest_paged_stop.argtypes = [ctypes.c_int] * 3
    return lib


def run(lib, q, kp, vp, table, cs, cu, most, out, ws):
    """One call; the device status after it."""
    import torch as t
    o, lse = out
    P = lambda x: x.data_ptr()
    T, Hq, d = q.shape
    pages, page, Hkv, _ = kp.shape
    sp = t.cuda.current_stream().cuda_stream
    assert lib.fa_fwd_paged(P(q), P(kp), P(vp), P(table), P(cs), P(cu), P(o), P(lse), len(cs), Hq, Hkv, most, d, T, page,
                            pages, table.shape[1], d ** -0.5, 1, -1, None, fa.FA_FP32, P(ws), ws.numel(), sp) == 0
    return lib.fa_check_device_error(sp)


MIXES = [([1] * 6, [3000, 2500, 100, 4000, 1, 2222]),           # one-tile items alone, cut over many CTAs
         ([300, 1, 40, 1], [2300, 3000, 1000, 500])]            # items of both kinds


@pytest.mark.parametrize("new,lens", MIXES)
@pytest.mark.parametrize("cta,item", [(0, 0), (5, 0), (7, 1)])
@pytest.mark.parametrize("warp", [0, 6, PRODUCER, MMA])
def test_a_lost_item_ends_the_call(lib, warp, cta, item, new, lens):
    import torch as t
    Hq, Hkv, d = 8, 2, 128
    q, kp, vp, table, cs, cu = state(new, lens, 16, Hq, Hkv, d, 3)
    T = sum(new)
    new_out = lambda: (t.full((T, Hq, d), 5.0, device="cuda"), t.full((Hq, T), 5.0, device="cuda"))
    ws = t.ones(fa.fa_fwd_paged_workspace_size(Hq, Hkv, max(new), d) // 4, device="cuda").view(t.uint8)
    args = (q, kp, vp, table, cs, cu, max(new))
    lib.fa_selftest_paged_stop(-1, -1, -1)
    good = new_out()
    assert run(lib, *args, good, ws) == 0
    lib.fa_selftest_paged_stop(warp, cta, item)
    t0 = time.time()
    status = run(lib, *args, new_out(), ws)
    assert time.time() - t0 < 10.0
    lib.fa_selftest_paged_stop(-1, -1, -1)
    again = new_out()
    assert run(lib, *args, again, ws) == 0
    assert all(t.equal(a, b) for a, b in zip(good, again))
    assert status == 7


@pytest.mark.parametrize("new,lens", MIXES)
@pytest.mark.parametrize("cta,item", [(0, 0), (5, 0), (7, 1), (30, 0)])
@pytest.mark.parametrize("warp", [0, 6, PRODUCER, MMA])
def test_rows_are_right_or_left_alone(lib, warp, cta, item, new, lens):
    """What the workspace held (here numbers that would pass for parts) never gets into a row."""
    import torch as t
    Hq, Hkv, d = 8, 2, 128
    q, kp, vp, table, cs, cu = state(new, lens, 16, Hq, Hkv, d, 3)
    T = sum(new)
    outs = []
    for at in ((-1, -1, -1), (warp, cta, item)):
        ws = t.ones(fa.fa_fwd_paged_workspace_size(Hq, Hkv, max(new), d) // 4, device="cuda").view(t.uint8)
        out = t.full((T, Hq, d), 5.0, device="cuda"), t.full((Hq, T), 5.0, device="cuda")
        lib.fa_selftest_paged_stop(*at)
        status = run(lib, q, kp, vp, table, cs, cu, max(new), out, ws)
        lib.fa_selftest_paged_stop(-1, -1, -1)
        assert status == (7 if warp in at else 0)
        outs.append(out)
    (good, lgood), (o, lse) = outs
    right, left = (o == good).all(-1), (o == 5).all(-1)
    assert bool((right ^ left).all())
    assert bool(((lse.T == lgood.T) == right).all()) and bool(((lse.T == 5) == left).all())
    assert bool(left.any()) and bool(right.any())
