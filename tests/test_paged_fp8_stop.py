"""The paged forward over e4m3 codes when a wait runs out (GPU).

Built with FA_PAGED_STOP, one warp of one CTA of one of the call's two kernels
waits for an item on a barrier that nothing arrives on, a millisecond long: to
the kernel an arrival that got lost.  Every other wait of that CTA then has to
end too, the call has to return with FA_ERR_DEVICE_TIMEOUT in the status word,
its rows have to be right or as they were, and the next call has to be as ever.
Nothing here faults, traps or hangs a GPU.
"""
import ctypes
import time

import pytest

from exact_io_aware_36_gb300 import build, fa
from tests.test_paged_fp8 import state

pytestmark = pytest.mark.gpu

MMA, TURN, VALUES = 9, 10, 11   # of many rows; 11: brings the values' codes to 8 rows of the other kernel


@pytest.fixture(scope="module")
def lib():
    lib = fa.load(build.build_variant("pagedfp8stop", ["FA_PAGED_STOP=1"], ("fa_fwd_paged_fp8.cu", "fa_fwd_paged_few.cu")))
    for name in ("fa_selftest_paged_fp8_stop", "fa_selftest_paged_few_stop"):
        getattr(lib, name).argtypes = [ctypes.c_int] * 3
    return lib


def run(lib, st, most, out, ws):
    """One call; the device status after it."""
    import torch as t
    q, codes, scales, table, cs, cu = st
    P = lambda x: x.data_ptr()
    T, Hq, d = q.shape
    pages, page, Hkv, _ = codes[0].shape
    sp = t.cuda.current_stream().cuda_stream
    assert lib.fa_fwd_paged_fp8(P(q), *map(P, codes), *map(P, scales), P(table), P(cs), P(cu), *map(P, out), len(cs), Hq, Hkv,
                                most, d, T, page, pages, table.shape[1], d ** -0.5, 1, -1, None, fa.FA_FP32, P(ws),
                                ws.numel(), sp) == 0
    return lib.fa_check_device_error(sp)


MIXES = [([300, 1, 40, 1], [2300, 3000, 1000, 500]),            # both kernels, items of both kinds in one
         ([20] * 6, [3000, 2500, 100, 4000, 20, 2222]),         # one-tile items alone, cut over many CTAs
         ([1] * 6, [3000, 2500, 100, 4000, 1, 2222])]           # the kernel for few rows alone


@pytest.mark.parametrize("mix,kernel,warps", [(0, "fp8", (0, 6, MMA, TURN)), (1, "fp8", (0, 6, MMA, TURN)), (0, "few", (0, 5, VALUES)),
                                              (2, "few", (0, 5, VALUES))])
@pytest.mark.parametrize("cta,item", [(0, 0), (5, 0), (7, 1)])
def test_rows_are_right_or_left_alone(lib, mix, kernel, warps, cta, item):
    """What the workspace held (here numbers that would pass for parts) never gets into a row."""
    import torch as t
    new, lens = MIXES[mix]
    Hq, Hkv, d = 8, 2, 128
    st = state(new, lens, 16, Hq, Hkv, d, 3)
    T, most = sum(new), max(new)
    stop = getattr(lib, "fa_selftest_paged_%s_stop" % kernel)
    size = lib.fa_fwd_paged_fp8_workspace_size(Hq, Hkv, most, d, T)

    def call(*at):
        ws = t.ones(size // 4, device="cuda").view(t.uint8)
        out = t.full((T, Hq, d), 5.0, device="cuda"), t.full((Hq, T), 5.0, device="cuda")
        stop(*at)
        t0 = time.time()
        status = run(lib, st, most, out, ws)
        assert time.time() - t0 < 20.0
        stop(-1, -1, -1)
        return out, status

    (good, lgood), status = call(-1, -1, -1)
    assert status == 0
    seen = []
    for warp in warps:
        (o, lse), status = call(warp, cta, item)
        right, left = (o == good).all(-1), (o == 5).all(-1)
        assert bool((right ^ left).all())
        assert bool(((lse.T == lgood.T) == right).all()) and bool(((lse.T == 5) == left).all())
        assert bool(right.any()) and (status == 7 or not bool(left.any()))
        seen.append(status)
        again, status = call(-1, -1, -1)
        assert status == 0 and all(t.equal(a, b) for a, b in zip((good, lgood), again))
    if item == 0:
        assert seen == [7] * len(warps)
