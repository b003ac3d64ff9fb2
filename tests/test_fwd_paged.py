"""Attention of new tokens over a cache in pages against plain fp64.

Every slot that holds no token, and every page no sequence uses, is NaN, so a
read that reaches a result shows.  Tolerances per element, with A = sum p |v|:
  scores   a bf16 product is exact in float32; d additions and what follows
           lose at most e = (d + 8) 2^-23 |q| |k| scale + 2^-21 (|lse| + 8)
  LSE      2 e + 2^-22 |lse|
  O        2 e A for the scores, 2 * 2^-8 A for P in one bf16 part (its own
           rounding and the sum's it is divided by) or 2 * 2^-16 A in two parts
           (at most 128 rows), 2^-20 A for the sums, half a step of o's type.
"""
import numpy as np
import pytest

from exact_io_aware_36_gb300 import fa
from oracle import paged_fp64 as P
from tests.test_cache_pages import cache
from tests.test_norm_rope import npf

A_ = 0x10000   # a fake, 256-byte aligned device address (never dereferenced)


def call(**kw):
    a = dict(q=A_, k=A_, v=A_, bt=A_, cs=A_, cu=None, o=A_, lse=A_, B=2, Hq=8, Hkv=2, N=3, d=128, T=0, P=16, np=8, mp=4,
             scale=0.1, causal=1, window=-1, alibi=None, odt=fa.FA_BF16, ws=A_, wsb=1 << 40)
    a.update(kw)
    return fa.fa_fwd_paged(a["q"], a["k"], a["v"], a["bt"], a["cs"], a["cu"], a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"],
                           a["N"], a["d"], a["T"], a["P"], a["np"], a["mp"], a["scale"], a["causal"], a["window"],
                           a["alibi"], a["odt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 2), (dict(N=-1), 2), (dict(Hq=7), 2), (dict(Hkv=0), 2), (dict(T=5), 2), (dict(np=0), 2), (dict(mp=-1), 2),
    (dict(d=96), 3), (dict(P=24), 3), (dict(P=8), 3), (dict(Hq=258, Hkv=2), 3), (dict(B=8193), 3), (dict(scale=0.0), 3),
    (dict(scale=float("inf")), 3), (dict(causal=2), 3), (dict(causal=0, window=5), 3), (dict(causal=0, alibi=A_), 3),
    (dict(odt=5), 3), (dict(np=1 << 27), 3), (dict(q=None), 1), (dict(bt=None), 1), (dict(cs=None), 1), (dict(lse=None), 1),
    (dict(q=A_ + 8), 4), (dict(o=A_ + 4), 4), (dict(o=A_ + 16), 4), (dict(lse=A_ + 2), 4), (dict(ws=A_ + 16), 4), (dict(ws=None), 5),
    (dict(wsb=1000), 5), (dict(B=0), 0), (dict(N=0), 0), (dict(cu=A_, T=0), 0)])
def test_refuses_before_launch(kw, code):
    assert call(**kw) == code


def test_workspace_size():
    r = lambda x: (x + 255) // 256 * 256
    for Hq, Hkv, N, d, rows in ((32, 8, 1, 128, 4), (32, 8, 500, 128, 256), (7, 1, 500, 64, 252), (128, 1, 9, 64, 256)):
        assert fa.fa_fwd_paged_workspace_size(Hq, Hkv, N, d) == r(304 * rows * d * 4) + r(304 * rows * 16) + r(304 * 16)
    assert fa.fa_fwd_paged_workspace_size(6, 4, 1, 64) == 0 and fa.fa_fwd_paged_workspace_size(129, 1, 1, 64) == 0


def test_oracle_rows_of_a_whole_sequence():
    """The paged oracle equals softmax attention written out, whatever the split into cached and new tokens."""
    g = np.random.default_rng(0)
    L, d, page = 21, 8, 4
    k, v, q = (g.standard_normal((L, 1, d)) for _ in range(3))
    table = g.permutation(8)[None, :6]
    pools = [np.full((8, page, 1, d), np.nan) for _ in range(2)]
    for pool, x in zip(pools, (k, v)):
        pool.reshape(-1, 1, d)[P.slots(table[0], L, page)] = x
    s = q[:, 0] @ k[:, 0].T
    s[np.triu_indices(L, 1)] = -np.inf
    p = np.exp(s)
    want = p @ v[:, 0] / p.sum(1, keepdims=True)
    for n in (1, 5, L):
        O, lse = P.attention(q[L - n:], *pools, table, [L], [0, n], page, 1.0)
        assert np.allclose(O[:, 0], want[L - n:]) and np.allclose(lse[0], np.log(p.sum(1))[L - n:])


# -------------------------------------------------------------------------------------- on the GPU

def state(new, lens, page, Hq, Hkv, d, seed, causal=True, window=None, gain=1.0, tail=0):
    """(q, pools, table, lengths, cu), NaN wherever no key that a row sees lies."""
    import torch as t
    kp, vp, table, cs, cu, g = cache(new, lens, page, Hkv, d, seed)
    seen = t.zeros(kp.shape[0] * page, dtype=t.bool)
    tab = table.cpu().numpy().copy()
    for b, (n, L) in enumerate(zip(new, lens)):
        lo = max(0, L - n - window) if window is not None and causal else 0
        if n:
            seen[t.from_numpy(P.slots(tab[b], L, page)[lo:])] = True
            tab[b, :lo // page] = -7                       # released pages
        else:
            tab[b] = -7
    for pool in (kp, vp):
        pool.view(-1, Hkv, d)[~seen.cuda()] = float("nan")
    q = (gain * t.randn(sum(new) + tail, Hq, d, generator=g)).bfloat16().cuda()
    return q, kp, vp, t.from_numpy(tab).cuda(), cs, cu


def check(out, q, kp, vp, table, lens, cu, page, causal=True, window=None, slopes=None, scale=None):
    import torch as t
    O, lse = out
    T, Hq, d = q.shape
    Hkv = kp.shape[2]
    scale = scale or d ** -0.5
    cun = cu.cpu().numpy()
    tab = np.where(table.cpu().numpy() < 0, 0, table.cpu().numpy())
    k, v, qf = npf(kp), npf(vp), npf(q)
    args = (tab, lens, cun, page, scale, causal, window, npf(slopes))
    Or, lr = P.attention(qf, k, v, *args)
    A = P.attention(qf, k, np.abs(v), *args)[0]
    kn = np.sqrt(np.nan_to_num((k * k).sum(-1))).max()
    live = cun[-1]
    two = np.zeros(T, bool)                                  # rows of items with two tiles
    tpt = 128 // (Hq // Hkv)
    for b in range(len(lens)):
        n = cun[b + 1] - cun[b]
        for i in range(n):
            two[cun[b] + i] = n - i // (2 * tpt) * 2 * tpt > tpt
    qn = np.sqrt((qf * qf).sum(-1))[:live]
    lref = lr.T[:live]
    seen = np.isfinite(lref)
    e = (d + 8) * 2.0 ** -23 * qn * kn * scale + 2.0 ** -21 * (np.where(seen, np.abs(lref), 0) + 8)
    got = npf(lse).T[:live]
    assert (got[~seen] == -np.inf).all()
    el = np.abs(got[seen] - lref[seen]) - (2 * e[seen] + 2.0 ** -22 * np.abs(lref[seen]))
    assert el.size == 0 or el.max() <= 0, float(el.max())
    pp = np.where(two, 2.0 ** -7, 2.0 ** -15)[:live, None, None]
    u = 2.0 ** -8 if O.dtype == t.bfloat16 else 2.0 ** -24
    tol = (2 * e[..., None] + pp + 2.0 ** -20) * A[:live] + u * np.abs(Or[:live])
    eo = np.abs(npf(O)[:live] - Or[:live]) - tol
    assert eo.max() <= 0, float(eo.max())                    # NaN fails too


CASES = [  # new, lens, page, Hq, Hkv, d
    ([1], [1], 16, 1, 1, 64), ([1], [777], 16, 16, 16, 64), ([1, 1, 1], [5, 128, 129], 32, 8, 2, 128),
    ([1] * 5, [4000, 1, 63, 1999, 700], 64, 8, 1, 128), ([3, 1, 0, 8], [3, 40, 0, 513], 16, 6, 2, 64),
    ([128], [128], 128, 1, 1, 128), ([129], [129], 256, 1, 1, 64), ([130, 1, 300], [700, 2000, 300], 64, 4, 2, 128),
    ([33, 64, 65], [33, 1000, 66], 16, 8, 2, 64), ([500], [3001], 32, 4, 1, 128), ([17], [5000], 16, 7, 1, 64),
    ([19, 37], [600, 37], 128, 14, 2, 128), ([1, 5], [300, 260], 16, 128, 1, 64), ([2], [257], 16, 100, 1, 128),
    ([1] * 300, [1 + (37 * i) % 400 for i in range(300)], 16, 4, 2, 64), ([0, 0, 2, 0], [9, 0, 20, 0], 16, 2, 2, 128),
    ([1500], [1500], 16, 2, 1, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,page,Hq,Hkv,d", CASES)
@pytest.mark.parametrize("odt", ["fp32", "bf16"])
def test_causal(new, lens, page, Hq, Hkv, d, odt):
    import torch as t
    q, kp, vp, table, cs, cu = state(new, lens, page, Hq, Hkv, d, len(lens) + lens[0])
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), check=True,
                                     out_dtype=t.float32 if odt == "fp32" else None)
    check(out, q, kp, vp, table, lens, cu, page)


@pytest.mark.gpu
@pytest.mark.parametrize("window,alibi", [(0, False), (1, True), (17, False), (127, True), (128, False), (500, True),
                                          (100000, False), (None, True)])
@pytest.mark.parametrize("new,lens,page,Hq,Hkv,d", [([1, 1, 3], [900, 64, 2000], 16, 8, 2, 128), ([200, 1, 40], [1300, 700, 40], 64, 6, 2, 64),
                                                    ([300], [300], 256, 2, 1, 128)])
def test_window_and_alibi(new, lens, page, Hq, Hkv, d, window, alibi):
    import torch as t
    q, kp, vp, table, cs, cu = state(new, lens, page, Hq, Hkv, d, 5, window=window)
    slopes = t.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device="cuda") if alibi else None
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), window=window,
                                     alibi_slopes=slopes, out_dtype=t.float32, check=True)
    check(out, q, kp, vp, table, lens, cu, page, window=window, slopes=slopes)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", [([5], [300]), ([200, 1, 4, 0], [70, 1000, 0, 5]), ([300, 2], [128, 129]), ([4], [0])])
@pytest.mark.parametrize("page,Hq,Hkv,d", [(16, 4, 4, 64), (64, 8, 2, 128)])
def test_not_causal(new, lens, page, Hq, Hkv, d):
    import torch as t
    q, kp, vp, table, cs, cu = state(new, lens, page, Hq, Hkv, d, 8, causal=False)
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), causal=False,
                                     out_dtype=t.float32, check=True)
    check(out, q, kp, vp, table, lens, cu, page, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("gain", [6.0, 25.0])
@pytest.mark.parametrize("new,lens", [([1, 2], [3000, 900]), ([150], [2000])])
def test_peaked_scores(gain, new, lens):
    """Scores whose max keeps rising over the visited tiles: the reference is raised again and again."""
    import torch as t
    q, kp, vp, table, cs, cu = state(new, lens, 32, 4, 2, 128, 3, gain=gain)
    tab = table.cpu().numpy()
    for b, L in enumerate(lens):                            # older keys larger: the visit goes backwards
        rows = t.from_numpy(P.slots(tab[b], L, 32)).cuda()
        kp.view(-1, 2, 128)[rows] *= t.linspace(3, 0.2, L, device="cuda").bfloat16()[:, None, None]
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check(out, q, kp, vp, table, lens, cu, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,bad", [([1, 2], [20000, 60], [0, 2]), ([1, 5, 1], [300, 900, 1], [0, 3, 6]),
                                          ([150], [9000], [0, 70, 149])])
def test_nan_rows_stay_nan_and_alone(new, lens, bad):
    """A row of q with a NaN gives NaN, in one part or in many, and no other row takes notice."""
    import torch as t
    q, kp, vp, table, cs, cu = state(new, lens, 64, 8, 2, 128, 21)
    run = lambda x: fa.attention_forward_paged(x, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    O, lse = run(q)
    x = q.clone()
    x[bad, 3, 5] = float("nan")
    On, ln = run(x)
    assert bool(On[bad, 3].isnan().all()) and bool(ln[3, bad].isnan().all())
    On[bad, 3], ln[3, bad] = O[bad, 3], lse[3, bad]
    check((On, ln), q, kp, vp, table, lens, cu, 64)


@pytest.mark.gpu
def test_no_sequences():
    import torch as t
    e = lambda *s, dtype=t.bfloat16: t.empty(s, dtype=dtype, device="cuda")
    pools = e(4, 16, 2, 64), e(4, 16, 2, 64)
    lengths = e(0, 3, dtype=t.int32), e(0, dtype=t.int32)
    O, lse = fa.attention_forward_paged(e(0, 4, 64), *pools, *lengths, check=True)
    assert O.shape == (0, 4, 64) and lse.shape == (4, 0)
    fa.cache_append(e(0, 2, 64), e(0, 2, 64), *pools, *lengths, check=True)
    with pytest.raises(ValueError):
        fa.cache_append(e(2, 2, 64), e(2, 2, 64), *pools, *lengths)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_random_mixes(seed):
    """Sequences that bring nothing, one token, a few or a chunk, in one call, over any cut of the work."""
    import torch as t
    g = np.random.default_rng(seed)
    Hkv = int(g.choice([1, 2, 3, 8]))
    Hq, d, page = Hkv * int(g.choice([1, 2, 3, 4, 7, 16])), int(g.choice([64, 128])), int(g.choice([16, 32, 128, 256]))
    B = int(g.integers(1, 24))
    new = [int(g.choice([0, 1, 1, 1, int(g.integers(2, 40)), int(g.integers(40, 400))])) for _ in range(B)]
    new[0] = max(new[0], 1)
    lens = [n + int(g.choice([0, 1, int(g.integers(0, 300)), int(g.integers(0, 2500))])) for n in new]
    window = int(g.integers(0, 1500)) if seed % 3 == 0 else None
    slopes = t.tensor(2.0 ** (-8 * (np.arange(Hq) + 1) / Hq), dtype=t.float32, device="cuda") if seed % 4 == 1 else None
    q, kp, vp, table, cs, cu = state(new, lens, page, Hq, Hkv, d, seed, window=window, gain=float(g.choice([1.0, 4.0])))
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new) + seed % 2, window=window,
                                     alibi_slopes=slopes, out_dtype=t.float32, check=True)
    check(out, q, kp, vp, table, lens, cu, page, window=window, slopes=slopes)


@pytest.mark.gpu
def test_thousands_of_sequences():
    """More sequences than the block that plans has threads, most of them idle."""
    import torch as t
    new = [1 if b % 7 == 3 else 0 for b in range(5000)]
    lens = [1 + (11 * b) % 97 if n else 0 for b, n in enumerate(new)]
    q, kp, vp, table, cs, cu = state(new, lens, 16, 2, 1, 64, 1)
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=1, out_dtype=t.float32, check=True)
    check(out, q, kp, vp, table, lens, cu, 16)


@pytest.mark.gpu
def test_pools_past_32_bits():
    """Pages whose elements lie past 2^31 in the pool give what the same pages give in a small one."""
    import torch as t
    page, Hkv, d = 256, 8, 128
    pages = (1 << 31) // (page * Hkv * d) + 4
    lens, new = [700, 300], [1, 70]
    q, kp, vp, table, cs, cu = state(new, lens, page, 16, Hkv, d, 2)
    kp.nan_to_num_()
    vp.nan_to_num_()
    big = [t.empty(pages, page, Hkv, d, dtype=t.bfloat16, device="cuda") for _ in range(2)]
    n = kp.shape[0]
    big[0][-n:], big[1][-n:] = kp, vp
    kw = dict(cu_seqlens=cu, max_seqlen=70, check=True)
    want = fa.attention_forward_paged(q, kp, vp, table, cs, **kw)
    got = fa.attention_forward_paged(q, *big, t.where(table < 0, table, table + pages - n), cs, **kw)
    assert all(t.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_rows_behind_the_last_sequence_and_repeats():
    """A padded batch: rows from cu[B] on are left as they were; the same call twice gives the same bits."""
    import torch as t
    new, lens = [1, 40, 1], [2500, 100, 60]
    q, kp, vp, table, cs, cu = state(new, lens, 16, 8, 2, 128, 4, tail=9)
    q[42:] = float("nan")
    o = t.full((51, 8, 128), 5.0, device="cuda")
    lse = t.full((8, 51), 5.0, device="cuda")
    out = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=40, out=o, lse=lse, check=True)
    assert bool((o[42:] == 5).all()) and bool((lse[:, 42:] == 5).all())
    q0 = q.clone()
    q0[42:] = 0
    check(out, q0, kp, vp, table, lens, cu, 16)
    for _ in range(3):
        o2, l2 = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=40, out_dtype=t.float32)
        assert t.equal(o2[:42], o[:42]) and t.equal(l2[:, :42], lse[:, :42])


@pytest.mark.gpu
@pytest.mark.parametrize("what,status", [("short", 8), ("long", 8), ("max", 8), ("page", 9), ("cu", 8)])
def test_reports_and_skips(what, status):
    import torch as t
    new, lens = [2, 3, 1], [200, 300, 100]
    q, kp, vp, table, cs, cu = state(new, lens, 16, 4, 2, 64, 7)
    mx, bad = 3, slice(2, 5)
    good = fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=mx, out_dtype=t.float32, check=True)[0]
    if what == "short":
        cs[1] = 2
    elif what == "long":
        cs[1] = 16 * table.shape[1] + 1
    elif what == "max":
        mx = 2
    elif what == "page":
        table[1, 3] = kp.shape[0]
    else:
        cu[1], bad = -4, slice(0, 5)        # both neighbours are malformed
    o = t.full((6, 4, 64), 5.0, device="cuda")
    fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=mx, out=o)
    sp = t.cuda.current_stream().cuda_stream
    assert fa.fa_check_device_error(sp) == status and fa.fa_check_device_error(sp) == 0
    if what != "page":
        assert bool((o[bad] == 5).all())
    assert t.allclose(o[5], good[5], rtol=1e-3, atol=1e-4) and (bad.start == 0 or t.allclose(o[:2], good[:2], rtol=1e-3, atol=1e-4))


@pytest.mark.gpu
def test_captured_calls_share_a_workspace_and_replay_with_other_lengths():
    import torch as t
    new = [1, 1, 1]
    q, kp, vp, table, cs, cu = state(new, [900, 300, 3000], 32, 8, 2, 128, 2)
    kp.nan_to_num_()
    vp.nan_to_num_()
    ws = t.empty(fa.fa_fwd_paged_workspace_size(8, 2, 1, 128), dtype=t.uint8, device="cuda")
    q2 = (q * 2).contiguous()
    graphs, outs = [], []
    fa.attention_forward_paged(q, kp, vp, table, cs)                # load the kernels before the capture
    for x in (q, q2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            outs.append(fa.attention_forward_paged(x, kp, vp, table, cs, workspace=ws, out_dtype=t.float32))
        graphs.append(g)
    for lens in ([900, 300, 3000], [1, 290, 2000]):
        cs.copy_(t.tensor(lens, dtype=t.int32))
        for g in graphs:
            g.replay()
        t.cuda.synchronize()
        for x, out in zip((q, q2), outs):
            check(out, x, kp, vp, table, lens, cu, 32)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    o, lse = fa.attention_forward_paged(q, kp, vp, table, cs, out_dtype=t.float32, stream=side)
    side.synchronize()
    assert t.equal(o, outs[0][0]) and t.equal(lse, outs[0][1])


@pytest.mark.gpu
def test_binding_refuses():
    import torch as t
    q, kp, vp, table, cs, cu = state([2], [40], 16, 4, 2, 64, 1)
    f = lambda *a, **k: fa.attention_forward_paged(*a, **k)
    for bad in ((q.float(), kp, vp, table, cs), (q, kp.float(), vp, table, cs), (q, kp, vp, table.long(), cs)):
        with pytest.raises(TypeError):
            f(*bad)
    for bad in ((q, kp, vp[:1], table, cs), (q, kp, vp, table, cs.cpu()), (q[:, :, ::2], kp, vp, table, cs),
                (q, kp, vp, table[:, ::2], cs), (q[:, :, :32], kp, vp, table, cs)):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(q, kp, vp, table, cs, cu_seqlens=cu)
    with pytest.raises(fa.FAError):
        f(q, kp, vp, table, cs, causal=False, window=3)


@pytest.mark.gpu
def test_a_serving_loop():
    """Prompts in chunks, then single tokens, then a fork, as a server runs
    them: norm + rotation + append, attention over the pages, page copies.
    Compared with attention_forward over the whole sequences' normed, rotated q
    and k: both round the same q and k, so they differ by the two forwards'
    own errors only (O: 2 (2^-7 + 2^-8) A, A <= max |v|)."""
    import torch as t
    g = t.Generator().manual_seed(0)
    Hq, Hkv, d, page = 8, 2, 128, 16
    lens = [150, 37, 300]
    total = [L + 6 for L in lens]
    w = (1 + 0.1 * t.randn(2, d, generator=g)).cuda()
    ang = t.arange(400, dtype=t.float64)[:, None] * 10000.0 ** (-t.arange(0, d, 2, dtype=t.float64) / d)
    kw = dict(q_weight=w[0], k_weight=w[1], cos=ang.cos().float().cuda(), sin=ang.sin().float().cuda())
    qkv = [t.randn(n, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda() for n in total]
    pages = 80
    kp, vp = (t.full((pages, page, Hkv, d), float("nan"), dtype=t.bfloat16, device="cuda") for _ in range(2))
    order = t.randperm(pages, generator=g).int()
    table = order[:66].reshape(3, 22).contiguous().cuda()
    got = [t.zeros(n, Hq, d, device="cuda") for n in total]
    at = [0, 0, 0]
    while any(a < n for a, n in zip(at, total)):
        new = [min(64 if a < L else 1, (L if a < L else n) - a) for a, L, n in zip(at, lens, total)]
        at = [a + m for a, m in zip(at, new)]
        x = t.cat([s[a - m:a] for s, a, m in zip(qkv, at, new)])
        cs = t.tensor(at, dtype=t.int32, device="cuda")
        cu = t.tensor([0] + list(np.cumsum(new)), dtype=t.int32, device="cuda")
        a = dict(cu_seqlens=cu, max_seqlen=max(new), check=True)
        q = fa.qk_norm_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kp, vp, table, cs, **a, **kw)
        o, _ = fa.attention_forward_paged(q, kp, vp, table, cs, out_dtype=t.float32, **a)
        for b, part in enumerate(o.split(new)):
            got[b][at[b] - new[b]:at[b]] = part
    want = []
    for b, s in enumerate(qkv):
        pos = t.arange(total[b], dtype=t.int32, device="cuda")
        q, k = fa.qk_norm_rope(s[:, :Hq], s[:, Hq:Hq + Hkv], positions=pos, **kw)
        want.append(fa.attention_forward(q, k, s[:, Hq + Hkv:].contiguous(), causal=True, out_dtype=t.float32)[0])
        vmax = float(s[:, Hq + Hkv:].float().abs().max())
        assert float((got[b] - want[b]).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -8) * vmax
    # fork sequence 0: full pages are shared, the last one copied; both go on with other tokens
    full = total[0] // page
    row = table[0].clone()
    spare = int(order[70])
    fa.cache_copy(kp, vp, table[0, full:full + 1].contiguous(), t.tensor([spare], dtype=t.int32, device="cuda"), check=True)
    row[full] = spare
    two = t.stack([table[0], row])
    cs = t.tensor([total[0] + 1] * 2, dtype=t.int32, device="cuda")
    x = t.randn(2, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q = fa.qk_norm_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kp, vp, two, cs, check=True, **kw)
    out = fa.attention_forward_paged(q, kp, vp, two, cs, out_dtype=t.float32, check=True)
    check(out, q, kp, vp, two, [total[0] + 1] * 2, t.tensor([0, 1, 2]), page)


@pytest.mark.gpu
def test_a_training_step():
    """norm + rotation, attention, and both backward passes against fp64 through the whole chain.
    The chain's gradient is checked along random directions: the bf16
    roundings of z, of O and of the attention gradients (each 2^-8 of its
    tensor at most, and independent) stay within 5 * 2^-8 of the norm
    |grad| |direction| / sqrt(size), times 8 for the sample."""
    import torch as t
    from oracle import attention_fp64 as Aor
    g = t.Generator().manual_seed(3)
    T, Hq, Hkv, d = 200, 4, 2, 64
    qkv = t.randn(T, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:].contiguous()
    w = (1 + 0.1 * t.randn(2, d, generator=g)).cuda()
    ang = t.arange(T, dtype=t.float64)[:, None] * 10000.0 ** (-t.arange(0, d, 2, dtype=t.float64) / d)
    pos = t.arange(T, dtype=t.int32).cuda()
    kw = dict(q_weight=w[0], k_weight=w[1], cos=ang.cos().float().cuda(), sin=ang.sin().float().cuda(), positions=pos)
    do = t.randn(T, Hq, d, generator=g).bfloat16().cuda()
    zq, zk = fa.qk_norm_rope(q, k, **kw)
    o, lse = fa.attention_forward(zq, zk, v, causal=True, out_dtype=t.float32)
    dzq, dzk, dv = fa.attention_backward(zq, zk, v, o, do, lse, causal=True, check=True)
    dqkv = t.empty_like(qkv)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dzq, dzk, dq=dqkv[:, :Hq], dk=dqkv[:, Hq:Hq + Hkv], check=True, **kw)
    pn, cn, sn = pos.cpu().numpy(), npf(kw["cos"]), npf(kw["sin"])
    norm = lambda x, ww: P.norm_rope(npf(x), npf(ww), 1e-6, pn, cn, sn, False)
    cu = np.array([0, T], np.int32)
    rq, rk = Aor.attention_backward(norm(q, w[0]), norm(k, w[1]), npf(v), npf(do), d ** -0.5, True, cu, None)[:2]
    rng = np.random.default_rng(0)
    for x, ww, rz, dx, dw in ((q, w[0], rq, dq, dwq), (k, w[1], rk, dk, dwk)):
        want, wantw = P.norm_rope_backward(npf(x), rz, npf(ww), 1e-6, pn, cn, sn, False)
        for a, b in ((npf(dx), want), (npf(dw), wantw)):
            for _ in range(4):
                r = rng.standard_normal(b.shape)
                bound = 8 * 5 * 2.0 ** -8 * np.linalg.norm(b) * np.linalg.norm(r) / np.sqrt(b.size)
                assert abs(((a - b) * r).sum()) <= bound


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,b,entry,left,causal", [
    ([2, 3, 1], [200, 300, 100], 1, 3, range(2, 5), True),              # a few rows of one CTA
    ([1, 1, 1], [20000, 30000, 500], 1, 900, range(1, 2), True),        # parts in many CTAs, one of them meets it
    ([1, 1, 1], [20000, 30000, 500], 0, 1249, range(0, 1), True),       # ... the first tile of all
    ([600, 1], [600, 40], 0, 20, range(320, 600), True),                # blocks of 64 tokens before it see nothing of it
    ([70, 3], [2000, 900], 0, 77, range(0, 70), False),
])
@pytest.mark.parametrize("page", [-1, "past"])
def test_a_page_outside_the_pool_leaves_its_rows_alone(new, lens, b, entry, left, causal, page):
    import torch as t
    q, kp, vp, table, cs, cu = state(new, lens, 16, 8, 2, 64, 13, causal=causal)
    T = sum(new)
    kw = dict(cu_seqlens=cu, max_seqlen=max(new), causal=causal)
    good, lgood = fa.attention_forward_paged(q, kp, vp, table, cs, out_dtype=t.float32, check=True, **kw)
    table[b, entry] = kp.shape[0] if page == "past" else page
    o, lse = t.full((T, 8, 64), 5.0, device="cuda"), t.full((8, T), 5.0, device="cuda")
    fa.attention_forward_paged(q, kp, vp, table, cs, out=o, lse=lse, **kw)
    assert fa.fa_check_device_error(t.cuda.current_stream().cuda_stream) == 9
    good[left], lgood[:, left] = 5.0, 5.0
    assert t.equal(o, good) and t.equal(lse, lgood)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[0, 0], [2, 0], [0, 3]])
def test_tokens_with_a_largest_number_of_zero(new):
    """max_seqlen 0: a sequence that brings tokens all the same is reported and nothing is written; padding alone is fine."""
    import torch as t
    q, kp, vp, table, cs, cu = state([max(n, 1) for n in new], [40, 70], 16, 4, 2, 64, 1)
    cu.copy_(t.tensor([0, new[0], sum(new)], dtype=t.int32))
    q = t.randn(6, 4, 64, device="cuda").bfloat16()
    k = t.randn(6, 2, 64, device="cuda").bfloat16()
    kw = dict(cu_seqlens=cu, max_seqlen=0)
    outs = [t.full((6, 4, 64), 5.0, device="cuda"), t.full((4, 6), 5.0, device="cuda"), t.full_like(q, 5.0)]
    pools = [x.nan_to_num_().clone() for x in (kp, vp)]
    one = t.ones(100, 16, device="cuda")
    for call in (lambda: fa.attention_forward_paged(q, kp, vp, table, cs, out=outs[0], lse=outs[1], **kw),
                 lambda: fa.cache_append(k, k, kp, vp, table, cs, **kw),
                 lambda: fa.qk_norm_rope_append(q, k, k, kp, vp, table, cs, q_out=outs[2], cos=one, sin=one, **kw)):
        call()
        assert fa.fa_check_device_error(t.cuda.current_stream().cuda_stream) == (8 if sum(new) else 0)
    assert all(bool((x == 5).all()) for x in outs)
    assert t.equal(kp, pools[0]) and t.equal(vp, pools[1])


@pytest.mark.gpu
def test_numbers_past_32_bits_are_not_cut():
    """A window past every length is no window; a largest number of new tokens past 32 bits is refused, or as good as any."""
    import torch as t
    q, kp, vp, table, cs, cu = state([2, 1], [300, 40], 16, 4, 2, 64, 1)
    kw = dict(cu_seqlens=cu, max_seqlen=2)
    want = fa.attention_forward_paged(q, kp, vp, table, cs, **kw)
    for window in (2 ** 31 - 1, 2 ** 32, 2 ** 40 + 7):
        got = fa.attention_forward_paged(q, kp, vp, table, cs, window=window, check=True, **kw)
        assert all(t.equal(a, b) for a, b in zip(want, got))
    for most, status in ((2 ** 32 + 2, 3), (2 ** 31, 3), (-2 ** 32 + 2, 2), (-1, 2)):
        with pytest.raises(fa.FAError) as e:
            fa.attention_forward_paged(q, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=most)
        assert e.value.status == status
    k = t.randn(3, 2, 64, device="cuda").bfloat16()
    pools = [[x.clone() for x in (kp, vp)] for _ in range(2)]
    for pool, most in zip(pools, (2, 2 ** 32)):
        fa.cache_append(k, k, *pool, table, cs, cu_seqlens=cu, max_seqlen=most, check=True)
    assert all(t.equal(a.view(t.int16), b.view(t.int16)) for a, b in zip(*pools))


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot,il", [(64, 32, True), (128, 128, False)])
def test_a_training_steps_gradients_by_norm(d, rot, il):
    """The chain of norm + rotation, attention and both backward passes on packed sequences, head by head.

    Roundings to bf16 on the way, each off by at most 2^-8 of its own tensor:
    z (which enters the scores in the forward and the backward pass, and dS K
    or dS^T Q once more: three times), P, dS, dz and dx.  Together 7 * 2^-8 =
    0.027 of the gradient's norm.  A 5 % error in a factor, or the gradient of
    the norm without its mean, is more than that."""
    import torch as t
    from oracle import attention_fp64 as Aor
    g = t.Generator().manual_seed(d)
    Hq, Hkv, cu = 6, 2, np.array([0, 150, 151, 260], np.int32)
    T = int(cu[-1])
    qkv = t.randn(T, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:].contiguous()
    w = (1 + 0.3 * t.randn(2, d, generator=g)).cuda()
    ang = t.arange(T, dtype=t.float64)[:, None] * 10000.0 ** (-t.arange(0, rot, 2, dtype=t.float64) / rot)
    pos = np.concatenate([np.arange(b - a) for a, b in zip(cu, cu[1:])]).astype(np.int32)
    kw = dict(q_weight=w[0], k_weight=w[1], cos=ang.cos().float().cuda(), sin=ang.sin().float().cuda(),
              positions=t.from_numpy(pos).cuda(), interleaved=il)
    do = t.randn(T, Hq, d, generator=g).bfloat16().cuda()
    seqs = dict(causal=True, cu_seqlens=t.from_numpy(cu).cuda(), max_seqlen=150)
    zq, zk = fa.qk_norm_rope(q, k, **kw)
    o, lse = fa.attention_forward(zq, zk, v, out_dtype=t.float32, **seqs)
    dzq, dzk, _ = fa.attention_backward(zq, zk, v, o, do, lse, check=True, **seqs)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dzq, dzk, check=True, **kw)
    args = (1e-6, pos, npf(kw["cos"]), npf(kw["sin"]), il)
    norm = lambda x, ww: P.norm_rope(npf(x), npf(ww), *args)
    rz = Aor.attention_backward(norm(q, w[0]), norm(k, w[1]), npf(v), npf(do), d ** -0.5, True, cu, None)[:2]
    bound = 7 * 2.0 ** -8
    off = lambda a, b: np.sqrt(((a - b) ** 2).sum() / (b ** 2).sum())
    for x, ww, z, dx, dw in ((q, w[0], rz[0], dq, dwq), (k, w[1], rz[1], dk, dwk)):
        want, wantw = P.norm_rope_backward(npf(x), z, npf(ww), *args)
        per_head = [off(npf(dx)[:, h], want[:, h]) for h in range(want.shape[1])]
        assert max(per_head) <= bound, per_head
        assert off(npf(dw), wantw) <= bound
        # what the bound tells apart: no mean in the norm's gradient, one wrong sign in the rotation's
        r = 1 / np.sqrt((npf(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        dy = P.rotate(z, *args[1:], transposed=True)
        assert off(r * dy * npf(ww), want) > bound
        assert off(P.norm_rope_backward(npf(x), P.rotate(P.rotate(z, *args[1:]), *args[1:]), npf(ww), *args)[0], want) > bound


@pytest.mark.gpu
def test_two_streams_side_by_side():
    """Calls in flight on two streams, each with a workspace of its own, give what they give alone."""
    import torch as t
    cases = [([1] * 9, [9000, 300, 5000, 1, 128, 7000, 2000, 64, 4000]), ([400, 1, 70], [3000, 6000, 70])]
    calls, want = [], []
    for seed, (new, lens) in enumerate(cases):
        q, kp, vp, table, cs, cu = state(new, lens, 32, 8, 2, 128, seed)
        ws = t.empty(fa.fa_fwd_paged_workspace_size(8, 2, max(new), 128), dtype=t.uint8, device="cuda")
        calls.append(lambda stream, a=(q, kp, vp, table, cs), cu=cu, n=max(new), ws=ws: fa.attention_forward_paged(
            *a, cu_seqlens=cu, max_seqlen=n, workspace=ws, out_dtype=t.float32, stream=stream))
        want.append(calls[-1](None))
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(20):
        for i, (call, stream) in enumerate(zip(calls, streams)):
            got[i].append(call(stream))
    t.cuda.synchronize()
    assert fa.fa_check_device_error(None) == 0
    for outs, (o, lse) in zip(got, want):
        assert all(t.equal(a, o) and t.equal(b, lse) for a, b in outs)
