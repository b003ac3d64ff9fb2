"""Norm and rotation of q and k and its gradient against plain fp64.

Tolerances, per element, with u the half step of the stored type (2^-8 bf16,
2^-24 fp32) and e = 2^-24: a result is off by u |result| from its one rounding
plus what float32 arithmetic loses on the way.  Forward: the mean of d squares
is a sum of d / 8 lanes' 8-term chains (13 roundings, halved by the root),
rsqrt 4, two products and the rotation's two: below 32 e of the pair's
magnitude |a| + |b|.  Backward: the same with a second sum of d products:
below 64 e of r (|g| + |xh| mean |g xh|), magnitudes before any cancellation.
A weight's gradient adds N = T H rows: each lane's chain of 2 ceil(units /
4864) rows, then 3 + 8 + 76 + 8 terms, 8 more for each term's own error.
"""
import numpy as np
import pytest

from exact_io_aware_36_gb300 import fa
from oracle import paged_fp64 as P

E32 = 2.0 ** -24


# ------------------------------------------------------------------------ the oracle itself (CPU)

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_oracle_gradient_matches_differences(interleaved, norm):
    g = np.random.default_rng(3)
    x, dz = g.standard_normal((4, 2, 16)), g.standard_normal((4, 2, 16))
    w = 1 + 0.1 * g.standard_normal(16) if norm else None
    pos = np.array([0, 3, 1, 2])
    ang = g.standard_normal((4, 4))
    args = (1e-3, pos, np.cos(ang), np.sin(ang), interleaved)
    loss = lambda x, w: float((P.norm_rope(x, w, *args) * dz).sum())
    dx, dw = P.norm_rope_backward(x, dz, w, *args)
    v, h = g.standard_normal(x.shape), 1e-6
    assert abs((loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h) - (dx * v).sum()) < 1e-7
    if norm:
        v = g.standard_normal(16)
        assert abs((loss(x, w + h * v) - loss(x, w - h * v)) / (2 * h) - (dw * v).sum()) < 1e-7
    else:
        assert dw is None


# ------------------------------------------------------------------------------ refusals (CPU)

A = 0x10000   # a fake, 256-byte aligned device address (never dereferenced)


def fwd(**kw):
    a = dict(q=A, k=A, qo=A, ko=A, qs=512, ks=256, qw=A, kw=A, eps=1e-6, cos=A, sin=A, pos=A, T=4, Hq=4,
             Hkv=2, d=128, rot=128, mp=64, il=0, dt=fa.FA_BF16)
    a.update(kw)
    return fa.fa_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["qs"], a["ks"], a["qw"], a["kw"], a["eps"],
                              a["cos"], a["sin"], a["pos"], a["T"], a["Hq"], a["Hkv"], a["d"], a["rot"],
                              a["mp"], a["il"], a["dt"], None)


def bwd(**kw):
    a = dict(q=A, k=A, dqo=A, dko=A, qs=512, ks=256, qw=A, kw=A, eps=1e-6, cos=A, sin=A, pos=A, dq=A, dk=A,
             dqs=512, dks=256, dqw=A, dkw=A, T=4, Hq=4, Hkv=2, d=128, rot=128, mp=64, il=0, dt=fa.FA_BF16,
             ws=A, wsb=1 << 30)
    a.update(kw)
    return fa.fa_qk_norm_rope_bwd(a["q"], a["k"], a["dqo"], a["dko"], a["qs"], a["ks"], a["qw"], a["kw"],
                                  a["eps"], a["cos"], a["sin"], a["pos"], a["dq"], a["dk"], a["dqs"], a["dks"],
                                  a["dqw"], a["dkw"], a["T"], a["Hq"], a["Hkv"], a["d"], a["rot"], a["mp"],
                                  a["il"], a["dt"], a["ws"], a["wsb"], None)


BAD = [(dict(T=-1), 2), (dict(Hq=-1), 2), (dict(Hq=0, Hkv=0), 2), (dict(d=0), 2), (dict(d=96, rot=64), 3), (dict(d=256), 3),
       (dict(rot=8), 3), (dict(rot=144), 2), (dict(rot=-16), 2), (dict(il=2), 3), (dict(dt=7), 3),
       (dict(eps=-1.0), 3), (dict(eps=float("nan")), 3), (dict(eps=float("inf")), 3),
       (dict(qw=None, kw=None, rot=0), 3), (dict(qw=None), 1), (dict(kw=None), 1), (dict(q=None), 1),
       (dict(cos=None), 1), (dict(sin=None), 1), (dict(pos=None), 1),
       (dict(qs=511), 2), (dict(qs=508), 2), (dict(ks=0), 2), (dict(qs=516), 4), (dict(q=A + 8), 4),
       (dict(qw=A + 4), 4), (dict(cos=A + 8), 4)]


@pytest.mark.parametrize("kw,code", BAD + [(dict(qo=None), 1), (dict(ko=A + 2), 4), (dict(T=0), 0)])
def test_forward_refuses(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", BAD + [(dict(dqo=None), 1), (dict(dk=A + 2), 4), (dict(dqs=500), 2), (dict(dqw=None), 1),
                                           (dict(dkw=A + 2), 4), (dict(ws=None), 5), (dict(wsb=100), 5),
                                           (dict(ws=A + 16), 4), (dict(T=0, qw=None, kw=None), 0)])
def test_backward_refuses(kw, code):
    assert bwd(**kw) == code


def test_binding_refuses_before_the_library():
    t = pytest.importorskip("torch")
    x = t.zeros(2, 1, 64)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, x, q_weight=t.ones(64), k_weight=t.ones(64))     # not on a GPU


# -------------------------------------------------------------------------------------- on the GPU

def make(T, Hq, Hkv, d, dtype, rot, norm, seed, strided=True, scale=1.0):
    import torch as t
    g = t.Generator().manual_seed(seed)
    qkv = (scale * t.randn(T, Hq + 2 * Hkv, d, generator=g)).to(dtype).cuda()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    qw, kw = ((1 + 0.2 * t.randn(2, d, generator=g)).cuda() if norm else (None, None))
    mp = 4096
    kw_ = dict(q_weight=qw, k_weight=kw, eps=1e-6)
    if rot:
        ang = t.arange(mp, dtype=t.float64)[:, None] * 10000.0 ** (-t.arange(0, rot, 2, dtype=t.float64) / rot)
        kw_.update(cos=ang.cos().float().cuda(), sin=ang.sin().float().cuda(),
                   positions=t.randint(0, mp, (T,), generator=g, dtype=t.int32).cuda())
    dz = [t.randn(T, H, d, generator=g).to(dtype).cuda() for H in (Hq, Hkv)]
    return q, k, kw_, dz


def npf(x):
    return None if x is None else x.detach().double().cpu().numpy()


def check_forward(x, w, kw, il, z, u):
    pos = kw["positions"].cpu().numpy() if "positions" in kw else None
    cos, sin = npf(kw.get("cos")), npf(kw.get("sin"))
    ref = P.norm_rope(npf(x), npf(w), kw["eps"], pos, cos, sin, il)
    y = np.abs(P.norm_rope(npf(x), npf(w), kw["eps"], None, None, None, il))
    mag = y + np.abs(mate(y, cos, il))
    err = np.abs(npf(z) - ref)
    assert (err <= u * np.abs(ref) + 32 * E32 * mag).all(), float((err - u * np.abs(ref) - 32 * E32 * mag).max())


def mate(y, cos, il):
    """The other member of every element's pair (0 where there is none)."""
    o = np.zeros_like(y)
    if cos is None:
        return o
    h = cos.shape[1]
    if il:
        o[..., 0:2 * h:2], o[..., 1:2 * h:2] = y[..., 1:2 * h:2], y[..., 0:2 * h:2]
    else:
        o[..., :h], o[..., h:2 * h] = y[..., h:2 * h], y[..., :h]
    return o


def check_backward(x, w, kw, il, dz, dx, dw, u):
    pos = kw["positions"].cpu().numpy() if "positions" in kw else None
    cos, sin = npf(kw.get("cos")), npf(kw.get("sin"))
    ref, refw = P.norm_rope_backward(npf(x), npf(dz), npf(w), kw["eps"], pos, cos, sin, il)
    a = np.abs(npf(dz))
    g = a + mate(a, cos, il)
    if w is None:
        mag = g
    else:
        r = 1 / np.sqrt((npf(x) ** 2).mean(-1, keepdims=True) + kw["eps"])
        xh = np.abs(npf(x)) * r
        gw = g * np.abs(npf(w))
        mag = r * (gw + xh * (gw * xh).mean(-1, keepdims=True))
        T, H, d = x.shape
        chain = 2 * -(-T * H // 4864) + 103
        ew = np.abs(npf(dw) - refw)
        assert (ew <= E32 * (np.abs(refw) + chain * (g * xh).sum((0, 1)))).all(), float(ew.max())
    err = np.abs(npf(dx) - ref)
    tol = u * np.abs(ref) + 64 * E32 * mag
    assert (err <= tol).all(), float((err - tol).max())


CASES = [  # T, Hq, Hkv, d, rot, norm, interleaved
    (1, 1, 1, 64, 64, True, False), (1, 8, 1, 128, 128, True, True), (5, 3, 2, 64, 16, True, False),
    (33, 4, 4, 128, 96, True, False), (7, 5, 1, 128, 48, True, True), (200, 32, 8, 128, 128, True, False),
    (17, 6, 3, 64, 0, True, False), (64, 8, 2, 64, 64, False, False), (65, 7, 7, 128, 32, False, True),
    (501, 12, 4, 64, 32, True, True), (40, 1, 0, 128, 128, True, False), (40, 0, 3, 64, 48, True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,norm,il", CASES)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_forward_and_backward(T, Hq, Hkv, d, rot, norm, il, dt):
    import torch as t
    dtype, u = (t.bfloat16, 2.0 ** -8) if dt == "bf16" else (t.float32, 2.0 ** -24)
    q, k, kw, (dzq, dzk) = make(T, Hq, Hkv, d, dtype, rot, norm, T + Hq)
    zq, zk = fa.qk_norm_rope(q, k, interleaved=il, check=True, **kw)
    check_forward(q, kw["q_weight"], kw, il, zq, u)
    check_forward(k, kw["k_weight"], kw, il, zk, u)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dzq, dzk, interleaved=il, check=True, **kw)
    check_backward(q, kw["q_weight"], kw, il, dzq, dq, dwq, u)
    check_backward(k, kw["k_weight"], kw, il, dzk, dk, dwk, u)
    again = fa.qk_norm_rope_backward(q, k, dzq, dzk, interleaved=il, **kw)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert a is b is None or t.equal(a, b)                     # the same from run to run


@pytest.mark.gpu
def test_gradient_matches_differences():
    """The kernel's float32 gradient along a direction against central
    differences of the fp64 form: 1e-5 of the sum of |gradient * direction|
    covers the gradient's 64 e and the differences' 1e-8."""
    import torch as t
    q, k, kw, (dzq, dzk) = make(9, 4, 2, 64, t.float32, 64, True, 5, strided=False)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dzq, dzk, **kw)
    g = np.random.default_rng(1)
    pos, cos, sin = kw["positions"].cpu().numpy(), npf(kw["cos"]), npf(kw["sin"])
    for x, w, dz, dx, dw in ((q, kw["q_weight"], dzq, dq, dwq), (k, kw["k_weight"], dzk, dk, dwk)):
        loss = lambda x, w: float((P.norm_rope(x, w, 1e-6, pos, cos, sin, False) * npf(dz)).sum())
        h = 1e-6
        v = g.standard_normal(x.shape)
        d = (loss(npf(x) + h * v, npf(w)) - loss(npf(x) - h * v, npf(w))) / (2 * h)
        assert abs(d - (npf(dx) * v).sum()) <= 1e-5 * np.abs(npf(dx) * v).sum()
        v = g.standard_normal(w.shape)
        d = (loss(npf(x), npf(w) + h * v) - loss(npf(x), npf(w) - h * v)) / (2 * h)
        assert abs(d - (npf(dw) * v).sum()) <= 1e-5 * np.abs(npf(dw) * v).sum()


@pytest.mark.gpu
def test_in_place_and_into_parts_of_one_buffer():
    import torch as t
    q, k, kw, (dzq, dzk) = make(70, 6, 2, 128, t.bfloat16, 128, True, 9, strided=False)
    zq, zk = fa.qk_norm_rope(q, k, **kw)
    q2, k2 = q.clone(), k.clone()
    fa.qk_norm_rope(q2, k2, q_out=q2, k_out=k2, **kw)
    assert t.equal(q2, zq) and t.equal(k2, zk)
    dq, dk, _, _ = fa.qk_norm_rope_backward(q, k, dzq, dzk, **kw)
    buf = t.full((70, 10, 128), 7.0, dtype=t.bfloat16, device="cuda")
    fa.qk_norm_rope_backward(q, k, dzq, dzk, dq=buf[:, :6], dk=buf[:, 6:8], **kw)
    assert t.equal(buf[:, :6], dq) and t.equal(buf[:, 6:8], dk) and bool((buf[:, 8:] == 7).all())


@pytest.mark.gpu
def test_values_out_of_the_ordinary():
    """Rows of zeros (r = eps^-1/2), of infinities and NaN, tiny and huge rows: each stays in its own row."""
    import torch as t
    q, k, kw, (dzq, dzk) = make(8, 4, 2, 64, t.float32, 64, True, 2, strided=False)
    q[0], q[1], q[2] = 0, 1e-30, 1e15
    bad = q.clone()
    bad[5, 1, 3], bad[6, 2, 0] = float("nan"), float("inf")
    zq, _ = fa.qk_norm_rope(q, k, **kw)
    check_forward(q, kw["q_weight"], kw, False, zq, E32)
    zb, _ = fa.qk_norm_rope(bad, k, **kw)
    same = t.ones(8, 4, dtype=t.bool)
    same[5, 1] = same[6, 2] = False
    assert t.equal(zb[same], zq[same]) and bool(zb[5, 1].isnan().all()) and bool(zb[6, 2].isnan().any())
    dq = fa.qk_norm_rope_backward(bad, k, dzq, dzk, **kw)[0]
    assert t.equal(dq[same], fa.qk_norm_rope_backward(q, k, dzq, dzk, **kw)[0][same])


@pytest.mark.gpu
def test_positions_out_of_range_are_reported_and_skipped():
    import torch as t
    q, k, kw, (dzq, dzk) = make(6, 2, 1, 64, t.bfloat16, 64, True, 4)
    good_q, good_k = fa.qk_norm_rope(q, k, **kw)
    pos = kw["positions"].clone()
    pos[1], pos[4] = -1, 4096
    qo, ko = t.full((6, 2, 64), 3.0, dtype=q.dtype, device="cuda"), t.full((6, 1, 64), 3.0, dtype=q.dtype, device="cuda")
    bad = dict(kw, positions=pos)
    with pytest.raises(fa.FAError) as e:
        fa.qk_norm_rope(q, k, q_out=qo, k_out=ko, check=True, **bad)
    assert e.value.status == 10
    keep = t.tensor([0, 2, 3, 5])
    for out, good in ((qo, good_q), (ko, good_k)):
        assert bool((out[[1, 4]] == 3).all()) and t.equal(out[keep], good[keep])
    got = fa.qk_norm_rope_backward(q, k, dzq, dzk, **bad)
    assert fa.fa_check_device_error(t.cuda.current_stream().cuda_stream) == 10
    sub = {**kw, "positions": kw["positions"][keep.cuda()].contiguous()}
    ref = P.norm_rope_backward(npf(q[keep]), npf(dzq[keep]), npf(kw["q_weight"]), 1e-6,
                               sub["positions"].cpu().numpy(), npf(kw["cos"]), npf(kw["sin"]), False)[1]
    assert np.abs(npf(got[2]) - ref).max() <= 1e-4 * np.abs(ref).max()
    assert fa.fa_check_device_error(t.cuda.current_stream().cuda_stream) == 0


@pytest.mark.gpu
def test_no_tokens():
    import torch as t
    z = t.empty(0, 4, 64, device="cuda", dtype=t.bfloat16)
    w = t.ones(64, device="cuda")
    q, k = fa.qk_norm_rope(z, z, q_weight=w, k_weight=w, check=True)
    assert q.shape == k.shape == (0, 4, 64)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(z, z, z, z, q_weight=w, k_weight=w, check=True)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    import torch as t
    T, H, d = 131072 + 3, 128, 128                      # more than 2^31 elements of q
    q = t.zeros(T, H, d, dtype=t.bfloat16, device="cuda")
    k = t.zeros(T, 1, d, dtype=t.bfloat16, device="cuda")
    rows = t.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    q[rows] = t.randn(5, H, d, device="cuda").bfloat16()
    kw = make(T, 1, 1, d, t.bfloat16, 128, True, 1)[2]
    zq, _ = fa.qk_norm_rope(q, k, check=True, **kw)
    sub = dict(kw, positions=kw["positions"][rows].contiguous())
    check_forward(q[rows], kw["q_weight"], sub, False, zq[rows], 2.0 ** -8)
    dq = fa.qk_norm_rope_backward(q, k, zq, k, check=True, **kw)[0]
    few = fa.qk_norm_rope_backward(q[rows], k[rows], zq[rows], k[rows], **sub)[0]
    assert t.equal(dq[rows], few)


@pytest.mark.gpu
def test_streams_and_graphs():
    """Another stream's call, and two captured backward passes that share a workspace."""
    import torch as t
    q, k, kw, (dzq, dzk) = make(300, 8, 2, 64, t.bfloat16, 64, True, 11)
    ref = [*fa.qk_norm_rope(q, k, **kw), *fa.qk_norm_rope_backward(q, k, dzq, dzk, **kw)]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    got = [*fa.qk_norm_rope(q, k, stream=side, **kw), *fa.qk_norm_rope_backward(q, k, dzq, dzk, stream=side, **kw)]
    side.synchronize()
    assert all(t.equal(a, b) for a, b in zip(ref, got))
    ws = t.empty(fa.fa_qk_norm_rope_bwd_workspace_size(64), dtype=t.uint8, device="cuda")
    dz2 = dzq * 2
    graphs, outs = [], []
    for dz in (dzq, dz2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            outs.append(fa.qk_norm_rope_backward(q, k, dz, dzk, workspace=ws, **kw))
        graphs.append(g)
    want2 = fa.qk_norm_rope_backward(q, k, dz2, dzk, **kw)
    for _ in range(2):
        for g in graphs:
            g.replay()
    t.cuda.synchronize()
    assert all(t.equal(a, b) for a, b in zip(outs[0], ref[2:])) and all(t.equal(a, b) for a, b in zip(outs[1], want2))
