"""A cache in 8 bits: quantizing writes, page copies and attention over the pages.

Writes without norm and rotation and copies are compared bit for bit.  Behind
norm and rotation a key carries the float32 error that test_norm_rope.py bounds
(32 2^-24 of its pair's magnitude), so its code is off by half a step of e4m3
and that, and its block's exponent may be the neighbour's where the largest
element lies that close to the border.

Attention, per element of a row, with A = sum p |v| (codes times their scale are
exact in bf16 and float32):
  scores   a product is exact in float32; d additions and what follows lose at
           most e = (d + 8) 2^-23 |q| |k| scale + 2^-21 (|lse| + 8)
  LSE      2 e + 2^-22 |lse|
  O        2 e A for the scores, for P 2^-7 A (one bf16 part: its rounding and
           that of the sum it is divided by), 2^-15 A (two bf16 parts: items of
           at most 128 rows) or 2^-11 A (fp16, divided by the unrounded sum:
           sequences of few rows), 2^-20 A for the sums, half a step of o's type.
           In fp16 2^7 P of a row's largest key is at least 2^7, and steps below
           2^-14 are 2^-24: a key's P is off by 2^-25 / 2^7 at most, in units of
           the largest scale, whose codes are at most 448: 2^-32 448 2^e per key.
"""
import numpy as np
import pytest

from exact_io_aware_36_gb300 import fa
from oracle import paged_fp64 as P
from oracle import paged_fp8 as P8
from tests.test_cache_pages import LAYOUTS, cache
from tests.test_norm_rope import check_forward, npf

A = 0x10000   # a fake, 256-byte aligned device address (never dereferenced)


# -------------------------------------------------------------------------------- the oracle (CPU)

def test_oracle_codes():
    """Every code stands for what torch's e4m3 says, and encoding gives it back; rounding agrees with torch's."""
    import torch as t
    every = np.arange(256, dtype=np.uint8)
    want = t.from_numpy(every).view(t.float8_e4m3fn).double().numpy()
    assert np.array_equal(P8.VALUES, want, equal_nan=True)
    fine = ~np.isnan(want)
    assert (P8.encode(want[fine]) == every[fine]).all()
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * s for s in (1e-3, 0.1, 10, 300)])
    got = P8.encode(np.float32(x).astype(np.float64))
    clamped = t.from_numpy(np.float32(x)).clamp(-448, 448).to(t.float8_e4m3fn).view(t.uint8).numpy()
    assert (got == clamped).all()
    assert np.isnan(P8.VALUES[P8.encode(np.array([np.inf, -np.inf, np.nan]))]).all()


def test_oracle_appends():
    """A block's scale is the least that holds what is written, never falls below older tokens' and rescales their codes."""
    codes, scales = np.zeros((2, 16, 1, 64), np.uint8), np.full((2, 1, 1), 200, np.uint8)
    table = np.array([[1]])
    x = np.ones((3, 1, 64))
    c, s = P8.append(codes, scales, 448.0 * x, table, [3], [0, 3], 16)
    assert s[1, 0, 0] == 127 and (P8.values(c, s)[1, :3] == 448).all() and s[0, 0, 0] == 200
    c, s = P8.append(c, s, 448.5 * x[:1], table, [4], [0, 1], 16)
    assert s[1, 0, 0] == 128 and (P8.values(c, s)[1, :4] == 448).all()
    c, s = P8.append(c, s, 1.0 * x[:1], table, [5], [0, 1], 16)
    assert s[1, 0, 0] == 128 and (P8.values(c, s)[1, 4] == 1).all()
    c, s = P8.append(c, s, 1.0 * x[:1], table, [1], [0, 1], 16)         # the block begins anew
    assert s[1, 0, 0] == 119 and (P8.values(c, s)[1, 0] == 1).all()
    c, s = P8.append(c, s, 0 * x[:1], table, [1], [0, 1], 16)
    assert s[1, 0, 0] == 27


# ------------------------------------------------------------------------------------ refusals (CPU)

def app(**kw):
    a = dict(k=A, v=A, kp=A, vp=A, sk=A, sv=A, ks=256, vs=256, bt=A, cs=A, cu=None, B=2, Hkv=2, N=1, d=128, T=0, P=16, np=8, mp=4)
    a.update(kw)
    return fa.fa_cache_append_fp8(a["k"], a["v"], a["kp"], a["vp"], a["sk"], a["sv"], a["ks"], a["vs"], a["bt"], a["cs"],
                                  a["cu"], a["B"], a["Hkv"], a["N"], a["d"], a["T"], a["P"], a["np"], a["mp"], None)


def napp(**kw):
    a = dict(q=A, k=A, v=A, qo=A, kp=A, vp=A, sk=A, sv=A, qs=512, ks=256, vs=256, qw=A, kw=A, eps=0.0, cos=A, sin=A, bt=A,
             cs=A, cu=None, B=2, Hq=4, Hkv=2, N=1, d=128, T=0, rot=128, mpos=64, il=0, P=16, np=8, mp=4)
    a.update(kw)
    return fa.fa_qk_norm_rope_append_fp8(a["q"], a["k"], a["v"], a["qo"], a["kp"], a["vp"], a["sk"], a["sv"], a["qs"], a["ks"],
                                         a["vs"], a["qw"], a["kw"], a["eps"], a["cos"], a["sin"], a["bt"], a["cs"], a["cu"],
                                         a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["T"], a["rot"], a["mpos"], a["il"],
                                         a["P"], a["np"], a["mp"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 2), (dict(N=-1), 2), (dict(Hkv=0), 2), (dict(T=7), 2), (dict(P=0), 2), (dict(np=-1), 2), (dict(mp=-2), 2),
    (dict(P=8), 3), (dict(P=48), 3), (dict(P=512), 3), (dict(d=32, rot=0), 3), (dict(np=1 << 27), 3), (dict(mp=1 << 26), 3),
    (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(sk=None), 1), (dict(sv=None), 1), (dict(bt=None), 1),
    (dict(cs=None), 1), (dict(vp=A + 8), 4), (dict(sk=A + 4), 4), (dict(sv=A + 8), 4), (dict(ks=260), 4), (dict(vs=100), 2),
    (dict(B=0), 0), (dict(N=0), 0), (dict(cu=A, T=0), 0), (dict(B=65536, N=65536), 3)])
def test_append_refuses(kw, code):
    assert app(**{k: v for k, v in kw.items() if k != "rot"}) == code
    assert napp(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(Hq=0), 2), (dict(q=None), 1), (dict(qo=None), 1), (dict(qo=A + 8), 4), (dict(rot=24), 3),
                                     (dict(qw=None), 1), (dict(qw=None, kw=None, rot=0), 3), (dict(cos=None), 1)])
def test_norm_rope_append_refuses(kw, code):
    assert napp(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(n=-1), 2), (dict(H=0), 2), (dict(np=-1), 2), (dict(P=24), 3), (dict(d=96), 3), (dict(n=131073), 3),
                                     (dict(k=None), 1), (dict(sk=None), 1), (dict(sv=None), 1), (dict(s=None), 1), (dict(v=A + 4), 4),
                                     (dict(sk=A + 1), 4), (dict(n=0, k=None), 0)])
def test_copy_refuses(kw, code):
    a = dict(k=A, v=A, sk=A, sv=A, s=A, d_=A, n=3, np=8, P=16, H=2, d=128)
    a.update(kw)
    assert fa.fa_cache_copy_fp8(a["k"], a["v"], a["sk"], a["sv"], a["s"], a["d_"], a["n"], a["np"], a["P"], a["H"], a["d"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 2), (dict(N=-1), 2), (dict(Hq=7), 2), (dict(Hkv=0), 2), (dict(T=5), 2), (dict(np=0), 2), (dict(mp=-1), 2),
    (dict(d=96), 3), (dict(P=24), 3), (dict(P=8), 3), (dict(Hq=258, Hkv=2), 3), (dict(B=8193), 3), (dict(scale=0.0), 3),
    (dict(scale=float("inf")), 3), (dict(causal=2), 3), (dict(causal=0, window=5), 3), (dict(causal=0, alibi=A), 3),
    (dict(odt=5), 3), (dict(np=1 << 27), 3), (dict(q=None), 1), (dict(sk=None), 1), (dict(sv=None), 1), (dict(bt=None), 1),
    (dict(cs=None), 1), (dict(lse=None), 1), (dict(q=A + 8), 4), (dict(sk=A + 8), 4), (dict(o=A + 16), 4), (dict(lse=A + 2), 4),
    (dict(ws=A + 16), 4), (dict(ws=None), 5), (dict(wsb=1000), 5), (dict(B=0), 0), (dict(N=0), 0), (dict(cu=A, T=0), 0)])
def test_attention_refuses(kw, code):
    a = dict(q=A, k=A, v=A, sk=A, sv=A, bt=A, cs=A, cu=None, o=A, lse=A, B=2, Hq=8, Hkv=2, N=3, d=128, T=0, P=16, np=8, mp=4,
             scale=0.1, causal=1, window=-1, alibi=None, odt=fa.FA_BF16, ws=A, wsb=1 << 40)
    a.update(kw)
    assert fa.fa_fwd_paged_fp8(a["q"], a["k"], a["v"], a["sk"], a["sv"], a["bt"], a["cs"], a["cu"], a["o"], a["lse"], a["B"],
                               a["Hq"], a["Hkv"], a["N"], a["d"], a["T"], a["P"], a["np"], a["mp"], a["scale"], a["causal"],
                               a["window"], a["alibi"], a["odt"], a["ws"], a["wsb"], None) == code


# -------------------------------------------------------------------------------------- on the GPU

def pools(kp, g, spread=4):
    """(codes, scales) for pools of kp's shape: codes of normal values, scales that differ between blocks."""
    import torch as t
    n, page, H, d = kp.shape
    codes = [(100 * t.randn(n, page, H, d, generator=g)).clamp(-448, 448).to(t.float8_e4m3fn).cuda() for _ in range(2)]
    scales = [t.randint(119, 119 + spread, (n, page // 16, H), generator=g).to(t.uint8).cuda() for _ in range(2)]
    return codes, scales


def raw(x):
    import torch as t
    return x.view(t.uint8).cpu().numpy()


def same_codes(got, want):
    """Equal bytes; a NaN's sign does not matter."""
    return ((got == want) | ((got & 0x7f) == 0x7f) & ((want & 0x7f) == 0x7f)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", LAYOUTS + [([30, 2, 9], [1000, 35, 12])])
@pytest.mark.parametrize("page,Hkv,d", [(16, 2, 64), (64, 3, 128), (256, 1, 64)])
@pytest.mark.parametrize("gain", [0.02, 1.0, 50.0])
def test_append(new, lens, page, Hkv, d, gain):
    """Gains below and above what the blocks hold: older codes stay, or are rounded to a larger scale."""
    import torch as t
    kp, _, table, cs, cu, g = cache(new, lens, page, Hkv, d, 3)
    (kc, vc), (ks, vs) = pools(kp, g)
    T = sum(new)
    kv = (gain * t.randn(T + 2, 2 * Hkv, d, generator=g) * 2.0 ** t.randint(-3, 4, (T + 2, 1, 1), generator=g)).bfloat16().cuda()
    k, v = kv[:, :Hkv], kv[:, Hkv:]                        # two rows behind the last sequence
    args = (table.cpu().numpy(), lens, cu.cpu().numpy(), page)
    want = [P8.append(raw(c), raw(s), npf(x), *args) for c, s, x in ((kc, ks, k), (vc, vs, v))]
    fa.cache_append_fp8(k, v, kc, vc, ks, vs, table, cs, cu_seqlens=cu, max_seqlen=max(new), check=True)
    for c, s, w in ((kc, ks, want[0]), (vc, vs, want[1])):
        assert (raw(s) == w[1]).all() and same_codes(raw(c), w[0])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_every_bit_pattern(d):
    """Each of the 65536 bf16 patterns as a key and as a value: zeros of both signs, subnormals, the largest, infinities, NaN."""
    import torch as t
    n = 65536 // (4 * d)
    kp, _, table, cs, cu, g = cache([n], [n + 5], 32, 4, d, 9)
    (kc, vc), (ks, vs) = pools(kp, g)
    every = t.arange(65536, dtype=t.int32).to(t.int16).view(t.bfloat16)
    for k in (every.view(n, 4, d), every.view(4, d, n).permute(2, 0, 1).contiguous()):
        k, v = k.cuda(), k.flip(0).contiguous().cuda()
        args = (table.cpu().numpy(), [n + 5], [0, n], 32)
        want = [P8.append(raw(c), raw(s), npf(x), *args) for c, s, x in ((kc, ks, k), (vc, vs, v))]
        fa.cache_append_fp8(k, v, kc, vc, ks, vs, table, cs, check=True)
        for c, s, w in ((kc, ks, want[0]), (vc, vs, want[1])):
            assert (raw(s) == w[1]).all() and same_codes(raw(c), w[0])


@pytest.mark.gpu
def test_append_scales_at_the_borders():
    """The largest element at, just below and just above 448 2^e, for every e; blocks of zeros; scales outside the range they take."""
    import torch as t
    n, d = 230, 64
    kp, _, table, cs, cu, g = cache([n * 16], [n * 16], 256, 1, d, 5)
    (kc, vc), (ks, vs) = pools(kp, g)
    tops = t.tensor([1.75, 1.7421875, 1.7578125, 1.0, 1.9921875])[t.arange(n) % 5] * 2.0 ** (t.arange(n, dtype=t.float64) - 101)
    x = t.zeros(n, 16, 1, d, dtype=t.float64)
    x[t.arange(n), t.arange(n) % 16, 0, t.arange(n) % d] = tops * (1 - 2.0 * (t.arange(n) % 2))
    x[7] = 0
    k = x.view(n * 16, 1, d).bfloat16().cuda()
    args = (table.cpu().numpy(), [n * 16], [0, n * 16], 256)
    want = P8.append(raw(kc), raw(ks), npf(k), *args)
    fa.cache_append_fp8(k, k, kc, vc, ks, vs, table, cs, check=True)
    assert (raw(ks) == want[1]).all() and (raw(kc) == want[0]).all()
    # one more token each behind scales of 0 and 255 and codes of every pattern
    for byte in (0, 26, 247, 255):
        ks.fill_(byte)
        kc.view(t.uint8).copy_(t.arange(kc.numel(), device="cuda").view(kc.shape) % 256)
        one = (3 * t.randn(1, 1, d, generator=g)).bfloat16().cuda()
        L = t.tensor([16 * 9 + 12], dtype=t.int32, device="cuda")
        want = P8.append(raw(kc), raw(ks), npf(one), args[0], [16 * 9 + 12], [0, 1], 256)
        fa.cache_append_fp8(one, one, kc, vc, ks, vs, table, L, check=True)
        assert (raw(ks) == want[1]).all() and same_codes(raw(kc), want[0])


def check_keys(codes, scales, before, k, w, kw, il, table, lens, cu, page):
    """Keys behind norm and rotation: exponents as the definition has them but at a border, codes within half a step."""
    a = dict(kw)
    pos = np.concatenate([np.arange(L - (cu[b + 1] - cu[b]), L) for b, L in enumerate(lens)]).astype(int)
    none = lambda x: None if x is None else npf(x)
    z = P.norm_rope(npf(k), none(w), a["eps"], pos, none(a["cos"]), none(a["sin"]), il)
    mag = np.abs(P.norm_rope(npf(k), none(w), a["eps"], pos, None, None, il)).max(-1, keepdims=True) * 2 + np.abs(z)
    err = 32 * 2.0 ** -24 * mag
    H, d = codes.shape[2:]
    got, sc = P8.values(codes, scales).reshape(-1, H, d), scales.reshape(-1, H).astype(int)
    old, so = P8.values(*before).reshape(-1, H, d), before[1].reshape(-1, H).astype(int)
    touched, blocks = np.zeros(len(got), bool), np.zeros(len(sc), bool)
    for b, L in enumerate(lens):
        n = int(cu[b + 1] - cu[b])
        at = P.slots(table[b], L, page)
        for first in range((L - n) // 16 * 16, L, 16) if n else ():
            lo, hi = max(first, L - n), min(first + 16, L)
            rows = slice(cu[b] + lo - (L - n), cu[b] + hi - (L - n))
            blk = at[first] // 16
            blocks[blk] = True
            touched[at[first:hi]] = True
            for h in range(H):
                low, top = (np.abs(z[rows, h]) - err[rows, h]).max(), (np.abs(z[rows, h]) + err[rows, h]).max()
                e = [P8.exponent(low), P8.exponent(top)]
                if lo > first:
                    e = [max(x, so[blk, h] - 127) for x in e]
                mine = sc[blk, h] - 127
                assert e[0] <= mine <= e[1]
                x = np.abs(z[rows, h]) + err[rows, h]
                step = np.ldexp(1.0, np.maximum(np.frexp(np.ldexp(x, -mine))[1] - 1, -6) - 3 + mine)
                assert (np.abs(got[at[lo:hi], h] - z[rows, h]) <= step / 2 + err[rows, h]).all()
                if lo > first:
                    again = P8.VALUES[P8.encode(np.ldexp(old[at[first:lo], h], -mine))] * 2.0 ** mine
                    assert np.array_equal(got[at[first:lo], h], again)
    c, co = codes.reshape(-1, H, d), before[0].reshape(-1, H, d)       # (a block's free slots keep their codes)
    assert (c[~touched] == co[~touched]).all() and (sc[~blocks] == so[~blocks]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", LAYOUTS)
@pytest.mark.parametrize("page,Hq,Hkv,d,rot,norm,il", [(16, 4, 2, 128, 128, True, False), (32, 5, 5, 64, 32, True, True),
                                                       (128, 7, 1, 128, 64, False, False), (64, 2, 1, 64, 0, True, False)])
def test_norm_rope_append(new, lens, page, Hq, Hkv, d, rot, norm, il):
    import torch as t
    kp, _, table, cs, cu, g = cache(new, lens, page, Hkv, d, 4)
    (kc, vc), (ks, vs) = pools(kp, g, 9)
    T = sum(new)
    qkv = t.randn(T + 1, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    qw, kw = (1 + 0.2 * t.randn(2, d, generator=g)).cuda() if norm else (None, None)
    ang = t.arange(800, dtype=t.float64)[:, None] * 10000.0 ** (-t.arange(0, rot, 2, dtype=t.float64) / max(rot, 1))
    a = dict(eps=1e-5, cos=ang.cos().float().cuda() if rot else None, sin=ang.sin().float().cuda() if rot else None)
    qo = t.full((T + 1, Hq, d), 9.0, dtype=q.dtype, device="cuda")
    before = [(raw(kc).copy(), raw(ks).copy()), (raw(vc).copy(), raw(vs).copy())]
    fa.qk_norm_rope_append_fp8(q, k, v, kc, vc, ks, vs, table, cs, cu_seqlens=cu, max_seqlen=max(new), interleaved=il, q_out=qo,
                               q_weight=qw, k_weight=kw, check=True, **a)
    tab, cun = table.cpu().numpy(), cu.cpu().numpy()
    want = P8.append(*before[1], npf(v), tab, lens, cun, page)
    assert (raw(vs) == want[1]).all() and same_codes(raw(vc), want[0])
    assert bool((qo[T:] == 9).all())
    pos = t.cat([t.arange(L - n, L) for n, L in zip(new, lens)]).int()
    pk = dict(a, positions=pos, q_weight=qw, k_weight=kw) if rot else dict(a, q_weight=qw, k_weight=kw)
    check_forward(q[:T], qw, pk, il, qo[:T], 2.0 ** -8)
    check_keys(raw(kc), raw(ks), before[0], k[:T], kw, a, il, tab, lens, cun, page)


@pytest.mark.gpu
def test_append_same_number_each_and_a_captured_call():
    import torch as t
    kp, _, table, cs, cu, g = cache([2, 2, 2], [2, 30, 64], 32, 2, 64, 6)
    (kc, vc), (ks, vs) = pools(kp, g)
    k, v = (t.randn(6, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    tab = table.cpu().numpy()
    k0, s0 = kc.clone(), ks.clone()
    want = P8.append(raw(kc), raw(ks), npf(k), tab, [2, 30, 64], [0, 2, 4, 6], 32)
    fa.cache_append_fp8(k, v, kc, vc, ks, vs, table, cs, check=True)
    assert (raw(kc) == want[0]).all() and (raw(ks) == want[1]).all()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        fa.cache_append_fp8(k, v, k0.view(t.uint8), vc.view(t.uint8), s0.view(t.float8_e8m0fnu), vs.view(t.float8_e8m0fnu), table, cs)
    cs -= 1                                                  # replayed with other lengths
    cs[0] = 2
    want = P8.append(raw(k0), raw(s0), npf(k), tab, [2, 29, 63], [0, 2, 4, 6], 32)
    graph.replay()
    t.cuda.synchronize()
    assert (raw(k0) == want[0]).all() and (raw(s0) == want[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("what,status", [("short", 8), ("long", 8), ("page", 9), ("negative", 9), ("cu", 8), ("max", 8), ("position", 10)])
@pytest.mark.parametrize("long", [0, 40])
def test_append_reports_and_skips(what, status, long):
    """Sequence 1's metadata is wrong: its tokens are not written, the others' are."""
    import torch as t
    new, lens = [2, 3 + long, 1], [20, 33 + long, 10]
    T = sum(new)
    kp, _, table, cs, cu, g = cache(new, lens, 16, 2, 64, 7)
    (kc, vc), (ks, vs) = pools(kp, g)
    k, v = (t.randn(T, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    tab = table.cpu().numpy().copy()
    before = raw(kc).copy(), raw(ks).copy()
    want = P8.append(*P8.append(*before, npf(k), tab, lens[:1], [0, 2], 16), npf(k), tab[2:], lens[2:], [T - 1, T], 16)
    mx, cos = max(new), None
    if what == "short":
        cs[1] = 2
    elif what == "long":
        cs[1] = 16 * table.shape[1] + 1
    elif what == "page":
        table[1, 1:] = kc.shape[0]
    elif what == "negative":
        table[1, 1:] = -1
    elif what == "cu":
        cu[0] = 1                       # the sequences no longer start at row 0: nothing is written
        want = before
    elif what == "max":
        mx = 2
    if what == "position":
        one = t.ones(30, 16, device="cuda")
        q = t.full((T, 2, 64), 5.0, dtype=t.bfloat16, device="cuda")
        fa.qk_norm_rope_append_fp8(k, k, v, kc, vc, ks, vs, table, cs, cu_seqlens=cu, max_seqlen=mx, cos=one, sin=0 * one, q_out=q)
        assert t.equal(q[:2], k[:2]) and t.equal(q[-1], k[-1]) and bool((q[2:-1] == 5).all())
    else:
        fa.cache_append_fp8(k, v, kc, vc, ks, vs, table, cs, cu_seqlens=cu, max_seqlen=mx)
    sp = t.cuda.current_stream().cuda_stream
    assert fa.fa_check_device_error(sp) == status and fa.fa_check_device_error(sp) == 0
    if what == "position" or (what in ("page", "negative") and lens[1] - new[1] < 16):
        return                          # (a first block of sequence 1 that is in range is written)
    assert (raw(kc) == want[0]).all() and (raw(ks) == want[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("page,Hkv,d,pages,n", [(16, 1, 64, 9, 1), (16, 8, 128, 700, 300), (256, 3, 128, 20, 9), (64, 5, 64, 40, 0),
                                                (32, 2, 64, 6000, 2999), (256, 40, 64, 9, 4)])
def test_copy(page, Hkv, d, pages, n):
    import torch as t
    g = t.Generator().manual_seed(n)
    codes = [t.randint(0, 256, (pages, page, Hkv, d), generator=g).to(t.uint8).cuda() for _ in range(2)]
    scales = [t.randint(0, 256, (pages, page // 16, Hkv), generator=g).to(t.uint8).cuda() for _ in range(2)]
    order = t.randperm(pages, generator=g)
    src, dst = order[:n], order[n:2 * n]
    want = [raw(x).copy() for x in codes + scales]
    for w in want:
        w[dst.numpy()] = w[src.numpy()]
    fa.cache_copy_fp8(*codes, *scales, src.int().cuda(), dst.int().cuda(), check=True)
    assert all((raw(x) == w).all() for x, w in zip(codes + scales, want))


@pytest.mark.gpu
def test_copy_one_source_to_many_and_pairs_that_clash():
    import torch as t
    codes = [t.randint(0, 256, (12, 16, 2, 64)).to(t.uint8).cuda() for _ in range(2)]
    scales = [t.randint(0, 256, (12, 1, 2)).to(t.uint8).cuda() for _ in range(2)]
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")
    want = [raw(x).copy() for x in codes + scales]
    for w in want:
        w[[5, 6, 7]] = w[2]
    fa.cache_copy_fp8(*codes, *scales, i32(2, 2, 2, 3, 5), i32(5, 6, 7, 3, 5), check=True)
    assert all((raw(x) == w).all() for x, w in zip(codes + scales, want))
    with pytest.raises(fa.FAError) as e:
        fa.cache_copy_fp8(*codes, *scales, i32(0, 1, 3, 8, 9, -1, 10), i32(1, 2, 4, 4, 12, 9, 11), check=True)
    assert e.value.status == 9
    for w in want:
        w[11] = w[10]
    assert all((raw(x) == w).all() for x, w in zip(codes + scales, want))


# ------------------------------------------------------------------------------------------ attention

def state(new, lens, page, Hq, Hkv, d, seed, causal=True, window=None, gain=1.0, tail=0, spread=4):
    """(q, codes, scales, table, lengths, cu); NaN codes wherever no key that a row sees lies, scales of 255 in their blocks."""
    import torch as t
    kp, _, table, cs, cu, g = cache(new, lens, page, Hkv, d, seed)
    codes, scales = pools(kp, g, spread)
    seen = t.zeros(kp.shape[0] * page, dtype=t.bool)
    tab = table.cpu().numpy().copy()
    for b, (n, L) in enumerate(zip(new, lens)):
        lo = max(0, L - n - window) if window is not None and causal else 0
        if n:
            seen[t.from_numpy(P.slots(tab[b], L, page)[lo:])] = True
            tab[b, :lo // page] = -7                       # released pages
        else:
            tab[b] = -7
    blocks = seen.view(-1, 16).any(1).cuda()
    for c, s in zip(codes, scales):
        c.view(t.uint8).view(-1, Hkv, d)[~seen.cuda()] = 0x7f
        s.view(-1, Hkv)[~blocks] = 255
    q = (gain * t.randn(sum(new) + tail, Hq, d, generator=g)).bfloat16().cuda()
    return q, codes, scales, t.from_numpy(tab).cuda(), cs, cu


def parts(new, Hq, Hkv):
    """What rounding takes, of each row: of P, relative to it and of each key; of q's elements, relative to the largest.

    P in fp16: 2^-11, or half of fp16's least step, 2^-25, of P times a power of two:
    2^7 of P up to 1 where rows are few, 2^6 of P whose sum is 1/2 at least for
    others; a value over the largest power of two is a code, 448 at most.  q: few rows
    take it as it is; for others it is, times a power of two that brings its largest element to
    2^7 at least, two e4m3 parts.  What the first leaves of an element of 8 bits has
    4, so the second loses at most half of e4m3's least step, 2^-10, 2^-17 of 2^7.
    """
    G = Hq // Hkv
    most = max(new) * G if max(new) * G <= 32 else G
    few = next((r for r in (8, 16, 24, 32) if most <= r), 0)
    out = [(2.0 ** -11, 2.0 ** -32, 0.0) if n * G <= few else (2.0 ** -11, 2.0 ** -30, 2.0 ** -17) for n in new for _ in range(n)]
    return np.array(out)


def check(out, q, codes, scales, table, lens, new, page, causal=True, window=None, slopes=None, scale=None):
    import torch as t
    O, lse = out
    d = q.shape[2]
    Hq, Hkv = q.shape[1], codes[0].shape[2]
    scale = scale or d ** -0.5
    cun = np.concatenate([[0], np.cumsum(new)])
    live = cun[-1]
    tab = np.where(table.cpu().numpy() < 0, 0, table.cpu().numpy())
    k, v = (P8.values(raw(c), raw(s)) for c, s in zip(codes, scales))
    qf = npf(q)
    args = (tab, lens, cun, page, scale, causal, window, npf(slopes))
    Or, lr = P.attention(qf, k, v, *args)
    Ab = P.attention(qf, k, np.abs(v), *args)[0]
    kn = np.sqrt(np.nan_to_num((k * k).sum(-1))).max()
    qn = np.sqrt((qf * qf).sum(-1))[:live]
    pr, pk, pq = parts(new, Hq, Hkv).T[:, :, None]
    # a score's error by q's: sum_i |dq_i k_i| <= max|dq| sqrt(d) |k|
    qn = (d + 8) * 2.0 ** -23 * qn + pq * np.abs(qf[:live]).max(-1) * np.sqrt(d)
    lref = lr.T[:live]
    seen = np.isfinite(lref)
    e = qn * kn * scale + 2.0 ** -21 * (np.where(seen, np.abs(lref), 0) + 8)
    got = npf(lse).T[:live]
    assert (got[~seen] == -np.inf).all()
    el = np.abs(got[seen] - lref[seen]) - (2 * e[seen] + 2.0 ** -22 * np.abs(lref[seen]))
    assert el.size == 0 or el.max() <= 0, float(el.max())
    u = 2.0 ** -8 if O.dtype == t.bfloat16 else 2.0 ** -24
    tol = (2 * e[..., None] + pr[..., None] + 2.0 ** -20) * Ab[:live] + u * np.abs(Or[:live])
    top = max([int(x) for x in np.unique(raw(scales[1])) if x != 255], default=127) - 127
    tol += pk[..., None] * max(lens) * 448 * 2.0 ** top
    eo = np.abs(npf(O)[:live] - Or[:live]) - tol
    assert eo.max() <= 0, float(eo.max())                    # NaN fails too


def attend(q, codes, scales, table, cs, **kw):
    return fa.attention_forward_paged_fp8(q, *codes, *scales, table, cs, **kw)


CASES = [  # new, lens, page, Hq, Hkv, d
    ([1], [1], 16, 1, 1, 64), ([1], [777], 16, 16, 16, 64), ([1, 1, 1], [5, 128, 129], 32, 8, 2, 128),
    ([1] * 5, [4000, 1, 63, 1999, 700], 64, 8, 1, 128), ([3, 1, 0, 8], [3, 40, 0, 513], 16, 6, 2, 64),
    ([128], [128], 128, 1, 1, 128), ([129], [129], 256, 1, 1, 64), ([130, 1, 300], [700, 2000, 300], 64, 4, 2, 128),
    ([33, 64, 65], [33, 1000, 66], 16, 8, 2, 64), ([500], [3001], 32, 4, 1, 128), ([17], [5000], 16, 7, 1, 64),
    ([19, 37], [600, 37], 128, 14, 2, 128), ([1, 5], [300, 260], 16, 128, 1, 64), ([2], [257], 16, 100, 1, 128),
    ([1] * 300, [1 + (37 * i) % 400 for i in range(300)], 16, 4, 2, 64), ([0, 0, 2, 0], [9, 0, 20, 0], 16, 2, 2, 128),
    ([1500], [1500], 16, 2, 1, 128), ([4, 2, 1], [9000, 17, 100], 32, 12, 3, 128), ([1, 1], [33, 2000], 16, 16, 1, 128),
    ([16, 9, 1], [16, 1000, 48], 16, 3, 3, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,page,Hq,Hkv,d", CASES)
@pytest.mark.parametrize("odt", ["fp32", "bf16"])
def test_causal(new, lens, page, Hq, Hkv, d, odt):
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, page, Hq, Hkv, d, len(lens) + lens[0])
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), check=True,
                 out_dtype=t.float32 if odt == "fp32" else None)
    check(out, q, codes, scales, table, lens, new, page)


@pytest.mark.gpu
@pytest.mark.parametrize("window,alibi", [(0, False), (1, True), (17, False), (127, True), (128, False), (500, True),
                                          (100000, False), (None, True)])
@pytest.mark.parametrize("new,lens,page,Hq,Hkv,d", [([1, 1, 3], [900, 64, 2000], 16, 8, 2, 128), ([200, 1, 40], [1300, 700, 40], 64, 6, 2, 64),
                                                    ([300], [300], 256, 2, 1, 128), ([1, 1], [4000, 31], 32, 7, 1, 64)])
def test_window_and_alibi(new, lens, page, Hq, Hkv, d, window, alibi):
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, page, Hq, Hkv, d, 5, window=window)
    slopes = t.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device="cuda") if alibi else None
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), window=window, alibi_slopes=slopes,
                 out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, page, window=window, slopes=slopes)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", [([5], [300]), ([200, 1, 4, 0], [70, 1000, 0, 5]), ([300, 2], [128, 129]), ([4], [0]), ([2, 1], [50, 0])])
@pytest.mark.parametrize("page,Hq,Hkv,d", [(16, 4, 4, 64), (64, 8, 2, 128)])
def test_not_causal(new, lens, page, Hq, Hkv, d):
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, page, Hq, Hkv, d, 8, causal=False)
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), causal=False, out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, page, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("gain", [6.0, 25.0])
@pytest.mark.parametrize("new,lens", [([1, 2], [3000, 900]), ([150], [2000])])
def test_peaked_scores(gain, new, lens):
    """Scores whose max keeps rising over the visited tiles: the reference is raised again and again."""
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, 32, 4, 2, 128, 3, gain=gain)
    tab = table.cpu().numpy()
    for b, L in enumerate(lens):                            # older keys larger: the visit goes backwards
        rows = t.from_numpy(P.slots(tab[b], L, 32)).cuda()
        scales[0].view(-1, 2)[rows[::16] // 16] += t.linspace(3, 0, len(rows[::16]), device="cuda").to(t.uint8)[:, None]
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", [([1, 1], [2000, 300]), ([5], [700]), ([300], [900])])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_far_apart(new, lens, d):
    """Blocks of values 2^30 and 2^-20, blocks of zeros under the least scale, and keys whose blocks differ as much."""
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, 16, 4, 2, d, 3, gain=1e-3)
    g = t.Generator().manual_seed(1)
    live = scales[1] != 255
    pick = t.tensor([27, 100, 119, 127, 150], dtype=t.uint8)[t.randint(0, 5, scales[1].shape, generator=g)].cuda()
    scales[1] = t.where(live, pick, scales[1])
    zero = (scales[1] == 27)[:, :, None, :, None].expand(-1, -1, 16, -1, d).reshape(codes[1].shape)
    c = codes[1].view(t.uint8)
    c[zero & (c != 0x7f)] = 0
    scales[0] = t.where(live, t.tensor([60, 117, 121], dtype=t.uint8)[t.randint(0, 3, live.shape, generator=g)].cuda(), scales[0])
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_every_code_and_scale(d):
    """One key in view: O is its value exactly, for every code and every scale that a write makes."""
    import torch as t
    B, H = 220, 4
    codes = t.arange(256, dtype=t.int32).to(t.uint8)
    for lo in range(0, 256, H * d):
        vals = codes.roll(-lo)[:min(256, H * d)].repeat(-(-H * d // 256))[:H * d].view(H, d)
        pool = vals.expand(B, 16, H, d).contiguous().cuda()
        scales = t.arange(27, 27 + B, dtype=t.uint8)[:, None, None].expand(B, 1, H).contiguous().cuda()
        table = t.arange(B, dtype=t.int32, device="cuda")[:, None].contiguous()
        q = t.zeros(B, H, d, dtype=t.bfloat16, device="cuda")
        one = t.full((B,), 1, dtype=t.int32, device="cuda")
        zero = t.zeros_like(pool)
        o, _ = fa.attention_forward_paged_fp8(q, zero, pool, scales, scales, table, one, out_dtype=t.float32, check=True)
        want = P8.values(pool.cpu().numpy(), scales.cpu().numpy())[:, 0]
        assert np.array_equal(npf(o), want, equal_nan=True)
        q[:, :, 0] = 1                                       # and as a key: the score of element 0
        pool[:, :, :, 1:] = 0
        pool[:, 0, 0, 0] = t.arange(B, dtype=t.int32, device="cuda").to(t.uint8)
        value = P8.values(pool.cpu().numpy(), scales.cpu().numpy())[:, 0, :, 0].T
        # The score's way into the LSE: times scale log2(e), times ln 2, each constant rounded too, and one
        # sum: below 6 2^-24 of it.  (float32 holds neither the smallest nor, to a unit, the largest.)
        for scale in (2.0 ** -115, 2.0 ** -10, 2.0 ** 90):
            _, lse = fa.attention_forward_paged_fp8(q, pool, zero, scales, scales, table, one, scale=scale, check=True)
            got, want = npf(lse), value * scale
            assert np.isnan(got[np.isnan(want)]).all()
            held = (np.abs(want) < 2.0 ** 12) & (np.abs(want) > 2.0 ** -100)
            assert held.any() and (np.abs(got - want)[held] <= 6 * 2.0 ** -24 * np.abs(want[held])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [40, 150])
def test_every_code_and_scale_under_many_rows(d, n):
    """The same for sequences that bring one tile of rows and more."""
    import torch as t
    B, H = 220, 4
    codes = t.arange(256, dtype=t.int32).to(t.uint8)
    vals = codes.repeat(-(-H * d // 256))[:H * d].view(H, d) if H * d >= 256 else codes[:H * d].view(H, d)
    pool = vals.expand(B, 16, H, d).contiguous().cuda()
    scales = t.arange(27, 27 + B, dtype=t.uint8)[:, None, None].expand(B, 1, H).contiguous().cuda()
    table = t.arange(B, dtype=t.int32, device="cuda")[:, None].contiguous()
    q = t.zeros(B * n, H, d, dtype=t.bfloat16, device="cuda")
    one = t.full((B,), 1, dtype=t.int32, device="cuda")
    o, lse = fa.attention_forward_paged_fp8(q, t.zeros_like(pool), pool, scales, scales, table, one, causal=False,
                                            out_dtype=t.float32, check=True)
    want = t.from_numpy(P8.values(pool.cpu().numpy(), scales.cpu().numpy())[:, 0]).cuda()
    assert t.equal(t.nan_to_num(o.double(), 1e300).view(B, n, H, d), t.nan_to_num(want, 1e300)[:, None].expand(-1, n, -1, -1))
    assert bool((lse == 0).all())
    q[..., 0] = 1                                            # and as a key: the score of element 0
    key = t.zeros_like(pool)
    key[:, 0, :, 0] = t.arange(B, dtype=t.int32, device="cuda").to(t.uint8)[:, None]
    _, lse = fa.attention_forward_paged_fp8(q, key, t.zeros_like(pool), scales.fill_(120), scales, table, one, causal=False, check=True)
    score = P8.values(key.cpu().numpy(), scales.cpu().numpy())[:, 0, 0, 0] * d ** -0.5
    got = npf(lse)[0].reshape(B, n)
    # relative: the scale's, log2 e's, ln 2's and the products' roundings, 6 2^-24; absolute: m - 6 (2^-22), exp2 and log2
    # as the device has them (2^-22 relative and absolute)
    assert np.allclose(got, score[:, None], rtol=2.0 ** -21, atol=2.0 ** -20, equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", [([1, 1], [900, 300]), ([150], [900]), ([40, 1], [700, 300]), ([300], [300])])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_far_apart(new, lens, d):
    """Rows of 2^20 down to 2^-100, rows of zeros, and rows whose elements lie 2^-16 apart."""
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, 16, 4, 2, d, 7)
    g = t.Generator().manual_seed(2)
    live = scales[0] != 255
    scales[0] = t.where(live, scales[0] - 20, scales[0])
    far = t.tensor([2.0 ** 20, 2.0 ** 18, 1.0, 2.0 ** -100, 0.0])[t.randint(0, 5, q.shape[:2], generator=g)].cuda()
    q = (q.float() * far[..., None]).bfloat16()
    near = t.tensor([1.0, 2.0 ** -8, 2.0 ** -11, 2.0 ** -16])[t.randint(0, 4, q.shape, generator=g)].cuda()
    q[:, ::2] = (q.float() * near).bfloat16()[:, ::2]
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,bad", [([1, 2], [20000, 60], [0, 2]), ([1, 5, 1], [300, 900, 1], [0, 3, 6]),
                                          ([150], [9000], [0, 70, 149]), ([1, 1], [5000, 60], [1])])
def test_nan_rows_stay_nan_and_alone(new, lens, bad):
    """A row of q with a NaN gives NaN, in one part or in many, and no other row takes notice."""
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, 64, 8, 2, 128, 21)
    run = lambda x: attend(x, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    O, lse = run(q)
    x = q.clone()
    x[bad, 3, 5] = float("nan")
    On, ln = run(x)
    assert bool(On[bad, 3].isnan().all()) and bool(ln[3, bad].isnan().all())
    On[bad, 3], ln[3, bad] = O[bad, 3], lse[3, bad]
    check((On, ln), q, codes, scales, table, lens, new, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", [([1, 1], [5000, 60]), ([40], [900])])
def test_nan_keys_and_values_reach_the_rows_that_see_them(new, lens):
    import torch as t
    q, codes, scales, table, cs, cu = state(new, lens, 16, 4, 2, 64, 2)
    tab = table.cpu().numpy()
    run = lambda: attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    good, lgood = run()
    at = int(P.slots(tab[0], lens[0], 16)[lens[0] // 2])
    for i in range(2):
        c = codes[i].view(t.uint8).view(-1, 2, 64)
        was = c[at, 1, 7].clone()
        c[at, 1, 7] = 0xff
        O, lse = run()
        n = new[0]
        if i == 0:
            assert bool(O[:n, 2:].isnan().all()) and bool(lse[2:, :n].isnan().all())
        else:
            assert bool(O[:n, 2:, 7].isnan().all()) and t.equal(lse, lgood)
            O[:n, 2:, 7] = good[:n, 2:, 7]
        if i == 0:
            O[:n, 2:] = good[:n, 2:]
        assert t.equal(O, good)
        c[at, 1, 7] = was


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
    if seed % 2:
        new = [min(n, 2) for n in new]
    lens = [n + int(g.choice([0, 1, int(g.integers(0, 300)), int(g.integers(0, 2500))])) for n in new]
    window = int(g.integers(0, 1500)) if seed % 3 == 0 else None
    slopes = t.tensor(2.0 ** (-8 * (np.arange(Hq) + 1) / Hq), dtype=t.float32, device="cuda") if seed % 4 == 1 else None
    q, codes, scales, table, cs, cu = state(new, lens, page, Hq, Hkv, d, seed, window=window, gain=float(g.choice([1.0, 4.0])))
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), window=window, alibi_slopes=slopes,
                 out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, page, window=window, slopes=slopes)


@pytest.mark.gpu
def test_thousands_of_sequences():
    """More sequences than the block that plans has threads, most of them idle."""
    import torch as t
    new = [1 if b % 7 == 3 else 0 for b in range(5000)]
    lens = [1 + (11 * b) % 97 if n else 0 for b, n in enumerate(new)]
    for Hq in (2, 40):
        q, codes, scales, table, cs, cu = state(new, lens, 16, Hq, 1, 64, 1)
        out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=1, out_dtype=t.float32, check=True)
        check(out, q, codes, scales, table, lens, new, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 70], [1, 1]])
def test_pools_past_32_bits(new):
    """Pages whose codes lie past 2^32 in the pool: attention, writes and copies do what they do in a small one."""
    import torch as t
    page, Hkv, d = 256, 8, 128
    pages = (1 << 32) // (page * Hkv * d) + 4
    lens = [700, 300]
    q, codes, scales, table, cs, cu = state(new, lens, page, 16, Hkv, d, 2)
    k, v = (t.randn(sum(new), Hkv, d, device="cuda").bfloat16() for _ in range(2))
    n = codes[0].shape[0]
    big = [t.zeros(pages, page, Hkv, d, dtype=t.uint8, device="cuda") for _ in range(2)]
    bigs = [t.zeros(pages, page // 16, Hkv, dtype=t.uint8, device="cuda") for _ in range(2)]
    for a, b in zip(big + bigs, codes + scales):
        a[-n:] = b.view(t.uint8)
    kw = dict(cu_seqlens=cu, max_seqlen=max(new), check=True)
    small = [c.view(t.uint8) for c in codes]
    far = t.where(table < 0, table, table + pages - n)
    fa.cache_append_fp8(k, v, *small, *scales, table, cs, **kw)
    fa.cache_append_fp8(k, v, *big, *bigs, far, cs, **kw)
    assert all(t.equal(a[-n:], b) for a, b in zip(big + bigs, small + scales))
    want = attend(q, small, scales, table, cs, **kw)
    got = attend(q, big, bigs, far, cs, **kw)
    assert all(t.equal(a, b) for a, b in zip(want, got))
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")
    fa.cache_copy_fp8(*big, *bigs, i32(pages - 1), i32(0), check=True)
    assert all(t.equal(a[0], b[-1]) for a, b in zip(big + bigs, small + scales))


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 40, 1], [1, 1, 1]])
def test_rows_behind_the_last_sequence_and_repeats(new):
    """A padded batch: rows from cu[B] on are left as they were; the same call twice gives the same bits."""
    import torch as t
    lens, T = [2500, 100, 60], sum(new)
    q, codes, scales, table, cs, cu = state(new, lens, 16, 8, 2, 128, 4, tail=9)
    q[T:] = float("nan")
    o = t.full((T + 9, 8, 128), 5.0, device="cuda")
    lse = t.full((8, T + 9), 5.0, device="cuda")
    kw = dict(cu_seqlens=cu, max_seqlen=max(new))
    out = attend(q, codes, scales, table, cs, out=o, lse=lse, check=True, **kw)
    assert bool((o[T:] == 5).all()) and bool((lse[:, T:] == 5).all())
    q0 = q.clone()
    q0[T:] = 0
    check(out, q0, codes, scales, table, lens, new, 16)
    for _ in range(3):
        o2, l2 = attend(q, codes, scales, table, cs, out_dtype=t.float32, **kw)
        assert t.equal(o2[:T], o[:T]) and t.equal(l2[:, :T], lse[:, :T])


@pytest.mark.gpu
@pytest.mark.parametrize("what,status", [("short", 8), ("long", 8), ("max", 8), ("page", 9), ("cu", 8)])
@pytest.mark.parametrize("Hq", [4, 64])
def test_reports_and_skips(what, status, Hq):
    import torch as t
    new, lens = [2, 3, 1], [200, 300, 100]
    q, codes, scales, table, cs, cu = state(new, lens, 16, Hq, 2, 64, 7)
    mx, bad = 3, slice(2, 5)
    good = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=mx, out_dtype=t.float32, check=True)[0]
    if what == "short":
        cs[1] = 2
    elif what == "long":
        cs[1] = 16 * table.shape[1] + 1
    elif what == "max":
        mx = 2
    elif what == "page":
        table[1, 3] = codes[0].shape[0]
    else:
        cu[1], bad = -4, slice(0, 5)        # both neighbours are malformed
    o = t.full((6, Hq, 64), 5.0, device="cuda")
    attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=mx, out=o)
    sp = t.cuda.current_stream().cuda_stream
    assert fa.fa_check_device_error(sp) == status and fa.fa_check_device_error(sp) == 0
    assert bool((o[bad] == 5).all())
    assert t.allclose(o[5], good[5], rtol=1e-3, atol=1e-3) and (bad.start == 0 or t.allclose(o[:2], good[:2], rtol=1e-3, atol=1e-3))


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
    q, codes, scales, table, cs, cu = state(new, lens, 16, 8, 2, 64, 13, causal=causal)
    T = sum(new)
    kw = dict(cu_seqlens=cu, max_seqlen=max(new), causal=causal)
    good, lgood = attend(q, codes, scales, table, cs, out_dtype=t.float32, check=True, **kw)
    table[b, entry] = codes[0].shape[0] if page == "past" else page
    o, lse = t.full((T, 8, 64), 5.0, device="cuda"), t.full((8, T), 5.0, device="cuda")
    attend(q, codes, scales, table, cs, out=o, lse=lse, **kw)
    assert fa.fa_check_device_error(t.cuda.current_stream().cuda_stream) == 9
    good[left], lgood[:, left] = 5.0, 5.0
    assert t.equal(o, good) and t.equal(lse, lgood)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 9])
def test_captured_calls_share_a_workspace_and_replay_with_other_lengths(n):
    import torch as t
    new = [n] * 3
    q, codes, scales, table, cs, cu = state(new, [900, 300, 3000], 32, 8, 2, 128, 2)
    ws = t.empty(fa.fa_fwd_paged_fp8_workspace_size(8, 2, n, 128, 3 * n), dtype=t.uint8, device="cuda")
    q2 = (q * 2).contiguous()
    graphs, outs = [], []
    attend(q, codes, scales, table, cs)                             # load the kernels before the capture
    for x in (q, q2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            outs.append(attend(x, codes, scales, table, cs, workspace=ws, out_dtype=t.float32))
        graphs.append(g)
    for lens in ([900, 300, 3000], [n, 290, 2000]):
        cs.copy_(t.tensor(lens, dtype=t.int32))
        for g in graphs:
            g.replay()
        t.cuda.synchronize()
        for x, out in zip((q, q2), outs):
            check(out, x, codes, scales, table, lens, new, 32)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    o, lse = attend(q, codes, scales, table, cs, out_dtype=t.float32, stream=side)
    side.synchronize()
    assert t.equal(o, outs[0][0]) and t.equal(lse, outs[0][1])


@pytest.mark.gpu
def test_two_streams_side_by_side():
    """Calls in flight on two streams, each with a workspace of its own, give what they give alone."""
    import torch as t
    cases = [([1] * 9, [9000, 300, 5000, 1, 128, 7000, 2000, 64, 4000]), ([400, 1, 70], [3000, 6000, 70])]
    calls, want = [], []
    for seed, (new, lens) in enumerate(cases):
        q, codes, scales, table, cs, cu = state(new, lens, 32, 8, 2, 128, seed)
        ws = t.empty(fa.fa_fwd_paged_fp8_workspace_size(8, 2, max(new), 128, sum(new)), dtype=t.uint8, device="cuda")
        calls.append(lambda stream, a=(q, codes, scales, table, cs), cu=cu, n=max(new), ws=ws: attend(
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


@pytest.mark.gpu
def test_no_sequences():
    import torch as t
    e = lambda *s, dtype=t.bfloat16: t.empty(s, dtype=dtype, device="cuda")
    cache8 = (e(4, 16, 2, 64, dtype=t.float8_e4m3fn), e(4, 16, 2, 64, dtype=t.float8_e4m3fn), e(4, 1, 2, dtype=t.uint8), e(4, 1, 2, dtype=t.uint8))
    lengths = e(0, 3, dtype=t.int32), e(0, dtype=t.int32)
    O, lse = fa.attention_forward_paged_fp8(e(0, 4, 64), *cache8, *lengths, check=True)
    assert O.shape == (0, 4, 64) and lse.shape == (4, 0)
    fa.cache_append_fp8(e(0, 2, 64), e(0, 2, 64), *cache8, *lengths, check=True)
    with pytest.raises(ValueError):
        fa.cache_append_fp8(e(2, 2, 64), e(2, 2, 64), *cache8, *lengths)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[0, 0], [2, 0], [0, 3]])
def test_tokens_with_a_largest_number_of_zero(new):
    """max_seqlen 0: a sequence that brings tokens all the same is reported and nothing is written; padding alone is fine."""
    import torch as t
    q, codes, scales, table, cs, cu = state([max(n, 1) for n in new], [40, 70], 16, 4, 2, 64, 1)
    cu.copy_(t.tensor([0, new[0], sum(new)], dtype=t.int32))
    q, k = t.randn(6, 4, 64, device="cuda").bfloat16(), t.randn(6, 2, 64, device="cuda").bfloat16()
    kw = dict(cu_seqlens=cu, max_seqlen=0)
    outs = [t.full((6, 4, 64), 5.0, device="cuda"), t.full((4, 6), 5.0, device="cuda"), t.full_like(q, 5.0)]
    before = [raw(x).copy() for x in codes + scales]
    one = t.ones(100, 16, device="cuda")
    for call in (lambda: attend(q, codes, scales, table, cs, out=outs[0], lse=outs[1], **kw),
                 lambda: fa.cache_append_fp8(k, k, *codes, *scales, table, cs, **kw),
                 lambda: fa.qk_norm_rope_append_fp8(q, k, k, *codes, *scales, table, cs, q_out=outs[2], cos=one, sin=one, **kw)):
        call()
        assert fa.fa_check_device_error(t.cuda.current_stream().cuda_stream) == (8 if sum(new) else 0)
    assert all(bool((x == 5).all()) for x in outs)
    assert all((raw(x) == b).all() for x, b in zip(codes + scales, before))


@pytest.mark.gpu
def test_binding_refuses():
    import torch as t
    q, codes, scales, table, cs, cu = state([2], [40], 16, 4, 2, 64, 1)
    f = fa.attention_forward_paged_fp8
    good = (q, *codes, *scales, table, cs)
    put = lambda i, x: good[:i] + (x,) + good[i + 1:]
    for bad in (put(0, q.float()), put(1, codes[0].float()), put(2, codes[1].view(t.uint8)), put(3, scales[0].int()),
                put(4, scales[1].view(t.float8_e8m0fnu)), put(5, table.long())):
        with pytest.raises(TypeError):
            f(*bad)
    for bad in (put(2, codes[1][:1]), put(3, scales[0][:1]), put(3, scales[0].repeat(1, 2, 1)), put(6, cs.cpu()), put(0, q[:, :, ::2]),
                put(4, scales[1].cpu()), put(5, table[:, ::2]), put(0, q[:, :, :32].contiguous())):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(*good, cu_seqlens=cu)
    with pytest.raises(fa.FAError):
        f(*good, causal=False, window=3)
    with pytest.raises(ValueError):
        fa.cache_copy_fp8(*codes, scales[0], scales[1][:1], cs, cs)


@pytest.mark.gpu
def test_a_serving_loop():
    """Prompts in chunks, then single tokens, then a fork, as a server runs them, with the cache in 8 bits.

    Each step's attention is checked against fp64 over what the pages hold, and the pages' values against the normed
    and rotated keys in fp64: a code is off by half a step of e4m3 (2^-4 of the value, or of 2^-6 of the scale) when
    it is written and again when its block's scale rises, at most as often as tokens follow it in its block; a scale
    is at most twice the least that holds its block, so all of it stays below 2^-4 |x| + 16 * 2^-10 2^e, and
    2^e <= 2 * max|x| / 224."""
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
    codes = [t.full((pages, page, Hkv, d), 0x7f, dtype=t.uint8, device="cuda").view(t.float8_e4m3fn) for _ in range(2)]
    scales = [t.full((pages, 1, Hkv), 255, dtype=t.uint8, device="cuda") for _ in range(2)]
    order = t.randperm(pages, generator=g).int()
    table = order[:66].reshape(3, 22).contiguous().cuda()
    at = [0, 0, 0]
    while any(a < n for a, n in zip(at, total)):
        new = [min(64 if a < L else 1, (L if a < L else n) - a) for a, L, n in zip(at, lens, total)]
        at = [a + m for a, m in zip(at, new)]
        x = t.cat([s[a - m:a] for s, a, m in zip(qkv, at, new)])
        cs = t.tensor(at, dtype=t.int32, device="cuda")
        cu = t.tensor([0] + list(np.cumsum(new)), dtype=t.int32, device="cuda")
        a = dict(cu_seqlens=cu, max_seqlen=max(new), check=True)
        q = fa.qk_norm_rope_append_fp8(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *codes, *scales, table, cs, **a, **kw)
        out = attend(q, codes, scales, table, cs, out_dtype=t.float32, **a)
        check(out, q, codes, scales, table, at, new, page)
    tab = table.cpu().numpy()
    held = [P8.values(raw(c), raw(s)).reshape(-1, Hkv, d) for c, s in zip(codes, scales)]
    for b, s in enumerate(qkv):
        rows = P.slots(tab[b], total[b], page)
        key = P.norm_rope(npf(s[:, Hq:Hq + Hkv]), npf(w[1]), 1e-6, np.arange(total[b]), npf(kw["cos"]), npf(kw["sin"]), False)
        for pool, x in zip(held, (key, npf(s[:, Hq + Hkv:]))):
            assert (np.abs(pool[rows] - x) <= 2.0 ** -4 * np.abs(x) + 16 * 2.0 ** -10 * 2 * np.abs(x).max() / 224).all()
    # fork sequence 0: full pages are shared, the last one copied; both go on with other tokens
    full = total[0] // page
    row = table[0].clone()
    spare = int(order[70])
    fa.cache_copy_fp8(*codes, *scales, table[0, full:full + 1].contiguous(), t.tensor([spare], dtype=t.int32, device="cuda"), check=True)
    row[full] = spare
    two = t.stack([table[0], row])
    cs = t.tensor([total[0] + 1] * 2, dtype=t.int32, device="cuda")
    x = t.randn(2, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q = fa.qk_norm_rope_append_fp8(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *codes, *scales, two, cs, check=True, **kw)
    out = attend(q, codes, scales, two, cs, out_dtype=t.float32, check=True)
    check(out, q, codes, scales, two, [total[0] + 1] * 2, [1, 1], page)
