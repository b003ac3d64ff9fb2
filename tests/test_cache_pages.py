"""A cache in pages: writing new tokens (plain, and with norm and rotation) and
copying pages.  Plain writes and copies are compared bit for bit; normed and
rotated rows within the bounds that test_norm_rope.py derives."""
import numpy as np
import pytest

from exact_io_aware_36_gb300 import fa
from oracle import paged_fp64 as P
from tests.test_norm_rope import check_forward, npf

A = 0x10000   # a fake, 256-byte aligned device address (never dereferenced)


def app(**kw):
    a = dict(k=A, v=A, kp=A, vp=A, ks=256, vs=256, bt=A, cs=A, cu=None, B=2, Hkv=2, N=1, d=128, T=0, P=16, np=8, mp=4)
    a.update(kw)
    return fa.fa_cache_append(a["k"], a["v"], a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["cs"], a["cu"],
                              a["B"], a["Hkv"], a["N"], a["d"], a["T"], a["P"], a["np"], a["mp"], None)


def napp(**kw):
    a = dict(q=A, k=A, v=A, qo=A, kp=A, vp=A, qs=512, ks=256, vs=256, qw=A, kw=A, eps=0.0, cos=A, sin=A, bt=A, cs=A,
             cu=None, B=2, Hq=4, Hkv=2, N=1, d=128, T=0, rot=128, mpos=64, il=0, P=16, np=8, mp=4)
    a.update(kw)
    return fa.fa_qk_norm_rope_append(a["q"], a["k"], a["v"], a["qo"], a["kp"], a["vp"], a["qs"], a["ks"], a["vs"],
                                     a["qw"], a["kw"], a["eps"], a["cos"], a["sin"], a["bt"], a["cs"], a["cu"],
                                     a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["T"], a["rot"], a["mpos"],
                                     a["il"], a["P"], a["np"], a["mp"], None)


BAD = [(dict(B=-1), 2), (dict(N=-1), 2), (dict(Hkv=0), 2), (dict(T=7), 2), (dict(P=0), 2), (dict(np=-1), 2),
       (dict(mp=-2), 2), (dict(P=8), 3), (dict(P=48), 3), (dict(P=512), 3), (dict(d=32, rot=0), 3),
       (dict(np=1 << 27), 3), (dict(mp=1 << 26), 3), (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1),
       (dict(bt=None), 1), (dict(cs=None), 1), (dict(vp=A + 8), 4), (dict(ks=260), 4), (dict(vs=100), 2), (dict(B=0), 0),
       (dict(N=0), 0), (dict(cu=A, T=0), 0), (dict(B=65536, N=65536), 3)]


@pytest.mark.parametrize("kw,code", BAD)
def test_append_refuses(kw, code):
    assert app(**{k: v for k, v in kw.items() if k != "rot"}) == code
    assert napp(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(Hq=0), 2), (dict(q=None), 1), (dict(qo=None), 1), (dict(qo=A + 8), 4), (dict(rot=24), 3),
                                     (dict(qw=None), 1), (dict(qw=None, kw=None, rot=0), 3), (dict(cos=None), 1)])
def test_norm_rope_append_refuses(kw, code):
    assert napp(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(n=-1), 2), (dict(H=0), 2), (dict(np=-1), 2), (dict(P=24), 3), (dict(d=96), 3),
                                     (dict(n=131073), 3), (dict(k=None), 1), (dict(s=None), 1), (dict(v=A + 4), 4), (dict(n=0, k=None), 0)])
def test_copy_refuses(kw, code):
    a = dict(k=A, v=A, s=A, d_=A, n=3, np=8, P=16, H=2, d=128)
    a.update(kw)
    assert fa.fa_cache_copy(a["k"], a["v"], a["s"], a["d_"], a["n"], a["np"], a["P"], a["H"], a["d"], None) == code


# -------------------------------------------------------------------------------------- on the GPU

def cache(new, lens, page, Hkv, d, seed, spare=2, slack=1):
    """Pools, a table of random pages (-1 behind each sequence's last) and the lengths."""
    import torch as t
    g = t.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    order = t.randperm(pages, generator=g).int()
    table = t.full((len(lens), max(used + [1]) + slack), -1, dtype=t.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    kp, vp = (t.randn(pages, page, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    cu = t.tensor([0] + list(np.cumsum(new)), dtype=t.int32)
    return kp, vp, table.cuda(), t.tensor(lens, dtype=t.int32).cuda(), cu.cuda(), g


def bits(x):
    import torch as t
    return x.view(t.int16).cpu().numpy()


LAYOUTS = [([1], [1]), ([1, 1, 1], [5, 16, 17]), ([3, 0, 17, 1], [3, 40, 33, 256]), ([0, 0, 5], [0, 7, 300]),
           ([40, 1, 0, 64, 2], [41, 700, 3, 64, 129]), ([1] * 70, list(range(1, 71)))]


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", LAYOUTS)
@pytest.mark.parametrize("page,Hkv,d", [(16, 2, 64), (64, 3, 128), (256, 1, 64)])
def test_append(new, lens, page, Hkv, d):
    import torch as t
    kp, vp, table, cs, cu, g = cache(new, lens, page, Hkv, d, 3)
    T = sum(new)
    kv = t.randn(T + 2, 2 * Hkv, d, generator=g).bfloat16().cuda()     # two rows behind the last sequence
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    args = (table.cpu().numpy(), lens, cu.cpu().numpy(), page)
    want = [P.append(bits(p), bits(x.contiguous()), *args) for p, x in ((kp, k), (vp, v))]
    fa.cache_append(k, v, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), check=True)
    assert (bits(kp) == want[0]).all() and (bits(vp) == want[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", LAYOUTS)
@pytest.mark.parametrize("page,Hq,Hkv,d,rot,norm,il", [(16, 4, 2, 128, 128, True, False), (32, 5, 5, 64, 32, True, True),
                                                       (128, 7, 1, 128, 64, False, False), (64, 2, 1, 64, 0, True, False)])
def test_norm_rope_append(new, lens, page, Hq, Hkv, d, rot, norm, il):
    import torch as t
    kp, vp, table, cs, cu, g = cache(new, lens, page, Hkv, d, 4)
    T = sum(new)
    qkv = t.randn(T + 1, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    qw, kw = (1 + 0.2 * t.randn(2, d, generator=g)).cuda() if norm else (None, None)
    ang = t.arange(800, dtype=t.float64)[:, None] * 10000.0 ** (-t.arange(0, rot, 2, dtype=t.float64) / max(rot, 1))
    a = dict(q_weight=qw, k_weight=kw, eps=1e-5, cos=ang.cos().float().cuda() if rot else None,
             sin=ang.sin().float().cuda() if rot else None)
    qo = t.full((T + 1, Hq, d), 9.0, dtype=q.dtype, device="cuda")
    before = [bits(kp).copy(), bits(vp)]
    fa.qk_norm_rope_append(q, k, v, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=max(new), interleaved=il, q_out=qo,
                           check=True, **a)
    tab, cun = table.cpu().numpy(), cu.cpu().numpy()
    assert (bits(vp) == P.append(before[1], bits(v.contiguous()), tab, lens, cun, page)).all()
    assert bool((qo[T:] == 9).all())
    rows = t.zeros(T, dtype=t.int64)
    pos = t.zeros(T, dtype=t.int32)
    for b, (n, L) in enumerate(zip(new, lens)):
        rows[cun[b]:cun[b + 1]] = t.from_numpy(P.slots(tab[b], L, page)[L - n:])
        pos[cun[b]:cun[b + 1]] = t.arange(L - n, L)
    got = kp.view(-1, Hkv, d)[rows.cuda()]
    pk = dict(a, positions=pos) if rot else a
    check_forward(q[:T], qw, pk, il, qo[:T], 2.0 ** -8)
    check_forward(k[:T], kw, pk, il, got, 2.0 ** -8)
    left = np.ones(kp.shape[0] * page, bool)
    left[rows.numpy()] = False
    after = bits(kp).reshape(-1, Hkv, d)
    assert (after[left] == before[0].reshape(-1, Hkv, d)[left]).all()          # every other slot as it was


@pytest.mark.gpu
def test_append_same_number_each_and_a_captured_call():
    import torch as t
    kp, vp, table, cs, cu, g = cache([2, 2, 2], [2, 30, 64], 32, 2, 64, 6)
    k, v = (t.randn(6, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    want = P.append(bits(kp), bits(k), table.cpu().numpy(), [2, 30, 64], [0, 2, 4, 6], 32)
    k0 = kp.clone()
    fa.cache_append(k, v, kp, vp, table, cs, check=True)
    assert (bits(kp) == want).all()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        fa.cache_append(k, v, k0, vp, table, cs)
    cs -= 1                                                  # replayed with other lengths
    cs[0] = 2
    want = P.append(bits(k0), bits(k), table.cpu().numpy(), [2, 29, 63], [0, 2, 4, 6], 32)
    graph.replay()
    t.cuda.synchronize()
    assert (bits(k0) == want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("what,status", [("short", 8), ("long", 8), ("page", 9), ("negative", 9), ("cu", 8), ("max", 8), ("position", 10)])
def test_append_reports_and_skips(what, status):
    """Sequence 1's metadata is wrong: its tokens are not written, the others' are."""
    import torch as t
    new, lens = [2, 3, 1], [20, 33, 10]
    kp, vp, table, cs, cu, g = cache(new, lens, 16, 2, 64, 7)
    k, v = (t.randn(6, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    tab = table.cpu().numpy().copy()
    want = P.append(P.append(bits(kp), bits(k), tab, lens[:1], [0, 2], 16), bits(k), tab[2:], lens[2:], [5, 6], 16)
    mx, cos = 3, None
    if what == "short":
        cs[1] = 2
    elif what == "long":
        cs[1] = 16 * table.shape[1] + 1
    elif what == "page":
        table[1, 1:3] = kp.shape[0]
    elif what == "negative":
        table[1, 1:3] = -1
    elif what == "cu":
        cu[0] = 1                       # the sequences no longer start at row 0: nothing is written
        want = bits(kp).copy()
    elif what == "max":
        mx = 2
    if what == "position":
        one = t.ones(30, 16, device="cuda")
        q = fa.qk_norm_rope_append(k, k, v, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=mx, cos=one, sin=0 * one)
    else:
        fa.cache_append(k, v, kp, vp, table, cs, cu_seqlens=cu, max_seqlen=mx)
    sp = t.cuda.current_stream().cuda_stream
    assert fa.fa_check_device_error(sp) == status and fa.fa_check_device_error(sp) == 0
    assert (bits(kp) == want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("page,Hkv,d,pages,n", [(16, 1, 64, 9, 1), (16, 8, 128, 700, 300), (256, 3, 128, 20, 9), (64, 5, 64, 40, 0),
                                                (32, 2, 64, 6000, 2999)])
def test_copy(page, Hkv, d, pages, n):
    import torch as t
    g = t.Generator().manual_seed(n)
    kp, vp = (t.randn(pages, page, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    order = t.randperm(pages, generator=g)
    src, dst = order[:n], order[n:2 * n]
    want = [bits(x).copy() for x in (kp, vp)]
    for w in want:
        w[dst.numpy()] = w[src.numpy()]
    fa.cache_copy(kp, vp, src.int().cuda(), dst.int().cuda(), check=True)
    assert (bits(kp) == want[0]).all() and (bits(vp) == want[1]).all()


@pytest.mark.gpu
def test_copy_one_source_to_many_and_pairs_that_clash():
    import torch as t
    kp, vp = (t.randn(12, 16, 2, 64).bfloat16().cuda() for _ in range(2))
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")
    want = bits(kp).copy()
    want[[5, 6, 7]] = want[2]
    fa.cache_copy(kp, vp, i32(2, 2, 2, 3, 5), i32(5, 6, 7, 3, 5), check=True)      # 3 -> 3 and 5 -> 5 do nothing
    assert (bits(kp) == want).all()
    #  0 -> 1 with 1 -> 2 (read and written), 3 -> 4 with 8 -> 4 (written twice),
    #  9 -> 12 and -1 -> 9 (outside); 10 -> 11 alone is sound
    with pytest.raises(fa.FAError) as e:
        fa.cache_copy(kp, vp, i32(0, 1, 3, 8, 9, -1, 10), i32(1, 2, 4, 4, 12, 9, 11), check=True)
    assert e.value.status == 9
    want[11] = want[10]
    assert (bits(kp) == want).all()


@pytest.mark.gpu
def test_pools_past_32_bits():
    """Pages whose elements lie past 2^31 in the pool."""
    import torch as t
    page, Hkv, d = 256, 8, 128
    pages = (1 << 31) // (page * Hkv * d) + 3
    kp, vp = (t.zeros(pages, page, Hkv, d, dtype=t.bfloat16, device="cuda") for _ in range(2))
    table = t.tensor([[pages - 1, pages - 2]], dtype=t.int32, device="cuda")
    k, v = (t.randn(300, Hkv, d, device="cuda").bfloat16() for _ in range(2))
    fa.cache_append(k, v, kp, vp, table, t.tensor([300], dtype=t.int32, device="cuda"), check=True)
    assert t.equal(kp[pages - 1], k[:256]) and t.equal(vp[pages - 2, :44], v[256:])
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")
    fa.cache_copy(kp, vp, i32(pages - 1, pages - 2), i32(0, pages - 3), check=True)
    assert t.equal(kp[0], k[:256]) and t.equal(vp[pages - 3, :44], v[256:]) and not bool(kp[1].any())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_keeps_every_bit_pattern(d):
    """Each of the 65536 bf16 patterns, -0 and every NaN among them, as a key and as a value."""
    import torch as t
    n = 65536 // (4 * d)
    kp, vp, table, cs, cu, g = cache([n], [n + 5], 32, 4, d, 9)
    every = t.arange(65536, dtype=t.int32).to(t.int16)
    k, v = (x.view(t.bfloat16).view(n, 4, d).cuda() for x in (every, every.flip(0).contiguous()))
    want = [P.append(bits(p), bits(x), table.cpu().numpy(), [n + 5], [0, n], 32) for p, x in ((kp, k), (vp, v))]
    fa.cache_append(k, v, kp, vp, table, cs, check=True)
    assert (bits(kp) == want[0]).all() and (bits(vp) == want[1]).all()
