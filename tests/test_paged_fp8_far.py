"""A cache in 8 bits at the ends of its ranges: blocks of values very far apart,
scales below and at the largest that a write makes, sequences of any number of
new tokens.  Bounds are those that test_paged_fp8.py derives."""
import numpy as np
import pytest

from exact_io_aware_36_gb300 import fa
from oracle import paged_fp64 as P
from oracle import paged_fp8 as P8
from tests.test_cache_pages import cache
from tests.test_norm_rope import npf
from tests.test_paged_fp8 import attend, check, parts, pools, raw, same_codes, state


def value_scales(codes, scales, table, lens, page, step, bytes_of, zero):
    """Every `step` slots of a sequence get one of `bytes_of` as the scale of their values, at random; those with `zero`
    hold zeros."""
    import torch as t
    g = t.Generator().manual_seed(5)
    H = scales[1].shape[2]
    tab = table.cpu().numpy()
    c, s = codes[1].view(t.uint8).view(-1, 16, *codes[1].shape[2:]), scales[1].view(-1, H)
    for b, L in enumerate(lens):
        blocks = t.from_numpy(P.slots(tab[b], L, page)[::16] // 16).cuda()
        pick = t.randint(0, len(bytes_of), (-(-L // step), H), generator=g)
        kind = t.tensor(bytes_of, dtype=t.uint8)[pick].repeat_interleave(step // 16, 0)[:len(blocks)].cuda()
        s[blocks] = kind
        x = c[blocks]
        x[(kind == zero)[:, None, :, None].expand_as(x) & (x != 0x7f)] = 0
        c[blocks] = x


# one token of 8, 16, 24 and 32 heads, three of 8, five of 8 beside one of a chunk, five of 8 alone, a chunk
MIXES = [([1] * 6, 8), ([1] * 6, 16), ([1] * 6, 24), ([1] * 6, 32), ([3] * 6, 8), ([5, 1, 1, 300, 1, 1], 8), ([5] * 6, 8),
         ([300] * 2, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("new,group", MIXES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [100, 107, 110, 119])
def test_zeros_beside_values_of_any_size_count_in_the_sum(new, group, d, e):
    """Blocks of zeros take the least scale; the keys they stand for weigh what they do beside ordinary values."""
    import torch as t
    lens, page, Hkv = [3000 - 111 * b for b in range(len(new))], 32, 2
    q, codes, scales, table, cs, cu = state(new, lens, page, Hkv * group, Hkv, d, e, gain=2.0)
    kw = dict(cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    _, lse = attend(q, codes, scales, table, cs, **kw)
    value_scales(codes, scales, table, lens, page, 32, [127 + e, 27, 27], 27)
    if e >= 110:                                       # (a sum of many such values is past float32)
        c = codes[1].view(t.uint8)
        c[(c != 0) & (c != 0x7f)] = 1
    O, got = attend(q, codes, scales, table, cs, **kw)
    # the same scores, so each LSE is off by its own sum's share, 2^-20 (|lse| + 8) + 2^-22 |lse|
    assert t.allclose(got, lse, rtol=2.0 ** -18, atol=2.0 ** -16)
    check((O, got), q, codes, scales, table, lens, new, page)


@pytest.mark.gpu
@pytest.mark.parametrize("most", [2**31 - 1, 2**31 - 14, 2**31 - 15])
@pytest.mark.parametrize("B,Hkv", [(1, 2), (16, 8), (64, 8), (64, 2)])
def test_writes_without_a_bound_on_the_new_tokens(most, B, Hkv):
    """A max_seqlen that bounds nothing: every sequence's tokens are written."""
    import torch as t
    new = [1 + b % 5 for b in range(B)]
    lens = [n + 7 * (b % 9) for b, n in enumerate(new)]
    kp, _, table, cs, cu, g = cache(new, lens, 16, Hkv, 64, 8)
    k, v = (t.randn(sum(new), Hkv, 64, generator=g).bfloat16().cuda() for _ in range(2))
    one = t.ones(max(lens), 16, device="cuda")
    q = t.full_like(k, 5.0)
    kw = dict(cu_seqlens=cu, max_seqlen=most, check=True)
    for write in (lambda *c: fa.cache_append_fp8(k, v, *c, table, cs, **kw),
                  lambda *c: fa.qk_norm_rope_append_fp8(k, k, v, *c, table, cs, cos=one, sin=0 * one, q_out=q, **kw)):
        (kc, vc), (ks, vs) = pools(kp, g)
        args = (table.cpu().numpy(), lens, cu.cpu().numpy(), 16)
        want = [P8.append(raw(c), raw(s), npf(x), *args) for c, s, x in ((kc, ks, k), (vc, vs, v))]
        write(kc, vc, ks, vs)
        for c, s, w in ((kc, ks, want[0]), (vc, vs, want[1])):
            assert (raw(s) == w[1]).all() and same_codes(raw(c), w[0])
    assert t.equal(q, k)


@pytest.mark.gpu
@pytest.mark.parametrize("n,group", [(1, 1), (2, 8), (3, 8), (4, 8), (40, 1), (150, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_below_those_that_a_write_makes(n, group, d):
    """One key in view: O is its value exactly under scales of 2^-127 to 2^-101 too."""
    import torch as t
    B, Hkv = 27, 2
    vals = t.arange(256, dtype=t.int32).to(t.uint8)
    for lo in range(0, 256, Hkv * d):
        pool = vals.roll(-lo)[:Hkv * d].view(Hkv, d).expand(B, 16, Hkv, d).contiguous().cuda()
        scales = t.arange(B, dtype=t.uint8)[:, None, None].expand(B, 1, Hkv).contiguous().cuda()
        table = t.arange(B, dtype=t.int32, device="cuda")[:, None].contiguous()
        q = t.zeros(B * n, Hkv * group, d, dtype=t.bfloat16, device="cuda")
        one = t.full((B,), 1, dtype=t.int32, device="cuda")
        o, _ = fa.attention_forward_paged_fp8(q, t.zeros_like(pool), pool, scales, scales, table, one, causal=False,
                                              out_dtype=t.float32, check=True)
        want = P8.values(pool.cpu().numpy(), scales.cpu().numpy())[:, 0].repeat(group, 1)
        assert np.array_equal(npf(o).reshape(B, n, Hkv * group, d), want[:, None].repeat(n, 1), equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("new,group", MIXES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("byte", [246, 245, 3])
def test_many_values_at_the_ends_of_the_scales(new, group, d, byte):
    """O lies within the values, so it is as good as ever, whether the sum of p v is past float32 or not."""
    import torch as t
    lens, page, Hkv = [2000 - 111 * b for b in range(len(new))], 32, 2
    q, codes, scales, table, cs, cu = state(new, lens, page, Hkv * group, Hkv, d, byte)
    c = codes[1].view(t.uint8)
    c[..., ::2] &= 0x7f                                # half of the elements: no sign
    value_scales(codes, scales, table, lens, page, 16, [byte, byte, byte - 1, byte - 3], 255)
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, page)


@pytest.mark.gpu
@pytest.mark.parametrize("new,group", MIXES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bytes_of", [(27, 246), (0, 246), (27, 100, 200, 246)])
def test_the_largest_values_beside_the_smallest(new, group, d, bytes_of):
    """O goes on in the units of small values where large ones came before, and is as good as ever in the end."""
    import torch as t
    lens, page, Hkv = [2000 - 111 * b for b in range(len(new))], 32, 2
    q, codes, scales, table, cs, cu = state(new, lens, page, Hkv * group, Hkv, d, len(bytes_of))
    value_scales(codes, scales, table, lens, page, 16, list(bytes_of), 255)
    out = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check(out, q, codes, scales, table, lens, new, page)


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [0, 10, 26])
@pytest.mark.parametrize("size", [2.0 ** -118, 2.0 ** -110, 2.0 ** -90, 1.0])
def test_older_tokens_under_scales_that_no_write_makes(byte, size):
    """A block whose own scale lies below the least of a write: its older codes are rounded to the new one."""
    import torch as t
    kp, _, table, cs, cu, g = cache([3, 1], [12, 40], 16, 2, 64, 8)
    (kc, vc), (ks, vs) = pools(kp, g)
    for c, s in ((kc, ks), (vc, vs)):
        c.view(t.uint8).copy_(t.arange(c.numel(), device="cuda").view(c.shape) % 256)
        s.fill_(byte)
    k, v = (size * t.randn(4, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    args = (table.cpu().numpy(), [12, 40], cu.cpu().numpy(), 16)
    want = [P8.append(raw(c), raw(s), npf(x), *args) for c, s, x in ((kc, ks, k), (vc, vs, v))]
    fa.cache_append_fp8(k, v, kc, vc, ks, vs, table, cs, cu_seqlens=cu, max_seqlen=3, check=True)
    for c, s, w in ((kc, ks, want[0]), (vc, vs, want[1])):
        assert (raw(s) == w[1]).all() and same_codes(raw(c), w[0])


@pytest.mark.gpu
@pytest.mark.parametrize("new,group", MIXES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gaps", [(8,), (9,), (10,), (16,), (20,), (1, 9, 10), (3, 12, 18)])
def test_small_values_beside_large_ones(new, group, d, gaps):
    """Columns in which the blocks of the largest scale hold zeros: O there is made of the smaller ones alone.

    Scores are flat (gain 2^-10), so a row's keys weigh alike, the reference is within 2^s of every key, s = 2 |q| |k|
    scale log2 e, and its sum is at least 2^-s of the number of its keys.  Of a key's P at most half of fp16's least
    step is lost, 2^-25, over 2^6 at least, times a code of the largest scale: over the row 2^s 2^-31 448 2^e.  (More than
    20 apart, P over the largest scale is below fp16's normal numbers where rows are many.)"""
    import torch as t
    lens, page, Hkv = [2000 - 111 * b for b in range(len(new))], 32, 2
    top = 140
    q, codes, scales, table, cs, cu = state(new, lens, page, Hkv * group, Hkv, d, sum(gaps), gain=2.0 ** -10)
    scales[0][scales[0] != 255] -= 3                   # (|k| below 2^9)
    value_scales(codes, scales, table, lens, page, 16, [top] + [top - g for g in gaps], 255)
    c = codes[1].view(t.uint8).view(-1, 16, Hkv, d)
    large = (scales[1].view(-1, Hkv) == top)[:, None, :, None].expand_as(c) & (c != 0x7f)
    large[..., ::2] = False
    c[large] = 0
    O, lse = attend(q, codes, scales, table, cs, cu_seqlens=cu, max_seqlen=max(new), out_dtype=t.float32, check=True)
    check((O, lse), q, codes, scales, table, lens, new, page)
    k, v = (P8.values(raw(c), raw(s)) for c, s in zip(codes, scales))
    args = (np.where(table.cpu().numpy() < 0, 0, table.cpu().numpy()), lens, np.concatenate([[0], np.cumsum(new)]), page, d ** -0.5)
    Or, lr = P.attention(npf(q), k, v, *args)
    Ab = P.attention(npf(q), k, np.abs(v), *args)[0]
    pr, _, pq = parts(new, Hkv * group, Hkv).T[:, :, None]
    kn, qn = np.sqrt(np.nan_to_num((k * k).sum(-1))).max(), np.sqrt((npf(q) ** 2).sum(-1))
    e = ((d + 8) * 2.0 ** -23 * qn + pq * np.abs(npf(q)).max(-1) * np.sqrt(d)) * kn * d ** -0.5 + 2.0 ** -21 * (np.abs(lr.T) + 8)
    lost = 2.0 ** (2 * qn * kn * d ** -0.5 * np.log2(np.e)) * 2.0 ** -31 * 448 * 2.0 ** (top - 127)
    tol = (2 * e[..., None] + pr[..., None] + 2.0 ** -20) * Ab + 2.0 ** -24 * np.abs(Or) + lost[..., None]
    off = np.abs(npf(O) - Or)[..., 1::2] - tol[..., 1::2]
    assert off.max() <= 0, float(off.max())
    # And the bound says something: without the smaller blocks O would be past it nearly everywhere.  (20 apart, half of
    # 2000 keys: O is of 100 2^-7 1000^1/2 / 2000 = 0.012, the bound 448 2^-18 = 0.0017 and less than a tenth of that, so
    # |O| is below it with a probability of 0.12.)
    assert (np.abs(Or) > tol)[..., 1::2].mean() > 0.75
