"""The serving operators over a cache held in 8 bits, as cases to measure.

Keys and values lie in pages as e4m3 codes, [pages, page, Hkv, d], with one power of two for every 16 slots and
head, [pages, page / 16, Hkv], held as its exponent plus 127 in a byte.  A case names one call:

  write    new tokens' keys and values quantized into the pages
  append   norm and rotation of the new tokens' q and k, then k and v quantized into the pages
  copy     whole pages with their scales copied to other pages (the fork of a sequence, a compaction)
  paged    attention of each sequence's newest tokens over its pages

A block of 16 slots that a call writes gets the smallest power of two 2^e with max|x| <= 448 2^e over the tokens
written, -100 <= e <= 119; where older tokens precede them in the block, it does not fall below the block's own, and
where it rises the older codes are rounded to it anew.

`run` computes a case in its plain form, or through the library where `own` is true; `exact` gives the values of the
definition in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BLOCK = 16                       # slots that share a scale
LOW, HIGH, BIAS = -100, 119, 127


# --------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One serving step of 64 sequences, one new token each, before the attention: the smallest of calls.
        dict(name="append_decode", op="append", B=64, new="1", lo=100, hi=4000, Hq=32, Hkv=8, d=128, rot=128,
             pairs="half", page=16, layout=21),
        # A step that takes in prompts: five ragged chunks of up to 2048 tokens behind cached prefixes.
        dict(name="append_chunks", op="append", B=5, new="1100-2048", lo=2048, hi=9000, Hq=32, Hkv=8, d=128, rot=128,
             pairs="half", page=64, layout=22),
        # Keys that come rotated, long prompts: bound by the bytes of the projection.
        dict(name="write_prompts", op="write", B=8, new="4096", lo=4096, hi=6000, Hkv=8, d=128, page=64, layout=23),
        # A few accepted tokens of each sequence, in the middle of blocks that hold older tokens; small heads.
        dict(name="write_accepted", op="write", B=48, new="1-7", lo=40, hi=3000, Hkv=4, d=64, page=32, layout=24),
        # Forks of a few sequences: the last, partly filled page of each is copied.
        dict(name="copy_fork", op="copy", n=24, pages=512, page=16, Hkv=8, d=128, layout=25),
        # A compaction that moves thousands of pages.
        dict(name="copy_compact", op="copy", n=4096, pages=9001, page=16, Hkv=8, d=128, layout=26),
        # One decode step over long caches (16 sequences of 1024 to 32768 tokens, 32 query heads on 8 key heads):
        # bound by the bytes of the cache.
        dict(name="paged_decode", op="paged", B=16, new="1", lo=1024, hi=32768, Hq=32, Hkv=8, d=128, page=64,
             causal=True, window=-1, alibi=False, layout=27),
        # One sequence, one new token, a short cache, small heads: latency alone.
        dict(name="paged_one", op="paged", B=1, new="1", lo=777, hi=777, Hq=16, Hkv=16, d=64, page=16,
             causal=True, window=-1, alibi=False, layout=28),
        # A decode step of many sequences with a sliding window and ALiBi, an odd number of key heads.
        dict(name="paged_window", op="paged", B=120, new="1", lo=200, hi=9000, Hq=21, Hkv=3, d=64, page=32,
             causal=True, window=2000, alibi=True, layout=29),
        # A step that verifies five proposed tokens of each sequence.
        dict(name="paged_verify", op="paged", B=32, new="5", lo=1000, hi=12000, Hq=32, Hkv=8, d=128, page=32,
             causal=True, window=-1, alibi=False, layout=30),
        # A mixed serving step: most sequences bring one token, some a ragged chunk of a prompt.
        dict(name="paged_mixed", op="paged", B=24, new="1,1,1,1,1,97-512", lo=600, hi=6000, Hq=32, Hkv=8, d=128, page=16,
             causal=True, window=-1, alibi=False, layout=31),
        # Chunks of 2048 new tokens behind long prefixes: bound by the tensor cores.
        dict(name="paged_chunk", op="paged", B=2, new="2048", lo=24000, hi=32768, Hq=32, Hkv=8, d=128, page=64,
             causal=True, window=-1, alibi=False, layout=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "append", "copy", "paged", "paged", "paged", "paged"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hq = min(Hkv * group, 32 // Hkv * Hkv)
    page = rng.choice([16, 32, 64, 128, 256])
    layout = rng.randrange(1, 1 << 30)
    if op == "copy":
        n = _log(rng, 1, 2000 * 16 // page)
        return dict(op=op, n=n, pages=2 * n + _log(rng, 1, 500), page=page, Hkv=Hkv, d=d, layout=layout)
    shape = rng.choice(["decode", "verify", "mixed", "chunk"])
    if shape == "decode":
        B, new, lo, hi = _log(rng, 1, 100), "1", 1, _log(rng, 20, 5000)
    elif shape == "verify":     # a few proposed tokens for each sequence
        B, new, lo, hi = _log(rng, 1, 48), str(rng.randrange(2, 9)), 8, _log(rng, 20, 5000)
    elif shape == "mixed":
        B, new, lo, hi = _log(rng, 2, 32), "1,1,1,0,2-%d" % _log(rng, 3, 400), 400, _log(rng, 401, 5000)
    else:
        c = _log(rng, 17, 1500)
        B, new, lo, hi = rng.randrange(1, 4), "%d-%d" % (max(1, c // 2), c), c, c + _log(rng, 1, 8000)
    case = dict(op=op, B=B, new=new, lo=lo, hi=hi, Hkv=Hkv, d=d, page=page, layout=layout)
    if op != "write":
        case.update(Hq=Hq)
    if op == "append":
        case.update(rot=rng.choice([0, 16, d // 2, d]), pairs=rng.choice(["half", "neighbours"]))
    if op == "paged":
        causal = rng.random() < 0.85
        case.update(causal=causal, window=_log(rng, 1, 4000) if causal and rng.random() < 0.4 else -1,
                    alibi=causal and rng.random() < 0.3)
    return case


def _lengths(case):
    """New tokens and cached tokens (the new ones included) of every sequence: part of the case, not of the seed."""
    r = random.Random(case["layout"])
    forms = case["new"].split(",")
    new, total = [], []
    for b in range(case["B"]):
        lo, _, hi = forms[b % len(forms)].partition("-")
        new.append(r.randint(int(lo), int(hi or lo)))
        total.append(max(new[-1], r.randint(case["lo"], case["hi"])))
    return new, total


# -------------------------------------------------------------------------------------------- inputs

def _tables(n, rot):
    """cos and sin of position times frequency, float32 [n, rot / 2], the angles in float64."""
    if rot == 0:
        return None, None
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["layout"] % 1000003)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    op, d, H, P, s = case["op"], case["d"], case["Hkv"], case["page"], dict(case=case)

    def pool(pages):
        """Codes of normal values, and scales that differ by factors of up to 8 between blocks."""
        codes = (normal(pages, P, H, d, dtype=torch.float32) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        scales = torch.randint(BIAS - 8, BIAS - 4, (pages, P // BLOCK, H), generator=g, device="cuda")
        return codes, scales.to(torch.uint8)

    if op == "copy":
        order = torch.randperm(case["pages"], generator=g, device="cuda").int()
        s["src"], s["dst"] = order[:case["n"]].clone(), order[case["n"]:2 * case["n"]].clone()
        s["k_pages"], s["k_scales"] = pool(case["pages"])
        s["v_pages"], s["v_scales"] = pool(case["pages"])
        return s
    new, total = _lengths(case)
    used = [-(-n // P) for n in total]
    width, pages = max(used) + 1, sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((case["B"], width), -1, dtype=torch.int32)
    at, order = 0, order.cpu()
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["table"], s["new"], s["total"], s["at"] = table.cuda(), new, total, cu
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["k_pages"], s["k_scales"] = pool(pages)
    s["v_pages"], s["v_scales"] = pool(pages)
    if op == "paged":
        s["q"] = normal(cu[-1], case["Hq"], d)
        if case["alibi"]:
            s["slopes"] = torch.tensor([2.0 ** (-8 * (h + 1) / case["Hq"]) for h in range(case["Hq"])], device="cuda")
        return s
    Hq = case.get("Hq", 0)
    s["qkv"] = normal(cu[-1], Hq + 2 * H, d)         # the parts of one fused projection's output, so rows are strided
    s["q"], s["k"], s["v"] = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + H], s["qkv"][:, Hq + H:]
    if op == "append":
        s["qw"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["kw"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["cos"], s["sin"] = _tables(max(total), case["rot"])
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _pow2(e):
    """2^e in float32, made of its bits: exact, -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _norm_rope(x, w, cos, sin, pairs):
    """float32 in and out; the first 2 * cos.shape[1] elements rotated by the angles of cos and sin [T, rot / 2]."""
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    if cos is None:
        return y
    h, c, s = cos.shape[1], cos[:, None], sin[:, None]
    first, second = (slice(0, h), slice(h, 2 * h)) if pairs == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    a, b = y[..., first], y[..., second]
    z = y.clone()
    z[..., first], z[..., second] = a * c - b * s, b * c + a * s
    return z


def _slots(s):
    """Position and slot (page * page size + place in it) of every new token, and of every sequence's first one."""
    P = s["case"]["page"]
    n = s["cu"].long().diff()
    start = s["lens"].long() - n
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["at"][-1])
    pos = torch.arange(s["at"][-1], device="cuda") - s["cu"].long()[seq] + start[seq]
    slot = s["table"][seq, pos // P].long() * P + pos % P
    first = s["table"][torch.arange(len(n), device="cuda"), start // P].long() * P + start % P
    return pos, slot, first, n > 0


def _write(pages, scales, slot, first, brings, x):
    """x [T, H, d] float32 into the slots, quantized; `first`: the first new slot of every sequence that brings any."""
    H, d = x.shape[1:]
    codes, sc = pages.view(torch.uint8).view(-1, BLOCK, H, d), scales.view(-1, H)
    top = torch.zeros(sc.shape, device="cuda").index_reduce_(0, slot // BLOCK, x.abs().amax(-1), "amax")
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875)).clamp(LOW, HIGH).masked_fill(top == 0, LOW)
    # blocks that hold older tokens: at most one of each sequence
    at, older = torch.where(brings, first // BLOCK, 0), torch.where(brings, first % BLOCK, 0)
    was, mine = sc[at].int() - BIAS, e[at]
    now = torch.where((older > 0)[:, None], torch.maximum(was, mine), mine)
    e.index_reduce_(0, at, torch.where(brings[:, None], now, LOW), "amax")
    old = codes[at].view(torch.float8_e4m3fn).float() * _pow2((was - now).clamp(min=-126))[:, None, :, None]
    keep = torch.arange(BLOCK, device="cuda") < older[:, None]
    t = codes.view(-1, H, d)
    place = torch.where(keep, at[:, None] * BLOCK + torch.arange(BLOCK, device="cuda"), slot[0])
    t[place] = old.to(torch.float8_e4m3fn).view(torch.uint8)          # slot[0] is written below, whatever it gets here
    y = x * _pow2(-e[slot // BLOCK])[..., None]
    t[slot] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    sc[slot // BLOCK] = (e[slot // BLOCK] + BIAS).to(torch.uint8)


def _plain_append(s):
    case = s["case"]
    pos, slot, first, brings = _slots(s)
    k, q = s["k"].float(), None
    if case["op"] == "append":
        cos, sin = (None, None) if s["cos"] is None else (s["cos"][pos], s["sin"][pos])
        q = _norm_rope(s["q"], s["qw"], cos, sin, case["pairs"]).to(s["q"].dtype)
        k = _norm_rope(s["k"], s["kw"], cos, sin, case["pairs"])
    _write(s["k_pages"], s["k_scales"], slot, first, brings, k)
    _write(s["v_pages"], s["v_scales"], slot, first, brings, s["v"].float())
    return q


def _gather(pages, scales, page, place):
    """Values at [page, place], float32."""
    x = pages.view(torch.uint8)[page, place].view(torch.float8_e4m3fn).float()
    return x * _pow2(scales[page, place // BLOCK].int() - BIAS)[..., None]


def _attend(s, bs, o, lse):
    """The sequences bs, padded to the longest of them."""
    case = s["case"]
    Hq, H, d, P = case["Hq"], case["Hkv"], case["d"], case["page"]
    G, M, n = Hq // H, max(s["new"][b] for b in bs), max(s["total"][b] for b in bs)
    ids = torch.tensor(bs, device="cuda")
    new, total = s["cu"].long().diff()[ids], s["lens"].long()[ids]
    at = torch.arange(n, device="cuda")
    page, place = s["table"][ids][:, at // P].long().clamp(min=0), (at % P).expand(len(bs), n)
    i = torch.arange(M, device="cuda")
    rows = (s["cu"].long()[ids][:, None] + i).clamp(max=s["q"].shape[0] - 1)
    live = i < new[:, None]
    dist = (total - new)[:, None, None] + i[:, None] - at                      # [b, M, n]
    hidden = (at >= total[:, None])[:, None].expand(dist.shape)
    if case["causal"]:
        hidden = hidden | (dist < 0)
    if case["window"] >= 0:
        hidden = hidden | (dist > case["window"])
    k = _gather(s["k_pages"], s["k_scales"], page, place).permute(0, 2, 3, 1)    # [b, H, d, n]
    v = _gather(s["v_pages"], s["v_scales"], page, place).transpose(1, 2)
    q = s["q"][rows].float().view(len(bs), M, H, G, d).permute(0, 2, 3, 1, 4)    # [b, H, G, M, d]
    step = max(1, min(H, (1 << 28) // (len(bs) * G * M * n)))                    # key heads at a time, by the scores' size
    for h in range(0, H, step):
        e = min(H, h + step)
        x = torch.matmul(q[:, h:e].reshape(len(bs), e - h, G * M, d), k[:, h:e]).mul_(d ** -0.5).view(len(bs), e - h, G, M, n)
        if case["alibi"]:
            x -= s["slopes"][h * G:e * G].view(1, e - h, G, 1, 1) * dist[:, None, None]
        x.masked_fill_(hidden[:, None, None], float("-inf"))
        top = x.amax(-1, keepdim=True)
        x = x.sub_(top).exp_()
        z = x.sum(-1, keepdim=True)
        y = torch.matmul(x.view(len(bs), e - h, G * M, n), v[:, h:e]).view(len(bs), e - h, G, M, d) / z
        o[rows[live], h * G:e * G] = y.permute(0, 3, 1, 2, 4).reshape(len(bs), M, -1, d)[live].to(o.dtype)
        lse[h * G:e * G, rows[live]] = (top + torch.log(z)).permute(0, 3, 1, 2, 4).reshape(len(bs), M, -1)[live].T


def _plain_paged(s):
    case = s["case"]
    T = s["q"].shape[0]
    o = torch.empty(T, case["Hq"], case["d"], dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(case["Hq"], T, dtype=torch.float32, device="cuda")
    # together what is of a size: one token each, then those with more, a few at a time
    left = sorted((b for b in range(case["B"]) if s["new"][b]), key=lambda b: (s["new"][b], s["total"][b]))
    while left:
        m, n = s["new"][left[0]], 2 * s["total"][left[0]]
        few = [b for b in left if s["new"][b] <= max(8, 2 * m) and s["total"][b] <= max(n, 20000000 // (case["Hkv"] * case["d"]))]
        few = few[:max(1, (1 << 29) // (case["Hkv"] * case["d"] * max(s["total"][b] for b in few)))]
        _attend(s, few, o, lse)
        left = [b for b in left if b not in set(few)]
    return o, lse


def _run_plain(s):
    op = s["case"]["op"]
    if op == "paged":
        return _plain_paged(s)
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        for pool in (s["k_pages"].view(torch.uint8), s["v_pages"].view(torch.uint8), s["k_scales"], s["v_scales"]):
            pool[dst] = pool[src]
        return None
    return _plain_append(s)


# ----------------------------------------------------------------------------------- the library's calls

def _run_own(s):
    from exact_io_aware_36_gb300 import fa
    case = s["case"]
    op = case["op"]
    cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    if op == "copy":
        return fa.cache_copy_fp8(*cache, s["src"], s["dst"])
    kw = dict(cu_seqlens=s["cu"], max_seqlen=max(s["new"]))
    if op == "write":
        return fa.cache_append_fp8(s["k"], s["v"], *cache, s["table"], s["lens"], **kw)
    if op == "append":
        return fa.qk_norm_rope_append_fp8(s["q"], s["k"], s["v"], *cache, s["table"], s["lens"], q_weight=s["qw"],
                                          k_weight=s["kw"], eps=EPS, cos=s["cos"], sin=s["sin"],
                                          interleaved=case["pairs"] == "neighbours", **kw)
    return fa.attention_forward_paged_fp8(s["q"], *cache, s["table"], s["lens"], causal=case["causal"],
                                          window=case["window"] if case["window"] >= 0 else None,
                                          alibi_slopes=s.get("slopes"), **kw)


def run(state):
    out = _run_own(state) if own else _run_plain(state)
    if state["case"]["op"] == "paged":
        return out
    # the cache as it is now: the codes' values, and the powers of two that they are multiplied with
    cache = dict(k=state["k_pages"], v=state["v_pages"], k_scale=state["k_scales"].view(torch.float8_e8m0fnu),
                 v_scale=state["v_scales"].view(torch.float8_e8m0fnu))
    return cache if out is None else dict(cache, q=out)


# ---------------------------------------------------------------------------------------------- work

def work(case):
    op, d, H = case["op"], case["d"], case["Hkv"]
    if op == "copy":
        return dict(bytes=4 * case["n"] * case["page"] * H * (d + 1 / BLOCK), flops=0)
    new, total = _lengths(case)
    T, Hq = sum(new), case.get("Hq", 0)
    if op in ("append", "write"):
        blocks = sum(-(-n // BLOCK) - (n - m) // BLOCK for m, n in zip(new, total) if m)
        moved = T * H * d * 2 * 3 + blocks * H * 2 + 4 * T          # keys and values read and written as codes, scales, table
        if op == "write":
            return dict(bytes=moved, flops=4 * T * H * d)
        return dict(bytes=moved + T * Hq * d * 4 + T * case["rot"] * 4, flops=8 * T * (Hq + 2 * H) * d)
    keys = pairs = 0
    for m, n in zip(new, total):
        if m == 0:
            continue
        w = case["window"] if case["window"] >= 0 else n
        keys += min(n, m + w)
        pairs += m * n if not case["causal"] else sum(min(p, w) + 1 for p in range(n - m, n))
    return dict(bytes=keys * H * 2 * (d + 1 / BLOCK) + 4 * T * Hq * d + 4 * T * Hq, flops=4 * pairs * Hq * d)


# --------------------------------------------------------------------------------------------- exact

def _power(e):
    """2^e in float64, made of its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(y):
    """Float64 values rounded to the nearest of e4m3 (4 bits, the least step 2^-9, at most 448), ties to even."""
    step = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_rows(x, w, pos, case, s):
    y = x.double()
    y = y / (y.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    rot = case["rot"]
    if rot:
        i = torch.arange(rot // 2, device="cuda")
        a, b = (i, i + rot // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(y[..., a], y[..., b]) * torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_write(s, pages, scales, x):
    """Sequence by sequence, block by block."""
    P = s["case"]["page"]
    codes, power = pages.double(), scales.long() - BIAS
    table = s["table"].tolist()
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        p, t = n - m, s["at"][b]
        while p < n:
            end = min(n, (p // BLOCK + 1) * BLOCK)
            rows, page, lo = x[t:t + end - p], table[b][p // P], p % P
            j = lo // BLOCK
            size = rows.abs().amax((0, 2))
            e = torch.ceil(torch.log2(size / 448)).clamp(LOW, HIGH).long()
            if lo % BLOCK:
                was = power[page, j].clone()
                e = torch.maximum(e, was)
                old = codes[page, j * BLOCK:lo]
                old.copy_(_e4m3(old * _power(was - e)[:, None]))
            power[page, j] = e
            codes[page, lo:lo + end - p] = _e4m3(rows * _power(-e)[:, None])
            t, p = t + end - p, end
    return codes, _power(power)


def _exact_paged(s):
    case = s["case"]
    Hq, H, d, P = case["Hq"], case["Hkv"], case["d"], case["page"]
    T = s["q"].shape[0]
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(Hq, T, dtype=torch.float64, device="cuda")
    k_powers, v_powers = _power(s["k_scales"].long() - BIAS), _power(s["v_scales"].long() - BIAS)
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        at = torch.arange(n, device="cuda")
        page, off = s["table"][b].long()[at // P], at % P
        kb = s["k_pages"].view(torch.uint8)[page, off].view(torch.float8_e4m3fn).double() * k_powers[page, off // BLOCK][..., None]
        vb = s["v_pages"].view(torch.uint8)[page, off].view(torch.float8_e4m3fn).double() * v_powers[page, off // BLOCK][..., None]
        for h in range(Hq):
            k, v = kb[:, h * H // Hq], vb[:, h * H // Hq]
            for i in range(0, m, 512):                       # rows in blocks, one head at a time
                r = torch.arange(i, min(m, i + 512), device="cuda")
                row, t = (n - m + r)[:, None], s["at"][b] + r
                x = s["q"][t, h].double() @ k.T / math.sqrt(d)
                if case["alibi"]:
                    x = x + s["slopes"][h].double() * (at[None] - row)
                seen = torch.ones(len(r), n, dtype=torch.bool, device="cuda")
                if case["causal"]:
                    seen &= at[None] <= row
                if case["window"] >= 0:
                    seen &= at[None] >= row - case["window"]
                x = x.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[h, t] = z
                o[t, h] = torch.exp(x - z[:, None]) @ v
    return o, lse


def exact(case, seed):
    if case["op"] == "paged" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "paged":
        return _exact_paged(s)
    names = ("k_pages", "v_pages", "k_scales", "v_scales")
    if op == "copy":
        out = [s[n].double() if n[2] == "p" else _power(s[n].long() - BIAS) for n in names]
        for pool in out:
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                pool[b].copy_(pool[a])
        return dict(zip(("k", "v", "k_scale", "v_scale"), out))
    k, out = s["k"].double(), {}
    if op == "append":
        pos = torch.tensor([p for m, n in zip(s["new"], s["total"]) for p in range(n - m, n)], device="cuda")
        out["q"] = _exact_rows(s["q"], s["qw"], pos, case, s)
        k = _exact_rows(s["k"], s["kw"], pos, case, s)
    out["k"], out["k_scale"] = _exact_write(s, s["k_pages"], s["k_scales"], k)
    out["v"], out["v_scale"] = _exact_write(s, s["v_pages"], s["v_scales"], s["v"].double())
    return out
