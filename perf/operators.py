"""The serving and training operators around exact attention, as cases to measure.

A case names one call:

  norm_rope      RMS norm of every query and key head and the rotation by position, one pass over q and k
  norm_rope_bwd  its gradient: dq, dk and the two weights' gradients
  append         norm and rotation of the new tokens' q and k, k and v written into the pages of a cache
  copy           whole pages of a cache copied to other pages (the fork of a sequence, a compaction)
  paged          attention of each sequence's newest tokens over its pages

`run` computes a case in its plain form, or through the library where `own` is true; `exact` gives the values
of the definition in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # A training micro-batch of packed sequences: 32 query and 8 key heads of 128, the q and k parts of one
        # fused projection's output (so their rows are strided).
        dict(name="norm_rope_train", op="norm_rope", T=16384, Hq=32, Hkv=8, d=128, rot=128, pairs="half",
             dtype="bf16", layout=1),
        # An odd number of tokens in float32, half of each head rotated, neighbouring elements paired.
        dict(name="norm_rope_fp32_part", op="norm_rope", T=3001, Hq=12, Hkv=4, d=64, rot=32, pairs="neighbours",
             dtype="fp32", layout=2),
        # The backward pass of the training micro-batch.
        dict(name="norm_rope_bwd_train", op="norm_rope_bwd", T=16384, Hq=32, Hkv=8, d=128, rot=128, pairs="half",
             dtype="bf16", layout=1),
        # The backward pass of a short, odd batch: few tokens, where the weights' sums cost as much as the rows.
        dict(name="norm_rope_bwd_short", op="norm_rope_bwd", T=777, Hq=16, Hkv=8, d=64, rot=64, pairs="half",
             dtype="bf16", layout=3),
        # One serving step of 64 sequences, one new token each, before the attention: the smallest of calls.
        dict(name="append_decode", op="append", B=64, new="1", lo=100, hi=4000, Hq=32, Hkv=8, d=128, rot=128,
             pairs="half", page=16, layout=4),
        # A step that takes in prompts: five ragged chunks of up to 2048 tokens behind cached prefixes.
        dict(name="append_chunks", op="append", B=5, new="1100-2048", lo=2048, hi=9000, Hq=32, Hkv=8, d=128, rot=128,
             pairs="half", page=64, layout=5),
        # Forks of a few sequences: the last, partly filled page of each is copied.
        dict(name="copy_fork", op="copy", n=24, pages=512, page=16, Hkv=8, d=128, layout=6),
        # A compaction that moves thousands of pages.
        dict(name="copy_compact", op="copy", n=4096, pages=9001, page=16, Hkv=8, d=128, layout=7),
        # One decode step over long caches (16 sequences of 1024 to 32768 tokens, 32 query heads on 8 key heads):
        # bound by the bytes of the cache.
        dict(name="paged_decode", op="paged", B=16, new="1", lo=1024, hi=32768, Hq=32, Hkv=8, d=128, page=64,
             causal=True, window=-1, alibi=False, layout=8),
        # One sequence, one new token, a short cache, small heads: latency alone.
        dict(name="paged_one", op="paged", B=1, new="1", lo=777, hi=777, Hq=16, Hkv=16, d=64, page=16,
             causal=True, window=-1, alibi=False, layout=9),
        # A mixed serving step: most sequences bring one token, some a ragged chunk of a prompt.
        dict(name="paged_mixed", op="paged", B=24, new="1,1,1,1,1,97-512", lo=600, hi=6000, Hq=32, Hkv=8, d=128, page=16,
             causal=True, window=-1, alibi=False, layout=10),
        # Chunks of 2048 new tokens behind long prefixes: bound by the tensor cores.
        dict(name="paged_chunk", op="paged", B=2, new="2048", lo=24000, hi=32768, Hq=32, Hkv=8, d=128, page=64,
             causal=True, window=-1, alibi=False, layout=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "copy", "paged", "paged", "paged"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    layout = rng.randrange(1, 1 << 30)
    if op in ("norm_rope", "norm_rope_bwd"):
        Hq = min(Hkv * group, 32 // Hkv * Hkv)
        return dict(op=op, T=_log(rng, 1, 12000), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([0, 16, d // 2, d]),
                    pairs=rng.choice(["half", "neighbours"]), dtype=rng.choice(["bf16", "bf16", "fp32"]), layout=layout)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "copy":
        n = _log(rng, 1, 2000 * 16 // page)
        return dict(op=op, n=n, pages=2 * n + _log(rng, 1, 500), page=page, Hkv=Hkv, d=d, layout=layout)
    Hq = min(Hkv * group, 32 // Hkv * Hkv)
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
    case = dict(op=op, B=B, new=new, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, layout=layout)
    if op == "append":
        case.update(rot=rng.choice([0, 16, d // 2, d]), pairs=rng.choice(["half", "neighbours"]))
    else:
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


def _runs(case):
    """Lengths of the packed sequences of a training batch."""
    r, left, out = random.Random(case["layout"]), case["T"], []
    while left:
        out.append(min(left, r.randint(1, 4096)))
        left -= out[-1]
    return out


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

    op, d, Hkv, s = case["op"], case["d"], case["Hkv"], dict(case=case)
    if op in ("norm_rope", "norm_rope_bwd", "append"):
        Hq = case["Hq"]
        dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
        T = case["T"] if op != "append" else sum(_lengths(case)[0])
        s["qkv"] = normal(T, Hq + 2 * Hkv, d, dtype=dtype)
        s["q"], s["k"], s["v"] = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
        s["qw"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["kw"] = 1 + 0.1 * normal(d, dtype=torch.float32)
    if op in ("norm_rope", "norm_rope_bwd"):
        runs = _runs(case)
        s["cos"], s["sin"] = _tables(max(runs), case["rot"])
        s["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in runs]).cuda()
        if op == "norm_rope_bwd":
            s["dzq"], s["dzk"] = normal(T, Hq, d, dtype=dtype), normal(T, Hkv, d, dtype=dtype)
        return s
    if op == "copy":
        order = torch.randperm(case["pages"], generator=g, device="cuda").int()
        s["src"], s["dst"] = order[:case["n"]].clone(), order[case["n"]:2 * case["n"]].clone()
        s["k_pages"] = normal(case["pages"], case["page"], Hkv, d)
        s["v_pages"] = normal(case["pages"], case["page"], Hkv, d)
        return s
    new, total = _lengths(case)
    P = case["page"]
    used = [-(-n // P) for n in total]
    width, pages = max(used) + 1, sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["new"], s["total"] = table, new, total
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["k_pages"] = normal(pages, P, Hkv, d)
    s["v_pages"] = normal(pages, P, Hkv, d)
    if op == "append":
        s["cos"], s["sin"] = _tables(max(total), case["rot"])
    else:
        s["q"] = normal(cu[-1], case["Hq"], d)
        if case["alibi"]:
            s["slopes"] = torch.tensor([2.0 ** (-8 * (h + 1) / case["Hq"]) for h in range(case["Hq"])], device="cuda")
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, pairs):
    """x [T, H, d] float32; its first 2 * cos.shape[1] elements rotated by the angles of cos and sin [T, rot / 2]."""
    if cos is None:
        return x
    h = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * c - b * s, b * c + a * s
    return y


def _norm_rope(x, w, cos, sin, pairs):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    return _rotate(f * r * w, cos, sin, pairs).to(x.dtype)


def _norm_rope_bwd(x, dz, w, cos, sin, pairs):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    dy = _rotate(dz.float(), cos, None if sin is None else -sin, pairs)
    hat = f * r
    dw = (dy * hat).sum((0, 1), dtype=torch.float64).float()
    dhat = dy * w
    dx = r * (dhat - hat * (dhat * hat).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _at(s, pos):
    return (None, None) if s["cos"] is None else (s["cos"][pos], s["sin"][pos])


def _plain_append(s):
    case = s["case"]
    P = case["page"]
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(s["new"], s["total"])]).cuda()
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(s["new"])]).cuda()
    cos, sin = _at(s, pos)
    page = s["table"][seq, pos // P].long()
    s["k_pages"][page, pos % P] = _norm_rope(s["k"], s["kw"], cos, sin, case["pairs"])
    s["v_pages"][page, pos % P] = s["v"]
    return _norm_rope(s["q"], s["qw"], cos, sin, case["pairs"]), s["k_pages"], s["v_pages"]


def _plain_paged(s):
    case = s["case"]
    Hq, Hkv, d, P = case["Hq"], case["Hkv"], case["d"], case["page"]
    G, scale = Hq // Hkv, d ** -0.5
    T = s["q"].shape[0]
    o = torch.empty(T, Hq, d, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(Hq, T, dtype=torch.float32, device="cuda")
    t0 = 0
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        if m == 0:
            continue
        ids = s["table"][b, :-(-n // P)].long()
        k = s["k_pages"][ids].reshape(-1, Hkv, d)[:n].float()
        v = s["v_pages"][ids].reshape(-1, Hkv, d)[:n].float()
        q = s["q"][t0:t0 + m].float()
        dist = torch.arange(n - m, n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None]
        hidden = torch.zeros_like(dist, dtype=torch.bool)
        if case["causal"]:
            hidden |= dist < 0
        if case["window"] >= 0:
            hidden |= dist > case["window"]
        step = max(1, min(Hkv, (1 << 28) // (G * m * n)))        # key heads at a time, by the scores' size
        for g in range(0, Hkv, step):
            e = min(Hkv, g + step)
            x = q[:, g * G:e * G].reshape(m, e - g, G, d).permute(1, 2, 0, 3).reshape(e - g, G * m, d)
            x = torch.matmul(x, k[:, g:e].permute(1, 2, 0)).mul_(scale).view(e - g, G, m, n)
            if case["alibi"]:
                x -= s["slopes"][g * G:e * G].view(e - g, G, 1, 1) * dist
            x.masked_fill_(hidden, float("-inf"))
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            z = x.sum(-1, keepdim=True)
            y = torch.matmul(x.view(e - g, G * m, n), v[:, g:e].transpose(0, 1)).view(e - g, G, m, d) / z
            o[t0:t0 + m, g * G:e * G] = y.permute(2, 0, 1, 3).reshape(m, (e - g) * G, d).to(o.dtype)
            lse[g * G:e * G, t0:t0 + m] = (top + torch.log(z)).view((e - g) * G, m)
        t0 += m
    return o, lse


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_rope":
        cos, sin = _at(s, s["pos"].long())
        return (_norm_rope(s["q"], s["qw"], cos, sin, case["pairs"]),
                _norm_rope(s["k"], s["kw"], cos, sin, case["pairs"]))
    if op == "norm_rope_bwd":
        cos, sin = _at(s, s["pos"].long())
        dq, dqw = _norm_rope_bwd(s["q"], s["dzq"], s["qw"], cos, sin, case["pairs"])
        dk, dkw = _norm_rope_bwd(s["k"], s["dzk"], s["kw"], cos, sin, case["pairs"])
        return dq, dk, dqw, dkw
    if op == "append":
        return _plain_append(s)
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        s["k_pages"][dst] = s["k_pages"][src]
        s["v_pages"][dst] = s["v_pages"][src]
        return s["k_pages"], s["v_pages"]
    return _plain_paged(s)


# ----------------------------------------------------------------------------------- the library's calls

def _run_own(s):
    from exact_io_aware_36_gb300 import fa
    case = s["case"]
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd", "append"):
        kw = dict(q_weight=s["qw"], k_weight=s["kw"], eps=EPS, cos=s["cos"], sin=s["sin"],
                  interleaved=case["pairs"] == "neighbours")
    if op == "norm_rope":
        return fa.qk_norm_rope(s["q"], s["k"], positions=s["pos"], **kw)
    if op == "norm_rope_bwd":
        return fa.qk_norm_rope_backward(s["q"], s["k"], s["dzq"], s["dzk"], positions=s["pos"], **kw)
    if op == "append":
        q = fa.qk_norm_rope_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                   cu_seqlens=s["cu"], max_seqlen=max(s["new"]), **kw)
        return q, s["k_pages"], s["v_pages"]
    if op == "copy":
        fa.cache_copy(s["k_pages"], s["v_pages"], s["src"], s["dst"])
        return s["k_pages"], s["v_pages"]
    return fa.attention_forward_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], cu_seqlens=s["cu"],
                                      max_seqlen=max(s["new"]), causal=case["causal"],
                                      window=case["window"] if case["window"] >= 0 else None,
                                      alibi_slopes=s.get("slopes"))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------- work

def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op in ("norm_rope", "norm_rope_bwd"):
        e = 4 if case["dtype"] == "fp32" else 2
        elems = case["T"] * (case["Hq"] + Hkv) * d
        tables = max(_runs(case)) * case["rot"] * 4 + case["T"] * 4
        if op == "norm_rope":
            return dict(bytes=2 * elems * e + tables + 8 * d, flops=8 * elems)
        return dict(bytes=3 * elems * e + tables + 16 * d, flops=18 * elems)
    if op == "copy":
        return dict(bytes=4 * case["n"] * case["page"] * Hkv * d * 2, flops=0)
    new, total = _lengths(case)
    T, Hq = sum(new), case["Hq"]
    if op == "append":
        angles = sum(new) * case["rot"] * 4
        return dict(bytes=2 * T * (Hq + 2 * Hkv) * d * 2 + angles + 12 * T, flops=8 * T * (Hq + Hkv) * d)
    keys = pairs = 0
    for m, n in zip(new, total):
        if m == 0:
            continue
        w = case["window"] if case["window"] >= 0 else n
        keys += min(n, m + w)
        pairs += m * n if not case["causal"] else sum(min(p, w) + 1 for p in range(n - m, n))
    return dict(bytes=4 * keys * Hkv * d + 4 * T * Hq * d + 4 * T * Hq, flops=4 * pairs * Hq * d)


# --------------------------------------------------------------------------------------------- exact

def _turn(pos, rot, pairs, d, cos, sin):
    """The rotation of every token as complex factors, and the element pairs they act on."""
    i = torch.arange(rot // 2, device="cuda")
    first, second = (i, i + rot // 2) if pairs == "half" else (2 * i, 2 * i + 1)
    return first, second, torch.complex(cos.double(), sin.double())[pos]


def _exact_rows(x, w, turn):
    y = x.double()
    y = y / (y.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    if turn is not None:
        first, second, factor = turn
        z = torch.complex(y[..., first], y[..., second]) * factor[:, None]
        y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_grad(x, dz, w, turn):
    """By the Jacobian of x / rms: with n = mean(x^2) + eps, d(x_i n^-1/2)/dx_j = n^-1/2 (delta - x_i x_j / (d n))."""
    x, dy, w = x.double(), dz.double().clone(), w.double()
    if turn is not None:
        first, second, factor = turn
        z = torch.complex(dy[..., first], dy[..., second]) * factor[:, None].conj()
        dy[..., first], dy[..., second] = z.real, z.imag
    n = x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS
    dw = torch.einsum("thd,thd->d", dy, x * n.pow(-0.5))
    gw = dy * w
    inner = torch.einsum("thd,thd->th", gw, x)[..., None]
    return n.pow(-0.5) * gw - n.pow(-1.5) * x * inner / x.shape[-1], dw


def _exact_paged(s):
    case = s["case"]
    Hq, Hkv, d, P = case["Hq"], case["Hkv"], case["d"], case["page"]
    T = s["q"].shape[0]
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(Hq, T, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        at = torch.arange(n, device="cuda")
        page = s["table"][b].long()[at // P]
        for h in range(Hq):
            k, v = s["k_pages"][page, at % P, h * Hkv // Hq].double(), s["v_pages"][page, at % P, h * Hkv // Hq].double()
            for i in range(0, m, 512):                       # rows in blocks, one head at a time
                r = torch.arange(i, min(m, i + 512), device="cuda")
                row = (n - m + r)[:, None]
                x = s["q"][t0 + r, h].double() @ k.T / math.sqrt(d)
                if case["alibi"]:
                    x = x + s["slopes"][h].double() * (at[None] - row)
                seen = torch.ones(len(r), n, dtype=torch.bool, device="cuda")
                if case["causal"]:
                    seen &= at[None] <= row
                if case["window"] >= 0:
                    seen &= at[None] >= row - case["window"]
                x = x.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[h, t0 + r] = z
                o[t0 + r, h] = torch.exp(x - z[:, None]) @ v
        t0 += m
    return o, lse


def exact(case, seed):
    if case["op"] == "paged" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "copy":
        out = []
        for pool in (s["k_pages"], s["v_pages"]):
            pool = pool.double()
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                pool[b].copy_(pool[a])
            out.append(pool)
        return tuple(out)
    if op == "paged":
        return _exact_paged(s)
    if op == "append":
        pos = torch.tensor([p for m, n in zip(s["new"], s["total"]) for p in range(n - m, n)], device="cuda")
    else:
        pos = s["pos"].long()
    turn = _turn(pos, case["rot"], case["pairs"], case["d"], s["cos"], s["sin"]) if case["rot"] else None
    if op == "norm_rope":
        return _exact_rows(s["q"], s["qw"], turn), _exact_rows(s["k"], s["kw"], turn)
    if op == "norm_rope_bwd":
        dq, dqw = _exact_grad(s["q"], s["dzq"], s["qw"], turn)
        dk, dkw = _exact_grad(s["k"], s["dzk"], s["kw"], turn)
        return dq, dk, dqw, dkw
    k, v = s["k_pages"].double(), s["v_pages"].double()
    rows, t, P = _exact_rows(s["k"], s["kw"], turn), 0, case["page"]
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        at = torch.arange(n - m, n, device="cuda")
        slot = s["table"][b].long()[at // P] * P + at % P
        k.view(-1, *k.shape[2:])[slot], v.view(-1, *v.shape[2:])[slot] = rows[t:t + m], s["v"][t:t + m].double()
        t += m
    return _exact_rows(s["q"], s["qw"], turn), k, v
