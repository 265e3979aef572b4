"""Measured cases of the paged key/value cache and of the attention that reads it.

A serving loop keeps the keys and values of its sequences in pages of a common pool.  Each step it
rotates the new queries and keys by their positions, appends keys and values to the pages
(``kv_append``) and lets the queries attend to everything the pages hold (``attention_paged``).
The pool is bf16, or e4m3 (8 bits) with one scale per page and head.

Conventions: query and key/value heads [B, H, Nq, d]; pools [n_pages, Hkv, page, d]; page_table
[B, max_pages]; key_lens[b] keys in sequence b after the append, new_lens[b] of them new (the last
ones); query i of sequence b stands at position key_lens[b] - new_lens[b] + i.  Heads are shared in
groups of Hq / Hkv.  Scales of e4m3 pages are powers of two, the smallest with |x| <= 448 * scale.
"""
import math

import torch

own = False

MAX_POS = 131072   # rows of the rotation tables


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's first answers: a short cache, one token; what counts is latency
        attention("attention bf16, 1 x 1000 keys", "bf16", B=1, Hq=32, Hkv=8, Nq=1, lo=1000, hi=1000, d=128, page=16),
        # an ordinary decode step of a busy server: many sequences of every length, grouped heads
        attention("attention bf16, 64 ragged", "bf16", B=64, Hq=32, Hkv=8, Nq=1, lo=100, hi=4000, d=128, page=16),
        # the repository's decode workload (16 heads, 8 rows, 65,536 keys) with its cache in pages
        attention("attention bf16, 64k keys", "bf16", B=1, Hq=16, Hkv=16, Nq=8, lo=65536, hi=65536, d=128, page=64),
        # a chunk of a long prompt against what the cache holds already
        attention("attention bf16, chunk of 512", "bf16", B=4, Hq=32, Hkv=8, Nq=512, lo=4097, hi=8100, d=128, page=64),
        # the busy server with its cache in 8 bits
        attention("attention e4m3, 64 ragged", "e4m3", B=64, Hq=32, Hkv=8, Nq=1, lo=100, hi=4000, d=128, page=32),
        # long contexts, wide groups
        attention("attention e4m3, 8 x 32k keys", "e4m3", B=8, Hq=64, Hkv=8, Nq=1, lo=32768, hi=32768, d=128, page=64),
        # five drafted tokens checked at once, small heads
        attention("attention e4m3, 5 drafted", "e4m3", B=16, Hq=16, Hkv=4, Nq=5, lo=1000, hi=9001, d=64, page=16),
        # the chunk of a long prompt, cache in 8 bits
        attention("attention e4m3, chunk of 256", "e4m3", B=3, Hq=32, Hkv=8, Nq=256, lo=3000, hi=8001, d=128, page=64),
        # one token of each of 64 sequences: latency
        append("append bf16, 64 x 1", "bf16", B=64, Hq=32, Hkv=8, Nq=1, lo=100, hi=4000, d=128, page=16),
        # prompts of up to 2048 tokens, padded to the longest
        append("append bf16, 8 x 2048", "bf16", B=8, Hq=32, Hkv=8, Nq=2048, lo=1500, hi=9000, d=128, page=64, short=500),
        append("append e4m3, 64 x 1", "e4m3", B=64, Hq=32, Hkv=8, Nq=1, lo=100, hi=4000, d=128, page=32),
        append("append e4m3, 8 x 2048", "e4m3", B=8, Hq=32, Hkv=8, Nq=2048, lo=1500, hi=9000, d=128, page=64, short=500),
    ]


def attention(name, cache, B, Hq, Hkv, Nq, lo, hi, d, page, short=0, causal=True):
    return {"name": name, "op": "attention", "cache": cache, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "lo": lo, "hi": hi, "d": d,
            "page": page, "short": short, "causal": causal}


def append(name, cache, B, Hq, Hkv, Nq, lo, hi, d, page, short=0, rot=0, interleaved=False):
    return {"name": name, "op": "append", "cache": cache, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "lo": lo, "hi": hi, "d": d,
            "page": page, "short": short, "rot": rot or d, "interleaved": interleaved}


def draw(rng):
    """One more case: sequences 1-128, heads in groups of 1-8, lengths 1-65,536, 1-512 (attention) or
    1-2048 (append) new tokens, pages of 16-128 tokens, both head sizes and both caches."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["attention", "append"])
        Hkv, g = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 6, 7, 8])
        B, Nq = spread(1, 128), rng.choice([1, 1, spread(2, 8), spread(9, 512 if op == "attention" else 2048)])
        hi = spread(max(Nq, 2), 65536)
        lo = max(Nq, spread(1, hi))
        c = {"cache": rng.choice(["bf16", "e4m3"]), "B": B, "Hq": Hkv * g, "Hkv": Hkv, "Nq": Nq, "lo": lo, "hi": max(lo, hi),
             "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128])}
        if op == "attention":
            c = attention("", short=rng.choice([0, Nq - 1]), causal=rng.choice([True, True, False]), **c)
        else:
            c = append("", short=rng.choice([0, Nq]), rot=rng.choice([c["d"], c["d"] // 2]), interleaved=rng.choice([False, True]), **c)
        del c["name"]
        w, held = work(c), sum(-(-n // c["page"]) for n in lengths(c)[0]) * c["page"] * Hkv * c["d"]
        if w["bytes"] <= 5.5e8 and w["flops"] <= 2.0e11 and held <= 2.7e8 and Hkv * g <= 64:
            return c


# ----------------------------------------------------------------------------- a case's lengths
def lengths(c):
    """(key_lens, new_lens): spread over lo..hi and over Nq - short..Nq, the same for every seed."""
    B, turn = c["B"], 0.6180339887498949
    kl = [c["lo"] + int((c["hi"] - c["lo"]) * math.fmod(0.5 + turn * b, 1.0)) for b in range(B)]
    nl = [c["Nq"] - int(round(c["short"] * math.fmod(turn * b, 1.0))) for b in range(B)]
    return kl, nl


def work(c):
    kl, nl = lengths(c)
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    e = 2 if c["cache"] == "bf16" else 1
    pages = [-(-n // c["page"]) for n in kl]
    scales = 0 if e == 2 else 2 * 4 * Hkv
    if c["op"] == "attention":
        rows = c["B"] * Hq * c["Nq"]
        used = [p if n else 0 for p, n in zip(pages, nl)]
        keys = [k if n else 0 for k, n in zip(kl, nl)]
        pairs = sum(n * k - (n * (n - 1) // 2 if c["causal"] else 0) for n, k in zip(nl, kl))
        return {"bytes": 2 * e * Hkv * d * sum(keys) + scales * sum(used) + 4 * sum(used) + 8 * c["B"] + rows * (4 * d + 4),
                "flops": 4 * d * Hq * pairs}
    new = sum(nl)
    touched = sum((k - 1) // c["page"] - (k - n) // c["page"] + 1 for k, n in zip(kl, nl) if n)
    # each new key and value read and written, each query read and written; one row of the tables per token
    return {"bytes": new * (Hkv * d * (2 * 2 + 2 * e) + Hq * d * 4 + 4 * c["rot"]) + 2 * scales * touched + 4 * touched + 8 * c["B"],
            "flops": new * (Hq + Hkv) * c["rot"] * 3}


# ----------------------------------------------------------------------------- inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kl, nl = lengths(c)
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    n = [-(-x // page) for x in kl]
    width, n_pages = max(n) + 1, sum(n) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda")[: sum(n)].to(torch.int32)
    first = torch.tensor(n, device="cuda").cumsum(0) - torch.tensor(n, device="cuda")
    at = torch.arange(width, device="cuda")
    used = at < torch.tensor(n, device="cuda")[:, None]
    table = torch.where(used, order[(first[:, None] + at).clamp(max=sum(n) - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    s = {"case": c, "page_table": table.contiguous(), "key_lens": torch.tensor(kl, dtype=torch.int32, device="cuda"),
         "new_lens": torch.tensor(nl, dtype=torch.int32, device="cuda") if c["short"] else None, "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        # activations of uneven size: every page and head has an amplitude of its own
        x = torch.randn((n_pages, Hkv, page, d), generator=g, device="cuda")
        if c["cache"] == "e4m3":
            x *= torch.exp(0.5 * torch.randn((n_pages, Hkv, 1, 1), generator=g, device="cuda"))
            scale = power_of_two(x.abs().amax((2, 3)))
            s[name + "_cache"] = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn)
            s[name + "_scale"] = scale
        else:
            s[name + "_cache"] = x.to(torch.bfloat16)
        del x
    if c["op"] == "attention":
        s["q"] = (1.5 * torch.randn((B, c["Hq"], c["Nq"], d), generator=g, device="cuda")).to(torch.bfloat16)
    else:
        # q, k and v as a projection leaves them: [B, Nq, (Hq + 2 Hkv) d], seen as heads
        x = torch.randn((B, c["Nq"], c["Hq"] + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
        s["q"], s["k"], s["v"] = x[:, : c["Hq"]], x[:, c["Hq"]: c["Hq"] + Hkv], x[:, c["Hq"] + Hkv:]
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        angle = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * freq
        s["rope"] = (angle.cos().float().contiguous(), angle.sin().float().contiguous())
    return s


def power_of_two(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-117."""
    m, e = torch.frexp(amax)   # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-117))


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import exact_io_aware_68_b200 as fa
        if c["op"] == "attention":
            return fa.attention_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["key_lens"], causal=c["causal"],
                                      new_lens=s["new_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        q = fa.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["key_lens"], new_lens=s["new_lens"],
                         rope=s["rope"], interleaved=c["interleaved"], q=s["q"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return pools(s, q)
    return plain_attention(s) if c["op"] == "attention" else plain_append(s)


def pools(s, q):
    new = {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return new if s["k_scale"] is None else {**new, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def new_of(s):
    """The number of new tokens of each sequence."""
    return torch.full_like(s["key_lens"], s["case"]["Nq"]) if s["new_lens"] is None else s["new_lens"]


def gathered(s, name):
    """A pool's pages in each sequence's order, fp32 [B, Hkv, keys, d]."""
    x = s[name + "_cache"][s["page_table"].long()] if s[name + "_scale"] is None else \
        s[name + "_cache"].view(torch.uint8)[s["page_table"].long()].view(torch.float8_e4m3fn)
    x = x.float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][s["page_table"].long()][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def plain_attention(s):
    c = s["case"]
    B, Hkv, Nq, d = c["B"], c["Hkv"], c["Nq"], c["d"]
    k, v = gathered(s, "k"), gathered(s, "v")
    i, j = torch.arange(Nq, device="cuda")[:, None], torch.arange(k.shape[2], device="cuda")
    L, n = s["key_lens"][:, None, None], new_of(s)[:, None, None]
    seen = (j < L) & (i < n)
    if c["causal"]:
        seen = seen & (j <= L - n + i)
    seen = seen[:, None, None]                                   # [B, 1, 1, Nq, keys]
    x = s["q"].float().view(B, Hkv, -1, d) @ k.transpose(2, 3) * (1 / math.sqrt(d))
    x = x.view(B, Hkv, -1, Nq, k.shape[2]).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = torch.where((j < L[:, 0])[:, None, :, None], v, 0.0)
    o = (p.view(B, Hkv, -1, p.shape[-1]) @ v).view(B, Hkv, -1, Nq, d) / torch.where(total > 0, total, 1.0)
    return o.view(B, -1, Nq, d).to(torch.bfloat16), (m + torch.log(total)).view(B, -1, Nq)


def rotated(s, x, position):
    """x [B, H, T, d] fp32 with its first rot features turned by the angles of position [B, T]."""
    c = s["case"]
    r = c["rot"]
    cos, sin = (t[position][:, None] for t in s["rope"])         # [B, 1, T, rot / 2]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., r:]), -1)


def plain_append(s):
    c = s["case"]
    Nq, page = c["Nq"], c["page"]
    L, n = s["key_lens"].long()[:, None], new_of(s).long()[:, None]
    i = torch.arange(Nq, device="cuda")
    # rotated queries; rows that hold no token are zero
    position = (L - n + i).clamp(0, MAX_POS - 1)
    q = torch.where((i < n)[:, None, :, None], rotated(s, s["q"].float(), position), 0.0).to(torch.bfloat16)
    new = {"k": rotated(s, s["k"].float(), position), "v": s["v"].float()}
    if s["k_scale"] is None:
        # rows without a token repeat the last token's write; a sequence without any rewrites what position 0 holds
        last = i.minimum((n - 1).clamp(min=0))
        at = (L - n + last) * (n > 0)
        to = torch.gather(s["page_table"].long(), 1, at // page)
        for name, x in new.items():
            pool = s[name + "_cache"]
            x = torch.gather(x, 2, last[:, None, :, None].expand_as(x)).transpose(1, 2)     # [B, T, Hkv, d]
            pool[to, :, at % page] = torch.where((n > 0)[..., None, None], x.to(torch.bfloat16), pool[to, :, at % page])
        return pools(s, q)
    # e4m3: the pages that get new tokens, whole.  A page beyond the last such one repeats that one.
    start = L - n
    first, end = start // page, (L - 1).clamp(min=0) // page
    at = (first + torch.arange((Nq + page - 2) // page + 1, device="cuda")).minimum(end.maximum(first))
    at = at.clamp(max=s["page_table"].shape[1] - 1)
    to = torch.gather(s["page_table"].long(), 1, at)                                        # [B, P]
    slot = at[..., None] * page + torch.arange(page, device="cuda")                         # [B, P, page]: positions
    fresh = ((slot >= start[..., None]) & (slot < L[..., None]))[:, :, None, :, None]
    held = (slot < start[..., None])[:, :, None, :, None]
    row = (slot - start[..., None]).clamp(0, Nq - 1).flatten(1)
    for name, x in new.items():
        codes, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        x = torch.gather(x, 2, row[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3]))
        x = x.unflatten(2, slot.shape[1:]).transpose(1, 2)                                  # [B, P, Hkv, page, d]
        amax = torch.where(fresh & x.isfinite(), x.abs(), 0.0).amax((3, 4))
        before = torch.where(held.any(3)[..., 0], scale[to], 0.0)
        after = torch.where(fresh.any(3)[..., 0], power_of_two(amax).maximum(before), scale[to])
        old = codes[to]
        y = torch.where(fresh, x, old.view(torch.float8_e4m3fn).float() * before[..., None, None]) / after[..., None, None]
        y = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[to] = torch.where(fresh | (held & fresh.any(3, keepdim=True)), y, old)
        scale[to] = after
    return pools(s, q)


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    kl, nl = lengths(c)
    if c["op"] == "attention":
        return exact_attention(c, s, kl, nl)
    return exact_append(c, s, kl, nl)


def exact_attention(c, s, kl, nl):
    Hq, Hkv, Nq, d = c["Hq"], c["Hkv"], c["Nq"], c["d"]
    g = Hq // Hkv
    o = torch.zeros((c["B"], Hq, Nq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(kl, nl)):
        ids = s["page_table"][b, : -(-L // c["page"])].long()
        for h in range(Hkv):
            k, v = (s[x + "_cache"][:, h].view(torch.uint8)[ids].view(s[x + "_cache"].dtype).double() for x in ("k", "v"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][ids, h].double()[:, None, None], v * s["v_scale"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, d)[:L], v.reshape(-1, d)[:L]
            for r in range(g):
                x = torch.einsum("id,jd->ij", s["q"][b, h * g + r, :n].double(), k) / math.sqrt(d)
                if c["causal"] and n > 1:
                    x[:, L - n:] += torch.full((n, n), -math.inf, dtype=torch.float64, device="cuda").triu(1)
                lse[b, h * g + r, :n] = torch.logsumexp(x, 1)
                o[b, h * g + r, :n] = torch.softmax(x, 1) @ v
    return o, lse


def exact_append(c, s, kl, nl):
    page, r = c["page"], c["rot"]
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    out = {"q": q}
    for x in ("k", "v"):
        out[x + "_cache"] = s[x + "_cache"].double()
        if s["k_scale"] is not None:
            out[x + "_scale"] = s[x + "_scale"].double()
    cos, sin = (t.double() for t in s["rope"])

    def turned(x, at):
        z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else torch.complex(x[..., : r // 2], x[..., r // 2: r])
        z = z * torch.complex(cos[at], sin[at])
        x = x.clone()
        if c["interleaved"]:
            x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
        else:
            x[..., :r] = torch.cat((z.real, z.imag), -1)
        return x

    for b, (L, n) in enumerate(zip(kl, nl)):
        if n == 0:
            continue
        at = torch.arange(L - n, L, device="cuda")
        q[b, :, :n] = turned(s["q"][b, :, :n].double(), at)
        for name, x in (("k", turned(s["k"][b, :, :n].double(), at)), ("v", s["v"][b, :, :n].double())):
            cache = out[name + "_cache"]
            if s["k_scale"] is None:
                cache[s["page_table"][b, at // page].long(), :, at % page] = x.transpose(0, 1)
                continue
            scale = out[name + "_scale"]
            for p in range((L - n) // page, (L - 1) // page + 1):
                lo, hi = max(p * page, L - n), min((p + 1) * page, L)
                i = s["page_table"][b, p].long()
                y = x[:, lo - (L - n): hi - (L - n)]
                need = torch.ceil(torch.log2(y.abs().amax((1, 2)) / 448.0)).clamp(min=-117.0).exp2()
                old = lo - p * page
                after = torch.maximum(need, scale[i]) if old else need
                cache[i, :, :old] = e4m3(cache[i, :, :old] * (scale[i] / after)[:, None, None])
                cache[i, :, old: hi - p * page] = e4m3(y / after[:, None, None])
                scale[i] = after
    return out


def e4m3(x):
    """Each value (at most 448) at the nearest e4m3 number, ties to the even one."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step
