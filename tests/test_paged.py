"""The paged key/value cache: appending (``kv_append``) and attending (``attention_paged``) against the
fp64 oracle, their refusals, and both together as a serving loop uses them."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import exact_io_aware_68_b200 as fa
from exact_io_aware_68_b200 import _lib
from exact_io_aware_68_b200.build import build

NAN = float("nan")


# ----------------------------------------------------------------------------- a cache to test on
class Cache:
    """Pools whose every unused place is NaN (rows past a sequence's end, pages of nobody, their scales), page
    numbers in random order, and table entries past the end that point nowhere."""

    def __init__(self, B, Hkv, d, page, lens, fp8, seed, room=0, split_pool=False):
        self.g = torch.Generator().manual_seed(seed)
        self.fp8, self.page = fp8, page
        self.lens = list(lens)
        n = [-(-(x + room) // page) for x in lens]
        self.n_pages = sum(n) + 3
        order = torch.randperm(self.n_pages, generator=self.g).tolist()
        self.table = torch.full((B, max(max(n), 1) + 2), 1 << 30, dtype=torch.int32)
        for b in range(B):
            for i in range(n[b]):
                self.table[b, i] = order.pop()
        shape = (self.n_pages, Hkv, page, d)
        x = {c: torch.full(shape, NAN) for c in "kv"}
        for b in range(B):
            for i in range(-(-lens[b] // page)):
                rows = min(page, lens[b] - i * page)
                for c in "kv":
                    amp = torch.exp(0.7 * torch.randn((Hkv, 1, 1), generator=self.g)) if fp8 else 1.0
                    x[c][self.table[b, i], :, :rows] = amp * torch.randn((Hkv, rows, d), generator=self.g)
        self.scale = {}
        self.pool, self.val = {}, {}
        for c in "kv":
            if fp8:
                held = torch.where(x[c].isnan(), 0.0, x[c]).abs().amax((2, 3))
                s = torch.tensor([[oracle.e4m3_scale(float(a)) if a > 0 else NAN for a in row] for row in held])
                codes = oracle.e4m3_encode((x[c] / s[:, :, None, None]).double().numpy())
                self.pool[c] = torch.from_numpy(codes).view(torch.float8_e4m3fn)
                self.scale[c] = s
                self.val[c] = oracle.E4M3[codes] * s.double().numpy()[:, :, None, None]
            else:
                self.pool[c] = x[c].to(torch.bfloat16)
                self.val[c] = self.pool[c].double().numpy()
        self.dev = {}
        if split_pool:   # one allocation holds both pools, page by page
            both = torch.stack((self.pool["k"].view(torch.uint8), self.pool["v"].view(torch.uint8)), 1).cuda()
            both = both.view(self.pool["k"].dtype)
            self.dev = {"k": both[:, 0], "v": both[:, 1]}
        else:
            self.dev = {c: self.pool[c].cuda() for c in "kv"}
        self.sdev = {c: s.cuda() for c, s in self.scale.items()}
        self.table_dev = self.table.cuda()

    def args(self):
        return self.dev["k"], self.dev["v"], self.table_dev

    def scales(self):
        return {"k_scale": self.sdev["k"], "v_scale": self.sdev["v"]} if self.fp8 else {}


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def bf16(x):
    return x.to(torch.bfloat16)


# ----------------------------------------------------------------------------- attention
def attention_bounds(q, cache, lens, news, scale, causal, R):
    """Elementwise allowances for O and lse, from the arithmetic of the kernels:
    * a score is an fp32 sum of d exact products: off by at most (d + 4) 2^-24 sum |q k| scale (the sum, the
      scale of the page, of the query row and the softmax, each rounded once): e_s;
    * a probability is then off by e_s + 2^-21 (ex2.approx, its argument's rounding) relative, and enters the
      matrix product in 16 bits: by half a step of bf16, 2^-8 of it, for more than 8 rows per K/V head; in
      two bf16 parts, 2^-16, for up to 8 rows; in f16 times its page's scale, 2^-11 + 2^-23, with e4m3;
    * e4m3 with more than 16 rows: a query's elements below 2^-17 of its largest one are off by up to 2^-21 of
      that one, so a score is off by at most 2^-21 max |q| sum |k| scale more;
    * fp32 sums over L keys add at most L 2^-24; O is rounded to bf16: half a step, 2^-8 |O|.
    So |dO| <= 2^-8 |O| + (2 e_p + c + 2 L 2^-24) sum P |V|, |dlse| <= e_p + L 2^-24 + 2^-21 + |lse| 2^-22."""
    absq, kval, vval = np.abs(q), np.abs(cache.val["k"]), np.abs(cache.val["v"])
    c = 2.0 ** -11 + 2.0 ** -22 if cache.fp8 else 2.0 ** -8 if R > 8 else 2.0 ** -16
    O, lse = oracle.forward_paged(q, cache.val["k"], cache.val["v"], cache.table.numpy(), lens, news, scale, causal)
    PV, _ = oracle.forward_paged(q, cache.val["k"], vval, cache.table.numpy(), lens, news, scale, causal)
    d = q.shape[3]
    kmax = np.zeros(q.shape[:3])
    g = q.shape[1] // kval.shape[1]
    for b, L in enumerate(lens):
        if L:
            keys = np.repeat(oracle.paged.sequence_keys(kval, cache.table.numpy(), b, L), g, 0)
            kmax[b] = np.einsum("hid,hjd->hij", absq[b], keys).max(-1) * scale
            if cache.fp8 and R > 16:
                kmax[b] += 2.0 ** -21 * absq[b].max(-1) * keys.sum(-1).max(-1)[:, None] * scale / ((d + 4) * 2.0 ** -24)
    e_p = (d + 4) * 2.0 ** -24 * kmax + 2.0 ** -21
    L = np.array(lens).reshape(-1, 1, 1) * 2.0 ** -24
    finite = np.where(np.isfinite(lse), lse, 0.0)
    return O, lse, 2.0 ** -8 * np.abs(O) + (2 * e_p + c + 2 * L)[..., None] * PV, e_p + L + 2.0 ** -21 + np.abs(finite) * 2.0 ** -22


def check_attention(cache, q, lens, news, causal, o, lse, R):
    scale = 1 / math.sqrt(q.shape[3])
    O, L, to, tl = attention_bounds(q.double().numpy(), cache, lens, news, scale, causal, R)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(L))
    dead = np.isneginf(L)
    assert not o[dead].any()
    live = ~dead
    assert np.isfinite(o).all()
    excess = (np.abs(o - O) - to)[live]
    assert not live.any() or excess.max() <= 0, f"O over its allowance by {excess.max():.3e}"
    excess = (np.abs(lse[live] - L[live]) - tl[live])
    assert not live.any() or excess.max() <= 0, f"lse over its allowance by {excess.max():.3e}"


# (B, Hkv, group, Nq, d, page, lens, new_lens, causal)
ATTENTION = [
    (1, 1, 1, 1, 64, 16, [1], None, False),
    (1, 2, 1, 1, 128, 16, [17], None, True),
    (3, 2, 4, 1, 128, 16, [0, 5, 1000], None, True),
    (4, 1, 8, 1, 64, 32, [300, 31, 32, 33], None, False),
    (2, 3, 7, 1, 128, 64, [65, 2049], None, True),
    (2, 2, 3, 3, 64, 16, [40, 700], [3, 1], True),
    (2, 2, 16, 1, 128, 128, [129, 1500], None, True),
    (3, 2, 4, 5, 128, 32, [5, 600, 0], [5, 4, 0], True),
    (2, 1, 5, 13, 64, 256, [13, 777], None, True),
    (2, 1, 2, 70, 128, 16, [70, 513], [70, 33], True),
    (1, 1, 8, 16, 64, 64, [500], None, False),
    (33, 1, 2, 1, 128, 16, [16 * (i % 5) + i for i in range(33)], None, True),
    (700, 1, 1, 1, 64, 16, [(7 * i) % 40 for i in range(700)], None, True),
    (2, 2, 8, 4, 64, 32, [400, 35], [4, 2], True),
    (2, 1, 6, 4, 128, 16, [300, 4], None, True),
    (2, 1, 1, 2, 64, 16, [1, 3], [2, 2], True),     # a query before position 0 sees nothing
    (2, 1, 3, 300, 128, 64, [300, 1000], [300, 211], True),
    (1, 1, 8, 40, 64, 16, [5000], None, True),
    (5, 2, 4, 33, 128, 32, [33, 0, 128, 129, 700], [33, 0, 1, 33, 20], True),
    (2, 1, 1, 600, 64, 256, [600, 1025], None, False),
    (3, 1, 20, 9, 128, 128, [4, 200, 9], [9, 9, 2], True),
    (1, 1, 130, 1, 64, 16, [77], None, True),       # more heads in a group than a tile has rows
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}q{c[3]}d{c[4]}p{c[5]}c{int(c[8])}")
def test_attention_matches_oracle(case, fp8):
    B, Hkv, group, Nq, d, page, lens, news, causal = case
    cache = Cache(B, Hkv, d, page, lens, fp8, seed=B + 7 * Nq + d + page)
    q = bf16(1.5 * torch.randn((B, Hkv * group, Nq, d), generator=cache.g))
    o, lse = fa.attention_paged(q.cuda(), *cache.args(), i32(lens), causal=causal, new_lens=None if news is None else i32(news),
                                **cache.scales())
    fa.check()
    check_attention(cache, q, lens, news or [Nq] * B, causal, o, lse, group * Nq)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_attention_long_cache(fp8):
    """A long sequence beside short ones, so that many warps share one and others own several."""
    lens = [30000, 3, 200, 0, 1, 4096, 17, 17]
    cache = Cache(8, 2, 128, 64, lens, fp8, seed=5)
    q = bf16(2 * torch.randn((8, 8, 1, 128), generator=cache.g))
    o, lse = fa.attention_paged(q.cuda(), *cache.args(), i32(lens), causal=True, **cache.scales())
    fa.check()
    check_attention(cache, q, lens, [1] * 8, True, o, lse, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("group,Nq", [(1, 4), (4, 4), (2, 40)])
def test_values_that_are_not_finite_stay_behind_the_mask(fp8, group, Nq):
    """NaN (and, bf16, infinite) keys and values in the last new token reach the last query alone."""
    lens = [100, 64]
    cache = Cache(2, 1, 64, 16, lens, fp8, seed=9)
    q = bf16(torch.randn((2, group, Nq, 64), generator=cache.g))
    args = (q.cuda(), *cache.args(), i32(lens))
    kw = dict(causal=True, **cache.scales())
    clean, clean_lse = fa.attention_paged(*args, **kw)
    # what every query but the last of sequence 0 sees is as it was (cache.val stays so)
    O, L, to, tl = attention_bounds(q.double().numpy(), cache, lens, [Nq, Nq], 1 / 8, True, group * Nq)

    def others_right(o, lse):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, rows in ((0, slice(0, Nq - 1)), (1, slice(0, Nq))):
            assert (np.abs(o - O)[b, :, rows] <= to[b, :, rows]).all() and (np.abs(lse - L)[b, :, rows] <= tl[b, :, rows]).all()

    others_right(clean, clean_lse)
    for c in "kv":
        raw = cache.dev[c].view(torch.uint8 if fp8 else torch.bfloat16)
        at = (cache.table[0, 99 // 16], 0, 99 % 16)
        raw[at] = 0x7F if fp8 else NAN
        if not fp8 and c == "v":
            raw[at][3], raw[at][5] = math.inf, -math.inf
    o, lse = fa.attention_paged(*args, **kw)
    fa.check()
    others_right(o, lse)
    assert torch.equal(o[1], clean[1]) and torch.equal(lse[1], clean_lse[1])
    assert o[0, :, -1].isnan().all() and lse[0, :, -1].isnan().all()
    # finite keys again: only the values are not
    raw = cache.dev["k"].view(torch.uint8 if fp8 else torch.bfloat16)
    raw[cache.table[0, 99 // 16], 0, 99 % 16] = 0 if fp8 else 0.0
    o, lse = fa.attention_paged(*args, **kw)
    fa.check()
    assert lse.isfinite().all()
    others_right(o, lse)
    last = o[0, :, -1].float()
    if fp8:
        assert last.isnan().all()
    else:
        assert (last[:, 3] == math.inf).all() and (last[:, 5] == -math.inf).all()
        assert last[:, [i for i in range(64) if i not in (3, 5)]].isnan().all()


@pytest.mark.gpu
def test_attention_equals_contiguous_decode():
    """One query head per K/V head, bf16: the same function as attention_decode over the gathered cache."""
    B, H, Nq, d, L = 2, 4, 3, 128, 1024
    cache = Cache(B, H, d, 64, [L, L], False, seed=3)
    q = bf16(torch.randn((B, H, Nq, d), generator=cache.g)).cuda()
    k, v = (cache.dev[c][cache.table_dev[:, : L // 64].long()].transpose(1, 2).reshape(B, H, L, d).contiguous() for c in "kv")
    o, lse = fa.attention_paged(q, *cache.args(), i32([L, L]), causal=True)
    o2, lse2 = fa.attention_decode(q, k, v, causal=True)
    fa.check()
    assert (o.float() - o2.float()).abs().max() <= 1e-2
    assert (lse - lse2).abs().max() <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Nq", [1, 2, 4, 30])
def test_attention_repeats_bit_for_bit(Nq, fp8):
    """No atomics: the same inputs give the same bits, also out of a workspace full of NaN."""
    lens = [5000, 300, 77]
    cache = Cache(3, 2, 64, 16, lens, fp8, seed=11)
    q = bf16(torch.randn((3, 12, Nq, 64), generator=cache.g)).cuda()
    ws = fa.paged_workspace(3, 12, 2, Nq, 64, "cuda")
    got = []
    for fill in (0, 0xFF):
        ws.fill_(fill)
        got.append(fa.attention_paged(q, *cache.args(), i32(lens), causal=True, workspace=ws, **cache.scales()))
    fa.check()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_pools_in_one_allocation_and_shared_pages(fp8):
    """Strided pages (keys and values interleaved page by page), and two sequences with a common prefix."""
    lens = [100, 90]
    cache = Cache(2, 2, 64, 16, lens, fp8, seed=21, split_pool=True)
    cache.table[1, :3] = cache.table[0, :3]
    cache.table_dev = cache.table.cuda()
    q = bf16(torch.randn((2, 4, 1, 64), generator=cache.g))
    o, lse = fa.attention_paged(q.cuda(), *cache.args(), i32(lens), **cache.scales())
    fa.check()
    check_attention(cache, q, lens, [1, 1], False, o, lse, 2)


# ----------------------------------------------------------------------------- append
def check_append(cache, q, k, v, lens, news, rope, interleaved, out):
    """Pools, scales and rotated queries against the definition; every byte that got no token as it was."""
    B, Hkv, Nq, d = k.shape
    page = cache.page
    cos, sin = (t.numpy() for t in rope) if rope is not None else (np.ones((1 << 16, 0)), np.zeros((1 << 16, 0)))
    touched = {c: np.zeros(cache.pool[c].shape[:3], bool) for c in "kv"}
    scaled = np.zeros(cache.pool["k"].shape[:2], bool)
    want = {c: cache.val[c].copy() for c in "kv"}
    slack = {c: np.zeros(cache.pool[c].shape[:3]) for c in "kv"}
    scale = {c: s.double().numpy().copy() for c, s in cache.scale.items()}
    for b in range(B):
        L, n = lens[b], news[b]
        pos = np.arange(L - n, L)
        for h in range(Hkv):
            for c, x in (("k", k), ("v", v)):
                y = x[b, h, :n].double().numpy()
                if c == "k":
                    y = oracle.rotate(y, pos, cos, sin, interleaved)
                # a rotated element: two products and their sum, each rounded to fp32 (2^-24 of |x| + |y|, twice)
                off = 2.0 ** -22 * np.abs(y).max(1) if n and c == "k" and cos.shape[1] else np.zeros(n)
                for j in range(n):
                    at = cache.table[b, pos[j] // page], h, pos[j] % page
                    touched[c][at] = True
                    want[c][at] = y[j]
                    slack[c][at] = off[j]
                if cache.fp8:
                    for p in sorted(set(pos // page)):
                        mine = y[pos // page == p]
                        i = int(cache.table[b, p])
                        fresh = oracle.e4m3_scale(np.abs(mine[np.isfinite(mine)]).max(initial=0.0))
                        start = max(L - n - p * page, 0)
                        scaled[i, h] = True
                        after = max(fresh, scale[c][i, h]) if start else fresh
                        if start and after > scale[c][i, h]:
                            touched[c][i, h, :start] = True
                        scale[c][i, h] = after
    for c in "kv":
        got = cache.dev[c].cpu()
        raw, was = got.view(torch.uint8).numpy(), cache.pool[c].view(torch.uint8).numpy()
        per = raw.reshape(*cache.pool[c].shape[:3], -1), was.reshape(*cache.pool[c].shape[:3], -1)
        assert np.array_equal(per[0][~touched[c]], per[1][~touched[c]]), f"{c}: bytes that got no token changed"
        if not cache.fp8:
            x, w = got.double().numpy()[touched[c]], want[c][touched[c]]
            assert np.array_equal(np.isnan(x), np.isnan(w))
            ok = np.isfinite(w)
            # half a step of bf16, 2^-8 of the value
            assert (np.abs(x - w)[ok] <= (2.0 ** -8 * np.abs(w) + slack[c][touched[c]][:, None])[ok]).all()
            assert np.array_equal(x[~ok & ~np.isnan(w)], w[~ok & ~np.isnan(w)])
            continue
        s = cache.sdev[c].cpu().double().numpy()
        assert np.array_equal(s[scaled], scale[c][scaled]), f"{c}: scales"
        assert np.array_equal(s[~scaled], cache.scale[c].double().numpy()[~scaled], equal_nan=True)
        codes, full = raw.reshape(cache.pool[c].shape), np.broadcast_to(scale[c][:, :, None, None], want[c].shape)
        t = touched[c]
        with np.errstate(invalid="ignore"):
            exact = oracle.e4m3_encode(want[c][t] / full[t])
            near = [oracle.e4m3_encode((want[c][t] + z * slack[c][t][:, None]) / full[t]) for z in (-1, 1)]
        # NaN has two codes
        exact, *near = (np.where(y == 0xFF, 0x7F, y) for y in (exact, *near))
        codes = np.where(codes == 0xFF, 0x7F, codes)
        # the nearest code, or where the fp32 rotation stands within its rounding of a border, the one beyond it
        assert ((codes[t] == exact) | (codes[t] == near[0]) | (codes[t] == near[1])).all(), f"{c}: codes"
    if q is None:
        assert out is None
        return
    w = np.zeros(q.shape)
    for b in range(B):
        n = news[b]
        for h in range(q.shape[1]):
            w[b, h, :n] = oracle.rotate(q[b, h, :n].double().numpy(), np.arange(lens[b] - n, lens[b]), cos, sin, interleaved)
    x = out.double().cpu().numpy()
    assert (np.abs(x - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -22 * np.abs(w).max(-1, keepdims=True)).all()
    for b in range(B):
        assert not x[b, :, news[b]:].any()


# (B, Hq (0: no queries), Hkv, Nq, d, page, key_lens after, new_lens, rot, interleaved)
APPEND = [
    (1, 1, 1, 1, 64, 16, [1], None, 64, False),
    (3, 8, 2, 1, 128, 16, [17, 16, 400], None, 128, False),
    (2, 4, 4, 1, 64, 32, [33, 64], None, 32, True),
    (4, 6, 2, 5, 128, 16, [5, 18, 40, 7], [5, 3, 0, 1], 128, True),
    (2, 0, 3, 40, 64, 16, [40, 133], [40, 39], 64, False),
    (2, 7, 1, 130, 128, 64, [130, 391], [130, 77], 64, False),
    (1, 2, 2, 300, 128, 256, [555], None, 0, False),
    (2, 3, 1, 150, 64, 128, [150, 150], [150, 0], 48, True),
    (1, 5, 5, 33, 128, 32, [64], None, 16, False),
]


def make_append(case, fp8, strided, split_pool=False):
    B, Hq, Hkv, Nq, d, page, lens, news, rot, inter = case
    news = news or [Nq] * B
    cache = Cache(B, Hkv, d, page, [x - n for x, n in zip(lens, news)], fp8, seed=sum(lens) + d, room=Nq, split_pool=split_pool)
    x = bf16(1.3 * torch.randn((B, Nq, Hq + 2 * Hkv, d), generator=cache.g)).transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    if not strided:
        q, k, v = (t.contiguous() for t in (q, k, v))
    rope = fa.rope_tables(max(lens), rot, device="cpu") if rot else None
    return cache, (q if Hq else None), k, v, lens, news, rope, inter


def run_append(cache, q, k, v, lens, news, rope, inter):
    x = torch.cat([t for t in (q, k, v) if t is not None], 1)
    strided = not k.is_contiguous()
    dev = x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if strided else x.cuda()
    h = 0 if q is None else q.shape[1]
    qd, kd, vd = dev[:, :h], dev[:, h: h + k.shape[1]], dev[:, h + k.shape[1]:]
    if not strided:
        qd, kd, vd = (t.contiguous() for t in (qd, kd, vd))
    out = fa.kv_append(kd, vd, *cache.args(), i32(lens), new_lens=i32(news), rope=None if rope is None else tuple(t.cuda() for t in rope),
                       interleaved=inter, q=qd if q is not None else None, **cache.scales())
    fa.check()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("strided", [False, True], ids=["contiguous", "views"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}n{c[3]}d{c[4]}p{c[5]}r{c[8]}i{int(c[9])}")
def test_append_matches_definition(case, fp8, strided):
    a = make_append(case, fp8, strided, split_pool=strided)
    check_append(*a, run_append(*a))


@pytest.mark.gpu
def test_append_e4m3_scale_rises_and_stays():
    """A louder token raises its page's scale and moves the held codes; a quieter one leaves both alone."""
    cache = Cache(1, 1, 64, 16, [5], True, seed=2, room=16)
    for amp, n in ((0.01, 1), (30.0, 1), (1.0, 2)):
        a = (cache, None, *(bf16(amp * torch.randn((1, 1, n, 64), generator=cache.g)) for _ in "kv"))
        lens = [cache.lens[0] + n]
        before = {c: cache.dev[c].view(torch.uint8).cpu().clone() for c in "kv"}
        out = run_append(*a, lens, [n], None, False)
        check_append(*a, lens, [n], None, False, out)
        if amp < 1:
            for c in "kv":
                i = int(cache.table[0, 0])
                assert torch.equal(cache.dev[c].view(torch.uint8).cpu()[i, :, :5], before[c][i, :, :5])
        for c in "kv":   # what the next append finds
            cache.pool[c], cache.scale[c] = cache.dev[c].cpu().clone(), cache.sdev[c].cpu().clone()
            cache.val[c] = oracle.E4M3[cache.pool[c].view(torch.uint8).numpy()] * cache.scale[c].double().numpy()[:, :, None, None]
        cache.lens = lens


@pytest.mark.gpu
def test_append_e4m3_zero_and_not_finite():
    """A page of zeros gets the least scale; infinities saturate and NaN stays, neither moves the scale."""
    cache = Cache(2, 1, 64, 16, [0, 0], True, seed=4, room=16)
    k, v = torch.zeros((2, 1, 3, 64)), torch.zeros((2, 1, 3, 64))
    k[1, 0, 0, 0], k[1, 0, 1, 1], k[1, 0, 2, 2], v[1, 0, 0, 5] = math.inf, NAN, -3.0, -math.inf
    a = (cache, None, bf16(k), bf16(v))
    check_append(*a, [3, 3], [3, 3], None, False, run_append(*a, [3, 3], [3, 3], None, False))
    i = int(cache.table[1, 0])
    codes = cache.dev["k"].view(torch.uint8)[i, 0].cpu()
    assert codes[0, 0] == 0x7E and codes[1, 1] & 0x7F == 0x7F and cache.sdev["k"][i, 0] == oracle.e4m3_scale(3.0)
    assert cache.sdev["k"][cache.table[0, 0], 0] == 2.0 ** -117


# ----------------------------------------------------------------------------- together
@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_serving_loop_in_a_captured_graph(fp8):
    """Prompts appended, then five decode steps replayed from one graph on another stream: each step's
    attention against the oracle on what the pools hold at that step."""
    B, Hq, Hkv, d, page = 3, 6, 2, 64, 16
    lens = [20, 1, 47]
    cache = Cache(B, Hkv, d, page, [0] * B, fp8, seed=8, room=64)
    cos, sin = (t.cuda() for t in fa.rope_tables(128, d, device="cpu"))
    g = cache.g

    def heads(n):
        x = bf16(torch.randn((B, n, Hq + 2 * Hkv, d), generator=g)).cuda().transpose(1, 2)
        return x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]

    def step(q, k, v, kl, nl):
        qr = fa.kv_append(k, v, *cache.args(), kl, new_lens=nl, rope=(cos, sin), q=q, **cache.scales())
        return (qr, *fa.attention_paged(qr, *cache.args(), kl, causal=True, new_lens=nl, **cache.scales()))

    def check(q, lens, news, o, lse):
        for c in "kv":
            if fp8:
                cache.val[c] = oracle.E4M3[cache.dev[c].view(torch.uint8).cpu().numpy()] * cache.sdev[c].double().cpu().numpy()[:, :, None, None]
            else:
                cache.val[c] = cache.dev[c].double().cpu().numpy()
        check_attention(cache, q.cpu(), lens, news, True, o, lse, Hq // Hkv * q.shape[2])

    q, k, v = heads(47)
    qr, o, lse = step(q, k, v, i32(lens), i32(lens))
    fa.check()
    check(qr, lens, lens, o, lse)
    kl = i32(lens)
    qs, ks, vs = (t.clone() for t in heads(1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kl += 1
        qr, o, lse = step(qs, ks, vs, kl, None)
    for i in range(5):
        for t, x in zip((qs, ks, vs), heads(1)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        fa.check()
        assert kl.tolist() == [x + i + 1 for x in lens]
        check(qr, kl.tolist(), [1] * B, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Nq", [1, 40])
def test_two_streams_with_workspaces_of_their_own(Nq, fp8):
    lens = [3000, 50]
    cache = Cache(2, 2, 128, 32, lens, fp8, seed=13)
    q = bf16(torch.randn((2, 8, Nq, 128), generator=cache.g)).cuda()
    want = fa.attention_paged(q, *cache.args(), i32(lens), causal=True, **cache.scales())
    kl = i32(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams * 4:
        with torch.cuda.stream(s):
            got.append(fa.attention_paged(q, *cache.args(), kl, causal=True, **cache.scales()))
    torch.cuda.synchronize()
    fa.check()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_chunks_of_a_prompt_in_a_captured_graph(fp8):
    """A prompt appended and attended to in padded chunks by one replayed graph, against the whole at once."""
    B, Hq, Hkv, d, page, chunk, steps = 2, 8, 2, 128, 64, 48, 3
    total = [chunk * steps, 100]   # the second prompt ends within the last chunk
    g = torch.Generator().manual_seed(31)
    x = bf16(torch.randn((B, chunk * steps, Hq + 2 * Hkv, d), generator=g)).cuda()
    rope = tuple(t.cuda() for t in fa.rope_tables(chunk * steps, d, device="cpu"))

    def heads(y):
        y = y.transpose(1, 2)
        return y[:, :Hq], y[:, Hq: Hq + Hkv], y[:, Hq + Hkv:]

    whole, parts = (Cache(B, Hkv, d, page, [0, 0], fp8, seed=17, room=chunk * steps) for _ in range(2))
    q, k, v = heads(x)
    kl = i32(total)
    qr = fa.kv_append(k, v, *whole.args(), kl, new_lens=kl, rope=rope, q=q, **whole.scales())
    want, want_lse = fa.attention_paged(qr, *whole.args(), kl, causal=True, new_lens=kl, **whole.scales())
    kl, nl, y = i32([0, 0]), i32([0, 0]), torch.zeros_like(x[:, :chunk])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        q, k, v = heads(y)
        qr = fa.kv_append(k, v, *parts.args(), kl, new_lens=nl, rope=rope, q=q, **parts.scales())
        o, lse = fa.attention_paged(qr, *parts.args(), kl, causal=True, new_lens=nl, **parts.scales())
    for i in range(steps):
        n = [max(0, min(chunk, t - i * chunk)) for t in total]
        nl.copy_(i32(n))
        kl.add_(nl)
        y.copy_(x[:, i * chunk: (i + 1) * chunk])
        graph.replay()
        torch.cuda.synchronize()
        fa.check()
        for b in range(B):
            a, w = o[b, :, : n[b]].float(), want[b, :, i * chunk: i * chunk + n[b]].float()
            assert not o[b, :, n[b]:].any() and torch.isneginf(lse[b, :, n[b]:]).all()
            if n[b] == 0:
                continue
            # the same function of the same values; e4m3 pages that grew by chunks hold codes that were re-rounded
            # (half a step of 2^-4 of a value, twice), bf16 ones the very same keys: two roundings of O, P in bf16
            tol = 0.25 if fp8 else 2.0 ** -6
            assert (a - w).abs().max() <= tol * w.abs().max().clamp(min=1)
            assert (a - w).norm() <= (0.06 if fp8 else 2.0 ** -7) * w.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_pools_beyond_32_bit_offsets(fp8, Nq):
    """Pages that lie more than 2^32 bytes into their pool."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    B, Hkv, group, d, page, lens = 2, 8, 4, 128, 64, [150, 64]
    small = Cache(B, Hkv, d, page, lens, fp8, seed=41)
    per = Hkv * page * d * (1 if fp8 else 2)
    far = (1 << 32) // per + 5   # page numbers from here on
    n = far + small.n_pages
    pools, scales = {}, {}
    for c in "kv":
        pools[c] = torch.zeros((n, Hkv, page, d), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        pools[c][far:] = small.dev[c].view(pools[c].dtype)
        pools[c] = pools[c].view(small.pool[c].dtype)
        if fp8:
            scales[c + "_scale"] = torch.ones((n, Hkv), device="cuda")
            scales[c + "_scale"][far:] = small.sdev[c]
    table = (small.table_dev + far).clamp(max=1 << 30)
    q = bf16(torch.randn((B, Hkv * group, Nq, d), generator=small.g))
    o, lse = fa.attention_paged(q.cuda(), pools["k"], pools["v"], table, i32(lens), causal=True, **scales)
    fa.check()
    check_attention(small, q, lens, [Nq] * B, True, o, lse, group * Nq)
    # and an append: the last row of sequence 0 again
    x = bf16(torch.randn((B, Hkv, 1, d), generator=small.g)).cuda()
    fa.kv_append(x, x, pools["k"], pools["v"], table, i32(lens), new_lens=i32([1, 0]), **scales)
    fa.check()
    at = (int(table[0, 149 // page]), slice(None), 149 % page)
    for c in "kv":
        if fp8:
            got = pools[c].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scales[c + "_scale"][at[0]][:, None]
            assert ((got - x[0, :, 0].float()).abs() <= 2.0 ** -4 * x[0, :, 0].float().abs() + scales[c + "_scale"][at[0]][:, None] * 2.0 ** -10).all()
        else:
            assert torch.equal(pools[c][at], x[0, :, 0])


@pytest.mark.gpu
def test_append_keeps_a_callers_scale():
    """A scale that is no power of two stays while it suffices, and its codes with it."""
    cache = Cache(1, 2, 64, 16, [3], True, seed=51, room=8)
    i = int(cache.table[0, 0])
    for c in "kv":
        cache.scale[c][i] = cache.scale[c][i] * 2.75
        cache.sdev[c] = cache.scale[c].cuda()
        cache.val[c][i] = oracle.E4M3[cache.pool[c].view(torch.uint8).numpy()[i]] * cache.scale[c][i].double().numpy()[:, None, None]
    k, v = (bf16(0.5 * torch.randn((1, 2, 2, 64), generator=cache.g)) for _ in "kv")
    check_append(cache, None, k, v, [5], [2], None, False, run_append(cache, None, k, v, [5], [2], None, False))
    k, v = (bf16(100 * torch.randn((1, 2, 2, 64), generator=cache.g)) for _ in "kv")
    for c in "kv":
        cache.pool[c], cache.scale[c] = cache.dev[c].cpu().clone(), cache.sdev[c].cpu().clone()
        cache.val[c] = oracle.E4M3[cache.pool[c].view(torch.uint8).numpy()] * cache.scale[c].double().numpy()[:, :, None, None]
    out = run_append(cache, None, k, v, [7], [2], None, False)
    # codes * (s / s'): the product with a scale that is no power of two is rounded to fp32 before it is encoded
    for c in "kv":
        cache.val[c] = np.float64(np.float32(cache.val[c]))
    check_append(cache, None, k, v, [7], [2], None, False, out)


# ----------------------------------------------------------------------------- refusals
FAKE = 0x2000


def c_attention(lib, fp8=False, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, o=FAKE, lse=FAKE, kp=1 << 20, vp=1 << 20, table=FAKE, lens=FAKE, new=None, B=1, Hq=2,
             Hkv=1, Nq=1, d=64, n_pages=4, page=16, max_pages=4, scale=0.125, causal=1, ws=0x10000, wsb=1 << 40)
    a.update(over)
    f = lib.fa_fwd_paged_e4m3 if fp8 else lib.fa_fwd_paged
    s = (a["ks"], a["vs"]) if fp8 else ()
    return f(a["q"], a["k"], a["v"], *s, a["o"], a["lse"], a["kp"], a["vp"], a["table"], a["lens"], a["new"], a["B"], a["Hq"], a["Hkv"],
             a["Nq"], a["d"], a["n_pages"], a["page"], a["max_pages"], a["scale"], a["causal"], a["ws"], a["wsb"], None)


def c_append(lib, fp8=False, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, strides=[64] * 9, qo=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, kp=1 << 20, vp=1 << 20, table=FAKE,
             lens=FAKE, new=None, cos=FAKE, sin=FAKE, max_pos=8, rot=32, inter=0, B=1, Hq=2, Hkv=1, Nq=1, d=64, n_pages=4, page=16, max_pages=4)
    a.update(over)
    f = lib.fa_kv_append_e4m3 if fp8 else lib.fa_kv_append
    s = (a["ks"], a["vs"]) if fp8 else ()
    st = None if a["strides"] is None else (ctypes.c_int64 * 9)(*a["strides"])
    return f(a["q"], a["k"], a["v"], st, a["qo"], a["kc"], a["vc"], *s, a["kp"], a["vp"], a["table"], a["lens"], a["new"], a["cos"], a["sin"],
             a["max_pos"], a["rot"], a["inter"], a["B"], a["Hq"], a["Hkv"], a["Nq"], a["d"], a["n_pages"], a["page"], a["max_pages"], None)


INV, UNS = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED
SHARED = [(dict(B=0), INV), (dict(Nq=0), INV), (dict(Hkv=0), INV), (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(Hq=3, Hkv=2), INV),
          (dict(d=96), UNS), (dict(d=256), UNS), (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=512), UNS), (dict(B=5000), UNS),
          (dict(B=4096, Hq=32), UNS), (dict(B=64, max_pages=1 << 21), UNS), (dict(kp=1023), INV), (dict(vp=1025), INV), (dict(kp=1 << 31), UNS), (dict(table=0), INV),
          (dict(lens=0), INV)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(scale=0.0), INV), (dict(scale=math.inf), INV), (dict(q=0), INV), (dict(q=0x2008), INV), (dict(k=0), INV), (dict(o=0), INV),
    (dict(lse=0x2004), INV), (dict(ws=0), INV), (dict(ws=0x10010), INV), (dict(wsb=100), INV), (dict(Hq=16, Nq=1 << 20, B=128), UNS)])
def test_attention_refuses_on_the_host(over, status, fp8):
    build()
    lib = _lib.load()
    assert c_attention(lib, fp8, **over) == status and lib.fa_get_error()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("over,status", SHARED + [
    (dict(strides=None), INV), (dict(strides=[64] * 8 + [12]), INV), (dict(strides=[-64] + [64] * 8), INV), (dict(k=0), INV), (dict(v=0x2002), INV),
    (dict(qo=0), INV), (dict(kc=0), INV), (dict(sin=None), INV), (dict(rot=8), UNS), (dict(rot=24), UNS), (dict(rot=80), UNS),
    (dict(max_pos=0), INV)])
def test_append_refuses_on_the_host(over, status, fp8):
    build()
    lib = _lib.load()
    assert c_append(lib, fp8, **over) == status and lib.fa_get_error()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_attention_refuses_o_over_q(fp8):
    build()
    lib = _lib.load()
    n = 2 * 64 * 2   # bytes of q and of o
    for o in (FAKE, FAKE + n - 16, FAKE - n + 16):
        assert c_attention(lib, fp8, o=o) == INV and b"overlaps" in lib.fa_get_error()
    for o in (FAKE + n, FAKE - n):   # side by side: refused for the next reason only
        assert c_attention(lib, fp8, o=o, ws=0) == INV and b"workspace" in lib.fa_get_error()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotates_a_contiguous_q_in_place(fp8, interleaved):
    g = torch.Generator().manual_seed(11)
    B, Hq, Hkv, Nq, d = 3, 6, 2, 5, 128
    q = bf16(torch.randn((B, Hq, Nq, d), generator=g)).cuda()
    k, v = (bf16(torch.randn((B, Hkv, Nq, d), generator=g)).cuda() for _ in range(2))
    rope = fa.rope_tables(64, 96)
    outs = []
    for in_place in (False, True):
        c = Cache(B, Hkv, d, 16, [40, 5, 17], fp8, seed=3)
        x = q.clone()
        y = fa.kv_append(k, v, *c.args(), i32([40, 5, 17]), i32([5, 5, 2]), rope=rope, interleaved=interleaved, q=x, **c.scales(),
                         q_out=x if in_place else None)
        assert (y is x) == in_place
        outs.append((y, *(t.view(torch.uint8) for t in c.args()[:2])))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and not outs[1][0][2, :, 2:].any()


@pytest.mark.parametrize("missing", ["ks", "vs"])
def test_e4m3_needs_scales(missing):
    build()
    lib = _lib.load()
    assert c_attention(lib, True, **{missing: 0}) == INV and c_append(lib, True, **{missing: 0}) == INV


def test_workspace_size_knows_its_arguments():
    build()
    size = _lib.load().fa_fwd_paged_workspace_size
    assert size(1, 8, 2, 1, 128) > 0 and size(1, 8, 2, 1, 128) % 256 == 0
    for bad in ((0, 8, 2, 1, 128), (1, 8, 3, 1, 128), (1, 8, 2, 0, 128), (1, 0, 2, 1, 128), (5000, 8, 2, 1, 128), (1, 8, 2, 1, 0)):
        assert size(*bad) == 0


def host_call(**over):
    a = dict(q=torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16), k_cache=torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16),
             v_cache=torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16), page_table=torch.zeros((2, 2), dtype=torch.int32),
             key_lens=torch.ones(2, dtype=torch.int32))
    a.update(over)
    return fa.attention_paged(**a)


def test_python_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        host_call()
    with pytest.raises(ValueError, match="q has shape"):
        host_call(q=torch.zeros((4, 64), dtype=torch.bfloat16))


@pytest.mark.gpu
def test_python_refuses_what_does_not_fit():
    c = Cache(2, 2, 64, 16, [20, 5], False, seed=1)
    good = dict(q=torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda"), k_cache=c.dev["k"], v_cache=c.dev["v"],
                page_table=c.table_dev, key_lens=i32([20, 5]))
    f32 = torch.zeros((c.n_pages, 2), device="cuda")
    for over, word in [(dict(q=good["q"].float()), "q must"), (dict(q=good["q"].expand(2, 4, 3, 64)), "q must"), (dict(v_cache=c.dev["v"][1:]), "same"),
                       (dict(v_cache=c.dev["v"].transpose(2, 3)), "same|contiguous"), (dict(key_lens=i32([1, 2, 3])), "key_lens"),
                       (dict(key_lens=torch.ones(2, device="cuda")), "key_lens"), (dict(page_table=c.table_dev[:1]), "page_table"),
                       (dict(new_lens=torch.ones(2, dtype=torch.int32)), "new_lens"), (dict(k_scale=f32, v_scale=f32), "scale"),
                       (dict(k_cache=c.dev["k"].float(), v_cache=c.dev["v"].float()), "bfloat16 or"), (dict(o=good["q"].float()), "o must"),
                       (dict(workspace=torch.zeros(64, device="cuda")), "workspace")]:
        with pytest.raises(ValueError, match=word):
            fa.attention_paged(**{**good, **over})
    with pytest.raises(_lib.FAError, match="workspace"):
        fa.attention_paged(**good, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    x = torch.zeros((2, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    rest = (c.dev["k"], c.dev["v"], c.table_dev, i32([20, 5]))
    for kw, word in [(dict(k=x, v=x[:, :1]), "same"), (dict(k=x[:, :1], v=x[:, :1]), "heads"), (dict(k=x, v=x, q=x[:1]), "q has"),
                     (dict(k=x.float(), v=x.float()), "k must"), (dict(k=x, v=x, q_out=x), "q_out"), (dict(k=x, v=x, rope=(f32, f32[1:])), "rope")]:
        with pytest.raises(ValueError, match=word):
            fa.kv_append(kw.pop("k"), kw.pop("v"), *rest, **kw)
    with pytest.raises(_lib.FAError, match="strides"):
        y = torch.zeros((2, 2, 1, 66), dtype=torch.bfloat16, device="cuda")[..., :64]
        fa.kv_append(y, y, *rest)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_device_reports_what_is_out_of_range(fp8):
    """Page numbers, lengths and positions outside the cache: skipped by the kernels' own checks, reported
    by check(), the other sequences right, and the next call clean."""
    lens = [40, 30]
    cache = Cache(2, 1, 64, 16, lens, fp8, seed=6, room=8)
    q = bf16(torch.randn((2, 2, 1, 64), generator=cache.g))
    kv = bf16(torch.randn((2, 1, 1, 64), generator=cache.g)).cuda()
    good, table = i32(lens), cache.table_dev
    bad = table.clone()
    bad[0, 1], bad[0, 2] = -5, cache.n_pages
    rope = tuple(t.cuda() for t in fa.rope_tables(35, 64, device="cpu"))
    want = fa.attention_paged(q.cuda(), *cache.args(), good, **cache.scales())
    fa.check()
    pools = [cache.dev[c].view(torch.uint8).clone() for c in "kv"]
    for tab, kl, nl in ((bad, good, None), (table, i32([1 << 20, 30]), None), (table, i32([-1, 30]), None), (table, good, i32([2, 1]))):
        o, _ = fa.attention_paged(q.cuda(), cache.dev["k"], cache.dev["v"], tab, kl, new_lens=nl, **cache.scales())
        with pytest.raises(_lib.FAError) as e:
            fa.check()
        assert e.value.status == _lib.FA_ERR_RANGE
        assert torch.equal(o[1], want[0][1])
    none = i32([1, 0])   # sequence 0 alone appends, and what it asks for is refused
    for tab, kl, r in ((bad, i32([41, 30]), None), (table, i32([1 << 20, 30]), None), (table, i32([0, 30]), None), (table, i32([41, 30]), rope)):
        fa.kv_append(kv, kv, cache.dev["k"], cache.dev["v"], tab, kl, new_lens=none, rope=r, **cache.scales())
        with pytest.raises(_lib.FAError) as e:
            fa.check()
        assert e.value.status == _lib.FA_ERR_RANGE
    assert all(torch.equal(cache.dev[c].view(torch.uint8), p) for c, p in zip("kv", pools))
    again = fa.attention_paged(q.cuda(), *cache.args(), good, **cache.scales())
    fa.check()
    assert torch.equal(again[0], want[0])


# ----------------------------------------------------------------------------- the oracle's own pins
def test_e4m3_oracle_against_torch():
    """Values by code and nearest-even codes, against torch's own casts on the CPU."""
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.E4M3, vals, equal_nan=True)
    g = torch.Generator().manual_seed(0)
    x = torch.cat((torch.randn(20000, generator=g) * 100, torch.randn(20000, generator=g) * 2.0 ** -7, torch.tensor([0.0, -0.0, 448.0, -448.0])))
    mid = torch.tensor([(vals[i] + vals[i + 1]) / 2 for i in range(125)])   # every tie
    x = torch.cat((x.clamp(-448, 448), mid.float(), -mid.float()))
    assert np.array_equal(oracle.e4m3_encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert oracle.e4m3_encode([math.inf, -math.inf, 1e9]).tolist() == [0x7E, 0xFE, 0x7E]


def test_scale_oracle():
    assert oracle.e4m3_scale(448.0) == 1.0 and oracle.e4m3_scale(448.0001) == 2.0 and oracle.e4m3_scale(0.0) == 2.0 ** -117
    assert oracle.e4m3_scale(3.5) == 2.0 ** -7 and oracle.e4m3_scale(3.51) == 2.0 ** -6


def test_rotation_oracle():
    """Rotations by position p and p' keep the products of pairs that are p - p' apart; norms stay."""
    rng = np.random.default_rng(1)
    cos, sin = (t.numpy() for t in fa.rope_tables(64, 32, device="cpu"))
    x, y = rng.standard_normal((1, 48)), rng.standard_normal((1, 48))
    for inter in (False, True):
        def r(z, p):
            return oracle.rotate(z, np.array([p]), cos, sin, inter)
        assert abs((r(x, 9) * r(y, 4)).sum() - (r(x, 30) * r(y, 25)).sum()) < 1e-5
        assert np.array_equal(r(x, 7)[:, 32:], x[:, 32:])
        assert np.allclose(r(x, 0), x)
        assert abs(np.linalg.norm(r(x, 50)) - np.linalg.norm(x)) < 1e-6


def test_paged_oracle_against_contiguous():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 2, 32, 8)), rng.standard_normal((2, 2, 32, 8))
    table = np.array([[3, 0], [1, 2]])
    pool = [np.zeros((4, 2, 16, 8)) for _ in "kv"]
    for p, x in zip(pool, (k, v)):
        for b in range(2):
            for i in range(2):
                p[table[b, i]] = x[b, :, 16 * i: 16 * i + 16]
    q = rng.standard_normal((2, 4, 3, 8))
    O, lse = oracle.forward_paged(q, *pool, table, [32, 20], [3, 3], 0.3, True)
    for b, L in enumerate((32, 20)):
        for h in range(4):
            for i in range(3):
                s = np.array([q[b, h, i] @ k[b, h // 2, j] * 0.3 for j in range(L - 3 + i + 1)])
                w = np.exp(s - s.max())
                assert np.allclose(O[b, h, i], (w / w.sum()) @ v[b, h // 2, : len(s)])
                assert abs(lse[b, h, i] - (s.max() + math.log(w.sum()))) < 1e-12
