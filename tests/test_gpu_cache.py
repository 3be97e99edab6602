"""The cache operators on the GPU: append with rotation, and the attention of
one new token over pages, against their definitions in 64 bits.

Tolerances (u = 2^-8, half a bf16 step relative to the value):
  append  copies are equal; a rotated element is two fp32 products and a sum
          (three roundings of 2^-24 relative to |a c| + |b s|) rounded once:
          |err| <= u |y| + 2^-22 (|a| + |b|).
  O       P and O are rounded once: |err| <= 1.25 (u sum P |v| + u |O|); the
          rest (fp32 sums, ex2 of 2^-22) is far below u.
  lse     |err| <= 2e-5 max(1, |lse|).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def fv():
    from block_sparse_attention_aware_b200 import build, fvattn
    build.build()
    assert torch.cuda.is_available(), "the CUDA path needs a GPU"
    fvattn.load()
    return fvattn


@pytest.fixture(scope="module")
def ca(fv):
    from block_sparse_attention_aware_b200 import cache
    return cache


def pool(ca, lens, hkv, D, page, seed, spare=2, width=None):
    """A pool of random tokens with the sequences' pages in random places; unused table entries are junk."""
    gen = torch.Generator().manual_seed(seed)
    n = [-(-x // page) for x in lens]
    total = sum(n) + spare
    place = torch.randperm(total, generator=gen)
    table = torch.full((len(lens), width or max(1, max(n))), 1 << 30, dtype=I32)
    at = 0
    for b, m in enumerate(n):
        table[b, :m] = place[at: at + m].to(I32)
        at += m
    dev = torch.Generator(device="cuda").manual_seed(seed)
    kp, vp = (torch.randn((total, hkv, page, D), generator=dev, device="cuda").to(BF16) for _ in range(2))
    return ca.PagedCache(kp, vp), table.cuda(), torch.tensor(lens, dtype=I32).cuda()


def attend_definition(c, q, table, lens, scale):
    B, hq, D = q.shape
    group = hq // c.Hkv
    o = torch.zeros((B, hq, D), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(o)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens.tolist()):
        if not n:
            continue
        pages = table[b, : -(-n // c.page)].long()
        k = c.k_pages[pages].transpose(0, 1).reshape(c.Hkv, -1, D)[:, :n].double()
        v = c.v_pages[pages].transpose(0, 1).reshape(c.Hkv, -1, D)[:, :n].double()
        x = q[b].double().view(c.Hkv, group, D) @ k.transpose(1, 2) * scale
        p = torch.softmax(x, -1)
        lse[b] = torch.logsumexp(x, -1).view(hq)
        o[b] = (p @ v).view(hq, D)
        bound[b] = 1.25 * U * ((p @ v.abs()).view(hq, D) + o[b].abs())
    return o, lse, bound


def check_attend(got, want):
    o, lse = got
    wo, wl, bound = want
    assert ((o.double() - wo).abs() <= bound).all(), float(((o.double() - wo).abs() / bound.clamp(min=1e-30)).max())
    assert torch.equal(lse.isinf(), wl.isinf())
    fine = ~wl.isinf()
    assert ((lse.double() - wl).abs()[fine] <= 2e-5 * wl.abs()[fine].clamp(min=1)).all()


ATTEND = [
    # lens, Hq, Hkv, D, page
    ([1], 1, 1, 64, 16),
    ([0, 1, 2, 15, 16, 17], 2, 2, 128, 16),
    ([63, 64, 65, 0, 127, 128, 129], 3, 1, 64, 32),
    ([1000], 40, 40, 128, 128),
    ([5000, 3, 0, 777], 8, 1, 128, 64),
    ([2500, 1, 130], 18, 2, 64, 128),
    ([300, 700], 17, 1, 128, 16),
    ([300, 700], 40, 1, 64, 16),
    ([33000], 4, 2, 128, 128),
    ([0], 4, 4, 64, 16),
]


@pytest.mark.parametrize("lens,hq,hkv,D,page", ATTEND)
def test_attend_against_the_definition(fv, ca, lens, hq, hkv, D, page):
    c, table, ln = pool(ca, lens, hkv, D, page, 3)
    q = (2.0 * torch.randn((len(lens), hq, D), generator=torch.Generator(device="cuda").manual_seed(4),
                           device="cuda")).to(BF16)
    want = attend_definition(c, q, table, ln, 1 / math.sqrt(D))
    got = c.attend(q, table, ln)
    assert fv.get_status() == 0
    check_attend(got, want)
    # any bound on the lengths gives a split that is right
    for longest in (max(lens), max(lens) + 1000):
        check_attend(c.attend(q, table, ln, longest=longest), want)
    assert fv.get_status() == 0


def rotate(x, cos, sin, halves):
    """In 64 bits, and the bound above."""
    x = x.double()
    n = x.shape[-1] // 2
    cos, sin = cos.double()[:, None], sin.double()[:, None]
    a, b = (x[..., :n], x[..., n:]) if halves else (x[..., ::2], x[..., 1::2])
    u, w = a * cos - b * sin, a * sin + b * cos
    s = a.abs() + b.abs()
    pack = (lambda p, r: torch.cat([p, r], -1)) if halves else (lambda p, r: torch.stack([p, r], -1).flatten(-2))
    y = pack(u, w)
    return y, U * y.abs() + 2.0 ** -22 * pack(s, s)


APPEND = [
    # new tokens, lengths with them, Hq, Hkv, D, page, axes, halves
    ([1], [1], 1, 1, 64, 16, (32,), False),
    ([1, 1, 1], [16, 17, 500], 5, 5, 128, 32, (64,), True),
    ([5, 1, 33, 16], [5, 128, 34, 700], 6, 2, 128, 16, (22, 21, 21), False),
    ([130, 7], [130, 135], 4, 4, 64, 128, (12, 10, 10), True),
    ([700], [1300], 40, 40, 128, 64, (30, 34), False),
    ([3, 0, 4], [3, 9, 8], 0, 3, 64, 16, None, False),
]


@pytest.mark.parametrize("new,lens,hq,hkv,D,page,axes,halves", APPEND)
def test_append_against_the_definition(fv, ca, new, lens, hq, hkv, D, page, axes, halves):
    c, table, ln = pool(ca, lens, hkv, D, page, 5)
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    gen = torch.Generator(device="cuda").manual_seed(6)
    spare = 4
    rows = sum(new) + spare
    qkv = torch.randn((rows, hq + 2 * hkv, D), generator=gen, device="cuda").to(BF16)
    q, k, v = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
    cu = torch.tensor([0] + new).cumsum(0).to(I32).cuda()
    kw = {}
    n_ax = len(axes) if axes else 0
    if axes:
        rot = ca.rotation_table(D, axes, 999)
        pos = torch.randint(0, 999, (rows, n_ax), generator=gen, device="cuda", dtype=I32)
        pos[sum(new):] = -5          # rows behind the last sequence: nothing of them is read
        kw = dict(rot=rot, pos=pos, axes=axes, halves=halves)
    if hq:
        kw.update(q=q, q_out=torch.full((rows, hq, D), 7.0, dtype=BF16, device="cuda"))
    got = c.append(k, v, table, ln, cu=cu, **kw)
    assert fv.get_status() == 0
    if axes:
        ax = torch.repeat_interleave(torch.arange(n_ax), torch.tensor(axes)).cuda()
        at = pos.clamp(min=0).long()[:, ax]
        i = torch.arange(D // 2, device="cuda")
        cos, sin = rot[at, i], rot[at, i + D // 2]
        kr, kb = rotate(k, cos, sin, halves)
    else:
        kr, kb = k.double(), torch.zeros_like(k).double()
    wk, wv, bk = k0.double(), v0.clone(), torch.zeros_like(k0).double()
    t = 0
    for b in range(len(new)):
        for n in range(lens[b] - new[b], lens[b]):
            pg = int(table[b, n // page])
            wk[pg, :, n % page], bk[pg, :, n % page], wv[pg, :, n % page] = kr[t], kb[t], v[t]
            t += 1
    assert torch.equal(c.v_pages, wv)
    assert ((c.k_pages.double() - wk).abs() <= bk).all()
    if hq:
        wq, bq = rotate(q, cos, sin, halves)
        used = sum(new)
        assert ((got[:used].double() - wq[:used]).abs() <= bq[:used]).all()
        assert (got[used:] == 7.0).all()
