"""The training operators on the GPU: the forward with its log-sum-exp and the
backward pass, against the definition in 64 bits.

Tolerances.  u = 2^-8 is bf16's unit roundoff (half a step relative to the
value), and a value v has an error of at most u |v| when it is rounded.
  lse: fp32 sums of at most a few thousand ex2 results of 2 ulp each, and a
       maximum in log2 units: |err| <= 2e-5 max(1, |lse|).
  O:   P and O are rounded once: |err_tc| <= u sum_u P |v_uc| + u |O_tc|.
  dV:  P and dV are rounded once: |err| <= u sum_t P |dO| + u |dV|.
  dQ:  dS and dQ are rounded once, and dS carries delta's error, which comes
       from O rounded to bf16: |d delta_t| <= u sum_c |dO_tc| |O_tc|.  So
       |err| <= scale (u sum_u |dS| |k| + sum_u P |d delta| |k|) + u |dQ|;
       dK likewise over t with |q|.
The remaining errors are of fp32 sums and of ex2 (2^-22 relative each), far
below u: the bounds are taken 1.25 times.
"""
import math

import pytest
import torch

from block_sparse_attention_aware_b200 import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
SLACK = 1.25


@pytest.fixture(scope="module")
def fv():
    from block_sparse_attention_aware_b200 import build, fvattn
    build.build()
    assert torch.cuda.is_available(), "the CUDA path needs a GPU"
    fvattn.load()
    return fvattn


@pytest.fixture(scope="module")
def tr(fv):
    from block_sparse_attention_aware_b200 import train
    return train


def real_rows(g):
    """Which tiled rows of a head are tokens (raster tile order)."""
    r = torch.arange(g.Npad)
    blk, off = r // g.bs, r % g.bs
    f = blk // (g.nby * g.nbx) * g.tf + off // (g.th * g.tw)
    y = blk // g.nbx % g.nby * g.th + off // g.tw % g.th
    x = blk % g.nbx * g.tw + off % g.tw
    return ((f < g.F) & (y < g.Hs) & (x < g.Ws)).cuda()


def random_lists(g, density, seed, empty=()):
    """Lists with uneven counts, ascending, junk behind each list's end."""
    gen = torch.Generator().manual_seed(seed)
    idx = torch.randint(-7, 10 ** 6, (g.B, g.H, g.nb, g.nb), generator=gen, dtype=torch.int32)
    cnt = torch.zeros((g.B, g.H, g.nb), dtype=torch.int32)
    for b in range(g.B):
        for h in range(g.H):
            for i in range(g.nb):
                n = max(1, min(g.nb, round(density * g.nb * (0.5 + torch.rand(1, generator=gen).item()))))
                if (b * g.H + h + i) % 5 in empty:
                    n = 0
                cnt[b, h, i] = n
                idx[b, h, i, :n] = torch.randperm(g.nb, generator=gen)[:n].sort().values
    return idx.cuda(), cnt.cuda()


def tiles(g, seed, scales=(1.0, 1.0, 1.0, 1.0)):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    real = real_rows(g)[:, None]
    return [(torch.randn((g.B, g.H, g.Npad, g.D), generator=gen, device="cuda") * s * real).to(torch.bfloat16)
            for s in scales]


def definition(g, q, k, v, do, idx, cnt, scale):
    """O, lse, dQ, dK, dV in 64 bits, and the bounds above for each."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    keep = torch.zeros((g.B, g.H, g.nb, g.nb), dtype=torch.bool)
    ci, cc = idx.cpu(), cnt.cpu()
    for b in range(g.B):
        for h in range(g.H):
            for i in range(g.nb):
                keep[b, h, i, ci[b, h, i, : cc[b, h, i]].long()] = True
    sees = keep.cuda().repeat_interleave(g.bs, 2).repeat_interleave(g.bs, 3) & real_rows(g)
    x = (q @ k.transpose(-1, -2)) * scale
    lse = torch.logsumexp(x.masked_fill(~sees, -math.inf), -1)
    z = torch.where(lse.isinf(), torch.zeros_like(lse), lse)
    p = torch.where(sees, (x - z[..., None]).exp(), torch.zeros_like(x))
    o = p @ v
    delta = (do * o).sum(-1, keepdim=True)
    ds = p * (do @ v.transpose(-1, -2) - delta)
    t = lambda m: m.transpose(-1, -2)  # noqa: E731
    out = dict(o=o, lse=lse, dq=ds @ k * scale, dk=t(ds) @ q * scale, dv=t(p) @ do)
    dd = U * (do.abs() * o.abs()).sum(-1, keepdim=True)
    e = U * ds.abs() + p * dd
    err = dict(o=U * (p @ v.abs()), lse=None, dq=scale * (e @ k.abs()), dk=scale * (t(e) @ q.abs()),
               dv=U * (t(p) @ do.abs()))
    real = real_rows(g)[:, None]
    for n in ("dq", "dk", "dv"):
        out[n] = out[n] * real
    return out, {n: None if v is None else SLACK * (v + U * out[n].abs()) + 1e-30 for n, v in err.items()}


def check(got, want, bound, name):
    got = got.double()
    if bound is None:
        assert torch.equal(got.isinf(), want.isinf()), name
        fine = ~want.isinf()
        got, want = got[fine], want[fine]
        bound = 2e-5 * want.abs().clamp(min=1.0)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(((got - want).abs() / bound).nan_to_num(1e9).max()))


GEOMS = [
    # B, H, D, F, Hs, Ws, tf, th, tw, density, rows left empty
    ("one-block", (1, 1, 128, 1, 8, 8, 2, 8, 8), 1.0, ()),
    ("one-token", (1, 1, 64, 1, 1, 1, 2, 2, 4), 1.0, ()),
    ("bs128-d128-pad", (1, 2, 128, 5, 19, 21, 2, 8, 8), 0.6, ()),
    ("bs128-d128-empty", (2, 1, 128, 4, 16, 24, 2, 8, 8), 0.4, (1, 3)),
    ("bs128-d64", (2, 2, 64, 3, 20, 16, 2, 8, 8), 0.7, (2,)),
    ("bs64-d128-odd", (1, 2, 128, 3, 8, 24, 1, 8, 8), 0.5, (0,)),
    ("bs64-d64-pad", (2, 2, 64, 3, 13, 21, 1, 8, 8), 0.4, ()),
    ("bs32-d64", (1, 3, 64, 2, 12, 16, 2, 4, 4), 0.3, (4,)),
    ("bs32-d128-pad", (1, 2, 128, 3, 9, 11, 1, 4, 8), 0.8, ()),
    ("bs16-d64-pad", (2, 3, 64, 3, 5, 7, 2, 2, 4), 0.5, (1,)),
    ("bs16-d128", (1, 2, 128, 4, 9, 14, 1, 4, 4), 0.2, (0, 1, 2)),
    ("all-empty", (1, 1, 128, 2, 8, 16, 2, 8, 8), 0.5, (0, 1, 2, 3, 4)),
]


@pytest.mark.parametrize("name,geo,density,empty", GEOMS, ids=[x[0] for x in GEOMS])
def test_forward_and_backward_against_the_definition(fv, tr, name, geo, density, empty):
    g = fv.geom(*geo)
    idx, cnt = random_lists(g, density, 5, empty)
    q, k, v, do = tiles(g, 6, (1.5, 1.0, 1.0, 1.0))
    scale = 1.0 / math.sqrt(g.D)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    assert fv.get_status() == 0
    want, bound = definition(g, q, k, v, do, idx, cnt, scale)
    check(o, want["o"], bound["o"], "o")
    check(lse, want["lse"], None, "lse")
    outs = [torch.full_like(q, float("nan")) for _ in range(3)]
    dq, dk, dv = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt, dq=outs[0], dk=outs[1], dv=outs[2])
    assert fv.get_status() == 0
    check(dv, want["dv"], bound["dv"], "dv")
    check(dq, want["dq"], bound["dq"], "dq")
    check(dk, want["dk"], bound["dk"], "dk")
