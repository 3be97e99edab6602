"""Training through the layer, and the calls around the gradient operators that
a training program makes: streams, graphs, several calls at once, bad lists,
concentrated rows.  Bounds are those of test_gpu_train (u = 2^-8, half a bf16
step); what is compared with another run of the same kernels has to have the
same bits."""
import math

import pytest
import torch

from tests.test_gpu_train import SLACK, U, check, definition, fv, random_lists, tiles, tr  # noqa: F401

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
GEO = (1, 2, 128, 3, 19, 21, 2, 8, 8)
GEO64 = (2, 2, 64, 3, 13, 21, 1, 8, 8)


def raster(g, seed, n=4, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn((g.B, g.N, g.H, g.D), generator=gen, device="cuda") * (scale if i == 0 else 1.0)).to(BF16)
            for i in range(n)]


def bits(t):
    return t.view(torch.int16)


def dense(q, k, v, do, scale):
    """O and gradients of dense attention on raster tensors in 64 bits, and test_gpu_train's bounds."""
    q, k, v, do = (t.double().transpose(1, 2) for t in (q, k, v, do))
    t = lambda m: m.transpose(-1, -2)  # noqa: E731
    p = torch.softmax(q @ t(k) * scale, -1)
    o = p @ v
    ds = p * (do @ t(v) - (do * o).sum(-1, keepdim=True))
    out = dict(o=o, dq=ds @ k * scale, dk=t(ds) @ q * scale, dv=t(p) @ do)
    e = U * ds.abs() + p * U * (do.abs() * o.abs()).sum(-1, keepdim=True)
    err = dict(o=U * (p @ v.abs()), dq=scale * (e @ k.abs()), dk=scale * (t(e) @ q.abs()), dv=U * (t(p) @ do.abs()))
    return ({n: x.transpose(1, 2) for n, x in out.items()},
            {n: (SLACK * (x + U * out[n].abs()) + 1e-30).transpose(1, 2) for n, x in err.items()})


@pytest.mark.parametrize("order", ["raster", "hilbert"])
@pytest.mark.parametrize("geo", [GEO, GEO64], ids=["bs128", "bs64"])
def test_layer_that_keeps_every_block_is_dense_attention(fv, tr, geo, order):  # noqa: F811
    g = fv.geom(*geo)
    q, k, v, do = raster(g, 1, scale=1.5)
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    layer = tr.TrainLayer(g, 1.0, 1, order=order)
    o = layer(q, k, v)
    o.backward(do)
    assert fv.get_status() == 0
    want, bound = dense(q.detach(), k.detach(), v.detach(), do, 1 / math.sqrt(g.D))
    for name, got in (("o", o.detach()), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        check(got, want[name], bound[name], name)


def test_gradients_agree_with_differences(fv, tr):  # noqa: F811
    """The kernel's gradients along random directions against central differences of the loss sum(O * dO) in 64 bits
    on the same lists.  Bound: the elements' bounds weighted with |direction|; the differences' own error is
    h^2 / 6 of a third derivative, with h = 1e-4 below 1e-6 of the terms' sizes."""
    g = fv.geom(*GEO64)
    idx, cnt = random_lists(g, 0.5, 3, (1,))
    q, k, v, do = tiles(g, 4, (1.5, 1.0, 1.0, 1.0))
    scale = 1 / math.sqrt(g.D)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    grads = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    _, bound = definition(g, q, k, v, do, idx, cnt, scale)
    gen = torch.Generator(device="cuda").manual_seed(9)
    h = 1e-4
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q.double(), k.double(), v.double()]
        real = (x[i].abs().sum(-1, keepdim=True) > 0)
        d = torch.randn(q.shape, generator=gen, device="cuda", dtype=torch.float64) * real

        def loss(s):
            y = list(x)
            y[i] = y[i] + s * h * d
            return (definition(g, *y, do, idx, cnt, scale)[0]["o"] * do.double()).sum().item()

        diff = (loss(1) - loss(-1)) / (2 * h)
        got = (grads[i].double() * d).sum().item()
        tol = (bound[name] * d.abs()).sum().item()
        assert abs(got - diff) <= tol + 1e-5 * abs(diff), name


def test_attention_function_is_the_operators_between_reorders(fv, tr):  # noqa: F811
    g = fv.geom(*GEO)
    idx, cnt = random_lists(g, 0.5, 6)
    q, k, v, do = raster(g, 7)
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    o = tr.attention(g, q, k, v, idx, cnt)
    got = torch.autograd.grad(o, (q, k, v), do)
    qt, kt, vt, dot = (fv.reorder(g, t.detach()) for t in (q, k, v, do))
    ot, lse = tr.sparse_attn_lse(g, qt, kt, vt, idx, cnt)
    assert torch.equal(bits(fv.inverse_reorder(g, ot)), bits(o.detach()))
    for a, b in zip(got, tr.sparse_attn_bwd(g, qt, kt, vt, ot, dot, lse, idx, cnt)):
        assert torch.equal(bits(a), bits(fv.inverse_reorder(g, b)))
    # the forward's bits are those of the inference call
    assert torch.equal(bits(ot), bits(fv.sparse_attn(g, qt, kt, vt, idx, cnt)))
    # a gradient that is not contiguous, and one input that needs none
    o = tr.attention(g, q, k.detach(), v, idx, cnt)
    wide = torch.zeros((g.B, g.N, g.H, 2 * g.D), dtype=BF16, device="cuda")
    wide[..., ::2] = do
    dq, dv = torch.autograd.grad(o, (q, v), wide[..., ::2])
    assert torch.equal(bits(dq), bits(got[0])) and torch.equal(bits(dv), bits(got[2]))


def test_concentrated_rows_lose_no_precision(fv, tr):  # noqa: F811
    """Scores of standard deviation 4: a row's softmax sits on a few keys, where dO . O from the rounded O would add
    an error as large as the rounding of the result.  r0 is that rounding's relative 2-norm (of the 64-bit result
    rounded to bf16); dS, rounded before its product, adds as much, independently, and tiles that keep to the rounded
    O at most a quarter: sqrt(2 + 1/16) r0, with 5% for chance."""
    g = fv.geom(1, 2, 64, 4, 16, 24, 2, 8, 8)
    idx, cnt = random_lists(g, 0.8, 2)
    q, k, v, do = tiles(g, 3, (4.0, 1.0, 1.0, 1.0))
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    got = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    want, bound = definition(g, q, k, v, do, idx, cnt, 1 / math.sqrt(g.D))
    for x, name in zip(got, ("dq", "dk", "dv")):
        check(x, want[name], bound[name], name)
        far = lambda y: ((y.double() - want[name]).norm() / want[name].norm()).item()  # noqa: B023, E731
        assert far(x) <= 1.05 * math.sqrt(2 + 1 / 16) * far(want[name].to(BF16)), name


def test_very_negative_scores(fv, tr):  # noqa: F811
    """Every score of some rows near -300: exp2(-lse) of the padding keys, which are zeros, would overflow if it were
    not masked there."""
    g = fv.geom(*GEO)
    idx, cnt = random_lists(g, 1.0, 2)
    q, k, v, do = tiles(g, 3)
    real = (k.abs().sum(-1, keepdim=True) > 0)
    k = (torch.ones_like(k) * 2 + 0.1 * k.float()).to(BF16) * real
    q = torch.where(torch.arange(g.Npad, device="cuda")[:, None] % 3 == 0, -13.0 - 0.0 * q, 0.3 * q).to(BF16)
    q = q * (real if g.order is None else 1)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    got = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    assert fv.get_status() == 0
    want, bound = definition(g, q, k, v, do, idx, cnt, 1 / math.sqrt(g.D))
    assert want["lse"][~want["lse"].isinf()].min() < -250
    # lse rounded to fp32 is off by 2^-24 * 300, which P = exp(s - lse) takes as a relative error of 2e-5 (and the
    # products of that size add as much again): far below u, with 1% on the bounds
    for x, name in zip(got, ("dq", "dk", "dv")):
        check(x, want[name], 1.01 * bound[name], name)


def test_two_streams_at_once_and_another_stream(fv, tr):  # noqa: F811
    g = fv.geom(*GEO)
    sets = []
    for s in range(2):
        idx, cnt = random_lists(g, 0.6, 20 + s)
        q, k, v, do = tiles(g, 30 + s)
        o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
        sets.append((q, k, v, o, do, lse, idx, cnt))
    want = [tr.sparse_attn_bwd(g, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        got = [tr.sparse_attn_bwd(g, *s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    assert fv.get_status() == 0
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(bits(x), bits(y))


def test_captured_operators_replay_on_new_inputs(fv, tr):  # noqa: F811
    g = fv.geom(*GEO64)
    idx, cnt = random_lists(g, 0.5, 1)
    ins = tiles(g, 2)
    q, k, v, do = (t.clone() for t in ins)
    aw, bw = fv.attn_workspace(g), tr.bwd_workspace(g)
    outs = [torch.empty_like(q) for _ in range(3)]
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt, workspace=aw)
    tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt, dq=outs[0], dk=outs[1], dv=outs[2], workspace=bw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.sparse_attn_lse(g, q, k, v, idx, cnt, out=o, lse=lse, workspace=aw)
        tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt, dq=outs[0], dk=outs[1], dv=outs[2], workspace=bw)
    for seed in (5, 6):
        new = tiles(g, seed, (2.0, 1.0, 1.0, 1.0))
        nidx, ncnt = random_lists(g, 0.7, seed, (2,))
        for t, n in zip((q, k, v, do, idx, cnt), (*new, nidx, ncnt)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        wo, wl = tr.sparse_attn_lse(g, *new[:3], nidx, ncnt)
        want = tr.sparse_attn_bwd(g, *new[:3], wo, new[3], wl, nidx, ncnt)
        for a, b in zip(outs, want):
            assert torch.equal(bits(a), bits(b))
    assert fv.get_status() == 0


def test_captured_training_step(fv, tr):  # noqa: F811
    """A whole step, routing to gradients, captured: autograd.grad on leaves that no eager graph uses."""
    g = fv.geom(*GEO)
    layer = tr.TrainLayer(g, 0.9, 2)
    buf = [t for t in raster(g, 3)]
    leaves = [t.detach().requires_grad_() for t in buf[:3]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(layer(*leaves), leaves, buf[3])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = layer(*leaves)
        got = torch.autograd.grad(o, leaves, buf[3])
    new = raster(g, 8, scale=2.0)
    with torch.no_grad():
        for t, n in zip(leaves + [buf[3]], new):
            t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    fresh = [t.clone().requires_grad_() for t in new[:3]]
    wo = layer(*fresh)
    want = torch.autograd.grad(wo, fresh, new[3])
    assert torch.equal(bits(o.detach()), bits(wo.detach()))
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    assert fv.get_status() == 0


def test_several_forwards_before_their_backwards(fv, tr):  # noqa: F811
    g = fv.geom(*GEO64)
    layer = tr.TrainLayer(g, 0.8, 2)
    sets = [raster(g, s) for s in (1, 2)]
    single = []
    for q, k, v, do in sets:
        x = [t.clone().requires_grad_() for t in (q, k, v)]
        single.append(torch.autograd.grad(layer(*x), x, do))
    xs = [[t.clone().requires_grad_() for t in s[:3]] for s in sets]
    os_ = [layer(*x) for x in xs]
    for x, o, s, want in reversed(list(zip(xs, os_, sets, single))):
        for a, b in zip(torch.autograd.grad(o, x, s[3]), want):
            assert torch.equal(bits(a), bits(b))
    # the same tensor as q, k and v: its gradient is the sum of the three
    x = sets[0][0].clone().requires_grad_()
    do = sets[0][3]
    (gx,) = torch.autograd.grad(layer(x, x, x), x, do)
    parts = [sets[0][0].clone().requires_grad_() for _ in range(3)]
    gp = torch.autograd.grad(layer(*parts), parts, do)
    # autograd adds two bf16 sums, each rounded: 2 u of the terms' sizes
    total = sum(t.double() for t in gp)
    assert ((gx.double() - total).abs() <= 2 * U * sum(t.double().abs() for t in gp) + 1e-30).all()


@pytest.mark.parametrize("what", ["count", "index", "twice"])
def test_bad_lists_are_reported(fv, tr, what):  # noqa: F811
    """Status word set; the bad entry is clamped, skipped or taken once; rows of other lists keep their results."""
    g = fv.geom(*GEO64)
    idx, cnt = random_lists(g, 0.6, 4)
    q, k, v, do = tiles(g, 5)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    want = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    assert fv.get_status() == 0
    bad_i, bad_c = idx.clone(), cnt.clone()
    n = int(cnt[0, 0, 1])
    if what == "count":
        bad_c[0, 0, 1] = -3
    elif what == "index":
        bad_i[0, 0, 1, n - 1] = g.nb
    else:
        bad_c[0, 0, 1] = n + 1
        bad_i[0, 0, 1, n] = bad_i[0, 0, 1, 0]
    got = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, bad_i, bad_c)
    assert fv.get_status() == fv.ERR_BOUNDS
    for a, b in zip(got, want):
        assert torch.equal(bits(a[:, 1:]), bits(b[:, 1:]))       # the other heads
    if what == "twice":
        for a, b in zip(got, want):
            assert torch.equal(bits(a), bits(b))
    if what == "count":
        assert (got[0][0, 0, g.bs: 2 * g.bs] == 0).all()


def test_blocks_that_nobody_keeps_may_hold_anything(fv, tr):  # noqa: F811
    """NaN and infinities in K and V blocks outside every list (128-token blocks): nothing of them is read."""
    g = fv.geom(1, 1, 128, 2, 16, 32, 2, 8, 8)
    idx, cnt = random_lists(g, 1.0, 1)
    keep = [0, 2, 3, 5, 7]
    cnt.fill_(len(keep))
    idx[..., : len(keep)] = torch.tensor(keep, dtype=torch.int32, device="cuda")
    q, k, v, do = tiles(g, 2)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    want = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    for j, x in ((1, float("nan")), (4, float("inf")), (6, -float("inf"))):
        k[:, :, j * g.bs: (j + 1) * g.bs] = x
        v[:, :, j * g.bs: (j + 1) * g.bs] = x
    o2, lse2 = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    assert torch.equal(bits(o), bits(o2)) and torch.equal(lse, lse2)
    got = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    # dK and dV of the blocks that nobody keeps are zero before and after; dQ reads kept blocks only.  (The choice of
    # the tiles that sum delta again goes by the mean of |V|^2, which is not finite now: the two dQ agree within
    # their bounds, not in their bits.)
    clean = [torch.where(t.isfinite(), t, torch.zeros_like(t)) for t in (k, v)]
    _, bound = definition(g, q, clean[0], clean[1], do, idx, cnt, 1 / math.sqrt(g.D))
    for a, b, name in zip(got, want, ("dq", "dk", "dv")):
        check(a, b.double(), 2 * bound[name], name)


def test_refusals_on_the_gpu(fv, tr):  # noqa: F811
    g = fv.geom(*GEO)
    idx, cnt = random_lists(g, 0.5, 6)
    q, k, v, do = tiles(g, 7)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    ok = dict(qt=q, kt=k, vt=v, ot=o, dot=do, lse=lse, kv_idx=idx, kv_cnt=cnt)
    for name, bad in (("qt", q[:, :1]), ("kt", k.float()), ("vt", v.transpose(2, 3)), ("ot", None), ("dot", do.cpu()),
                      ("lse", lse.double()), ("kv_idx", idx.long()), ("kv_cnt", cnt[..., :-1])):
        with pytest.raises(ValueError, match=name):
            tr.sparse_attn_bwd(g, **{**ok, name: bad})
    with pytest.raises(ValueError, match="distinct"):
        tr.sparse_attn_bwd(g, **ok, dq=q)
    with pytest.raises(ValueError, match="workspace"):
        tr.sparse_attn_bwd(g, **ok, workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        tr.sparse_attn_lse(g, q, k, v, idx, cnt, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="scale"):
        tr.sparse_attn_lse(g, q, k, v, idx, cnt, scale=-1.0)
    with pytest.raises(ValueError, match="input"):
        tr.sparse_attn_lse(g, q, k, v, idx, cnt, out=v)
    with pytest.raises(ValueError, match="order"):
        tr.attention(fv.with_order(g, fv.block_order(g)), *(torch.zeros((g.B, g.N, g.H, g.D), dtype=BF16, device="cuda"),) * 3,
                     idx, cnt)
    assert fv.get_status() == 0


def test_both_ways_through_the_binding_agree(fv, tr):  # noqa: F811
    """Without a stream argument a call is checked and marshalled by the extension, with one by the Python code."""
    g = fv.geom(*GEO64)
    idx, cnt = random_lists(g, 0.6, 4)
    q, k, v, do = tiles(g, 5)
    here = torch.cuda.current_stream()
    for kw in (dict(), dict(scale=0.2)):
        a, b = tr.sparse_attn_lse(g, q, k, v, idx, cnt, **kw), tr.sparse_attn_lse(g, q, k, v, idx, cnt, stream=here, **kw)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])
        x = tr.sparse_attn_bwd(g, q, k, v, a[0], do, a[1], idx, cnt, **kw)
        y = tr.sparse_attn_bwd(g, q, k, v, a[0], do, a[1], idx, cnt, stream=here, **kw)
        for s, t in zip(x, y):
            assert torch.equal(bits(s), bits(t))
    out, lse = torch.empty_like(q), torch.empty_like(a[1])
    got = tr.sparse_attn_lse(g, q, k, v, idx, cnt, scale=0.2, out=out, lse=lse, workspace=fv.attn_workspace(g))
    assert got[0] is out and got[1] is lse and torch.equal(bits(out), bits(a[0]))
    assert fv.get_status() == 0


LONG = [
    # few tiles, long lists: B, H, D, F, Hs, Ws, tf, th, tw, density, rows left empty, scale of Q
    ("bs16-d64", (1, 1, 64, 4, 16, 52, 1, 4, 4), 0.6, (), 1.5),
    ("bs16-d64-sparse", (1, 1, 64, 4, 16, 52, 1, 4, 4), 0.04, (1, 2), 1.5),
    ("bs128-d128", (1, 1, 128, 4, 40, 38, 2, 8, 8), 0.8, (3,), 1.5),
    ("bs32-d128-pad", (1, 2, 128, 3, 13, 21, 1, 4, 8), 0.9, (), 5.0),
    ("bs64-d64-empty", (1, 1, 64, 3, 20, 41, 1, 8, 8), 0.5, (0, 2, 4), 5.0),
    ("bs128-d64-all-kept", (2, 1, 64, 5, 23, 17, 2, 8, 8), 2.0, (), 1.0),
    # more tiles than SMs: some CTAs take a second one
    ("left-bs16-d64", (1, 8, 64, 4, 16, 52, 1, 4, 4), 0.3, (1,), 1.5),
    ("left-bs16-d128-sparse", (1, 7, 128, 4, 16, 50, 1, 4, 4), 0.02, (2, 4), 5.0),
    ("left-bs128-d64", (2, 2, 64, 5, 24, 40, 2, 8, 8), 0.7, (3,), 4.0),
    ("left-bs64-d128-pad", (1, 5, 128, 5, 23, 33, 1, 8, 8), 0.9, (), 0.5),
]


@pytest.mark.parametrize("name,geo,density,empty,qscale", LONG, ids=[x[0] for x in LONG])
def test_long_lists_against_the_definition(fv, tr, name, geo, density, empty, qscale):  # noqa: F811
    """Lists of tens of chunks; a workspace full of NaN; the same bits twice."""
    g = fv.geom(*geo)
    idx, cnt = random_lists(g, density, 11, empty)
    q, k, v, do = tiles(g, 12, (qscale, 1.0, 1.0, 1.0))
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    want, bound = definition(g, q, k, v, do, idx, cnt, 1 / math.sqrt(g.D))
    outs = [torch.full_like(q, float("nan")) for _ in range(3)]
    ws = tr.bwd_workspace(g).fill_(255)            # NaN in whatever is read before it is written
    tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    assert fv.get_status() == 0
    for x, n in zip(outs, ("dq", "dk", "dv")):
        check(x, want[n], bound[n], n)
    again = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt, workspace=ws)
    for a, b in zip(outs, again):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("D,keep", [(64, 1), (128, 1), (128, 2)])
def test_many_tiles_with_lists_of_a_chunk_or_two(fv, tr, D, keep):  # noqa: F811
    """Several tiles an SM, each with a list of `keep` blocks: the issuing warps are items ahead of the arithmetic.
    The same bits in every run, and those of the definition's bounds."""
    g = fv.geom(3, 8, D, 4, 16, 32, 2, 8, 8)
    idx, cnt = random_lists(g, 1.0, 3)
    cnt.fill_(keep)
    cnt[:, ::3, 1::2] = 3 - keep
    q, k, v, do = tiles(g, 4, (0.3, 1.0, 1.0, 1.0))
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    want, bound = definition(g, q, k, v, do, idx, cnt, 1 / math.sqrt(g.D))
    first = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
    for x, n in zip(first, ("dq", "dk", "dv")):
        check(x, want[n], bound[n], n)
    for _ in range(200):
        for a, b in zip(first, tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)):
            assert torch.equal(bits(a), bits(b))
    assert fv.get_status() == 0


@pytest.mark.parametrize("geo", [(1, 2, 64, 2, 8, 8, 2, 2, 4), GEO64, GEO], ids=["bs16", "bs64", "bs128"])
def test_calls_without_a_sync_between_them(fv, tr, geo):  # noqa: F811
    """Forward and backward passes of two sets of inputs in turn, many in flight, with one workspace for each
    operator: a call reads its own lists, orders and statistics there, not those of the call before."""
    g = fv.geom(*geo)
    sets = []
    for s in range(2):
        idx, cnt = random_lists(g, 0.3 + 0.5 * s, 40 + s, (s,))
        sets.append((*tiles(g, 50 + s, (1.0 + 3 * s, 1.0, 1.0, 1.0)), idx, cnt))
    aw, bw = fv.attn_workspace(g), tr.bwd_workspace(g)

    def step(q, k, v, do, idx, cnt):
        o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt, workspace=aw)
        return (o, lse, *tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt, workspace=bw))

    want = []
    for s in sets:
        torch.cuda.synchronize()
        want.append(step(*s))
        torch.cuda.synchronize()
    got = [step(*sets[i % 2]) for i in range(60)]
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % 2]):
            assert torch.equal(a, b)
    assert fv.get_status() == 0


@pytest.mark.parametrize("geo", [(2, 8, 64, 4, 16, 52, 1, 4, 4), (2, 12, 128, 4, 16, 48, 2, 4, 4), (2, 8, 64, 4, 40, 48, 1, 8, 8)],
                         ids=["bs16", "bs32", "bs64"])
def test_nan_stays_in_its_head(fv, tr, geo):  # noqa: F811
    """NaN in Q, K and V of some heads, more tiles than SMs, the other heads' lists filling half a chunk of
    128 keys: what a CTA's buffers keep of those heads reaches no other head's results, in no bit."""
    g = fv.geom(*geo)
    tile = 128 // g.bs
    idx = torch.zeros((g.B, g.H, g.nb, g.nb), dtype=torch.int32)
    gen = torch.Generator().manual_seed(21)
    idx[..., 0] = (torch.arange(g.nb) // tile * 5 + torch.randint(0, tile // 2, (g.B, g.H, g.nb), generator=gen)) % g.nb
    cnt = torch.ones((g.B, g.H, g.nb), dtype=torch.int32)
    cnt[:, :3], idx[:, :3, :, :tile] = tile, torch.arange(tile, dtype=torch.int32)
    idx, cnt = idx.cuda(), cnt.cuda()
    q, k, v, do = tiles(g, 22)

    def run():
        o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
        inference = fv.sparse_attn(g, q, k, v, idx, cnt)
        raster_o = fv.sparse_attn_raster(g, q, k, v, idx, cnt)
        return (o, lse[..., None], inference, raster_o.transpose(1, 2), *tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt))

    want = run()
    for i in range(3):
        for t in (q, k, v)[i:]:
            t[:, i] = float("nan")
    for _ in range(3):
        for a, b in zip(run(), want):
            assert torch.equal(a[:, 3:], b[:, 3:])
    assert fv.get_status() == 0


def test_values_that_no_list_holds_change_no_bit(fv, tr):  # noqa: F811
    """Concentrated rows, and values 25 times as large, or keys and values that are NaN, in the blocks that no list
    holds: the same bits."""
    for geo in ((1, 2, 64, 4, 16, 24, 2, 8, 8), (1, 2, 64, 4, 16, 24, 1, 4, 4)):
        g = fv.geom(*geo)
        last = g.nb - 128 // g.bs                   # whole tiles of blocks
        idx, cnt = random_lists(g, 0.9, 2)
        cnt = cnt.clamp(max=last)
        idx[..., :last] = torch.arange(last, dtype=torch.int32, device="cuda")
        q, k, v, do = tiles(g, 3, (3.0, 1.0, 1.0, 1.0))
        o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
        want = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)
        for factor in (25.0, float("nan")):
            v[:, :, last * g.bs:] *= factor
            k[:, :, last * g.bs:] *= factor / 25
            for a, b in zip(tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt), want):
                assert torch.equal(bits(a), bits(b))
        assert fv.get_status() == 0


@pytest.mark.parametrize("large", ["none", "no list holds them", "hardly weighted"])
def test_concentrated_rows_beside_large_values(fv, tr, large):  # noqa: F811
    """Scores of standard deviation 3 and some values 25 or 100 times the others', in blocks that no list holds, or
    on four keys that are zero, which rows give next to no weight.  dQ's error a row, relative to the row: the
    result's rounding r0 (measured on the 64-bit result), and independently dS's, r0 sqrt(sum_u |dS_tu k_u|^2),
    with up to a ninth more of it (in squares) in rows that take delta from the rounded O.  So the rows' root mean
    square is at most r0 sqrt(1 + (1 + 1/9) c), c the mean of sum_u |dS_tu k_u|^2 / |dQ_t|^2; 5% for chance.  Rows
    with a probability above 0.9 are left out: there dP - delta cancels further than fp32 goes."""
    g = fv.geom(1, 2, 64, 4, 16, 24, 2, 8, 8)
    idx, cnt = random_lists(g, 1.0, 2)
    last = g.nb - 1
    cnt.fill_(last)
    idx[..., :last] = torch.arange(last, dtype=torch.int32, device="cuda")
    q, k, v, do = tiles(g, 3, (3.0, 1.0, 1.0, 1.0))
    if large == "no list holds them":
        v[:, :, last * g.bs:] *= 25
    elif large == "hardly weighted":
        v[:, :, 700:704] *= 100
        k[:, :, 700:704] = 0
    scale = 1 / math.sqrt(g.D)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    got = tr.sparse_attn_bwd(g, q, k, v, o, do, lse, idx, cnt)[0].double()
    n = last * g.bs
    q, k, v, do = q.double(), k[:, :, :n].double(), v[:, :, :n].double(), do.double()
    p = torch.softmax(q @ k.transpose(-1, -2) * scale, -1)
    dp = do @ v.transpose(-1, -2)
    ds = scale * p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = ds @ k
    rows = p.amax(-1) < 0.9
    assert rows.double().mean() > 0.9
    rms = lambda e: ((e.square().sum(-1) / dq.square().sum(-1))[rows].mean().sqrt()).item()  # noqa: E731
    c = ((ds.square() @ k.square().sum(-1, keepdim=True)).squeeze(-1) / dq.square().sum(-1))[rows].mean().item()
    assert rms(got - dq) <= 1.05 * math.sqrt(1 + (1 + 1 / 9) * c) * rms(dq.to(BF16).double() - dq)
    assert fv.get_status() == 0


@pytest.mark.parametrize("keep", [1, 3], ids=["one chunk", "three chunks"])
def test_nan_scores_are_not_taken_for_an_empty_row(fv, tr, keep):  # noqa: F811
    """A row whose query holds a NaN, and rows that keep a block of keys with one: O and lse are NaN as the formula's
    are (O = 0 and lse = -inf are for rows that keep nothing); the other rows have the bits that they have without."""
    g = fv.geom(1, 1, 128, 2, 16, 64, 2, 8, 8)
    idx, cnt = random_lists(g, 1.0, 1)
    cnt.fill_(keep)
    cnt[0, 0, 5] = 0
    for i in range(g.nb):
        idx[0, 0, i, :keep] = torch.arange(keep, dtype=torch.int32) + (1 if i < 8 else 10)
    q, k, v, _ = tiles(g, 2)
    o, lse = tr.sparse_attn_lse(g, q, k, v, idx, cnt)
    rows = torch.arange(g.Npad, device="cuda")
    bad = (rows == 3) | ((rows >= 130) & (rows < 258)) | (rows == 5 * g.bs)
    q[0, 0, bad, 7] = float("nan")
    k[0, 0, 10 * g.bs + 9, 0] = float("nan")       # the blocks 8 .. keep it
    nan = ((bad & (rows // g.bs < 8)) | (rows >= 8 * g.bs)) & (rows // g.bs != 5)
    for got, l in ((tr.sparse_attn_lse(g, q, k, v, idx, cnt)), (fv.sparse_attn(g, q, k, v, idx, cnt.clamp(min=1)), None)):
        got, want = got[0, 0], o[0, 0]
        assert got[nan].isnan().all()
        fine = ~nan & (rows // g.bs != 5)
        assert torch.equal(bits(got[fine]), bits(want[fine]))
        if l is not None:
            assert l[0, 0, nan].isnan().all() and torch.equal(l[0, 0, ~nan], lse[0, 0, ~nan])
            assert (got[rows // g.bs == 5] == 0).all()
    assert fv.get_status() == 0


def test_a_gradient_that_starts_between_16_byte_boundaries(fv, tr):  # noqa: F811
    """Autograd hands over views: the gradient of a concatenation's part starts wherever that part does."""
    g = fv.geom(*GEO64)
    idx, cnt = random_lists(g, 0.5, 6)
    q, k, v, do = raster(g, 7)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    want = torch.autograd.grad(tr.attention(g, *leaves, idx, cnt), leaves, do)
    o = tr.attention(g, *leaves, idx, cnt)
    joined = torch.cat([torch.zeros(3, dtype=BF16, device="cuda"), o.flatten()])
    got = torch.autograd.grad(joined, leaves, torch.cat([torch.zeros(3, dtype=BF16, device="cuda"), do.flatten()]))
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    assert fv.get_status() == 0


def test_attention_takes_its_own_geometrys_order_only(fv, tr):  # noqa: F811
    g = fv.geom(*GEO)
    idx, cnt = random_lists(g, 0.5, 6)
    q, k, v, _ = raster(g, 7)
    mine, other = fv.block_order(g), fv.block_order(g)
    ordered = fv.with_order(g, mine)
    assert torch.equal(bits(tr.attention(ordered, q, k, v, idx, cnt, order=mine)), bits(tr.attention(
        fv.with_order(g, other), q, k, v, idx, cnt, order=other)))
    for geo, table in ((ordered, other), (ordered, None)):
        with pytest.raises(ValueError, match="order"):
            tr.attention(geo, q, k, v, idx, cnt, order=table)


def test_a_layers_block_order_is_on_its_tensors_device(fv, tr):  # noqa: F811
    """A table elsewhere would be read through an address that this GPU does not have: refused before any launch."""
    g = fv.geom(*GEO)
    q, k, v, _ = raster(g, 7)
    layer = tr.TrainLayer(g, 0.9, 2, order="hilbert")
    layer(q, k, v)
    layer.order_table = layer.order_table.cpu()
    with pytest.raises(ValueError, match="order"):
        layer(q, k, v)
    assert fv.get_status() == 0
