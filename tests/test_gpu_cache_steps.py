"""The cache operators as a generating program runs them: append and attend
step by step, captured, on other streams, with shared pages, bad tables and
long pools.  Bounds are those of test_gpu_cache."""
import math

import pytest
import torch

from tests.test_gpu_cache import BF16, I32, U, attend_definition, ca, check_attend, fv, pool, rotate  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16)


def normal(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * scale).to(BF16)


@pytest.mark.parametrize("hq,hkv,D,page,axes,halves", [(6, 2, 64, 16, (32,), True), (4, 4, 128, 64, (22, 21, 21), False)])
def test_generation(fv, ca, hq, hkv, D, page, axes, halves):  # noqa: F811
    """A first part of each sequence appended at once, then token after token; at every step the attention is that of
    the whole history, whose keys were rotated by their positions when they came."""
    B, first, steps = 3, [5, page * 2, 1], page + 3
    most = max(first) + steps
    width = -(-most // page)
    c = ca.PagedCache(*(torch.full((B * width, hkv, page, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2)))
    order = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).to(I32).view(B, width)
    table = torch.full((B, width), -1, dtype=I32, device="cuda")       # pages are handed out as they are needed
    rot = ca.rotation_table(D, axes, 512)
    n_ax = len(axes)
    ax = torch.repeat_interleave(torch.arange(n_ax), torch.tensor(axes)).cuda()
    col = torch.arange(D // 2, device="cuda")
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    lens = [0] * B
    for step in range(steps):
        new = first if step == 0 else [1] * B
        rows = sum(new)
        qkv = normal((rows, hq + 2 * hkv, D), 100 + step)
        q, k, v = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
        pos = torch.randint(0, 512, (rows, n_ax), generator=torch.Generator().manual_seed(step), dtype=I32).cuda()
        lens = [a + b for a, b in zip(lens, new)]
        for b in range(B):
            for p in range(-(-lens[b] // page)):
                table[b, p] = order[b, p]
        ln = torch.tensor(lens, dtype=I32, device="cuda")
        cu = torch.tensor([0] + new).cumsum(0).to(I32).cuda() if step == 0 else None
        qr = c.append(k, v, table, ln, cu=cu, q=q, pos=pos, rot=rot, axes=axes, halves=halves)
        at = pos.long()[:, ax]
        cos, sin = rot[at, col], rot[at, col + D // 2]
        kr, kb = rotate(k, cos, sin, halves)
        wq, qb = rotate(q, cos, sin, halves)
        assert ((qr.double() - wq).abs() <= qb).all()
        t, last = 0, []
        for b in range(B):
            for _ in range(new[b]):
                ks[b].append(kr[t].to(BF16))
                vs[b].append(v[t])
                t += 1
            last.append(t - 1)
        qn = qr[last].contiguous()
        o, lse = c.attend(qn, table, ln, longest=most)
        want = attend_definition(c, qn, table, ln, 1 / math.sqrt(D))
        check_attend((o, lse), want)
        # and the cache holds the history: V as it came, K within a rounding of the rotated key
        for b in range(B):
            pages = table[b, : -(-lens[b] // page)].long()
            hv = c.v_pages[pages].transpose(0, 1).reshape(hkv, -1, D)[:, : lens[b]]
            assert torch.equal(hv, torch.stack(vs[b], 1))
            hk = c.k_pages[pages].transpose(0, 1).reshape(hkv, -1, D)[:, : lens[b]].double()
            wk = torch.stack(ks[b], 1).double()
            # the kernel's rounding and the test's of the same sum: a step apart at most, plus the fp32 sum's error
            assert ((hk - wk).abs() <= 2 * U * wk.abs() + 2.0 ** -20).all()
    assert fv.get_status() == 0


def test_captured_step_reads_the_current_tables(fv, ca):  # noqa: F811
    hq, hkv, D, page, B = 8, 4, 128, 32, 4
    lens = [700, 33, 1, 320]
    c, table, ln = pool(ca, [x + 64 for x in lens], hkv, D, page, 3)
    longest = 800
    rot = ca.rotation_table(D, (64,), 1000)
    q, k, v = normal((B, hq, D), 1), normal((B, hkv, D), 2), normal((B, hkv, D), 3)
    qr, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((B, hq), device="cuda")
    pos = torch.zeros((B, 1), dtype=I32, device="cuda")
    ws = c.attend_workspace(B, hq, longest)
    ln.copy_(torch.tensor(lens, dtype=I32))

    def step():
        c.append(k, v, table, ln, q=q, q_out=qr, pos=pos, rot=rot)
        c.attend(qr, table, ln, longest=longest, out=o, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, 4):
        now = [x + 17 * i for x in lens]
        ln.copy_(torch.tensor(now, dtype=I32))
        pos.copy_((ln - 1).view(B, 1))
        for t, s in ((q, 10), (k, 20), (v, 30)):
            t.copy_(normal(t.shape, s + i))
        graph.replay()
        torch.cuda.synchronize()
        kp, vp = c.k_pages.clone(), c.v_pages.clone()
        want = attend_definition(c, qr, table, ln, 1 / math.sqrt(D))
        check_attend((o, lse), want)
        got = (o.clone(), lse.clone(), qr.clone())
        step()
        torch.cuda.synchronize()
        assert torch.equal(bits(c.k_pages), bits(kp)) and torch.equal(bits(c.v_pages), bits(vp))
        assert torch.equal(bits(o), bits(got[0])) and torch.equal(lse, got[1]) and torch.equal(bits(qr), bits(got[2]))
    assert fv.get_status() == 0


@pytest.mark.parametrize("page,longest", [(16, 40), (64, 3000)])
def test_many_sequences_some_empty(fv, ca, page, longest):  # noqa: F811
    """More sequences than a warp has lanes, runs of empty ones, split and not split."""
    B = 150
    lens = [0 if 40 < b < 75 or b % 7 == 0 or b > 146 else (b * 7919) % (longest + 1) for b in range(B)]
    lens[100] = longest
    c, table, ln = pool(ca, lens, 2, 64, page, 5)
    q = normal((B, 6, 64), 4, 2.0)
    got = c.attend(q, table, ln, longest=longest)
    assert fv.get_status() == 0
    check_attend(got, attend_definition(c, q, table, ln, 0.125))
    # a sequence's bits do not depend on the others: alone, with the same split
    parts = ca.load().fvattn_cache_attn_parts
    if parts(B, 6, 2, 64, longest, None) == parts(1, 6, 2, 64, longest, None) == 1:
        one = c.attend(q[100:101], table[100:101].contiguous(), ln[100:101].contiguous(), longest=longest)
        assert torch.equal(bits(one[0][0]), bits(got[0][100])) and torch.equal(one[1][0], got[1][100])


def test_results_do_not_depend_on_the_schedule(fv, ca):  # noqa: F811
    c, table, ln = pool(ca, [5000, 1, 2222, 700], 4, 128, 16, 5)
    q = normal((4, 16, 128), 4, 2.0)
    first = c.attend(q, table, ln, longest=5000)
    # lengths of the others change, the split (a host number) does not
    ln2 = ln.clone()
    ln2[1:] = torch.tensor([3, 1000, 0], dtype=I32)
    table2 = table.clone()
    table2[1] = table[0]
    second = c.attend(q, table2, ln2, longest=5000)
    for a, b in zip(first, second):
        assert torch.equal(a[0], b[0])
    for _ in range(5):
        again = c.attend(q, table, ln, longest=5000)
        assert torch.equal(bits(again[0]), bits(first[0])) and torch.equal(again[1], first[1])


def test_rows_past_the_end_may_hold_anything_and_scores_of_minus_infinity(fv, ca):  # noqa: F811
    lens = [1, 17, 64, 100, 130]
    c, table, ln = pool(ca, lens, 1, 64, 32, 7)
    q = normal((5, 1, 64), 8).abs() + 0.5
    want = attend_definition(c, q, table, ln, 0.125)
    for b, n in enumerate(lens):
        for p in range(-(-n // 32)):
            used = min(32, n - 32 * p)
            c.k_pages[table[b, p], :, used:] = float("nan")
            c.v_pages[table[b, p], :, used:] = float("inf")
    check_attend(c.attend(q, table, ln), want)
    # keys of -inf: their scores are -inf and their values take no part; a sequence of such keys only is like an empty one
    c.k_pages[table[0, 0], :, 0] = -float("inf")
    c.k_pages[table[3, 1], :, 3:9] = -float("inf")
    o, lse = c.attend(q, table, ln)
    keep = torch.ones(100, dtype=torch.bool)
    keep[35:41] = False
    k = c.k_pages[table[3, :4].long()].transpose(0, 1).reshape(-1, 64)[:100][keep].double()
    v = c.v_pages[table[3, :4].long()].transpose(0, 1).reshape(-1, 64)[:100][keep].double()
    p = torch.softmax(q[3].double() @ k.T * 0.125, -1)
    assert ((o[3].double() - p @ v).abs() <= 1.25 * U * (p @ v.abs() + (p @ v).abs())).all()
    assert (o[0] == 0).all() and lse[0, 0] == -math.inf
    assert fv.get_status() == 0


def test_bad_pages_and_lengths_are_reported(fv, ca):  # noqa: F811
    lens = [40, 50, 60]
    c, table, ln = pool(ca, lens, 2, 64, 16, 9)
    q, k, v = normal((3, 4, 64), 1), normal((3, 2, 64), 2), normal((3, 2, 64), 3)
    want = c.attend(q, table, ln, longest=64)
    k0 = c.k_pages.clone()
    for bad in (-1, c.pages, 1 << 30):
        t2 = table.clone()
        t2[1, 1] = bad
        got = c.attend(q, t2, ln, longest=64)
        assert fv.get_status() == fv.ERR_BOUNDS
        for b in (0, 2):
            assert torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b])
    t2 = table.clone()
    t2[1, 3] = -7                       # page of sequence 1's token 49
    c.append(k, v, t2, ln)
    assert fv.get_status() == fv.ERR_BOUNDS
    changed = (bits(c.k_pages) != bits(k0)).any(-1).any(1).nonzero()
    assert {(int(p), int(r)) for p, r in changed} == {(int(table[0, 2]), 7), (int(table[2, 3]), 11)}
    ln2 = ln.clone()
    ln2[1] = 65
    got = c.attend(q, table, ln2, longest=64)      # clamped to 64: of its 4 pages
    assert fv.get_status() == fv.ERR_BOUNDS
    assert torch.equal(got[0][0], c.attend(q, table, ln, longest=64)[0][0])
    ln2[1] = -1
    got = c.attend(q, table, ln2, longest=64)
    assert fv.get_status() == fv.ERR_BOUNDS
    assert (got[0][1] == 0).all() and (got[1][1] == -math.inf).all()
    # a position outside the rotation table: that token is not written, nor its query
    rot = ca.rotation_table(64, (32,), 100)
    pos = torch.tensor([[5], [100], [-1]], dtype=I32, device="cuda")
    k0, out = c.k_pages.clone(), torch.full_like(q, 3.0)
    c.append(k, v, table, ln, q=q, q_out=out, pos=pos, rot=rot)
    assert fv.get_status() == fv.ERR_BOUNDS
    changed = (bits(c.k_pages) != bits(k0)).any(-1).any(1).nonzero()
    assert {(int(p), int(r)) for p, r in changed} <= {(int(table[0, 2]), 7)}
    assert (out[1:] == 3.0).all() and not (out[0] == 3.0).all()
    assert fv.get_status() == 0


def test_shared_pages_strided_queries_and_another_stream(fv, ca):  # noqa: F811
    c, table, ln = pool(ca, [96, 96, 40], 2, 128, 32, 11)
    table[1, :2] = table[0, :2]                    # a common prefix of 64 tokens
    qkv = normal((3, 8 + 4, 128), 1)
    q = qkv[:, :8]
    want = attend_definition(c, q, table, ln, 1 / math.sqrt(128))
    check_attend(c.attend(q, table, ln), want)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.attend(q, table, ln, stream=st)
    torch.cuda.synchronize()
    check_attend(got, want)
    # in place: the rotated queries over the queries
    rot = ca.rotation_table(128, (30, 34), 50)
    pos = torch.randint(0, 50, (3, 2), dtype=I32, device="cuda")
    kw = dict(pos=pos, rot=rot, axes=(30, 34))
    out = c.append(qkv[:, 8:10], qkv[:, 10:], table, ln, q=q, **kw)
    same = c.append(qkv[:, 8:10], qkv[:, 10:], table, ln, q=q, q_out=q, **kw)
    assert same.data_ptr() == qkv.data_ptr() and torch.equal(bits(q.contiguous()), bits(out))
    assert fv.get_status() == 0


@pytest.mark.parametrize("rotated", [False, True])
def test_rows_outside_the_sequences_are_left_alone(fv, ca, rotated):  # noqa: F811
    """cu as a slice of a larger batch's: rows before its first entry and from its last one on belong to no sequence
    here, whatever their positions hold."""
    lens = [9, 20, 40]
    c, table, ln = pool(ca, lens, 2, 64, 16, 5)
    cu = torch.tensor([3, 5, 5, 8], dtype=I32, device="cuda")
    q, k, v = (normal((11, h, 64), 30 + h) for h in (4, 2, 6))
    v = v[:, :2]
    kp, vp, qo = c.k_pages.clone(), c.v_pages.clone(), normal((11, 4, 64), 40)
    want_q, args = qo.clone(), {}
    if rotated:      # by nothing: cosines of 1, and positions outside the table in rows of no sequence
        rot = torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1).cuda()
        pos = torch.full((11, 1), -7, dtype=I32, device="cuda")
        pos[3:8] = 2
        args = dict(pos=pos, rot=rot)
    for b, (first, past) in enumerate([(3, 5), (5, 5), (5, 8)]):
        for t in range(first, past):
            n = lens[b] - past + t
            page = int(table[b, n // 16])
            kp[page, :, n % 16], vp[page, :, n % 16] = k[t], v[t]
    want_q[3:8] = q[3:8]
    assert c.append(k, v, table, ln, cu=cu, q=q, q_out=qo, **args) is qo
    assert torch.equal(c.k_pages, kp) and torch.equal(c.v_pages, vp) and torch.equal(qo, want_q)
    assert fv.get_status() == 0


def test_nothing_to_append(fv, ca):  # noqa: F811
    c, table, ln = pool(ca, [10, 20], 2, 64, 16, 11)
    k0 = c.k_pages.clone()
    empty = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    zero = torch.zeros(3, dtype=I32, device="cuda")
    assert c.append(empty, empty, table, ln, cu=zero) is None
    k = normal((4, 2, 64), 1)
    c.append(k, k, table, ln, cu=zero)             # four rows, all behind the last sequence
    assert fv.get_status() == 0 and torch.equal(bits(c.k_pages), bits(k0))


def test_pool_past_two_gigaelements(fv, ca):  # noqa: F811
    """Pages whose elements lie past 2^31 (a pool of 4.3 GB a tensor)."""
    D, hkv, page = 128, 8, 128
    pages = (1 << 31) // (D * hkv * page) + 40
    c = ca.PagedCache.empty(pages, hkv, D, page)
    n, top = 700, 6
    table = torch.arange(pages - top, pages, dtype=I32, device="cuda").flip(0).view(1, top).contiguous()
    ln = torch.tensor([n], dtype=I32, device="cuda")
    k, v = normal((n, hkv, D), 1), normal((n, hkv, D), 2)
    c.append(k, v, table, ln, cu=torch.tensor([0, n], dtype=I32, device="cuda"))
    q = normal((1, 16, D), 3, 2.0)
    got = c.attend(q, table, ln)
    assert fv.get_status() == 0
    hk = c.k_pages[table[0].long()].transpose(0, 1).reshape(hkv, -1, D)[:, :n]
    assert torch.equal(hk, k.transpose(0, 1))
    check_attend(got, attend_definition(c, q, table, ln, 1 / math.sqrt(D)))


def test_cache_refusals_on_the_gpu(fv, ca):  # noqa: F811
    c, table, ln = pool(ca, [10, 20], 2, 64, 16, 11)
    k, q = normal((2, 2, 64), 1), normal((2, 4, 64), 1)
    for kw, match in ((dict(k=k.float()), "k:"), (dict(v=k[:, :1]), "v:"), (dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), "k:"),
                      (dict(table=table.long()), "table"), (dict(lens=ln[:1]), "lens"), (dict(cu=ln), "cu"), (dict(q_out=q), "q_out"),
                      (dict(pos=ln.view(2, 1)), "rot"), (dict(rot=torch.zeros((4, 32), device="cuda")), "rot"),
                      (dict(rot=torch.zeros((4, 64), device="cuda")), "pos"),
                      (dict(rot=torch.zeros((4, 64), device="cuda"), axes=(3, 4)), "axes")):
        with pytest.raises(ValueError, match=match):
            c.append(**{**dict(k=k, v=k, table=table, lens=ln), **kw})
    for kw, match in ((dict(q=q[:, :3]), "divide"), (dict(q=q[:1]), "q:"), (dict(scale=0.0), "scale"), (dict(longest=-1), "longest"),
                      (dict(out=q.float()), "out"), (dict(lse=q), "lse"), (dict(table=None), "table"),
                      (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), longest=5000), "workspace")):
        with pytest.raises(ValueError, match=match):
            c.attend(**{**dict(q=q, table=table, lens=ln), **kw})
    with pytest.raises(ValueError, match="distinct"):
        ca.PagedCache(c.k_pages, c.k_pages)
    with pytest.raises(ValueError, match="unsupported"):
        ca.PagedCache(*(torch.zeros((2, 2, 24, 64), dtype=BF16, device="cuda") for _ in range(2)))
    assert fv.get_status() == 0


def test_both_ways_through_the_binding_agree(fv, ca):  # noqa: F811
    """Without a stream argument a call is checked and marshalled by the extension, with one by the Python code."""
    here = torch.cuda.current_stream()
    c, table, ln = pool(ca, [300, 7, 0], 2, 64, 16, 3)
    q, k, v = normal((3, 8, 64), 1), normal((3, 2, 64), 2), normal((3, 2, 64), 3)
    rot, pos = ca.rotation_table(64, (20, 12), 50), torch.randint(0, 50, (3, 2), dtype=I32, device="cuda")
    ln[2] = 1
    table[2, 0] = c.pages - 1
    for kw in (dict(), dict(scale=0.3, longest=400), dict(out=torch.empty_like(q), lse=torch.empty((3, 8), device="cuda")),
               dict(workspace=c.attend_workspace(3, 8, 512), longest=512)):
        a = [t.clone() for t in c.attend(q, table, ln, **kw)]
        b = c.attend(q, table, ln, stream=here, **kw)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])
    for kw in (dict(), dict(q=q), dict(q=q, q_out=torch.empty_like(q), rot=rot, pos=pos, axes=(20, 12), halves=True),
               dict(rot=rot, pos=pos, axes=[20, 12]), dict(cu=torch.tensor([0, 1, 1, 3], dtype=I32, device="cuda"))):
        ways = []
        for extra in (dict(), dict(stream=here)):
            c.k_pages.zero_(), c.v_pages.zero_()
            out = c.append(k, v, table, ln + 2, **kw, **extra)
            ways.append((c.k_pages.clone(), c.v_pages.clone(), None if out is None else out.clone()))
        assert (ways[0][2] is None) == (ways[1][2] is None) == ("q" not in kw)
        for x, y in zip(*ways):
            assert x is None or torch.equal(bits(x), bits(y))
    assert fv.get_status() == 0


def test_capture_behind_copies_fills_and_another_stream(fv, ca):  # noqa: F811
    """The calls' first kernels may start while the work before them ends: behind a copy, a fill and an event of
    another stream, in a graph, they wait for it all the same."""
    c, table, ln = pool(ca, [90, 200], 2, 64, 16, 3)
    src = [normal((2, 2, 64), s) for s in (1, 2)] + [normal((2, 8, 64), 3)]
    k, v, q = (torch.zeros_like(t) for t in src)
    o, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
    ws = c.attend_workspace(2, 8, 300)
    other = torch.cuda.Stream()

    def step():
        k.copy_(src[0])
        c.k_pages.fill_(0.5)
        side = torch.cuda.current_stream()
        other.wait_stream(side)
        with torch.cuda.stream(other):
            v.copy_(src[1])
            c.v_pages.fill_(0.25)
            q.copy_(src[2])
        side.wait_stream(other)
        c.append(k, v, table, ln)
        c.attend(q, table, ln, longest=300, out=o, lse=lse, workspace=ws)
        return c.k_pages.sum(), o.float().sum()

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (c.k_pages, c.v_pages, o, lse)]
    check_attend((o, lse), attend_definition(c, q, table, ln, 0.125))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sums = step()
    for t in (k, v, q, o, lse, c.k_pages, c.v_pages):
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (c.k_pages, c.v_pages, o, lse)):
        assert torch.equal(a, b)
    assert torch.equal(sums[0], c.k_pages.sum()) and torch.equal(sums[1], o.float().sum())
    assert fv.get_status() == 0


@pytest.mark.parametrize("longest", [60, 900])
def test_steps_without_a_sync_between_them(fv, ca, longest):  # noqa: F811
    """Append and attention in turn, hundreds of them in flight, with one buffer for the rotated queries, one for the
    lengths and one workspace: every step reads what the one before it left there, not what an earlier one did."""
    hq, hkv, D, page, B, steps = 8, 2, 64, 16, 3, 300
    c, table, _ = pool(ca, [longest] * B, hkv, D, page, 3)
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    rot = ca.rotation_table(D, (D // 2,), 1000)
    ks, vs = normal((steps, B, hkv, D), 1), normal((steps, B, hkv, D), 2)
    qs = normal((steps, B, hq, D), 3, 2.0)
    gen = torch.Generator().manual_seed(4)
    lens = torch.randint(1, longest + 1, (steps, B), generator=gen, dtype=I32).cuda()
    pos = torch.randint(0, 1000, (steps, B, 1), generator=gen, dtype=I32).cuda()
    q = torch.zeros((B, hq, D), dtype=BF16, device="cuda")
    ws = c.attend_workspace(B, hq, longest)

    def run(sync):
        c.k_pages.copy_(k0)
        c.v_pages.copy_(v0)
        o = torch.zeros((steps, B, hq, D), dtype=BF16, device="cuda")
        lse = torch.zeros((steps, B, hq), device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            c.append(ks[i], vs[i], table, lens[i], q=qs[i], q_out=q, pos=pos[i], rot=rot)
            if sync:
                torch.cuda.synchronize()
            c.attend(q, table, lens[i], longest=longest, out=o[i], lse=lse[i], workspace=ws)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return o, lse, c.k_pages.clone(), c.v_pages.clone()

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    assert fv.get_status() == 0


@pytest.mark.parametrize("stream", [False, True], ids=["extension", "bindings"])
def test_rows_that_take_no_part_are_zero_in_queries_made_by_the_call(fv, ca, stream):  # noqa: F811
    """Rows outside the sequences and refused tokens: zero where the call makes q_out, left alone where it is given."""
    c, table, ln = pool(ca, [40, 7], 2, 64, 16, 3)
    rows, hq, D = 9, 4, 64
    k, v, q = normal((rows, 2, D), 1), normal((rows, 2, D), 2), normal((rows, hq, D), 3)
    cu = torch.tensor([2, 4, 7], dtype=I32, device="cuda")
    rot = ca.rotation_table(D, (32,), 100)
    pos = torch.arange(rows, dtype=I32, device="cuda").view(-1, 1)
    pos[5] = 100                                            # past the table: refused
    kw = dict(cu=cu, q=q, pos=pos, rot=rot, stream=torch.cuda.current_stream() if stream else None)
    out = torch.full_like(q, 7.0)
    assert c.append(k, v, table, ln, q_out=out, **kw) is out
    assert fv.get_status() == fv.ERR_BOUNDS
    junk = [torch.full_like(q, float("nan")) for _ in range(8)]      # what a fresh block of this size may hold
    del junk
    got = c.append(k, v, table, ln, **kw)
    assert fv.get_status() == fv.ERR_BOUNDS
    part = torch.tensor([i in (2, 3, 4, 6) for i in range(rows)], device="cuda")
    assert torch.equal(bits(got[part]), bits(out[part]))
    assert (got[~part] == 0).all() and (out[~part] == 7.0).all()


@pytest.mark.parametrize("way", ["extension", "bindings"])
def test_other_threads_run_while_a_call_waits_for_the_launch_queue(fv, ca, way):  # noqa: F811
    """A caller that runs ahead fills the stream's launch queue and waits in its next call until the GPU is through
    the work in front (half a second here); another Python thread goes on meanwhile."""
    import threading
    import time
    c, table, ln = pool(ca, [40, 7], 2, 64, 16, 3)
    k, v = normal((2, 2, 64), 1), normal((2, 2, 64), 2)
    here = torch.cuda.current_stream() if way == "bindings" else None
    c.append(k, v, table, ln, stream=here)
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), []

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    other = threading.Thread(target=tick)
    other.start()
    start = time.perf_counter()
    try:
        torch.cuda._sleep(1_000_000_000)         # clocks: over half a second at most 1965 MHz
        for _ in range(4000):                    # more launches than a queue holds (1024)
            c.append(k, v, table, ln, stream=here)
        ahead = time.perf_counter() - start
        torch.cuda.synchronize()
    finally:
        stop.set()
        other.join()
    assert ahead > 0.3                           # the calls did wait
    assert max(gaps) < 0.15
    assert fv.get_status() == 0
