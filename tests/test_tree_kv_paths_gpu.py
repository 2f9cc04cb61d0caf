"""The cache writes and reads and the tree attention on the GPU: uses that the
size-by-size tests do not make, against the plain 64-bit forms (treehelp)."""

import pytest

import treehelp as th

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import channel_token_sparse_b200 as ds  # noqa: E402
import test_tree_kv_gpu as sized  # noqa: E402
from test_tree_kv_gpu import caches, chain, cu, paged, quantised, randn  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ds.build()
    ds.lib()
    yield
    ds.check_device()


def test_dropped_handle_keeps_its_memory_until_another_stream_is_done():
    """Made on one stream, called on another behind work that takes a while,
    then dropped: what the first stream allocates meanwhile lies elsewhere."""
    b, t, hq, hkv, d, s = 2, 5, 8, 2, 128, 9000
    gen = torch.Generator().manual_seed(31)
    q = randn(gen, b, t, hq, d).bfloat16().cuda()
    k, v = cu(*caches(gen, "bf16", b, hkv, s + t, d)[:2])
    want = ds.tree_decode(q, k, v, s)
    first, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(first):
        call = ds.PreparedTreeDecode(q, k, v, s)
    size = ds.tree_decode_workspace(b, t, hq, hkv, s, d)
    at = call._args[-2]
    with torch.cuda.stream(other):
        torch.cuda._sleep(400_000_000)
        out = call()
        done = other.record_event()
    del call
    with torch.cuda.stream(first):
        new = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
        assert not done.query()  # else the memory was free to go
        for x in new:
            x.fill_(255)
    assert all(x.data_ptr() + size <= at or at + size <= x.data_ptr() for x in new)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# query rows a kv head (t * hq / hkv) that reach each kernel of 16-bit and 8-bit caches: the two of up
# to 32 rows, one row block, two, and two in several row tiles
ROWS = {"16": (4, 4), "32": (7, 4), "128": (24, 4), "256": (50, 4), "1024": (128, 8)}


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", ["key", "value"])
def test_infinite_scales(rows, d, where):
    """An infinite scale of a prefix row, then of a tree row: a key's makes the
    scores of the nodes that see it NaN, a value's their outputs infinite (NaN
    where the code is 0). Nodes that do not see the tree row keep their bits."""
    t, g = ROWS[rows]
    b, hkv, s, inf = 1, 2, 300, float("inf")
    gen = torch.Generator().manual_seed(41)
    k, v, ks, vs = caches(gen, "e4m3", b, hkv, s + t, d)
    k.view(torch.uint8)[0, :, 37, 0], v.view(torch.uint8)[0, :, 37, 0] = 0x38, 0
    q = randn(gen, b, t, g * hkv, d).bfloat16().cuda()
    see = torch.eye(t, dtype=torch.bool).repeat(b, 1, 1)
    see[:, :, 1] = torch.arange(t) % 3 == 1
    mask = th.bits_of(see).cuda()
    kd, vd, ksd, vsd = cu(k, v, ks, vs)

    def run():
        return ds.tree_decode(q, kd, vd, s, mask=mask, k_scale=ksd, v_scale=vsd).cpu()

    plain = run()
    assert bool(torch.isfinite(plain).all())
    scale = ksd if where == "key" else vsd
    keep = scale.clone()
    for row in (37, s + 1):
        scale.copy_(keep)
        scale[:, :, row] = inf
        got = run()
        seen = torch.ones(t, dtype=torch.bool) if row == 37 else see[0, :, 1]
        assert torch.equal(got[:, ~seen], plain[:, ~seen])
        if where == "key":
            assert bool(got[:, seen].isnan().all())
            continue
        want = (v[0, :, row].float() * inf).repeat_interleave(g, 0).expand(int(seen.sum()), -1, -1)
        assert torch.equal(got[0, seen].nan_to_num(7.0), want.nan_to_num(7.0))


def _not_finite(kind, rows, d, what, page=0):
    """Many short items, so that a CTA goes from items with rows that are not
    finite to items without: clean caches and the same ones with such rows."""
    t, g = ROWS[rows]
    hkv = 8 if t * g <= 32 else 4
    b, s = (24 if t * g <= 128 else 12), 150
    gen = torch.Generator().manual_seed(43)
    lens = [(37 * e) % (s + 1) for e in range(b)]
    nodes = [(t, max(t - 1, 0), min(t, 3), t, 0, t)[e % 6] for e in range(b)]
    k, v, ks, vs = caches(gen, kind, b, hkv, s + t + 5, d)
    q = randn(gen, b, t, g * hkv, d).to(torch.float32 if kind == "f32" else torch.bfloat16)
    see = torch.rand((b, t, t), generator=gen) < 0.4
    i = torch.arange(t)
    see[:, :, 1], see[:, :, 2] = i % 4 == 1, i % 3 == 2
    clean = [None if x is None else x.clone() for x in (k, v, ks, vs)]
    nan = float("nan")
    for e in range(b):
        behind = slice(lens[e] + nodes[e], None)
        if kind == "e4m3":
            for c, sc in ((k, ks), (v, vs)):
                c.view(torch.uint8)[e, :, behind], sc[e, :, behind] = 0x7f, what
        else:
            k[e, :, behind], v[e, :, behind] = what, what
        if e % 2 == 1 and nodes[e] > 2:  # a key
            if kind == "e4m3":
                ks[e, :, lens[e] + 2] = nan
            else:
                k[e, :, lens[e] + 2, 5] = nan
        if e % 3 == 0 and nodes[e] > 1:  # a value
            if kind == "e4m3":
                vs[e, :, lens[e] + 1] = what
            else:
                v[e, :, lens[e] + 1, 3::8] = what
    lens_d, nodes_d = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, nodes))
    outs = []
    for c in (clean, (k, v, ks, vs)):
        out = torch.full(q.shape, 7.0, device="cuda")
        kw = dict(mask=th.bits_of(see).cuda(), seq_lens=lens_d, node_lens=nodes_d, out=out)
        if page:
            pools, table = paged(c, page, torch.Generator().manual_seed(1))
            kd, vd, ksd, vsd = cu(*pools)
            ds.tree_decode_paged(q.cuda(), kd, vd, table.cuda(), s, k_scale=ksd, v_scale=vsd, **kw)
        else:
            kd, vd, ksd, vsd = cu(*c)
            ds.tree_decode(q.cuda(), kd, vd, s, k_scale=ksd, v_scale=vsd, **kw)
        outs.append(out.cpu())
    return q, clean, v, lens, nodes, see, g, outs


@pytest.mark.parametrize("kind,rows,d,page", [
    *[(kind, rows, d, 0) for kind in ("bf16", "e4m3") for rows in ROWS for d in (64, 128)],
    *[(kind, rows, 128, page) for kind in ("bf16", "e4m3") for rows, page in (("16", 16), ("128", 1), ("256", 64))],
    ("f32", "16", 128, 0), ("f32", "16", 64, 0), ("f32", "128", 128, 16), ("f32", "256", 64, 0)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite_in_every_kernel(kind, rows, d, page, what):
    """A node that does not see a row which is not finite keeps its bits, one
    that sees it gets what the formula gives, and rows past an entry's own nodes
    stay as they were."""
    q, clean, v, lens, nodes, see, g, (plain, got) = _not_finite(kind, rows, d, what, page)
    b, t = q.shape[:2]
    i = torch.arange(t)
    want = plain.clone()
    assert bool(torch.isfinite(plain).all())
    for e in range(b):
        n = nodes[e]
        assert bool((plain[e, n:] == 7.0).all())
        if e % 3 == 0 and n > 1:
            at = torch.nonzero(see[e, :n, 1] & (i[:n] >= 0)).flatten()
            if kind == "e4m3":
                x = v[e, :, lens[e] + 1].float() * what
                want[e, at] = x.repeat_interleave(g, 0)
            else:
                want[e, at, :, 3::8] = what
        if e % 2 == 1 and n > 2:
            want[e, torch.nonzero(see[e, :n, 2]).flatten()] = float("nan")
    # an infinite weight sum cannot be: infinities of one value row keep their sign
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(5.0, 1e30, -1e30), want.nan_to_num(5.0, 1e30, -1e30))
    # the clean call itself, for the first kv head of the first entries
    k0, v0 = (th.values(c[:6, :1], None if sc is None else sc[:6, :1]) for c, sc in ((clean[0], clean[2]), (clean[1], clean[3])))
    ref, bound = th.attention(q[:6, :, :1], k0, v0, lens[:6], nodes[:6], see, sloppy=kind != "f32")
    for e in range(6):
        ref[e, nodes[e]:], bound[e, nodes[e]:] = 7.0, 0.0
    th.check(plain[:6, :, :1], ref, bound)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_node_counts_that_leave_row_tiles_empty(kind):
    """The widest tree (256 nodes of 8 heads: eight row tiles or more), whose
    entries have all, few or none of the nodes."""
    b, t, hkv, g, d, s = 3, 256, 1, 8, 64, 200
    gen = torch.Generator().manual_seed(47)
    lens, nodes = [200, 0, 77], [256, 3, 0]
    k, v, ks, vs = caches(gen, kind, b, hkv, s + t, d)
    q = randn(gen, b, t, g, d).to(torch.float32 if kind == "f32" else torch.bfloat16)
    kd, vd, ksd, vsd = cu(k, v, ks, vs)
    lens_d, nodes_d = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, nodes))
    out = torch.full(q.shape, 7.0, device="cuda")
    ds.tree_decode(q.cuda(), kd, vd, s, seq_lens=lens_d, node_lens=nodes_d, k_scale=ksd, v_scale=vsd, out=out)
    h = [0, 7]
    want, bound = th.attention(q[:, :, h], th.values(k, ks), th.values(v, vs), lens, nodes, chain(b, t),
                               sloppy=kind != "f32")
    for e in range(b):
        want[e, nodes[e]:], bound[e, nodes[e]:] = 7.0, 0.0
        assert bool((out[e, nodes[e]:] == 7.0).all())
    th.check(out[:, :, h], want, bound)


@pytest.mark.parametrize("starts", [None, [0, 70001, 123456789]])
@pytest.mark.parametrize("page", [0, 8])
def test_rotation_by_the_rows_themselves(starts, page):
    """Without positions a token's position is its cache row (far ones lie
    outside the cache: their queries turn all the same)."""
    b, t, hq, hkv, d, cap = 3, 9, 4, 2, 64, 24
    gen = torch.Generator().manual_seed(53)
    x = randn(gen, b, t, hq + 2 * hkv, d)
    inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -2.0 * torch.arange(d // 2) / d).float()
    pos = (torch.tensor(starts or [0] * b)[:, None] + torch.arange(t)).to(torch.int32)
    shape, table = ((b, hkv, cap, d), None) if not page else ((9, hkv, page, d), torch.randperm(9, generator=gen).view(3, 3))
    kc, vc, _, _ = ds.new_kv_cache(shape, torch.float32)
    xd = x.cuda()
    got = ds.write_kv(xd[:, :, :hq], xd[:, :, hq:hq + hkv], xd[:, :, hq + hkv:], kc, vc, inv_freq=inv.cuda(),
                      starts=None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda(),
                      block_table=None if table is None else table.to(torch.int32).cuda())
    want, norms = th.heads(x[:, :, :hq], None, 0.0, pos, inv, False)
    th.check(got, want, th.HALF[torch.float32] * want.abs() + th.STEPS * norms, "q")
    want, norms = th.heads(x[:, :, hq:hq + hkv], None, 0.0, pos, inv, False)
    kk, vv = (th.gather(c, table) if page else c.cpu() for c in (kc, vc))
    for e in range(b):
        if int(pos[e, 0]) < cap:
            th.check(kk[e, :, :t], want[e].transpose(0, 1), (th.HALF[torch.float32] * want[e].abs() + th.STEPS * norms[e]).transpose(0, 1), "k")
            assert torch.equal(vv[e, :, :t], x[e, :, hq + hkv:].transpose(0, 1))
            assert bool((kk[e, :, t:] == 0).all()) and bool((vv[e, :, t:] == 0).all())
        else:
            assert bool((kk[e] == 0).all()) and bool((vv[e] == 0).all())


def _room(n):
    if torch.cuda.mem_get_info()[0] < n << 30:
        pytest.skip(f"needs {n} GB of device memory")


@pytest.mark.parametrize("page", [0, 1 << 16])
def test_writes_past_32_bits(page):
    """A cache of more than 2^32 elements: rows at its end, and no other."""
    b, hkv, d, t = 3, 8, 128, 2
    cap = 1 << 21
    _room(60)
    shape = (b, hkv, cap, d) if not page else (b * (cap // page), hkv, page, d)
    kc, vc, ks, vs = ds.new_kv_cache(shape, th.E4M3)
    gen = torch.Generator().manual_seed(59)
    x = randn(gen, b, t, 2 * hkv, d).bfloat16().cuda()
    table = torch.arange(b * (cap // page), dtype=torch.int32).view(b, -1).cuda() if page else None
    starts = torch.tensor([5, cap, cap - t], dtype=torch.int32).cuda()
    ds.write_kv(None, x[:, :, :hkv], x[:, :, hkv:], kc, vc, starts=starts, k_scale=ks, v_scale=vs, block_table=table)
    for c, sc, first in ((kc, ks, 0), (vc, vs, hkv)):
        for e, row in ((0, 5), (2, cap - t)):
            at = (e, slice(None), slice(row, row + t)) if not page else (
                e * (cap // page) + row // page, slice(None), slice(row % page, row % page + t))
            y = x[e, :, first:first + hkv].float().transpose(0, 1).cpu()
            codes, scale = quantised(y)
            assert torch.equal(sc[at].cpu(), scale)
            assert torch.equal(c[at].cpu().view(torch.uint8), codes.view(torch.uint8))
            sc[at] = 0
        assert not bool(sc.any())


def test_reads_past_32_bits():
    """A cache and outputs of more than 2^32 elements: the last entry's rows."""
    b, hkv, d, s = 3, 8, 128, 1 << 21
    _room(60)
    kc, vc, ks, vs = ds.new_kv_cache((b, hkv, s, d), th.E4M3)
    gen = torch.Generator().manual_seed(61)
    k, v, k_scale, v_scale = caches(gen, "e4m3", 1, hkv, 50, d)
    for c, x in ((kc, k), (vc, v)):
        c.view(torch.uint8)[2, :, -50:] = x[0].view(torch.uint8).cuda()
    ks[2, :, -50:], vs[2, :, -50:] = k_scale[0].cuda(), v_scale[0].cuda()
    outs = [torch.empty((b, hkv, s, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ds.read_kv(kc, vc, ks, vs, s, k_out=outs[0], v_out=outs[1])
    for o, x, sc in ((outs[0], k, k_scale), (outs[1], v, v_scale)):
        assert torch.equal(o[2, :, -50:].cpu(), (x[0].float() * sc[0, :, :, None]).bfloat16())
        assert not bool(o[2, :, -60:-50].any()) and not bool(o[0, 0, :1000].any())


def test_pieces_of_more_than_a_second():
    """So long a context that one CTA's piece of an item takes longer than a
    wait for a tile may: 105M tokens (all pages of the prefix are one block)
    under 2048 query rows."""
    page, blocks, t, g, d, b = 1 << 16, 1600, 256, 8, 64, 19
    gen = torch.Generator(device="cuda").manual_seed(67)
    k, v = (torch.randn((1, 1, page, d), generator=gen, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn((b, t, g, d), generator=gen, device="cuda").bfloat16()
    table = torch.zeros((b, blocks), dtype=torch.int32, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    out = ds.tree_decode_paged(q, k, v, table, blocks * page - t)
    end.record()
    ds.check_device()  # no wait gave up
    assert start.elapsed_time(end) > 1500.0
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("d", [64, 128])
def test_long_sums(kind, rows, d):
    """A million tokens an entry of values of one sign, all with the weight 1
    (the queries are 0), summed up by few CTAs: the output is the values' mean.
    The weights, their sums and (8-bit: scales that are powers of 2) the products
    are exact; what is off is the accumulation. A product adds 16 rows, in four
    steps at most, each cutting off less than 2^-23 of the sum so far: 2^-21 of
    it, half of that on average over a span of 128 tiles of 8 products. The spans
    themselves are added in fp32."""
    t, g = ROWS[rows]
    page, blocks = 1 << 15, 32
    b = 160 if t * g <= 256 else 40
    gen = torch.Generator(device="cuda").manual_seed(71)
    k = torch.randn((1, 1, page, d), generator=gen, device="cuda")
    v = 2.0 + torch.randn((1, 1, page, d), generator=gen, device="cuda")
    ks = vs = None
    if kind == "e4m3":
        k, v = k.to(th.E4M3), (v * 16).to(th.E4M3)
        ks, vs = torch.ones((1, 1, page), device="cuda"), torch.full((1, 1, page), 0.0625, device="cuda")
        values = v.double() / 16
    else:
        k, v = k.bfloat16(), v.bfloat16()
        values = v.double()
    q = torch.zeros((b, t, g, d), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((b, blocks), dtype=torch.int32, device="cuda")
    mask = torch.full((b, t, (t + 31) // 32), -1, dtype=torch.int32, device="cuda")
    out = ds.tree_decode_paged(q, k, v, table, blocks * page - t, mask=mask, k_scale=ks, v_scale=vs)
    ds.check_device()
    mean, size = values[0, 0].mean(0), values[0, 0].abs().mean(0)
    tiles = blocks * page // 128
    tol = (128 * 8 / 2 * 2.0 ** -21 + (tiles / 128 + 16) * 2.0 ** -24) * size
    assert bool(((out.double() - mean).abs() <= tol).all()), float(((out.double() - mean).abs() / tol).max())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", list(ROWS))
def test_maxima_that_move_late(kind, rows):
    """Two kinds of pages, the second with keys 2.5 times as large, met after
    thousands of tiles: what has been summed up by then, in both accumulators, is
    scaled down. The scores, weights and sums are off as in treehelp.attention
    (sums take a rounding a tile), the accumulation as in test_long_sums."""
    t, g = ROWS[rows]
    d, page, b = 128, 1 << 14, 80 if t * g <= 256 else 40
    order = torch.tensor([0] * 40 + [1] * 3 + [0] * 21)
    gen = torch.Generator(device="cuda").manual_seed(73)
    k = torch.randn((2, 1, page, d), generator=gen, device="cuda")
    v = 2.0 + torch.randn((2, 1, page, d), generator=gen, device="cuda")
    k[1] *= 2.5
    v[1] -= 3.0
    ks = vs = None
    if kind == "e4m3":
        (k, ks), (v, vs) = quantised(k), quantised(v)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    q = torch.randn((b, t, g, d), generator=gen, device="cuda").bfloat16()
    mask = torch.full((b, t, (t + 31) // 32), -1, dtype=torch.int32, device="cuda")
    s = len(order) * page - t
    out = ds.tree_decode_paged(q, k, v, order.to(torch.int32).repeat(b, 1).cuda(), s, mask=mask, k_scale=ks, v_scale=vs)
    ds.check_device()
    kk, vv = (c[:, 0].cuda() for c in (th.values(k, ks), th.values(v, vs)))
    times = torch.stack([(order == i).sum() for i in (0, 1)]).double().cuda()
    pick = q[:: b - 1, :: max(t - 1, 1), 1].double()  # the first and the last entry and node
    score = torch.einsum("btd,pnd->btpn", pick, kk) / d ** 0.5
    size = torch.einsum("btd,pnd->btpn", pick.abs(), kk.abs()) / d ** 0.5
    p = torch.softmax((score + times.log()[:, None]).flatten(2), -1).view_as(score)
    want = torch.einsum("btpn,pnd->btd", p, vv)
    sums = (s / 128 + 64) * th.F32
    rel = 2 * (d + 4) * th.F32 * size + sums
    bound = torch.einsum("btpn,pnd->btd", p * (rel + 2.0 ** -8 + 128 * 8 / 2 * 2.0 ** -21), vv.abs())
    bound += (p * rel).sum((2, 3))[..., None] * want.abs()
    th.check(out[:: b - 1, :: max(t - 1, 1), 1], want.cpu(), bound.cpu())


@pytest.mark.parametrize("case", [
    # either side of the row counts at which another kernel or row tile takes over
    ("f32", 2, 12, 2, 2, 128, 300, [300, 9], 0, "tree"), ("f32", 1, 25, 2, 2, 128, 300, None, 16, "tree"),
    ("f32", 2, 41, 2, 2, 128, 130, [0, 130], 0, "tree"), ("f32", 1, 49, 2, 2, 128, 200, None, 0, "tree"),
    ("f32", 2, 20, 4, 2, 64, 300, [300, 64], 0, "tree"), ("f32", 1, 49, 2, 2, 64, 300, None, 1, "tree"),
    ("bf16", 2, 16, 2, 2, 128, 400, [400, 200], 0, "tree"), ("bf16", 2, 17, 2, 2, 128, 400, [400, 200], 16, "tree"),
    ("bf16", 1, 32, 2, 2, 64, 400, None, 0, "tree"), ("bf16", 1, 128, 1, 1, 64, 300, None, 0, "tree"),
    ("bf16", 1, 129, 1, 1, 64, 300, None, 0, "tree"), ("e4m3", 1, 32, 2, 2, 64, 400, None, 0, "tree"),
    ("e4m3", 1, 33, 2, 2, 128, 400, None, 16, "tree"), ("e4m3", 1, 128, 1, 1, 64, 300, None, 0, "tree"),
    ("e4m3", 1, 129, 1, 1, 64, 300, None, 0, "tree"),
])
def test_borders_between_kernels(case):
    sized.test_tree_decode(*case)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("d", [64, 128])
def test_long_pieces_repeat(kind, rows, d):
    """Pieces of several spans with maxima that move: the same bits every time,
    whatever the workspace holds before, and captured."""
    t, g = ROWS[rows]
    page, blocks, b = 1 << 13, 32, 150 if t * g <= 256 else 40
    gen = torch.Generator(device="cuda").manual_seed(79)
    k, v = (torch.randn((blocks, 1, page, d), generator=gen, device="cuda") for _ in "kv")
    k *= torch.linspace(0.5, 2.0, blocks, device="cuda")[:, None, None, None]
    ks = vs = None
    if kind == "e4m3":
        (k, ks), (v, vs) = quantised(k), quantised(v)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    q = torch.randn((b, t, g, d), generator=gen, device="cuda").bfloat16()
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(b, 1)
    s = blocks * page - t
    ws = torch.empty(ds.tree_decode_workspace(b, t, g, 1, s, d, ds.DS_E4M3 if kind == "e4m3" else ds.DS_BF16),
                     dtype=torch.uint8, device="cuda")
    call = ds.PreparedTreeDecode(q, k, v, s, k_scale=ks, v_scale=vs, block_table=table, ws=ws)
    first = call().clone()
    assert bool(torch.isfinite(first).all())
    for fill in (0, 255, 127, 255):
        ws.fill_(fill)
        call.out.zero_()
        assert torch.equal(call(), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    call.out.zero_()
    graph.replay()
    assert torch.equal(call.out, first)
    ds.check_device()
