"""The cache writes and reads and the tree attention on the GPU, against plain
64-bit forms (treehelp), at the sizes, masks and layouts where they can go
wrong."""

import numpy as np
import pytest

import treehelp as th

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import channel_token_sparse_b200 as ds  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": th.E4M3}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ds.build()
    ds.lib()
    yield
    ds.check_device()


def randn(gen, *shape):
    return torch.randn(shape, generator=gen)


def quantised(x):
    """x [..., d] as 8-bit rows, by the definition: (codes, scales)."""
    sc = (x.abs().amax(-1) / torch.tensor(448.0)).clamp_min(2.0 ** -126)
    return (x / sc[..., None]).to(th.E4M3), sc


def caches(gen, kind, b, hkv, n, d, heavy=True):
    """Random caches (k, v, k_scale, v_scale) on the host, [b, hkv, n, d]."""
    k, v = randn(gen, b, hkv, n, d), randn(gen, b, hkv, n, d)
    if heavy:
        k[..., :4] *= 4
    if kind == "e4m3":
        (k, ks), (v, vs) = quantised(k), quantised(v)
        return k, v, ks, vs
    return k.to(TYPES[kind]), v.to(TYPES[kind]), None, None


def random_tree(gen, b, t):
    parents = (torch.rand((b, t), generator=gen) * (torch.arange(t) + 1)).long() - 1
    return parents


def sees_of(parents):
    b, t = parents.shape
    s = torch.zeros((b, t, t), dtype=torch.bool)
    for e in range(b):
        for i in range(t):
            j = i
            while j >= 0:
                s[e, i, j] = True
                j = int(parents[e, j])
    return s


def chain(b, t):
    return torch.tril(torch.ones((t, t), dtype=torch.bool)).repeat(b, 1, 1)


def cu(*ts):
    return [None if x is None else x.cuda() for x in ts]


def paged(x, page, gen):
    """A host cache [b, hkv, n, ...] as (pool, table), blocks in random order."""
    b, hkv, n = x[0].shape[:3]
    per = -(-n // page)
    table = torch.randperm(b * per + 2, generator=gen)[: b * per].view(b, per).to(torch.int32)
    pools = []
    for c in x:
        if c is None:
            pools.append(None)
            continue
        raw = c.view(torch.uint8) if c.dtype == th.E4M3 else c
        full = torch.zeros((b, hkv, per * page) + tuple(c.shape[3:]), dtype=raw.dtype)
        full[:, :, :n] = raw
        pool = torch.zeros((b * per + 2, hkv, page) + tuple(c.shape[3:]), dtype=raw.dtype)
        th.scatter(full, pool, table)
        pools.append(pool.view(c.dtype))
    return pools, table


# ------------------------------------------------------------- tree attention

TREE = [
    # kind, b, t, hq, hkv, d, s, lens, page, sees
    ("f32", 1, 4, 2, 2, 64, 512, None, 0, "tree"),
    ("f32", 2, 5, 6, 2, 128, 130, [130, 0], 0, "tree"),
    ("f32", 1, 33, 8, 1, 64, 63, None, 16, "tree"),
    ("f32", 3, 1, 2, 2, 128, 1000, [1000, 1, 0], 1, "chain"),
    ("f32", 2, 2, 8, 2, 128, 700, None, 64, "tree"),
    ("f32", 1, 5, 6, 2, 64, 200, None, 0, "tree"),
    ("f32", 2, 9, 8, 2, 128, 333, [333, 64], 0, "tree"),
    ("bf16", 1, 1, 1, 1, 128, 1, None, 0, "chain"),
    ("bf16", 1, 1, 4, 4, 128, 0, None, 0, "chain"),
    ("bf16", 2, 16, 8, 2, 128, 777, None, 0, "tree"),
    ("bf16", 3, 7, 10, 2, 64, 300, [300, 17, 128], 16, "tree"),
    ("bf16", 1, 64, 8, 2, 128, 1300, None, 64, "tree"),
    ("bf16", 1, 70, 16, 2, 128, 255, None, 0, "chain"),
    ("bf16", 2, 256, 3, 1, 64, 100, [100, 3], 0, "tree"),
    ("bf16", 4, 3, 8, 8, 128, 2000, [1999, 127, 128, 129], 256, "tree"),
    ("bf16", 70, 2, 2, 1, 64, 40, "many", 0, "tree"),
    ("e4m3", 1, 1, 2, 2, 128, 700, None, 0, "chain"),
    ("e4m3", 2, 8, 8, 4, 128, 513, [513, 100], 0, "tree"),
    ("e4m3", 2, 40, 15, 3, 64, 200, None, 1, "tree"),
    ("e4m3", 1, 64, 8, 1, 128, 390, None, 64, "tree"),
    ("e4m3", 5, 5, 4, 4, 64, 130, [0, 1, 123, 124, 130], 8, "tree"),
    ("bf16", 2, 6, 4, 2, 128, 333, [333, 40], 1, "tree"),
    ("bf16", 2, 11, 8, 2, 128, 300, None, 2, "tree"),
    ("bf16", 1, 9, 10, 2, 64, 260, None, 4, "tree"),
    ("bf16", 2, 20, 6, 2, 64, 500, [500, 130], 8, "tree"),
    ("bf16", 1, 17, 14, 2, 64, 777, None, 0, "tree"),
    ("e4m3", 2, 3, 4, 2, 64, 333, [333, 40], 1, "tree"),
    ("e4m3", 1, 10, 6, 2, 128, 300, None, 2, "tree"),
    ("e4m3", 2, 21, 6, 2, 128, 640, [640, 130], 32, "tree"),
    ("e4m3", 1, 33, 2, 2, 64, 1024, None, 0, "tree"),
    ("e4m3", 1, 40, 6, 2, 64, 1024, None, 4, "tree"),
]


def tree_case(kind, b, t, hq, hkv, d, s, lens, page, sees, seed=0):
    gen = torch.Generator().manual_seed(seed + 17)
    if lens == "many":
        lens = [int(x) for x in torch.randint(0, s + 1, (b,), generator=gen)]
    n = s + t + 3
    k, v, ks, vs = caches(gen, kind, b, hkv, n, d)
    q = randn(gen, b, t, hq, d).to(torch.float32 if kind == "f32" else torch.bfloat16)
    see = sees_of(random_tree(gen, b, t)) if sees == "tree" else chain(b, t)
    return gen, q, k, v, ks, vs, see, lens


@pytest.mark.parametrize("kind,b,t,hq,hkv,d,s,lens,page,sees", TREE)
def test_tree_decode(kind, b, t, hq, hkv, d, s, lens, page, sees):
    gen, q, k, v, ks, vs, see, lens = tree_case(kind, b, t, hq, hkv, d, s, lens, page, sees)
    want, bound = th.attention(q, th.values(k, ks), th.values(v, vs), lens or [s] * b, [t] * b, see,
                               sloppy=kind != "f32")
    mask = th.bits_of(see).cuda() if sees == "tree" else None
    sl = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    if page:
        pools, table = paged((k, v, ks, vs), page, gen)
        kd, vd, ksd, vsd = cu(*pools)
        out = ds.tree_decode_paged(q.cuda(), kd, vd, table.cuda(), s, mask=mask, seq_lens=sl, k_scale=ksd, v_scale=vsd)
    else:
        kd, vd, ksd, vsd = cu(k, v, ks, vs)
        out = ds.tree_decode(q.cuda(), kd, vd, s, mask=mask, seq_lens=sl, k_scale=ksd, v_scale=vsd)
    th.check(out, want, bound, "out")
    if kind != "f32" and not page:  # rounded once to bf16 from the same fp32 result
        o16 = ds.tree_decode(q.cuda(), kd, vd, s, mask=mask, seq_lens=sl, k_scale=ksd, v_scale=vsd,
                             out_dtype=torch.bfloat16)
        assert torch.equal(o16, out.bfloat16())


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_hidden_tokens_do_not_count(kind, what):
    """NaN and infinities in nodes that a node does not see, and in rows behind
    the sequence, reach no output of a node that does not see them."""
    b, t, hq, hkv, d, s = 2, 6, 4, 2, 128, 150
    gen, q, k, v, ks, vs, see, _ = tree_case(kind, b, t, hq, hkv, d, s, None, 0, "tree", 3)
    lens, nodes = [150, 121], [6, 4]
    see[:] = torch.eye(t, dtype=torch.bool)
    see[:, 3, 0] = True
    see[:, :, 2] = False  # node 2 is seen by none; it sees the prefix
    for e in range(b):
        for r in (lens[e] + 2, lens[e] + nodes[e], lens[e] + nodes[e] + 1):
            if kind == "e4m3":
                ks[e, :, r] = what
                vs[e, :, r] = what
            else:
                k[e, :, r] = what
                v[e, :, r, ::3] = what
    want, bound = th.attention(q, th.values(k, ks), th.values(v, vs), lens, nodes, see, sloppy=kind != "f32")
    kd, vd, ksd, vsd = cu(k, v, ks, vs)
    out = torch.full((b, t, hq, d), 7.0, device="cuda")
    ds.tree_decode(q.cuda(), kd, vd, s, mask=th.bits_of(see).cuda(), seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                   node_lens=torch.tensor(nodes, dtype=torch.int32).cuda(), k_scale=ksd, v_scale=vsd, out=out)
    want[1, 4:], bound[1, 4:] = 7.0, 0.0  # nodes past the entry's own stay as they were
    th.check(out, want, bound)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_seen_infinities_and_nans(kind):
    """A value that is infinite in one channel makes that channel of the nodes
    that see it infinite, and no other; a NaN key makes their rows NaN."""
    b, t, hq, hkv, d, s = 1, 4, 2, 1, 64, 140
    gen, q, k, v, ks, vs, see, _ = tree_case(kind, b, t, hq, hkv, d, s, None, 0, "tree", 4)
    see[:] = torch.eye(t, dtype=torch.bool)
    v[0, 0, s + 1, 5] = float("inf")
    k[0, 0, s + 2, 7] = float("nan")
    want, bound = th.attention(q, th.values(k), th.values(v), [s], [t], see, sloppy=kind != "f32")
    out = ds.tree_decode(q.cuda(), k.cuda(), v.cuda(), s, mask=th.bits_of(see).cuda()).cpu()
    assert bool(torch.isposinf(out[0, 1, :, 5]).all())
    assert bool(torch.isnan(out[0, 2]).all())
    fine = torch.isfinite(want)
    assert bool(torch.isfinite(out)[fine].all())
    th.check(torch.where(fine, out.double(), 0), torch.where(fine, want, 0), torch.where(fine, bound, 0))


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_rows_that_see_nothing_are_zero(kind):
    b, t, hq, hkv, d = 2, 40, 4, 2, 64
    gen, q, k, v, ks, vs, see, _ = tree_case(kind, b, t, hq, hkv, d, 8, None, 0, "tree", 5)
    see[:, 1::3] = False
    want, bound = th.attention(q, th.values(k, ks), th.values(v, vs), [0, 8], [t, t], see, sloppy=kind != "f32")
    kd, vd, ksd, vsd = cu(k, v, ks, vs)
    out = ds.tree_decode(q.cuda(), kd, vd, 8, mask=th.bits_of(see).cuda(),
                         seq_lens=torch.tensor([0, 8], dtype=torch.int32).cuda(), k_scale=ksd, v_scale=vsd)
    assert bool((out[0, 1::3] == 0).all())
    th.check(out, want, bound)


@pytest.mark.parametrize("kind,t,hq,hkv", [("bf16", 4, 32, 8), ("bf16", 48, 32, 8), ("e4m3", 4, 8, 8), ("f32", 4, 8, 8)])
def test_long_cache_splits(kind, t, hq, hkv):
    """Items split over many CTAs: against the same call in 64 bits on the GPU
    for some heads, and one scale that is far from the default."""
    b, d, s = 1, 128, 30011
    gen = torch.Generator().manual_seed(5)
    k, v, ks, vs = caches(gen, kind, b, hkv, s + t, d)
    q = randn(gen, b, t, hq, d).to(torch.float32 if kind == "f32" else torch.bfloat16)
    kd, vd, ksd, vsd = cu(k, v, ks, vs)
    for scale in (0.0, 0.31):
        out = ds.tree_decode(q.cuda(), kd, vd, s, k_scale=ksd, v_scale=vsd, sm_scale=scale)
        g = hq // hkv
        for h in (0, hq - 1):
            kk, vv = ((c[:, h // g:h // g + 1]) for c in (th.values(k, ks), th.values(v, vs)))
            want, bound = th.attention(q[:, :, h:h + 1], kk, vv, [s], [t], chain(b, t), scale or None, kind != "f32")
            th.check(out[:, :, h:h + 1], want, bound)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last entry's rows."""
    b, hkv, s, d = 3, 8, 1 << 21, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    k = torch.empty((b, hkv, s, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    n, t = 700, 3
    gen = torch.Generator().manual_seed(9)
    q = randn(gen, b, t, hkv, d).bfloat16()
    kh, vh, _, _ = caches(gen, "bf16", 1, hkv, n + t, d)
    k[2, :, :n + t], v[2, :, :n + t] = kh[0].cuda(), vh[0].cuda()
    lens = torch.tensor([0, 0, n], dtype=torch.int32).cuda()
    nodes = torch.tensor([0, 0, t], dtype=torch.int32).cuda()
    out = torch.zeros((b, t, hkv, d), device="cuda")
    ds.tree_decode(q.cuda(), k, v, n, seq_lens=lens, node_lens=nodes, out=out)
    want, bound = th.attention(q[2:], th.values(kh), th.values(vh), [n], [t], chain(1, t))
    th.check(out[2:], want, bound)
    assert bool((out[:2] == 0).all())


@pytest.mark.parametrize("kind,t,hq,hkv,d", [("e4m3", 1, 8, 8, 128), ("e4m3", 4, 32, 8, 128), ("e4m3", 12, 32, 8, 128),
                                             ("e4m3", 40, 32, 8, 128), ("e4m3", 3, 8, 8, 64), ("bf16", 1, 8, 8, 128),
                                             ("bf16", 7, 32, 8, 128), ("bf16", 16, 32, 8, 128), ("bf16", 64, 32, 8, 128)])
def test_long_runs_repeat(kind, t, hq, hkv, d):
    """Hundreds of tiles a CTA, many calls in a row: the same bits every time,
    and no wait that gave up."""
    b, s = 2, 100003
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((b, hkv, s + t, d), generator=gen, device="cuda") for _ in "kv")
    ks = vs = None
    if kind == "e4m3":
        (k, ks), (v, vs) = quantised(k), quantised(v)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    q = torch.randn((b, t, hq, d), generator=gen, device="cuda").bfloat16()
    call = ds.PreparedTreeDecode(q, k, v, s, k_scale=ks, v_scale=vs)
    first = call().clone()
    for _ in range(25):
        call.out.zero_()
        assert torch.equal(call(), first)
    ds.check_device()
    h = hq - 1
    kk, vv = th.values(k[:1, -1:], None if ks is None else ks[:1, -1:]), th.values(v[:1, -1:], None if vs is None else vs[:1, -1:])
    want, bound = th.attention(q[:1, :, h:], kk, vv, [s], [t], chain(1, t))
    th.check(first[:1, :, h:], want, bound)


def test_results_repeat_and_layouts_agree():
    """The same call gives the same bits, and so does the paged layout."""
    b, t, hq, hkv, d, s = 3, 9, 8, 2, 128, 1500
    for kind in ("bf16", "e4m3", "f32"):
        gen, q, k, v, ks, vs, see, _ = tree_case(kind, b, t, hq, hkv, d, s, None, 0, "tree", 6)
        kd, vd, ksd, vsd = cu(k, v, ks, vs)
        mask = th.bits_of(see).cuda()
        a = ds.tree_decode(q.cuda(), kd, vd, s, mask=mask, k_scale=ksd, v_scale=vsd)
        c = ds.tree_decode(q.cuda(), kd, vd, s, mask=mask, k_scale=ksd, v_scale=vsd)
        assert torch.equal(a, c)
        pools, table = paged((k, v, ks, vs), 32, gen)
        kp, vp, kps, vps = cu(*pools)
        e = ds.tree_decode_paged(q.cuda(), kp, vp, table.cuda(), s, mask=mask, k_scale=kps, v_scale=vps)
        assert torch.equal(a, e)


def test_one_token_matches_dense_decode():
    """A tree of one node is the dense decode step over s + 1 tokens."""
    b, hq, hkv, d, s = 2, 8, 2, 128, 900
    gen = torch.Generator().manual_seed(2)
    k, v, _, _ = caches(gen, "bf16", b, hkv, s + 1, d)
    q = randn(gen, b, 1, hq, d).bfloat16()
    out = ds.tree_decode(q.cuda(), k.cuda(), v.cuda(), s)
    dense = ds.dense_decode(q[:, 0].contiguous().cuda(), k.cuda(), v.cuda(), s + 1)
    want, bound = th.attention(q, th.values(k), th.values(v), [s] * b, [1] * b, chain(b, 1))
    th.check(out, want, bound)
    assert float((out[:, 0] - dense).abs().max()) <= 2e-3 * 2


# --------------------------------------------------------------- cache writes

WRITE = [
    # io, cache, b, t, hq, hkv, d, rot, inter, norm, page, lens
    ("bf16", "bf16", 2, 7, 8, 2, 128, 128, False, True, 0, None),
    ("bf16", "bf16", 1, 300, 3, 1, 64, 32, True, True, 16, None),
    ("bf16", "e4m3", 3, 5, 4, 4, 128, 64, False, True, 0, [5, 0, 2]),
    ("bf16", "e4m3", 1, 1, 0, 3, 64, 0, False, False, 8, None),
    ("f32", "f32", 2, 5, 4, 2, 64, 32, True, False, 0, None),
    ("f32", "f32", 1, 33, 5, 5, 128, 128, False, True, 1, [20]),
    ("f32", "e4m3", 2, 4, 2, 2, 128, 16, False, True, 0, None),
    ("bf16", "bf16", 40, 1, 32, 8, 128, 128, False, True, 64, None),
]


@pytest.mark.parametrize("io,cache,b,t,hq,hkv,d,rot,inter,norm,page,lens", WRITE)
def test_write_kv(io, cache, b, t, hq, hkv, d, rot, inter, norm, page, lens):
    gen = torch.Generator().manual_seed(b * 100 + t)
    dt = TYPES[io]
    cap = t + 41
    qkv = (randn(gen, b, t, hq + 2 * hkv + 1, d) * 3).to(dt)  # one projection with a head to spare
    q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:hq + 2 * hkv]
    w = [(1 + 0.3 * randn(gen, d)).to(dt) for _ in range(2)] if norm else [None, None]
    inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -2.0 * torch.arange(rot // 2) / rot).float() if rot else None
    starts = torch.randint(0, 40, (b,), generator=gen).to(torch.int32)
    pos = (starts[:, None] + torch.randint(0, 900000, (b, t), generator=gen)).to(torch.int32)
    # the cache before: something that must stay where nothing is written
    before = caches(gen, cache, b, hkv, cap, d)
    if page:
        pools, table = paged(before, page, gen)
    else:
        pools, table = before, None
    kd, vd, ksd, vsd = cu(*[None if x is None else x.clone() for x in pools])
    qkvd = qkv.cuda()
    args = dict(starts=starts.cuda(), positions=pos.cuda(), q_weight=cu(w[0])[0] if hq else None, k_weight=cu(w[1])[0],
                eps=1e-5, inv_freq=cu(inv)[0], rope=ds.DS_ROPE_INTERLEAVED if inter else ds.DS_ROPE_HALF, k_scale=ksd,
                v_scale=vsd, block_table=cu(table)[0], lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    q_out = torch.full((b, t, hq, d), 5.0, dtype=dt, device="cuda") if hq else None
    got_q = ds.write_kv(qkvd[:, :, :hq] if hq else None, qkvd[:, :, hq:hq + hkv], qkvd[:, :, hq + hkv:hq + 2 * hkv], kd, vd,
                        q_out=q_out, **args)
    assert torch.equal(qkvd.cpu(), qkv)
    after = [None if x is None else (th.gather(x, table)[:, :, :cap] if page else th.host(x)) for x in (kd, vd, ksd, vsd)]
    n = lens or [t] * b
    if hq:
        want, norms = th.heads(q, w[0], 1e-5, pos, inv, inter)
        bound = th.HALF[dt] * want.abs() + th.STEPS * norms * (1 + th.HALF[dt])
        for e in range(b):
            want[e, n[e]:], bound[e, n[e]:] = 5.0, 0.0
        th.check(got_q, want, bound, "q")
    else:
        assert got_q is None
    for name, x, wt, f, c0, sc0, c1, sc1 in (("k", k, w[1], inv, before[0], before[2], after[0], after[2]),
                                             ("v", v, None, None, before[1], before[3], after[1], after[3])):
        y, norms = th.heads(x, wt, 1e-5, pos, f, inter)
        want = th.values(c0, sc0)
        bound = torch.zeros_like(want)
        for e in range(b):
            rows = slice(int(starts[e]), int(starts[e]) + n[e])
            want[e, :, rows] = y[e, :n[e]].transpose(0, 1)
            b32 = th.STEPS * norms[e, :n[e]].transpose(0, 1) * (name == "k")
            if cache == "e4m3":
                sc = y[e, :n[e]].abs().amax(-1).transpose(0, 1)[..., None] / 448
                yy = want[e, :, rows].abs()
                bound[e, :, rows] = torch.maximum(2.0 ** -4 * yy, sc * 2.0 ** -10) + 1.1 * (b32 + 4 * th.F32 * yy)
            else:
                bound[e, :, rows] = (0 if name == "v" else th.HALF[dt]) * want[e, :, rows].abs() + b32 * (1 + th.HALF[dt])
        th.check(th.values(c1, sc1), want, bound, name)
        if name == "v" and cache == "e4m3":  # no norm, no rotation: the codes and scales by the definition, bit for bit
            for e in range(b):
                rows = slice(int(starts[e]), int(starts[e]) + n[e])
                codes, sc = quantised(v[e, :n[e]].float().transpose(0, 1))
                assert torch.equal(sc1[e, :, rows], sc)
                assert torch.equal(c1[e, :, rows].view(torch.uint8), codes.view(torch.uint8))


def test_write_rows_outside_the_cache():
    """Rows before 0 and from the capacity on, and blocks outside the pool, are
    not written; their queries are. Nothing else changes."""
    b, t, hkv, d, cap = 3, 6, 2, 64, 16
    gen = torch.Generator().manual_seed(1)
    k, v = (randn(gen, b, t, hkv, d).bfloat16().cuda() for _ in "kv")
    starts = torch.tensor([-3, cap - 2, 100], dtype=torch.int32).cuda()
    kc, vc = (torch.full((b, hkv, cap, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q = ds.write_kv(k, k, v, kc, vc, starts=starts)
    assert torch.equal(q, k)
    want = torch.full_like(kc, 9.0)
    want[0, :, :3] = k[0, 3:].transpose(0, 1)
    want[1, :, cap - 2:] = k[1, :2].transpose(0, 1)
    assert torch.equal(kc, want)
    table = torch.tensor([[0, -1], [7, 1], [2, 3]], dtype=torch.int32).cuda()
    kp, vp = (torch.full((4, hkv, 8, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ds.write_kv(None, k, v, kp, vp, starts=torch.tensor([4, 4, 12], dtype=torch.int32).cuda(), block_table=table)
    want = torch.full_like(kp, 9.0)
    want[0, :, 4:8] = k[0, :4].transpose(0, 1)
    want[1, :, 0:2] = k[1, 4:].transpose(0, 1)
    want[3, :, 4:8] = k[2, :4].transpose(0, 1)
    assert torch.equal(kp, want)


def test_write_in_place_and_padded_batch():
    """q_out may be q; k and v may be views with a batch stride of their own."""
    gen = torch.Generator().manual_seed(8)
    q = randn(gen, 2, 5, 4, 64).bfloat16().cuda()
    big = randn(gen, 2, 9, 3, 64).bfloat16().cuda()
    kc, vc, _, _ = ds.new_kv_cache((2, 3, 5, 64), torch.bfloat16)
    w = torch.full((64,), 2.0, dtype=torch.bfloat16, device="cuda")
    ref = ds.write_kv(q, big[:, :5], big[:, 4:], kc, vc, q_weight=w)
    assert torch.equal(kc, big[:, :5].transpose(1, 2)) and torch.equal(vc, big[:, 4:].transpose(1, 2))
    got = ds.write_kv(q, big[:, :5], big[:, 4:], kc, vc, q_weight=w, q_out=q)
    assert got is q and torch.equal(q, ref)


def test_quantised_edge_rows():
    """Zero rows, tiny rows, rows at the type's limits, NaN and infinity."""
    d = 64
    x = torch.zeros((1, 7, 1, d))
    x[0, 1] = 1e-44
    x[0, 2, 0, 0], x[0, 2, 0, 1] = 3e38, -1e37
    x[0, 3, 0, 3] = float("nan")
    x[0, 4, 0, 3] = float("inf")
    x[0, 5] = torch.linspace(-448, 448, d)
    x[0, 6, 0, 9] = -5e-7
    kc, vc, ks, vs = ds.new_kv_cache((1, 1, 7, d), th.E4M3)
    ds.write_kv(None, x.cuda(), x.cuda(), kc, vc, k_scale=ks, v_scale=vs)
    k, v = ds.read_kv(kc, vc, ks, vs, 7, dtype=torch.float32)
    assert torch.equal(k.isnan(), v.isnan())
    k = k.cpu()[0, 0]
    assert bool((k[0] == 0).all()) and bool(k[3].isnan().all()) and bool(k[4].isnan().all())
    for r in (1, 2, 5, 6):
        want = x[0, r, 0].double()
        sc = max(float(want.abs().max()) / 448, 2.0 ** -126)
        tol = torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(sc * 2.0 ** -10, dtype=torch.float64)) * (1 + 1e-6) + 2.0 ** -149
        assert bool(((k[r].double() - want).abs() <= tol).all()), r


@pytest.mark.parametrize("b,hkv,s,d,page,lens,dtype", [
    (2, 3, 37, 128, 0, [37, 5], torch.bfloat16),
    (1, 1, 1, 64, 0, None, torch.float32),
    (3, 2, 100, 64, 16, [100, 0, 33], torch.float32),
    (2, 4, 1000, 128, 1, None, torch.bfloat16),
])
def test_read_kv(b, hkv, s, d, page, lens, dtype):
    gen = torch.Generator().manual_seed(s)
    k, v, ks, vs = caches(gen, "e4m3", b, hkv, s + 2, d)
    src, table = ((k, v, ks, vs), None) if not page else paged((k, v, ks, vs), page, gen)
    outs = [torch.full((b, hkv, s + 3, d), 4.0, dtype=dtype, device="cuda") for _ in "kv"]
    got = ds.read_kv(*cu(*src), s, seq_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda(),
                     block_table=cu(table)[0], k_out=outs[0], v_out=outs[1])
    for o, c, sc in zip(got, (k, v), (ks, vs)):
        want = torch.full((b, hkv, s + 3, d), 4.0, dtype=dtype)
        for e in range(b):
            n = s if lens is None else lens[e]
            want[e, :, :n] = (c[e, :, :n].float() * sc[e, :, :n, None]).to(dtype)
        assert torch.equal(o.cpu(), want)
    alone, none = ds.read_kv(*cu(src[0]), None, *cu(src[2]), None, s, block_table=cu(table)[0], dtype=dtype)
    assert none is None and alone.shape == (b, hkv, s, d)
    assert torch.equal(ds.read_kv(*cu(*src), 0, block_table=cu(table)[0])[0], torch.empty((b, hkv, 0, d), dtype=torch.bfloat16, device="cuda"))


# --------------------------------------------------------------- used together

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_speculative_step_then_sparse_decode(kind):
    """A prompt and a drafted tree are written, the tree attends over the cache,
    the cache (read back where it is 8-bit) gets its labels and serves the
    sparse decode step: each stage against the plain forms of its inputs."""
    b, hq, hkv, d, s, t, page = 2, 8, 2, 128, 260, 6, 32
    gen = torch.Generator().manual_seed(11)
    lens = [260, 131]
    per = (s + t + page - 1) // page
    table = torch.randperm(b * per, generator=gen).view(b, per).to(torch.int32).cuda()
    kc, vc, ks, vs = ds.new_kv_cache((b * per, hkv, page, d), TYPES[kind])
    inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -2.0 * torch.arange(d // 2) / d).float().cuda()
    w = [(1 + 0.1 * randn(gen, d)).bfloat16().cuda() for _ in range(2)]
    kw = dict(inv_freq=inv, k_scale=ks, v_scale=vs, block_table=table, k_weight=w[1])
    prompt = randn(gen, b, s, 2 * hkv, d).bfloat16().cuda()
    lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
    ds.write_kv(None, prompt[:, :, :hkv], prompt[:, :, hkv:], kc, vc, lens=lens_d, **kw)
    parents = random_tree(gen, b, t)
    see = sees_of(parents)
    depth = see.sum(-1) - 1
    pos = (torch.tensor(lens)[:, None] + depth).to(torch.int32).cuda()
    x = randn(gen, b, t, hq + 2 * hkv, d).bfloat16().cuda()
    q = ds.write_kv(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], kc, vc, starts=lens_d, positions=pos,
                    q_weight=w[0], **kw)
    out = ds.tree_decode_paged(q, kc, vc, table, s, mask=ds.tree_mask(parents.cuda()), seq_lens=lens_d, k_scale=ks,
                               v_scale=vs)
    dense = [None if c is None else th.gather(c, table) for c in (kc, vc, ks, vs)]
    kv = [th.values(dense[0], dense[2]), th.values(dense[1], dense[3])]
    want, norms = th.heads(x[:, :, hq:hq + hkv], w[1], 1e-6, pos, inv, False)
    for e in range(b):  # the tree's keys are where the attention looks for them
        got = kv[0][e, :, lens[e]:lens[e] + t].transpose(0, 1)
        assert float((got - want[e]).abs().max()) <= (2.0 ** -8 if kind == "bf16" else 2.0 ** -4) * float(want.abs().max()) * 1.01
    ref, bound = th.attention(q, *kv, lens, [t] * b, see)
    th.check(out, ref, bound)
    # the sparse step of entry 0's prompt, over 16-bit rows
    if kind == "e4m3":
        kd, vd = ds.read_kv(kc, vc, ks, vs, s, block_table=table)
    else:
        kd, vd = (c[:, :, :s].contiguous().cuda() for c in dense[:2])
    idx = torch.arange(16, dtype=torch.int32, device="cuda").repeat(hkv, 1) * 8
    lab, _, _ = ds.new_label_cache(kd, 16)
    ds.build_label_cache(kd, idx, lens[0], lab)
    q1 = q[:, 0].contiguous()
    o = ds.sparse_decode(q1[:1], kd[:1].contiguous(), vd[:1].contiguous(), lab[:1].contiguous(), idx, lens[0], lens[0])
    ref, bound = th.attention(q1[:1, None], kd[:1].cpu().double(), vd[:1].cpu().double(), [lens[0]], [0 + 1],
                              torch.zeros((1, 1, 1), dtype=torch.bool))
    assert float((o.cpu().double() - ref[:, 0]).abs().max()) <= 2 * 2e-3


def test_prepared_calls_lengths_streams_and_graphs():
    """Prepared calls on another stream and captured: the replay sees new
    contents of the same buffers; two graphs with their own workspaces may run
    side by side; set_length moves the prefix."""
    b, t, hq, hkv, d, s = 2, 5, 8, 2, 128, 900
    gen = torch.Generator().manual_seed(21)
    k, v, _, _ = caches(gen, "bf16", b, hkv, s + t, d)
    q = randn(gen, b, t, hq, d).bfloat16()
    qd, kd, vd = cu(q, k, v)
    calls = [ds.PreparedTreeDecode(qd, kd, vd, s) for _ in range(2)]
    eager = ds.tree_decode(qd, kd, vd, s)
    streams = [torch.cuda.Stream() for _ in calls]
    graphs = []
    torch.cuda.synchronize()
    for c, st in zip(calls, streams):
        with torch.cuda.stream(st):
            c()
        st.synchronize()
        assert torch.equal(c.out, eager)
        c.out.zero_()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            c()
        graphs.append(g)
    qd.copy_(q.flip(1))
    kd.copy_(k.flip(0))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    want = ds.tree_decode(qd, kd, vd, s)
    for c in calls:
        assert torch.equal(c.out, want)
    calls[0].set_length(411)
    assert torch.equal(calls[0](), ds.tree_decode(qd, kd, vd, 411))
    with pytest.raises(ValueError):
        calls[0].set_length(s + 1)
    side = torch.cuda.Stream()
    got = ds.tree_decode(qd, kd, vd, s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    kc, vc, _, _ = ds.new_kv_cache((b, hkv, 16, d), torch.bfloat16)
    x = randn(gen, b, t, hkv, d).bfloat16().cuda()
    wr = ds.PreparedWriteKV(None, x, x, kc, vc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wr()
    x.copy_(x.flip(1))
    g.replay()
    assert torch.equal(kc[:, :, :t], x.transpose(1, 2)) and bool((kc[:, :, t:] == 0).all())
