"""The cache writes and reads and the tree attention on the GPU: uses that the
size-by-size tests do not make, against the plain 64-bit forms (treehelp)."""

import pytest

import treehelp as th

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import channel_token_sparse_b200 as ds  # noqa: E402
from test_tree_kv_gpu import caches, cu, randn  # noqa: E402


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
