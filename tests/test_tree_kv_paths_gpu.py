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
