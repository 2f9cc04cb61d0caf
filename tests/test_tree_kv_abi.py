"""Host-side checks of the cache writes and reads and of the tree attention (no
GPU needed): refusals before any launch, workspace sizes, masks."""

import ctypes as C

import pytest

import channel_token_sparse_b200 as ds

torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.lib()


TREE = dict(q=FAKE, k=FAKE, v=FAKE, kvdt=ds.DS_BF16, k_scale=None, v_scale=None, mask=None, seq_lens=None,
            node_lens=None, b=2, t=8, hq=8, hkv=2, s=100, s_cap=108, d=128, sm_scale=0.0, out=FAKE, out_dt=ds.DS_F32,
            ws=None, ws_bytes=0)
PAGED = dict(block_table=FAKE, max_blocks=7, page_size=16, num_blocks=14)


def tree(lib, **kw):
    a = {**TREE, **kw}
    return lib.ds_tree_decode(*[a[n] for n in TREE], None)


def tree_paged(lib, **kw):
    a = {**TREE, **PAGED, **kw}
    names = ["q", "k", "v", "kvdt", "k_scale", "v_scale", "mask", *PAGED, "seq_lens", "node_lens", "b", "t", "hq", "hkv",
             "s", "d", "sm_scale", "out", "out_dt", "ws", "ws_bytes"]
    return lib.ds_tree_decode_paged(*[a[n] for n in names], None)


@pytest.mark.parametrize("fault,expect", [
    ({}, ds.DS_ERR_WORKSPACE),  # all else is fine: no workspace
    (dict(q=None), ds.DS_ERR_INVALID_ARG),
    (dict(out=None), ds.DS_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), ds.DS_ERR_INVALID_ARG),
    (dict(mask=FAKE + 2), ds.DS_ERR_INVALID_ARG),
    (dict(b=0), ds.DS_ERR_INVALID_ARG),
    (dict(t=0), ds.DS_ERR_INVALID_ARG),
    (dict(t=257), ds.DS_ERR_UNSUPPORTED),
    (dict(hq=7), ds.DS_ERR_INVALID_ARG),
    (dict(hq=18), ds.DS_ERR_UNSUPPORTED),
    (dict(d=96), ds.DS_ERR_UNSUPPORTED),
    (dict(s=-1), ds.DS_ERR_INVALID_ARG),
    (dict(s=101), ds.DS_ERR_INVALID_ARG),                 # s + t > s_cap
    (dict(s=0x7fffffff, s_cap=0x7fffffff), ds.DS_ERR_UNSUPPORTED),
    (dict(kvdt=ds.DS_F16), ds.DS_ERR_UNSUPPORTED),
    (dict(kvdt=ds.DS_E4M3), ds.DS_ERR_INVALID_ARG),       # no scales
    (dict(kvdt=ds.DS_F32, out_dt=ds.DS_BF16), ds.DS_ERR_INVALID_ARG),
    (dict(out_dt=ds.DS_E4M3), ds.DS_ERR_INVALID_ARG),
    (dict(sm_scale=float("nan")), ds.DS_ERR_INVALID_ARG),
    (dict(ws=FAKE, ws_bytes=16), ds.DS_ERR_WORKSPACE),
    (dict(ws=FAKE + 4, ws_bytes=1 << 40), ds.DS_ERR_INVALID_ARG),
])
def test_tree_validation(lib, fault, expect):
    assert tree(lib, **fault) == expect, ds.last_error()
    assert ds.last_error()
    if "s_cap" not in fault and fault != dict(s=101):
        assert tree_paged(lib, **fault) == expect, ds.last_error()


@pytest.mark.parametrize("fault,expect", [
    (dict(block_table=None), ds.DS_ERR_INVALID_ARG),
    (dict(block_table=FAKE + 1), ds.DS_ERR_INVALID_ARG),
    (dict(page_size=24), ds.DS_ERR_INVALID_ARG),
    (dict(page_size=0), ds.DS_ERR_INVALID_ARG),
    (dict(page_size=1 << 17), ds.DS_ERR_INVALID_ARG),
    (dict(num_blocks=0), ds.DS_ERR_INVALID_ARG),
    (dict(max_blocks=6), ds.DS_ERR_INVALID_ARG),          # 96 rows < 108
    (dict(page_size=1 << 16, num_blocks=1 << 30), ds.DS_ERR_UNSUPPORTED),
])
def test_paged_validation(lib, fault, expect):
    assert tree_paged(lib, **fault) == expect, ds.last_error()


WRITE = dict(q=FAKE, q_bs=1024, q_ts=1024, k=FAKE, k_bs=256, k_ts=256, v=FAKE, v_bs=256, v_ts=256, dt=ds.DS_BF16,
             q_weight=FAKE, k_weight=FAKE, eps=1e-6, inv_freq=FAKE, rot_dim=128, rope=ds.DS_ROPE_HALF, positions=FAKE,
             starts=FAKE, lens=FAKE, b=2, t=1, hq=8, hkv=2, s_cap=64, d=128, q_out=FAKE, k_cache=FAKE, v_cache=FAKE,
             cache_dt=ds.DS_E4M3, k_scale=FAKE, v_scale=FAKE)


@pytest.mark.parametrize("fault,expect", [
    (dict(k=None), ds.DS_ERR_INVALID_ARG),
    (dict(v_cache=None), ds.DS_ERR_INVALID_ARG),
    (dict(q=None), ds.DS_ERR_INVALID_ARG),                # q_out without q
    (dict(q_out=None), ds.DS_ERR_INVALID_ARG),
    (dict(k_scale=None), ds.DS_ERR_INVALID_ARG),
    (dict(dt=ds.DS_F16), ds.DS_ERR_UNSUPPORTED),
    (dict(cache_dt=ds.DS_F32), ds.DS_ERR_UNSUPPORTED),
    (dict(d=80), ds.DS_ERR_UNSUPPORTED),
    (dict(t=0), ds.DS_ERR_INVALID_ARG),
    (dict(b=1 << 20, t=1 << 11), ds.DS_ERR_UNSUPPORTED),
    (dict(eps=-1.0), ds.DS_ERR_INVALID_ARG),
    (dict(eps=float("nan")), ds.DS_ERR_INVALID_ARG),
    (dict(rot_dim=24), ds.DS_ERR_INVALID_ARG),
    (dict(rot_dim=144), ds.DS_ERR_INVALID_ARG),
    (dict(rot_dim=0), ds.DS_ERR_INVALID_ARG),
    (dict(rope=2), ds.DS_ERR_INVALID_ARG),
    (dict(q_ts=1028), ds.DS_ERR_INVALID_ARG),
    (dict(v_bs=4), ds.DS_ERR_INVALID_ARG),
    (dict(k=FAKE + 4), ds.DS_ERR_INVALID_ARG),
    (dict(starts=FAKE + 2), ds.DS_ERR_INVALID_ARG),
    (dict(s_cap=0), ds.DS_ERR_INVALID_ARG),
    (dict(s_cap=0x7fffffff, b=1 << 20, hkv=1 << 10), ds.DS_ERR_UNSUPPORTED),
])
def test_write_validation(lib, fault, expect):
    a = {**WRITE, **fault}
    assert lib.ds_write_kv(*[a[n] for n in WRITE], None) == expect, ds.last_error()
    if "s_cap" not in fault:
        names = [n for n in WRITE if n != "s_cap"]
        assert lib.ds_write_kv_paged(*[a[n] for n in names], FAKE, 4, 16, 8, None) == expect, ds.last_error()
        assert lib.ds_write_kv_paged(*[{**WRITE}[n] for n in names], None, 4, 16, 8, None) == ds.DS_ERR_INVALID_ARG


READ = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, seq_lens=None, b=1, hkv=2, s=10, s_cap=16, d=64, k_out=FAKE,
            v_out=FAKE, out_dt=ds.DS_BF16, s_out_cap=16)


@pytest.mark.parametrize("fault,expect", [
    (dict(k=None), ds.DS_ERR_INVALID_ARG),
    (dict(k_scale=None), ds.DS_ERR_INVALID_ARG),
    (dict(v=None), ds.DS_ERR_INVALID_ARG),
    (dict(v_scale=None), ds.DS_ERR_INVALID_ARG),
    (dict(out_dt=ds.DS_E4M3), ds.DS_ERR_UNSUPPORTED),
    (dict(s=17), ds.DS_ERR_INVALID_ARG),
    (dict(s=-1), ds.DS_ERR_INVALID_ARG),
    (dict(s_out_cap=9), ds.DS_ERR_INVALID_ARG),
    (dict(d=32), ds.DS_ERR_UNSUPPORTED),
    (dict(k_out=FAKE + 8), ds.DS_ERR_INVALID_ARG),
    (dict(v_scale=FAKE + 2), ds.DS_ERR_INVALID_ARG),
    (dict(s=0), ds.DS_OK),                                # nothing to read: nothing is launched
])
def test_read_validation(lib, fault, expect):
    a = {**READ, **fault}
    assert lib.ds_read_kv(*[a[n] for n in READ], None) == expect, ds.last_error()


def test_workspace(lib):
    small = ds.tree_decode_workspace(1, 1, 1, 1, 0, 64)
    large = ds.tree_decode_workspace(1, 256, 8, 1, 100000, 128)
    assert 0 < small <= large <= 64 << 20
    assert small % 16 == 0 and large % 16 == 0
    n = C.c_size_t(77)
    assert lib.ds_tree_decode_workspace_size(1, 0, 1, 1, 0, 64, ds.DS_BF16, C.byref(n)) == ds.DS_ERR_INVALID_ARG
    assert n.value == 77
    assert lib.ds_tree_decode_workspace_size(1, 1, 1, 1, 0, 64, ds.DS_BF16, None) == ds.DS_ERR_INVALID_ARG


def test_tree_mask():
    m = ds.tree_mask(torch.tensor([[-1, 0, 0, 1, -1]]))
    assert m.dtype == torch.int32 and m.tolist() == [[[0b00001], [0b00011], [0b00101], [0b01011], [0b10000]]]
    line = torch.arange(40)[None] - 1
    m = ds.tree_mask(line)
    assert m.shape == (1, 40, 2) and m[0, 39].tolist() == [-1, 0xFF] and m[0, 31].tolist() == [-1, 0]
    for bad in ([[0]], [[-2]], [[-1, 1]]):
        with pytest.raises(ValueError):
            ds.tree_mask(torch.tensor(bad))


def test_host_tensors_are_refused(lib):
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ds.tree_decode(x, x, x, 0)
    with pytest.raises(ValueError):
        ds.write_kv(x, x, x, x, x)
    c = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        ds.read_kv(c, c, x[..., 0].float(), x[..., 0].float(), 1)
