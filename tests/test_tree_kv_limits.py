"""Sizes whose products do not fit 64 bits are refused before any launch (no GPU
needed), in the cache writes and reads and in the tree attention."""

import pytest

import channel_token_sparse_b200 as ds
from test_tree_kv_abi import FAKE, READ, TREE, WRITE, tree, tree_paged

BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.lib()


@pytest.mark.parametrize("size", [
    dict(b=BIG, hkv=BIG, s_cap=16, s=1, s_out_cap=1),             # rows of the cache: 2^64
    dict(b=BIG, hkv=1 << 16, s_cap=1 << 19, s=1, s_out_cap=1),    # 2^65
    dict(b=BIG, hkv=BIG, s_cap=16, s=1, s_out_cap=16),            # both
    dict(b=1 << 17, hkv=1 << 10, s_cap=1 << 7, s=1, s_out_cap=1 << 7),  # 2^34 rows of 64 channels: the first refused
])
def test_dense_read(lib, size):
    a = {**READ, **size}
    assert lib.ds_read_kv(*[a[n] for n in READ], None) == ds.DS_ERR_UNSUPPORTED, ds.last_error()


@pytest.mark.parametrize("b,hkv,s_out_cap,num_blocks,page", [
    (1, 1 << 20, 1, BIG, 1 << 16),          # rows of the pool: 2^66
    (1, BIG, 1, BIG, 16),                   # 2^64
    (BIG, BIG, 16, 1, 1),                   # rows of the output: 2^64
])
def test_paged_read(lib, b, hkv, s_out_cap, num_blocks, page):
    st = lib.ds_read_kv_paged(FAKE, FAKE, FAKE, FAKE, FAKE, 1, page, num_blocks, None, b, hkv, 1, 64, FAKE, FAKE, ds.DS_BF16,
                              s_out_cap, None)
    assert st == ds.DS_ERR_UNSUPPORTED, ds.last_error()


@pytest.mark.parametrize("size,pool", [
    (dict(b=BIG, hkv=1 << 20, s_cap=1 << 14), None),              # 2^64
    (dict(b=1, hkv=1 << 20), (1 << 16, BIG)),                     # 2^66
])
def test_write(lib, size, pool):
    a = {**WRITE, **size}
    if pool is None:
        st = lib.ds_write_kv(*[a[n] for n in WRITE], None)
    else:
        st = lib.ds_write_kv_paged(*[a[n] for n in WRITE if n != "s_cap"], FAKE, 4, *pool, None)
    assert st == ds.DS_ERR_UNSUPPORTED, ds.last_error()


@pytest.mark.parametrize("call,size", [
    (tree, dict(b=1 << 16, hq=1 << 10, hkv=1 << 10, s_cap=BIG)),                          # 2^56: no wrap
    (tree_paged, dict(b=1, hq=1 << 26, hkv=1 << 26, page_size=1 << 16, num_blocks=1 << 22)),  # 2^64
    (tree, dict(b=4, hq=64, hkv=64, s_cap=1 << 23)),                                      # 2^31 rows
])
def test_tree(lib, call, size):
    assert "s_cap" in TREE
    assert call(lib, **size, ws=FAKE, ws_bytes=1 << 50) == ds.DS_ERR_UNSUPPORTED, ds.last_error()


@pytest.mark.parametrize("t,g,d,tiles,per_cta", [
    (1, 8, 128, 8192, 0),       # up to 32 query rows: in tensor memory
    (8, 8, 128, 256, 0),        # up to 128: two streams of 128 tiles
    (8, 8, 128, 257, 2 * 128 * 128 * 4),
    (16, 8, 64, 257, 2 * 128 * 64 * 4),
    (17, 8, 128, 128, 0),       # more: each stream has every tile
    (17, 8, 128, 129, 2 * 128 * 128 * 4),
])
def test_workspace_of_long_pieces(lib, t, g, d, tiles, per_cta):
    """Second accumulators where a CTA's piece of an item may be longer than a
    span of 128 tiles a stream: 148 items, then one item shared by all CTAs."""
    rows = min(-(-t * g // 4) * 4, 256)
    parts = 148 * 2 * rows * (d + 2) * 4
    assert ds.tree_decode_workspace(148, t, g, 1, tiles * 128 - t, d) == parts + 148 * per_cta
    assert ds.tree_decode_workspace(1, t, g, 1, tiles * 128 - t, d) <= parts
