"""Outputs that share bytes with what other threads of the same call still read: refused on the host, before any
device is touched."""
import ctypes

import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from test_layer_host import A, L, cache  # noqa: F401  (L: the library, a fixture)
from test_tree_host import accept, pool

INVALID = kda.ERR_INVALID_ARG


def test_accept_refuses_lengths_that_overlap_its_inputs(L):
    """Three sequences of 9 nodes in all, a table of [3, 4] in rows of 6; every array at a place of its own, and
    lens_out moved over the ends of each."""
    at = dict(kv=2 * A, node=3 * A, cu=4 * A, parents=5 * A, table=6 * A)
    size = dict(kv=3, node=3, cu=4, parents=9, table=2 * 6 + 4)
    for name, n in size.items():
        for lens in {at[name] - 8, at[name] - 4, at[name], at[name] + 4, at[name] + 4 * (n - 1)}:
            c = cache(block_table=at["table"], table_stride=6, kv_lens=at["kv"])
            assert accept(L, c, node=at["node"], cu=at["cu"], parents=at["parents"], lens=lens, T=9, N=3) == INVALID, (name, lens)


# a pool of 10 pages and [3, 4] blocks in rows of 6, and lists of two, every one at a place of its own
PLACES = dict(refs=A, table=2 * A, lens=3 * A)
SIZES = dict(refs=10, table=2 * 6 + 4, lens=3, src=2, dst=2, fro=2, to=2)
LISTS = dict(src=4 * A, dst=5 * A, fro=6 * A, to=7 * A)


def over(places, sizes, name):
    """Addresses from which a list of two reaches into `name`."""
    return {places[name] - 4, places[name], places[name] + 4 * (sizes[name] - 1)}


@pytest.mark.parametrize("name", PLACES)
def test_free_refuses_rows_over_the_pool(L, name):
    for at in over(PLACES, SIZES, name):
        assert pool(L, "free", **PLACES, stride=6, list=at) == INVALID


@pytest.mark.parametrize("which", LISTS)
def test_fork_refuses_lists_over_the_pool_and_each_other(L, which):
    places = dict(PLACES, **LISTS)
    others = [x for x in places if x != which and (x in PLACES or {x, which} != {"src", "dst"})]
    for name in others:
        for at in over(places, SIZES, name):
            assert pool(L, "fork", **dict(places, **{which: at}), stride=6) == INVALID, name


@pytest.mark.gpu
def test_arrays_beside_each_other_are_none():
    """One buffer of kv_lens, accepted, lens_out, cu_seqlens and parents."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_pages import cache_of
    b = torch.tensor([20, 33, 2, -1, 7, 7, 0, 3, 7, -1, 0, 0, -1, -1, 1, 2], dtype=torch.int32, device="cuda")
    kv, node, lens, cu, parents = b[:2], b[2:4], b[4:6], b[6:9], b[9:]
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    got = kda.cache_accept(*cache_of(6, 2, 16, 1), table, kv, cu, parents, node, 4, lens_out=lens)
    assert got is lens and b.tolist() == [20, 33, 2, -1, 19, 29, 0, 3, 7, -1, 0, 0, -1, -1, 1, 2]
    # counts, lengths and lists; a list as src and dst both is read twice (its pairs are reported, not refused)
    b = torch.tensor([1, 0, 0, 0, 5, 0, 0, 1, 7, 7], dtype=torch.int32, device="cuda")
    refs, lens, src, dst, fro, to = b[:4], b[4:6], b[6:7], b[7:8], b[8:9], b[9:]
    table = torch.tensor([[0, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kda.fork_pages(refs, table, lens, src, dst, 16, from_pages=fro, to_pages=to, workspace=ws)
    assert kda.last_device_status(ws) == kda.OK
    assert b.tolist() == [1, 1, 0, 0, 5, 5, 0, 1, 0, 1] and table.tolist() == [[0, -1], [1, -1]]
    kda.free_pages(refs, table, lens, 16, rows=dst, workspace=ws)
    assert b.tolist() == [1, 0, 0, 0, 5, 0, 0, 1, 0, 1] and table.tolist() == [[0, -1], [-1, -1]]
    kda.fork_pages(refs, table, lens, src, src, 16, workspace=ws)
    assert kda.last_device_status(ws) == kda.ERR_BAD_CACHE_INDEX and lens.tolist() == [5, 0]
