"""Rows of the pool that are not as they should be before new tokens: what reserve_pages and fork_pages report,
what they leave, and that no other row's cached text is written."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import tree_ref as ref
from test_gpu_pages import on_gpu, pool_of, same, status_words
from test_gpu_tree_attention import i32

pytestmark = pytest.mark.gpu
BAD = kda.ERR_BAD_CACHE_INDEX


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def shared(len0=100, page=16, width=40, pages=60, seed=11):
    """A prompt in row 0 and a fork of it in row 1; row 2 by itself, rows 3 and 4 empty."""
    state = pool_of([len0, 0, 37, 0, 0], page, width, pages, seed)
    gpu, plain, ws = on_gpu(*state), ref.Pool(*state, page), status_words()
    kda.fork_pages(*gpu, i32([0]), i32([1]), page, workspace=ws)
    plain.fork([0], [1])
    assert kda.last_device_status(ws) == kda.OK
    same(gpu, plain)
    return gpu, plain, ws


@pytest.mark.parametrize("new", [1, 20, 300])       # (300: the row is looked at by a warp)
@pytest.mark.parametrize("trimmed", [False, True])
@pytest.mark.parametrize("cut", [20, 31, 95])
def test_a_row_set_back_into_a_shared_page(cut, trimmed, new):
    """Its next token would go into a page that row 0 reads: reported, and the row gets nothing; the rows
    beside it are served."""
    gpu, plain, ws = shared()
    gpu[2][1] = plain.lens[1] = cut
    if trimmed:
        kda.free_pages(*gpu, 16, workspace=ws)
        plain.free()
        same(gpu, plain)
    kda.reserve_pages(*gpu, i32([9, new, 30, 5, 0]), 16, workspace=ws)
    assert kda.last_device_status(ws) == BAD
    plain.reserve([9, 0, 30, 5, 0])
    same(gpu, plain)


def test_a_row_set_back_to_a_shared_pages_end():
    """Between pages: what lies behind has to be given back first, and then the row is like any other."""
    gpu, plain, ws = shared()
    gpu[2][1] = plain.lens[1] = 32
    kda.reserve_pages(*gpu, i32([0, 20, 0, 0, 0]), 16, workspace=ws)
    assert kda.last_device_status(ws) == BAD
    same(gpu, plain)
    kda.free_pages(*gpu, 16, workspace=ws)
    plain.free()
    ws.zero_()
    kda.reserve_pages(*gpu, i32([0, 20, 0, 0, 0]), 16, workspace=ws)
    plain.reserve([0, 20, 0, 0, 0])
    assert kda.last_device_status(ws) == kda.OK
    same(gpu, plain)


def test_a_row_set_back_goes_on_in_a_fork():
    """A fork of the row has a page of its own for the part that it keeps, and takes new tokens; so does the row
    once nobody else holds its page."""
    gpu, plain, ws = shared()
    gpu[2][1] = plain.lens[1] = 20
    kda.free_pages(*gpu, 16, workspace=ws)
    plain.free()
    got = kda.fork_pages(*gpu, i32([1]), i32([3]), 16, workspace=ws)
    want = plain.fork([1], [3])
    assert [x.tolist() for x in got] == list(want) and want[0] != want[1]
    kda.reserve_pages(*gpu, i32([0, 0, 0, 40, 0]), 16, workspace=ws)
    plain.reserve([0, 0, 0, 40, 0])
    same(gpu, plain)
    for rows in ([0], [3]):
        kda.free_pages(*gpu, 16, rows=i32(rows), workspace=ws)
        plain.free(rows)
    kda.reserve_pages(*gpu, i32([0, 40, 0, 0, 0]), 16, workspace=ws)
    plain.reserve([0, 40, 0, 0, 0])
    assert kda.last_device_status(ws) == kda.OK
    same(gpu, plain)


@pytest.mark.parametrize("new", [20, 300])
def test_blocks_that_hold_a_page_outside_the_pool_or_a_free_one(new):
    """A page number past the pool's end or below -1, and a page whose count says that it is free (which the call
    might give to another row): the row is reported and left out."""
    for what in (60, -2, 1 << 30, "free"):
        gpu, plain, ws = shared()
        if what == "free":
            gpu[0][plain.table[2][2]] = plain.refs[plain.table[2][2]] = 0
        else:
            gpu[1][2, 2] = plain.table[2][2] = what
        kda.reserve_pages(*gpu, i32([0, 0, new, 5, 0]), 16, workspace=ws)
        assert kda.last_device_status(ws) == BAD, what
        plain.reserve([0, 0, 0, 5, 0])
        same(gpu, plain)


def test_a_fork_that_found_too_few_pages():
    """The copy without its last page gets none from reserve_pages (an empty one would pass for cached text), also
    once there are free pages again; it is reported until it is ended or set down to its whole pages."""
    page, rows = 16, 5
    state = pool_of([20, 0, 0, 21, 0], page, 40, 5, 12)
    gpu, plain, ws = on_gpu(*state), ref.Pool(*state, page), status_words()
    got = kda.fork_pages(*gpu, i32([0, 0]), i32([1, 2]), page, workspace=ws)
    want = plain.fork([0, 0], [1, 2])
    assert kda.last_device_status(ws) == kda.ERR_OUT_OF_PAGES
    assert [x.tolist() for x in got] == list(want) and want[1][0] >= 0 and want[1][1] == -1
    same(gpu, plain)
    kda.free_pages(*gpu, page, rows=i32([3]), workspace=ws)
    plain.free([3])
    for new in (1, 300):
        ws.zero_()
        kda.reserve_pages(*gpu, i32([0, 0, new, 0, 10]), page, workspace=ws)
        assert kda.last_device_status(ws) == BAD
        plain.reserve([0, 0, 0, 0, 10])
        same(gpu, plain)
    gpu[2][2] = plain.lens[2] = 16
    ws.zero_()
    kda.reserve_pages(*gpu, i32([0, 0, 5, 0, 0]), page, workspace=ws)
    plain.reserve([0, 0, 5, 0, 0])
    assert kda.last_device_status(ws) == kda.OK
    same(gpu, plain)


@pytest.mark.parametrize("what", [-1, -5, 60, 1 << 30])
@pytest.mark.parametrize("block", [0, 3, 6])        # (6: the partly filled one)
def test_a_fork_of_a_row_with_a_page_outside_the_pool(block, what):
    """The copy has -1 there and is otherwise whole; the pair beside it is done, and where it is the last page, no
    page is taken for it and the copy gets none from reserve_pages."""
    state = pool_of([100, 0, 37, 0, 0], 16, 40, 60, 13)
    gpu, plain, ws = on_gpu(*state), ref.Pool(*state, 16), status_words()
    held = plain.table[0][block]
    gpu[1][0, block] = what
    fro, to = kda.fork_pages(*gpu, i32([0, 2]), i32([1, 3]), 16, workspace=ws)
    assert kda.last_device_status(ws) == BAD
    if block == 6:
        plain.lens[0] = 96                # (the definition of a source that ends there)
        want = plain.fork([0, 2], [1, 3])
        plain.lens[0] = plain.lens[1] = 100
        assert want[0][0] == want[1][0] == -1
    else:
        want = plain.fork([0, 2], [1, 3])
        plain.refs[held] -= 1             # (its copy's entry holds nothing)
        plain.table[1][block] = -1
    plain.table[0][block] = what
    assert [fro.tolist(), to.tolist()] == list(want)
    same(gpu, plain)
    if block == 6:
        ws.zero_()
        kda.reserve_pages(*gpu, i32([0, 5, 0, 40, 0]), 16, workspace=ws)
        assert kda.last_device_status(ws) == BAD
        plain.reserve([0, 0, 0, 40, 0])
        same(gpu, plain)


def test_entries_that_nobody_holds_are_given_back_as_nothing():
    """free_pages with a page behind an empty block: a page that is free stays free and is reported, one that the
    row holds goes back like the others."""
    for counted in (False, True):
        state = pool_of([40, 0, 20], 16, 6, 12, 14)
        free = state[0].index(0)
        state[1][1][3] = free
        state[0][free] = int(counted)
        gpu, plain, ws = on_gpu(*state), ref.Pool(*state, 16), status_words()
        kda.free_pages(*gpu, 16, workspace=ws)
        assert kda.last_device_status(ws) == (kda.OK if counted else BAD)
        plain.free()
        plain.refs[free] = 0
        same(gpu, plain)
