"""The page calls over pools that are not in order: entries outside the pool,
pages whose count does not fit. Whole numbers, entry by entry."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.test_gpu_pages import BLOCK, STATE, Pool, i32

pytestmark = pytest.mark.gpu


def fork(p, parents, children):
    dsa.pages_fork(p.d_refs, p.d_bt, p.d_seq, i32(parents), i32(children), p.dev, dev_err=p.err)


def lowest_free(p, n):
    return [int(x) for x in np.nonzero(p.refs == 0)[0][:n]]


@pytest.mark.parametrize("entry", [30, 2 ** 31 - 1, -1, -5])
def test_fork_of_a_part_filled_page_outside_the_pool(entry):
    p = Pool(21, 30, 7, [200, 200, 130])
    p.bt[0, 3] = entry
    p.up()
    fork(p, [0, 1, 0, 2], [3, 4, 5, 6])
    # rows 3 and 5 stay empty and take no page; the others take the lowest free ones
    p.fork([1, 2], [4, 6], run=False)
    p.same(BLOCK)
    assert p.seq[3] == 0 and p.seq[5] == 0 and p.seq[4] == 200


def test_fork_of_a_part_filled_page_without_users():
    # its bytes are anybody's: the page may be taken for another child of the same call
    for low in (False, True):
        p = Pool(22, 30, 7, [200, 200, 130])
        p.refs[p.bt[0, 3]] = 0
        if low:   # the lowest page of the pool that is free
            free = [b for b in lowest_free(p, 30) if b < p.bt[0, 3]]
            p.refs[free] = 1
        p.up()
        fork(p, [0, 1, 0, 2], [3, 4, 5, 6])
        p.fork([1, 2], [4, 6], run=False)
        p.same(STATE)
        if low:
            assert p.bt[4, 3] == p.bt[0, 3]


@pytest.mark.parametrize("count", [0, -2])
def test_fork_shares_a_page_without_users(count):
    p = Pool(23, 30, 6, [256, 200])
    page = int(p.bt[0, 1])
    free = [b for b in lowest_free(p, 30) if b < page]
    p.refs[free] = 1       # were its count 0, it would be the lowest free page
    p.refs[page] = count
    p.up()
    fork(p, [0], [3])      # whole pages alone: none is taken
    p.fork([0], [3], run=False)
    p.same(STATE)


@pytest.mark.parametrize("order", [[0, 1], [1, 0]])
def test_fork_shares_a_page_that_it_takes(order):
    # a full page of row 0 has count 0 and is the lowest free one: row 1's child takes it
    p = Pool(24, 30, 6, [256, 200])
    page = int(p.bt[0, 1])
    p.refs[[b for b in lowest_free(p, 30) if b < page]] = 1
    p.refs[page] = 0
    p.up()
    fork(p, order, [3, 4])
    child = 3 + order.index(1)
    assert int(p.d_bt[child, 3]) == page and int(p.d_refs[page]) == 2
    assert int(p.err.item()) == STATE


def test_fork_of_a_sound_pool_flags_nothing():
    # scratch from an earlier call says nothing of this one
    p = Pool(25, 300, 40, [64 * 5 + 3, 640, 64 * 2 + 1])
    ws = torch.zeros(dsa.pages_workspace_size(300, 12), dtype=torch.uint8, device="cuda")
    for at in (4, 16):
        par = [0, 1, 2] * 4
        dsa.pages_fork(p.d_refs, p.d_bt, p.d_seq, i32(par), i32(list(range(at, at + 12))), p.dev, ws=ws, dev_err=p.err)
        assert p.fork(par, list(range(at, at + 12)), run=False) == 0
        p.same()
        assert p.free([at + 1, at + 2, 0 if at == 16 else at + 3]) == 0
        p.same()


def test_free_flags_entries_that_are_no_pages():
    p = Pool(26, 40, 6, [300, 200, 64])
    pages = [int(b) for b in p.bt[0, :5]]
    p.bt[0, 1], p.bt[0, 3] = -2, -2 ** 31
    p.up()
    dsa.pages_free(p.d_refs, p.d_bt, p.d_seq, i32([0, 2]), dev_err=p.err)
    p.refs[[pages[0], pages[2], pages[4], int(p.bt[2, 0])]] -= 1
    p.bt[0, :5] = p.bt[2, :1] = -1
    p.seq[[0, 2]] = 0
    p.same(BLOCK)
    # -1 inside the length is an entry that another naming of the row has taken
    assert p.free([1, 1]) == 0
    p.same()
