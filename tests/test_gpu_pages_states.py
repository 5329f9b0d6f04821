"""The page calls over pools that are not in order: entries outside the pool.
Whole numbers, entry by entry."""
import pytest

import dsa_sparse_attention_quant_gb300 as dsa
from tests.test_gpu_pages import BLOCK, Pool, i32

pytestmark = pytest.mark.gpu


def fork(p, parents, children):
    dsa.pages_fork(p.d_refs, p.d_bt, p.d_seq, i32(parents), i32(children), p.dev, dev_err=p.err)


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
