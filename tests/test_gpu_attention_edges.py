"""Attention at its edges, against plain attention in 64 bits: rows that no
request owns."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import attend, check
from tests.test_gpu_attn_prompt import Prompts

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEQ = 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------ rows of nobody

def made(p, **kw):
    """p.run() with results that the call makes out of memory full of NaN: the
    allocator hands freed blocks of a size out again."""
    torch.cuda.synchronize()
    dirty = [torch.full(s, math.nan, dtype=t, device=DEV) for s, t in ((p.q.shape, p.dtype),
                                                                       (p.q.shape[:2], torch.float32))
             for _ in range(3)]
    del dirty
    return p.run(**kw)


def empty(out, lse):
    return bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("paged", [False, True])
def test_prompt_rows_behind_the_last_request(d, paged):
    # more tokens than the requests have: a padded batch
    p = Prompts(31, [100, 150], [100, 400], 4, 2, d, torch.bfloat16, paged)
    b = p.batch
    p.q = torch.cat([p.q, torch.full_like(p.q[:70], math.nan)])
    p.batch = dsa.Batch(b.query_start_loc, b.seq_lens, b.block_table, i32([0] * 100 + [1] * 150 + [-1] * 70), 0,
                        b.num_blocks, max_seq_len=400, num_decode_tokens=0)
    err = i32([0])
    out, lse = made(p, dev_err=err)
    assert int(err.item()) == 0
    p.check(out, lse)
    assert empty(out[250:], lse[250:])
    # passed results keep what they hold there
    out, lse = torch.full_like(p.q, 4.0), torch.full(p.q.shape[:2], 5.0, device=DEV)
    p.run(out=out, lse=lse)
    p.check(out, lse)
    assert bool((out[250:] == 4).all()) and bool((lse[250:] == 5).all())


def test_prompt_rows_of_requests_outside_the_batch():
    p = Prompts(32, [100, 200, 90], [100, 200, 90], 4, 2, 64, torch.bfloat16, True)
    p.batch.query_start_loc[2] = 10 ** 6   # request 1 ends behind the batch, request 2 begins there
    err = i32([0])
    out, lse = made(p, dev_err=err)
    assert int(err.item()) == SEQ
    p.check(out, lse, only=(0,))
    assert empty(out[100:], lse[100:])
    out, lse = torch.full_like(p.q, 4.0), torch.full(p.q.shape[:2], 5.0, device=DEV)
    p.run(out=out, lse=lse)
    p.check(out, lse, only=(0,))
    assert bool((out[100:] == 4).all()) and bool((lse[100:] == 5).all())


def test_rows_of_the_other_half_of_a_mixed_step():
    # results made by the call: the rows it does not write are empty rows
    p = Prompts(33, [130, 65], [130, 65], 4, 2, 128, torch.bfloat16, True, decodes=[70, 300])
    out, lse = made(p)
    p.check(out, lse)
    assert empty(out[:2], lse[:2])
    out, lse = dsa.attn_decode(p.batch, p.q, p.k, p.v)
    for t, n in enumerate([70, 300]):
        for e in range(4):
            check(out[t, e], lse[t, e], attend(p.q[t, e], p.kf[t][:, e // 2], p.vf[t][:, e // 2], 128 ** -0.5, p.dtype))
    assert empty(out[2:], lse[2:])
