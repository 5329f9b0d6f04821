"""Attention at its edges, against plain attention in 64 bits: rows that no
request owns, rows whose scores are all -infinity over values that are not
finite, sizes far from the usual ones."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import attend, check
from tests.test_gpu_attn_prompt import Prompts
from tests.test_gpu_attn_rows import Step, check_selected, selected_case

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


# ------------------------------------- scores of -infinity, values not finite

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("keys", [40, 3000])
@pytest.mark.parametrize("group", [2, 20])
def test_rows_of_minus_infinity_over_values_that_are_not_finite(dtype, keys, group):
    s = Step(41, [keys, keys, 5], [1] * 3, 2 * group, 2, 64, dtype)
    at = s.batch.block_table.long()
    s.q.abs_()
    for r, n in ((0, keys), (1, keys - 5)):     # request 0: every score, request 1: all but the last five
        for j in range(0, n, 64):
            s.k[at[r, j // 64], :min(64, n - j), 0] = -math.inf
        s.v[at[r, 0], 7, 0, 3], s.v[at[r, 0], 11, 0, 4] = math.nan, math.inf
    phys = torch.full((3, keys), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate([keys, keys, 5]):
        j = torch.arange(n, device=DEV)
        phys[r, :n] = (at[r][j // 64] * 64 + j % 64).to(torch.int32)
    for out, lse in (dsa.attn_decode(s.batch, s.q, s.k, s.v), dsa.attn_selected(s.q, s.k, s.v, phys)):
        assert empty(out[0, :group], lse[0, :group])
        # a visible NaN gives NaN, a visible infinity an infinity or NaN, however the keys are cut
        assert bool(torch.isnan(out[1, :group, 3]).all()) and not bool(torch.isfinite(out[1, :group, 4]).any())
        keep = [i for i in range(64) if i not in (3, 4)]
        for e in range(group):
            ref = attend(s.q[1, e], s.kf[1][-5:, 0], s.vf[1][-5:, 0], s.scale, dtype)
            check(out[1, e, keep], lse[1, e], (ref[0][keep], ref[1], ref[2][keep], ref[3]))
        assert bool(torch.isfinite(out[:, group:]).all()) and bool(torch.isfinite(out[2]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [2, 3])
def test_prompt_of_minus_infinity_over_values_that_are_not_finite(dtype, d, hq):
    n = 400
    p = Prompts(42, [n], [n], hq, 1, d, dtype, False, gap=0)
    p.q.abs_()
    p.k[:150] = -math.inf
    p.v[5, 0, 3], p.v[140, 0, 4], p.v[200, 0, 5] = math.nan, math.inf, math.inf
    out, lse = p.run()
    assert empty(out[:150], lse[:150])
    assert bool(torch.isnan(out[150:, :, 3]).all())
    assert not bool(torch.isfinite(out[150:, :, 4]).any()) and not bool(torch.isfinite(out[200:, :, 5]).any())
    keep = [i for i in range(d) if i not in (3, 4, 5)]
    assert bool(torch.isfinite(out[150:][..., keep]).all()) and bool(torch.isfinite(out[150:200, :, 5]).all())


# ----------------------------------------------------------- results over q

@pytest.mark.parametrize("keys", [[100, 300], [5000, 1200]])
def test_results_over_the_queries(keys):
    # out may be q's own memory
    s = Step(54, keys, [1, 1], 8, 2, 128, torch.bfloat16)
    want, wlse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    q = s.q.clone()
    out, lse = dsa.attn_decode(s.batch, q, s.k, s.v, out=q)
    assert out is q and torch.equal(q, want) and torch.equal(lse, wlse)
    for hq, hkv in ((4, 2), (3, 1)):
        p = Prompts(55, [300, 700], [400, 700], hq, hkv, 64, torch.float16, True)
        want, wlse = p.run()
        out, lse = p.run(out=p.q)
        assert torch.equal(out, want) and torch.equal(lse, wlse)


# ------------------------------------------------------------- unused metadata

def test_packed_prompts_without_a_block_table():
    p = Prompts(34, [300, 65], [300, 100], 4, 2, 64, torch.bfloat16, False)
    want, wlse = p.run()
    p.batch.c.block_table, p.batch.c.bt_stride = None, 0
    out, lse = p.run()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


# --------------------------------------------------------------------- sizes

@pytest.mark.parametrize("hq,hkv", [(72, 1), (128, 1), (256, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_many_heads(hq, hkv, d):
    # more than two passes over the keys, short rows and cut ones
    for keys in ([90, 0, 130], [2500, 1, 700]):
        s = Step(hq + d, keys, [1] * 3, hq, hkv, d, torch.bfloat16)
        out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
        s.check(out, lse)
    q, k, v, phys = selected_case(hq, 4, 900, hq, hkv, d, torch.float16)
    out, lse = dsa.attn_selected(q, k, v, phys)
    check_selected(q, k, v, phys, out, lse, torch.float16)


@pytest.mark.parametrize("hq,hkv", [(6, 2), (24, 1), (40, 1)])
def test_decode_several_long_tokens_per_request(hq, hkv):
    s = Step(51, [3000, 700, 1900], [4, 1, 7], hq, hkv, 64, torch.bfloat16)
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    s.check(out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_selected_for_the_tokens_of_a_prompt(dtype):
    # a row per prompt token; rows sampled over the whole length
    tokens, topk = 4099, 520
    q, k, v, phys = selected_case(52, tokens, topk, 8, 2, 128, dtype)
    phys[tokens - 1] = -1
    err = i32([0])
    out, lse = dsa.attn_selected(q, k, v, phys, dev_err=err)
    assert int(err.item()) == 0 and bool(torch.isfinite(out).all())
    rows = [0, 1, 303, 304, 1023, 2048, 2049, 3333, 4097, 4098]
    check_selected(q[rows], k, v, phys[rows], out[rows], lse[rows], dtype)
    again, _ = dsa.attn_selected(q, k, v, phys)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [64, 128])
def test_large_values(d):
    # O is summed before it is divided: with bf16, |v| < 2^98 / ceil(keys / 128) is
    # finite (here 2^96). The scores rise by 20 powers of two, so that weights get large.
    n = 500
    p = Prompts(53, [n], [n], 2, 1, d, torch.bfloat16, True)
    top = 20 * math.log(2) * d ** 0.5 / d
    p.q = torch.ones_like(p.q)
    up = (torch.arange(n, device=DEV) / n * top)[:, None, None].expand(n, 1, d).to(p.dtype)
    big = (p.vf[0].float().clamp(-2, 2) * 2.0 ** 94).to(p.dtype)
    for j in range(0, n, 64):
        page = p.bt[0][j // 64]
        p.k[page, :min(64, n - j)], p.v[page, :min(64, n - j)] = up[j:j + 64], big[j:j + 64]
    p.kf[0], p.vf[0] = up, big
    out, lse = p.run()
    p.check(out, lse)
    b = dsa.Batch(i32([0, 1]), i32([n]), i32(p.bt), i32([0]), 1, p.batch.num_blocks)
    rows, rlse = dsa.attn_decode(b, p.q[-1:].contiguous(), p.k, p.v)
    for e in range(2):
        check(rows[0, e], rlse[0, e], attend(p.q[-1, e], up[:, 0], big[:, 0], d ** -0.5, p.dtype))
