"""Attention over the 8-bit cache where V's scales of one row lie as far apart as the
writer makes them: every key keeps its share of the sum."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import check
from tests.kv8_ref import attend, value
from tests.test_gpu_attn_rows8 import DEV, Step8, check_lists, i32

pytestmark = pytest.mark.gpu


def spread(s, seed, low, high, zeros):
    """V's scales of a Step8: half of the blocks 2^-64 with codes of 0 (rows of zeros, as they are written), the
    others 2^low to 2^high; zeros: with codes of 0 above 2^2."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    none = torch.isnan(s.sc[..., 1])
    least = torch.rand(none.shape, generator=g, device=DEV) < 0.5
    e = torch.randint(low, high + 1, none.shape, generator=g, device=DEV).float()
    s.sc[..., 1] = torch.where(none, s.sc[..., 1], torch.where(least, 2.0 ** -64, torch.exp2(e)))
    gone = (least | (e > 2) if zeros else least).repeat_interleave(16, 1)[..., None].expand(s.v.shape)
    gone = gone & ~torch.isnan(s.v.float())
    s.v.view(torch.uint8)[gone] = 0


@pytest.mark.parametrize("low,high", [(72, 80), (60, 112), (105, 112), (-64, 112)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 4, 2), (64, 3, 3), (128, 24, 2), (64, 24, 2)])
@pytest.mark.parametrize("keys", [[40, 200], [3000, 70], [6000, 129, 700]])
def test_sum_over_values_of_far_scales(keys, d, hq, hkv, low, high):
    s = Step8(hq + d + high, keys, [1] * len(keys), hq, hkv, d, torch.bfloat16)
    spread(s, high, low, high, False)
    s.check(*s.run())
    phys = torch.full((len(keys), max(keys)), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate(keys):
        phys[r, :n] = torch.tensor(s.slots(r, n), dtype=torch.int32, device=DEV)
    s.check(*dsa.attn_selected8(s.q, s.k, s.v, s.sc, phys))


@pytest.mark.parametrize("low,high", [(72, 80), (105, 112), (-64, 112)])
@pytest.mark.parametrize("d", [64, 128])
def test_sum_split_over_the_length(d, low, high):
    # many slices of one token
    s = Step8(d + high, [50000], [1], 4, 2, d, torch.bfloat16)
    spread(s, high, low, high, False)
    s.check(*s.run())


@pytest.mark.parametrize("keys", [[200], [3000], [50000]])
def test_sum_whose_scales_rise_and_fall(keys):
    # from block to block ever larger, or ever smaller
    for sign in (1, -1):
        s = Step8(1, keys, [1], 8, 1, 64, torch.bfloat16)
        at = torch.tensor(s.slots(0, keys[0]), device=DEV)
        e = torch.linspace(-64, 112, keys[0], device=DEV).floor()
        s.sc[at // 64, at % 64 // 16, 0, 1] = torch.exp2(e if sign > 0 else e.flip(0))
        s.check(*s.run())
        s.check(*dsa.attn_selected8(s.q, s.k, s.v, s.sc, at.to(torch.int32)[None]))


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 16, 1)])
@pytest.mark.parametrize("keys", [[200], [3000], [20000]])
def test_sum_with_fp16_rows(keys, d, hq, hkv):
    # scales that an earlier, larger row has left behind: the codes there are 0
    s = Step8(hq + d, keys, [1], hq, hkv, d, torch.float16)
    spread(s, 5, -8, 112, True)
    s.check(*s.run())


def test_written_zeros_beside_large_values():
    # as the cache's writer leaves them: 32 rows of zeros, 32 of 2^90
    d = 64
    k, v, sc = dsa.new_kv_cache8(1, 1, d)
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.randn((64, 1, d), generator=g, device=DEV).to(torch.bfloat16)
    big = torch.where(torch.arange(64, device=DEV)[:, None, None] < 32, 0.0, 2.0 ** 90).to(torch.bfloat16)
    dsa.kv_write8(rows, big.expand(64, 1, d).contiguous(), torch.arange(64, device=DEV), k, v, sc)
    q = torch.zeros((1, 2, d), dtype=torch.bfloat16, device=DEV)   # every key counts alike
    batch = dsa.Batch(i32([0, 1]), i32([64]), i32([[0]]), i32([0]), 1, 1)
    out, lse = dsa.attn_decode8(batch, q, k, v, sc)
    assert bool((lse - math.log(64)).abs().max() < 1e-4)
    assert bool((out.float() == 2.0 ** 89).all())
    check_lists(q, k, v, sc, [torch.arange(64, device=DEV)], out, lse, torch.bfloat16, d ** -0.5)


@pytest.mark.parametrize("gap", [20.0, 45.0, 60.0, 75.0])
@pytest.mark.parametrize("keys", [100, 4000, 30000])
def test_scales_and_scores_far_apart(keys, gap):
    # the keys of V's least scales score e^gap above those of the largest: they may count as 2^-96 of these
    s = Step8(3, [keys], [1], 4, 1, 64, torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(4)
    at = torch.tensor(s.slots(0, keys), device=DEV)
    big = torch.rand(s.sc.shape[:2], generator=g, device=DEV) < 0.3
    big[s.bt[0][0], 0], big[s.bt[0][0], 1] = False, True
    s.q = torch.ones_like(s.q)
    ones = torch.ones((keys, 1, 64), device=DEV) * (1 - 2 * big[at // 64, at % 64 // 16].float())[:, None, None]
    s.k[at // 64, at % 64] = ones.to(torch.float8_e4m3fn)
    s.sc[at // 64, at % 64 // 16, :, 0] = 2.0 ** -3   # scores of 8 and -8, times scale
    s.sc[..., 1] = torch.where(torch.isnan(s.sc[..., 1]), s.sc[..., 1], torch.where(big, 2.0 ** 112, 2.0 ** -64)[..., None])
    scale = gap / 16
    out, lse = s.run(scale=scale)
    kk, vv = (value(c, s.sc[..., i]).flatten(0, 1)[at, 0] for i, c in enumerate((s.k, s.v)))
    sv = s.sc[..., 1].repeat_interleave(16, 1).flatten(0, 1)[at, 0]
    for e in range(4):
        ref, want, tol, ltol = attend(s.q[0, e], kk, vv, sv, scale, torch.bfloat16)
        check(out[0, e], lse[0, e], (ref, want, tol + 448 * 2.0 ** (112 - 96), ltol), f"head {e}")


@pytest.mark.parametrize("below", [10.2, 10.5, 11.0, 12.0, 14.0])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 2, 1), (64, 12, 1), (128, 12, 1)])
def test_small_share_of_keys_without_a_weight(d, hq, hkv, below):
    # 64 keys of V = 1 and 64 of zeros (the least scale), whose scores are 2^-below of the others': a share that
    # is the result's distance from 1. Every weight is a power of two, so that nothing else is rounded but scores of
    # the zeros (2^-19 of their share, which is 2^-10 at most) and the result
    k, v, sc = dsa.new_kv_cache8(2, hkv, d)
    k[1], v[0] = (torch.full((64, hkv, d), x, device=DEV).to(k.dtype) for x in (-1.0, 64.0))
    sc[..., 0] = 1.0
    sc[0, :, :, 1], sc[1, :, :, 1] = 2.0 ** -6, 2.0 ** -64
    q = torch.ones((1, hq, d), dtype=torch.float16, device=DEV)
    batch = dsa.Batch(i32([0, 1]), i32([128]), i32([[0, 1]]), i32([0]), 1, 2)
    slots = torch.arange(128, dtype=torch.int32, device=DEV)[None]
    scale = below * math.log(2) / d
    want = 1 / (1 + 2.0 ** -below)
    for out, _ in (dsa.attn_decode8(batch, q, k, v, sc, scale=scale),
                   dsa.attn_selected8(q, k, v, sc, slots, scale=scale)):
        assert float((out.double() - want).abs().max()) <= 2.0 ** -12 + 2.0 ** -20
