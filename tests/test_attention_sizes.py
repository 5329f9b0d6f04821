"""The longest rows that the calls over single query rows take, and those that they
refuse."""
import ctypes
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from dsa_sparse_attention_quant_gb300 import binding
from tests import test_attention_cpu as in16
from tests import test_kv8_cpu as in8
from tests.test_attention_cpu import EINVAL, batch, no_gpu

DEV = "cuda"
MOST = 2 ** 31 - 1


def test_more_tiles_than_are_counted_are_refused():
    lib = binding.load()
    # 512 tokens of 2^22 pages each are 2^31 tiles
    long = dict(num_reqs=512, num_decodes=512, num_tokens=512, num_decode_tokens=512, bt_stride=1 << 22,
                max_seq_len=1 << 28)
    for call in (in16.decode, in8.decode):
        assert call(b=batch(**long)) == EINVAL
        assert call(b=batch(**{**long, "max_seq_len": (1 << 28) - 63})) == EINVAL
    for size in (lib.dsa_attn_decode_workspace_size, lib.dsa_attn_decode8_workspace_size):
        assert size(ctypes.byref(batch(**long)), 8, 2, 128) == 0
        assert size(ctypes.byref(batch(**{**long, "max_seq_len": (1 << 28) - 64})), 8, 2, 128) > 0
    for call in (in16.selected, in8.selected):
        assert call(n=MOST, topk=65) == EINVAL and call(n=1 << 16, topk=MOST) == EINVAL
    for size in (lib.dsa_attn_selected_workspace_size, lib.dsa_attn_selected8_workspace_size):
        assert size(1 << 30, 65, 8, 2, 128) == 0 and size((1 << 30) - 1, 65, 8, 2, 128) > 0
        assert size(64, MOST, 8, 2, 128) == 0 and size(63, MOST, 8, 2, 128) > 0


@no_gpu
def test_the_longest_rows_are_taken():
    one = batch(num_decodes=1, num_decode_tokens=1, num_tokens=1, bt_stride=1 << 25, max_seq_len=MOST)
    for m in (in16, in8):
        assert m.decode(b=one) == binding.DSA_ENODEV and m.selected(n=3, topk=MOST) == binding.DSA_ENODEV


def cache(bits, g):
    """A page of 64 slots, one head of 64: (caches, K and V in 64 bits [64, 64])."""
    x = torch.randn((2, 1, 64, 1, 64), generator=g, device=DEV)
    if bits == 16:
        k, v = x.to(torch.bfloat16)
        return (k, v), (k[0, :, 0].double(), v[0, :, 0].double())
    k, v = (90 * x).clamp(-448, 448).to(torch.float8_e4m3fn)
    sc = torch.full((1, 4, 1, 2), 2.0 ** -6, device=DEV)
    return (k, v, sc), tuple(c[0, :, 0].float().double() * 2.0 ** -6 for c in (k, v))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [16, 8])
def test_selected_row_of_the_greatest_length(bits):
    # a list of 2^31 - 1 entries, all but a few of them -1
    g = torch.Generator(device=DEV).manual_seed(1)
    args, (k, v) = cache(bits, g)
    phys = torch.full((1, MOST), -1, dtype=torch.int32, device=DEV)
    at = {0: 5, 1 << 20: 7, MOST - 64: 11, MOST - 63: 30, MOST - 1: 63}
    for i, slot in at.items():
        phys[0, i] = slot
    q = torch.randn((1, 4, 64), generator=g, device=DEV).to(torch.bfloat16)
    out, lse = (dsa.attn_selected if bits == 16 else dsa.attn_selected8)(q, *args, phys)
    slots = torch.tensor(list(at.values()), device=DEV)
    s = q[0].double() @ k[slots].T / 8
    want = torch.softmax(s, 1) @ v[slots]
    # weights and result are rounded to bf16 (8 bits: weights to fp16): 2^-8 of sum p |v| each, and little besides
    assert bool(((out[0].double() - want).abs() <= 2.0 ** -6.9 * (torch.softmax(s, 1) @ v[slots].abs())).all())
    assert bool(((lse[0].double() - torch.logsumexp(s, 1)).abs() <= 2.0 ** -14 * (1 + s.abs().amax())).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [16, 8])
def test_decode_row_of_the_greatest_length(bits):
    # 2^31 - 1 keys: one page, 2^25 times
    g = torch.Generator(device=DEV).manual_seed(2)
    args, (k, v) = cache(bits, g)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.zeros((1, 1 << 25), dtype=torch.int32, device=DEV)
    b = dsa.Batch(i32([0, 1]), i32([MOST]), table, i32([0]), 1, 1, max_seq_len=MOST)
    q = torch.randn((1, 4, 64), generator=g, device=DEV).to(torch.bfloat16)
    out, lse = (dsa.attn_decode if bits == 16 else dsa.attn_decode8)(b, q, *args)
    s = q[0].double() @ k.T / 8
    want = torch.softmax(s, 1) @ v
    # a thread's fp32 sum of 2^31 / 2^6 / 300 / 2 keys or so, off by half a step at each: 2^-24 * 2^17 at most, and
    # the sums of 2^16 tiles in the MMAs, truncated: 2^-23 * 2^18
    mean = torch.softmax(s, 1) @ v.abs()
    assert bool(((out[0].double() - want).abs() <= (2.0 ** -5 + 2.0 ** -6.9 + 2.0 ** -7) * mean).all())
    assert bool(((lse[0].double() - torch.logsumexp(s, 1) - math.log(MOST / 64)).abs() <= 2.0 ** -6).all())


@pytest.mark.gpu
def test_prompt_behind_a_context_of_the_greatest_length():
    # 2^31 - 128 keys are the most that are read; a longer sequence is flagged and its rows are empty
    g = torch.Generator(device=DEV).manual_seed(3)
    args, _ = cache(16, g)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.zeros((2, 1 << 25), dtype=torch.int32, device=DEV)
    q = torch.randn((3, 4, 64), generator=g, device=DEV).to(torch.bfloat16)
    for n in (MOST, MOST - 126):
        b = dsa.Batch(i32([0, 2, 3]), i32([n, 5]), table, i32([0, 0, 1]), 0, 1, max_seq_len=MOST)
        err = i32([0])
        out, lse = dsa.attn_prompt(b, q, *args, dev_err=err)
        assert int(err.item()) == 16
        assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
        assert bool(torch.isfinite(lse[2]).all())
