"""Attention of single query rows over the 8-bit cache, against plain attention in
64 bits over what its codes and scales stand for: the decode tokens over their
pages, any token over selected slots."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import check
from tests.kv8_ref import F8, attend, value
from tests.test_gpu_kv8_cache import cache8

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALES = (-8, -3)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def codes(g, *shape):
    return (90 * torch.randn(shape, generator=g, device=DEV)).clamp(-448, 448).to(F8)


class Step8:
    """Decode requests of given key counts and query lengths over shuffled pages; every
    slot that holds no key has NaN codes, every block without one a NaN scale."""

    def __init__(self, seed, keys, qlens, hq, hkv, d, dtype, layout="pages", max_seq_len=None, scales=SCALES):
        g = torch.Generator(device=DEV).manual_seed(seed)
        need = [(n + 63) // 64 for n in keys]
        blocks = sum(need) + 2
        perm = torch.randperm(blocks, generator=g, device=DEV).tolist()
        bt = [[-7] * max(need + [1]) for _ in keys]   # entries behind a row's pages are never read
        self.k, self.v, self.sc = cache8(g, blocks, hkv, d, layout, filled=False)
        for c in (self.k, self.v):
            c.copy_(torch.full(c.shape, math.nan, device=DEV).to(F8))
        self.sc.fill_(math.nan)
        for r, n in enumerate(keys):
            for j in range(need[r]):
                p = perm.pop()
                bt[r][j] = p
                m = min(64, n - 64 * j)
                self.k[p, :m], self.v[p, :m] = codes(g, m, hkv, d), codes(g, m, hkv, d)
                b = (m + 15) // 16
                self.sc[p, :b] = 2.0 ** torch.randint(*scales, (b, hkv, 2), generator=g, device=DEV).float()
        self.bt = bt
        qsl = [0]
        for n in qlens:
            qsl.append(qsl[-1] + n)
        req = [r for r, n in enumerate(qlens) for _ in range(n)]
        self.batch = dsa.Batch(i32(qsl), i32(keys), i32(bt), i32(req), len(keys), blocks,
                               max_seq_len=max_seq_len or max(max(keys), 1), num_decode_tokens=qsl[-1])
        self.rows = [(r, max(0, keys[r] - qlens[r] + i + 1)) for r in range(len(keys)) for i in range(qlens[r])]
        self.q = torch.randn((qsl[-1], hq, d), generator=g, device=DEV).to(dtype)
        self.g, self.scale, self.dtype = hq // hkv, d ** -0.5, dtype

    def slots(self, r, n):
        return [self.bt[r][j // 64] * 64 + j % 64 for j in range(n)]

    def run(self, **kw):
        return dsa.attn_decode8(self.batch, self.q, self.k, self.v, self.sc, **kw)

    def check(self, out, lse, scale=None, only=None):
        lists = {r: torch.tensor(self.slots(r, max(n for q, n in self.rows if q == r)), dtype=torch.int64, device=DEV)
                 for r in {r for r, _ in self.rows}}
        check_lists(self.q, self.k, self.v, self.sc, [lists[r][:n] for r, n in self.rows], out, lse, self.dtype,
                    scale or self.scale, only)


def check_lists(q, k, v, sc, lists, out, lse, dtype, scale, only=None):
    """Rows of q against plain attention over these slots each."""
    k, v = (value(c, sc[..., i]).flatten(0, 1) for i, c in enumerate((k, v)))
    sv = sc[..., 1].repeat_interleave(16, 1).flatten(0, 1)
    grp = q.shape[1] // k.shape[1]
    for t in range(q.shape[0]) if only is None else only:
        at = lists[t]
        kk, vv, ss = k[at], v[at], sv[at]
        for e in range(q.shape[1]):
            h = e // grp
            check(out[t, e], lse[t, e], attend(q[t, e], kk[:, h], vv[:, h], ss[:, h], scale, dtype),
                  f"token {t} ({len(at)} keys) head {e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (16, 2), (7, 1), (32, 2), (20, 1), (40, 1), (6, 3), (40, 2)])
def test_decode_lengths_and_groups(dtype, d, hq, hkv):
    s = Step8(hq + d, [1, 0, 15, 16, 17, 64, 65, 300], [1] * 8, hq, hkv, d, dtype)
    err = i32([0])
    out, lse = s.run(dev_err=err)
    s.check(out, lse)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (24, 2), (24, 1), (16, 2), (9, 3)])
def test_decode_split_over_the_length(dtype, d, hq, hkv):
    s = Step8(7 * hq + d, [5000, 1, 0, 777, 64, 2049], [1] * 6, hq, hkv, d, dtype)
    err = i32([0])
    out, lse = s.run(dev_err=err)
    s.check(out, lse)
    assert int(err.item()) == 0
    # the same bits again, and with scratch full of NaN
    ws = torch.full((dsa.attn_decode8_workspace_size(s.batch, hq, hkv, d),), 255, dtype=torch.uint8, device=DEV)
    out2, lse2 = s.run(ws=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "joined", "loose"])
@pytest.mark.parametrize("keys", [[300, 64, 129], [3000, 64, 129], [6000, 64, 129]])
def test_decode_cache_layouts_and_strided_rows(layout, keys, d):
    s = Step8(3, keys, [1, 1, 1], 8, 2, d, torch.bfloat16, layout)
    wide = torch.zeros((3, 9, 200), dtype=torch.bfloat16, device=DEV)   # q and out as views of wider tensors
    q = wide[:, 1:, 8:8 + d]
    q.copy_(s.q)
    obuf = torch.full((3, 8, 160), 5.0, dtype=torch.bfloat16, device=DEV)
    out, lse = dsa.attn_decode8(s.batch, q, s.k, s.v, s.sc, out=obuf[:, :, 16:16 + d])
    s.check(out, lse)
    assert bool((obuf[:, :, :16] == 5).all()) and bool((obuf[:, :, 16 + d:] == 5).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1), (12, 1), (40, 2), (9, 3)])
@pytest.mark.parametrize("keys", [[257], [1000, 70, 0], [4096], [520, 1, 3000, 64, 2]])
def test_decode_tokens_that_clusters_share(dtype, d, hq, hkv, keys):
    s = Step8(hq + d + len(keys), keys, [1] * len(keys), hq, hkv, d, dtype)
    err = i32([0])
    out, lse = s.run(dev_err=err)
    s.check(out, lse)
    assert int(err.item()) == 0
    out2, lse2 = s.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_decode_several_tokens_per_request_and_padding():
    s = Step8(11, [700, 2, 65, 0], [3, 4, 2, 1], 8, 4, 64, torch.bfloat16)
    s.check(*s.run())


def test_decode_many_short_requests():
    s = Step8(12, [(37 * i) % 200 for i in range(300)], [1] * 300, 4, 2, 64, torch.float16, max_seq_len=3000)
    s.check(*s.run())


def test_decode_more_tokens_than_one_count():
    keys = [(53 * i) % 170 for i in range(900)]
    keys[17], keys[450], keys[899] = 5000, 0, 2100
    s = Step8(22, keys, [1 + i % 3 for i in range(900)], 2, 1, 64, torch.bfloat16)
    out, lse = s.run()
    s.check(out, lse, only=range(0, 1800, 7))
    t = [i for i, (r, _) in enumerate(s.rows) if r in (17, 450, 899)]
    s.check(out, lse, only=t)


def test_decode_rows_behind_stay_and_scale():
    s = Step8(13, [100, 600], [1, 1], 4, 1, 128, torch.float16)
    q = torch.cat([s.q, s.q])
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device=DEV)
    dsa.attn_decode8(s.batch, q, s.k, s.v, s.sc, scale=0.25, out=out, lse=lse)
    s.check(out[:2], lse[:2], 0.25)
    assert bool((out[2:] == 3).all()) and bool((lse[2:] == 3).all())
    out, lse = dsa.attn_decode8(s.batch, q, s.k, s.v, s.sc)
    assert bool((out[2:] == 0).all()) and bool((lse[2:] == -math.inf).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decode_result_over_q(dtype):
    s = Step8(19, [3000, 70], [1, 1], 16, 2, 64, dtype)
    q = s.q.clone()
    out, lse = dsa.attn_decode8(s.batch, q, s.k, s.v, s.sc, out=q)
    s.check(out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("factor", [2.0 ** -14, 16.0, 300.0])
def test_decode_sizes_of_q(dtype, factor):
    # scores of several hundred: the reference moves, weights underflow; rows of q near the type's ends
    s = Step8(14, [900, 70], [1, 1], 4, 2, 128, dtype)
    s.q = s.q * factor
    s.check(*s.run())


def test_decode_bf16_rows_far_from_fp16():
    for e in (-120, -60, 60, 100):
        up = max(-60, min(60, e))
        s = Step8(15, [300], [1], 4, 2, 64, torch.bfloat16, scales=(-up - 8, -up - 3))
        s.q = s.q * 2.0 ** e
        s.q[0, 1, 5] = 0.0
        s.q[0, 2] = 0.0
        s.sc[..., 1] = torch.where(torch.isnan(s.sc[..., 1]), s.sc[..., 1], 2.0 ** -6)
        s.check(*s.run(scale=1e-3), scale=1e-3)


@pytest.mark.parametrize("spread", [(-8, -3), (-40, 20), (-64, -30), (30, 100)])
@pytest.mark.parametrize("keys", [200, 3000, 6000])
def test_decode_values_of_uneven_scales(spread, keys):
    # V's scales far apart: the largest weight times scale leads, the sum does not
    s = Step8(20, [keys], [1], 8, 2, 64, torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(1)
    s.sc[..., 1] = torch.where(torch.isnan(s.sc[..., 1]), s.sc[..., 1],
                               2.0 ** torch.randint(*spread, s.sc.shape[:-1], generator=g, device=DEV).float())
    s.check(*s.run())


def test_decode_scales_that_are_no_powers_of_two():
    s = Step8(21, [900, 40], [1, 1], 8, 2, 128, torch.float16)
    g = torch.Generator(device=DEV).manual_seed(1)
    s.sc *= 1 + torch.rand(s.sc.shape, generator=g, device=DEV)
    s.check(*s.run())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decode_growing_scores_rescale(dtype):
    # later keys score ever higher, so the reference moves in most tiles
    s = Step8(15, [1500], [1], 2, 1, 64, dtype)
    s.q = torch.ones_like(s.q)
    for j in range(1500):
        p = s.bt[0][j // 64]
        s.k[p, j % 64] = 1.0
        s.sc[p, j % 64 // 16, :, 0] = j // 16 * 16 / 64
    s.sc[..., 0].clamp_(min=2.0 ** -10)
    s.check(*s.run())


def test_decode_zeroed_cache():
    # codes and scales as they are made: every value is 0
    k, v, sc = dsa.new_kv_cache8(3, 2, 64)
    batch = dsa.Batch(i32([0, 1]), i32([150]), i32([[2, 0, 1]]), i32([0]), 1, 3)
    q = torch.randn((1, 8, 64), device=DEV).to(torch.bfloat16)
    out, lse = dsa.attn_decode8(batch, q, k, v, sc)
    assert bool((out == 0).all()) and bool(((lse - math.log(150)).abs() < 1e-5).all())


@pytest.mark.parametrize("keys", [300, 3000, 5000])
def test_visible_nan_stays_in_its_rows(keys):
    s = Step8(16, [keys, 300], [1, 1], 4, 2, 64, torch.bfloat16)
    at = torch.tensor(s.slots(0, keys), dtype=torch.int32, device=DEV)
    phys = torch.full((2, keys), -1, dtype=torch.int32, device=DEV)
    phys[0] = at
    phys[1, :300] = torch.tensor(s.slots(1, 300), dtype=torch.int32, device=DEV)

    def both():
        yield s.run()
        yield dsa.attn_selected8(s.q, s.k, s.v, s.sc, phys)

    page = s.bt[0][1]
    s.v[page, 3, 0, 5] = math.nan
    for out, lse in both():
        bad = torch.isnan(out)
        assert bool(bad[0, :2, 5].all()) and int(bad.sum()) == 2 and not bool(torch.isnan(lse).any())
    s.k[page, 3, 0, 5] = math.nan
    for out, lse in both():
        assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isnan(lse[0, :2]).all())
        assert not bool(torch.isnan(out[0, 2:]).any()) and not bool(torch.isnan(out[1]).any())
    s.q[1, 3, 7] = math.inf
    for out, lse in both():
        assert not bool(torch.isfinite(out[1, 3]).any()) and bool(torch.isfinite(out[1, :3]).all())


def test_decode_bad_metadata_is_flagged():
    s = Step8(17, [100, 200, 300], [1, 1, 1], 4, 2, 64, torch.bfloat16)
    err = i32([0])
    s.batch.block_table[1, 2] = 10 ** 6   # outside the cache: the page's keys are left out
    out, lse = s.run(dev_err=err)
    assert int(err.item()) == 2
    lists = [torch.tensor([x for j, x in enumerate(s.slots(r, n)) if (r, j // 64) != (1, 2)], device=DEV)
             for r, n in s.rows]
    check_lists(s.q, s.k, s.v, s.sc, lists, out, lse, s.dtype, s.scale)
    for bad in (-1, 301):
        err.zero_()
        s.batch.seq_lens[0] = bad
        out, lse = s.run(dev_err=err)
        assert int(err.item()) & 16
        assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    s.batch.seq_lens[0] = 100
    err.zero_()
    s.batch.req_id_per_token[2] = 9
    out, lse = s.run(dev_err=err)
    assert int(err.item()) & 16 and bool((lse[2] == -math.inf).all())


# ------------------------------------------------------------------- selected

def selected_case(seed, tokens, topk, hq, hkv, d, dtype, blocks=40, none=0.2, layout="pages"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k, v, sc = cache8(g, blocks, hkv, d, layout)
    n = blocks * 64
    ids = (torch.rand(n, generator=g, device=DEV) < 0.7).nonzero()[:, 0]
    gone = torch.ones(n, dtype=torch.bool, device=DEV)
    gone[ids] = False
    gone = gone.nonzero()[:, 0]          # the other slots are NaN
    for c in (k, v):
        c[gone // 64, gone % 64] = torch.full((gone.numel(), hkv, d), math.nan, device=DEV).to(F8)
    pick = torch.randint(0, ids.numel(), (tokens, topk), generator=g, device=DEV)
    phys = ids[pick].to(torch.int32)
    phys[torch.rand((tokens, topk), generator=g, device=DEV) < none] = -1
    q = torch.randn((tokens, hq, d), generator=g, device=DEV).to(dtype)
    return q, k, v, sc, phys


def check_selected(q, k, v, sc, phys, out, lse, dtype):
    check_lists(q, k, v, sc, [p[p >= 0].long() for p in phys], out, lse, dtype, q.shape[2] ** -0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,topk,hq,hkv", [(3, 1, 4, 2), (2, 37, 8, 8), (5, 512, 24, 2), (3, 1030, 33, 1),
                                                (70, 600, 6, 2), (9, 300, 16, 16), (2, 2048, 40, 8)])
def test_selected_shapes(dtype, d, tokens, topk, hq, hkv):
    q, k, v, sc, phys = selected_case(tokens + topk, tokens, topk, hq, hkv, d, dtype)
    phys[1] = -1                       # a token with nothing selected
    if topk > 100:
        phys[0, 50:] = -1              # a short row's tail
    err = i32([0])
    out, lse = dsa.attn_selected8(q, k, v, sc, phys, dev_err=err)
    check_selected(q, k, v, sc, phys, out, lse, dtype)
    assert int(err.item()) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 4), (36, 4), (80, 4), (6, 6)])
@pytest.mark.parametrize("layout", ["pages", "heads", "joined", "loose"])
def test_selected_layouts_and_bad_slots(layout, hq, hkv, d):
    q, k, v, sc, phys = selected_case(5, 4, 900, hq, hkv, d, torch.bfloat16, layout=layout)
    bad = phys.clone()
    bad[2, 10], bad[2, 11], bad[3, 899] = 40 * 64, -2, 2 ** 31 - 1
    err = i32([0])
    out, lse = dsa.attn_selected8(q, k, v, sc, bad, dev_err=err)
    assert int(err.item()) == 4
    bad[2, 10] = bad[2, 11] = bad[3, 899] = -1
    check_selected(q, k, v, sc, bad, out, lse, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 4), (64, 16, 4), (64, 3, 3), (64, 24, 2), (128, 40, 2)])
def test_selected_slots_far_apart(dtype, d, hq, hkv):
    # K's pages are 8 MB apart, so that windows of the lists are brought into the cache's order
    tokens, topk, blocks = 150, 2500, 40
    q, k, v, sc, phys = selected_case(d + hq, tokens, topk, hq, hkv, d, dtype, blocks=blocks)
    far = torch.zeros(blocks << 23, dtype=torch.uint8, device=DEV).view(F8)
    far = torch.as_strided(far, k.shape, (1 << 23, hkv * d, d, 1))
    far.copy_(k)
    phys[1] = -1
    phys[2, 700:] = -1
    phys[3] = phys[3].clamp(max=64 * 8)      # many keys in the first stretch
    phys[4] = phys[4, :1]                    # one slot, or none
    phys[5] = phys[5].sort().values
    phys[3:6] = torch.where(torch.isin(phys[3:6], phys[:3]), phys[3:6], -1)  # (slots that hold a key)
    err = i32([0])
    out, lse = dsa.attn_selected8(q, far, v, sc, phys, dev_err=err)
    assert int(err.item()) == 0
    check_lists(q, k, v, sc, [p[p >= 0].long() for p in phys], out, lse, dtype, d ** -0.5,
                only=[0, 1, 2, 3, 4, 5, 77, 149])
    out2, lse2 = dsa.attn_selected8(q, far, v, sc, phys)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    bad = phys.clone()
    bad[7, 2400], bad[8, 1300], bad[9, 2499] = blocks * 64, -2, 2 ** 31 - 1
    out, lse = dsa.attn_selected8(q, far, v, sc, bad, dev_err=err)
    assert int(err.item()) == 4
    bad[7, 2400] = bad[8, 1300] = bad[9, 2499] = -1
    check_lists(q, k, v, sc, [p[p >= 0].long() for p in bad], out, lse, dtype, d ** -0.5, only=[7, 8, 9])


def test_selected_all_slots_is_decode():
    s = Step8(21, [700, 90], [1, 1], 8, 2, 128, torch.bfloat16)
    phys = torch.full((2, 704), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate([700, 90]):
        phys[r, :n] = torch.tensor(s.slots(r, n), dtype=torch.int32, device=DEV)
    s.check(*dsa.attn_selected8(s.q, s.k, s.v, s.sc, phys))


def test_rows_beyond_32_bit_offsets():
    # a cache of more than 2^32 codes: its last page is read there
    blocks, hkv, d = (1 << 32) // (64 * 8 * 128) + 3, 8, 128
    k, v, sc = dsa.new_kv_cache8(blocks, hkv, d)
    g = torch.Generator(device=DEV).manual_seed(2)
    slots = torch.arange((blocks - 1) * 64, blocks * 64, device=DEV)
    for c in (k, v):
        c[blocks - 1] = codes(g, 64, hkv, d)
    sc[blocks - 1] = 2.0 ** -6
    q = torch.randn((1, 16, d), generator=g, device=DEV).to(torch.bfloat16)
    batch = dsa.Batch(i32([0, 1]), i32([64]), i32([[blocks - 1]]), i32([0]), 1, blocks)
    last = (k[blocks - 1:], v[blocks - 1:], sc[blocks - 1:])
    phys = slots.to(torch.int32)[None]
    for out, lse in (dsa.attn_selected8(q, k, v, sc, phys), dsa.attn_decode8(batch, q, k, v, sc)):
        check_lists(q, *last, [torch.arange(64, device=DEV)], out, lse, torch.bfloat16, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 2])
def test_cache_of_one_page(d, hkv):
    # the page's stride is nothing's, the only head's neither
    g = torch.Generator(device=DEV).manual_seed(31)
    codes_of = codes(g, 64, hkv, d)
    k, v = (torch.as_strided(codes_of, (1, 64, hkv, d), (1, hkv * d, 3 if hkv == 1 else d, 1)) for _ in range(2))
    sc = torch.full((1, 4, hkv, 2), 2.0 ** -7, device=DEV)
    q = torch.randn((1, 4 * hkv, d), generator=g, device=DEV).to(torch.bfloat16)
    batch = dsa.Batch(i32([0, 1]), i32([50]), i32([[0]]), i32([0]), 1, 1)
    phys = torch.arange(50, dtype=torch.int32, device=DEV)[None]
    for out, lse in (dsa.attn_selected8(q, k, v, sc, phys), dsa.attn_decode8(batch, q, k, v, sc)):
        check_lists(q, k, v, sc, [torch.arange(50, device=DEV)], out, lse, torch.bfloat16, d ** -0.5)
    rows = [torch.randn((20, hkv, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    k, v = (torch.as_strided(torch.zeros((64, hkv, d), dtype=torch.uint8, device=DEV).view(F8), (1, 64, hkv, d),
                             (1, hkv * d, 3 if hkv == 1 else d, 1)) for _ in range(2))
    k2, v2, sc2 = dsa.new_kv_cache8(1, hkv, d)
    dsa.kv_write8(*rows, torch.arange(30, 50, device=DEV), k, v, sc)
    sc2.fill_(2.0 ** -7)
    dsa.kv_write8(*rows, torch.arange(30, 50, device=DEV), k2, v2, sc2)
    assert torch.equal(k.view(torch.uint8), k2.view(torch.uint8)) and torch.equal(sc, sc2)


# ----------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("keys", [3000, 7000])
def test_streams_and_captured_graphs(keys):
    s = Step8(30, [keys, 500, 77], [1] * 3, 16, 2, 128, torch.bfloat16)
    phys = torch.full((3, 900), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate([900, 500, 77]):
        phys[r, :n] = torch.tensor(s.slots(r, n), dtype=torch.int32, device=DEV)
    want = s.run(), dsa.attn_selected8(s.q, s.k, s.v, s.sc, phys)
    torch.cuda.synchronize()
    # two calls at once on two streams, each with its own scratch
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        got.append((s.run(stream=st), dsa.attn_selected8(s.q, s.k, s.v, s.sc, phys, stream=st)))
    torch.cuda.synchronize()
    for pair in got:
        for (o, l), (wo, wl) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    out, lse = torch.empty_like(s.q), torch.empty(s.q.shape[:2], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(out=out, lse=lse)
        sel = dsa.attn_selected8(s.q, s.k, s.v, s.sc, phys)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
    assert torch.equal(sel[0], want[1][0]) and torch.equal(sel[1], want[1][1])
