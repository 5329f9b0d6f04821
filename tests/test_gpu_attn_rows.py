"""Attention of single query rows over the paged cache, against plain attention
in 64 bits: the decode tokens over their pages, any token over selected slots."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import attend, check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def caches(gen, blocks, hkv, d, dtype, layout):
    """K and V [blocks, 64, hkv, d] filled with NaN, in one of several memory layouts."""
    if layout == "heads":      # [blocks, heads, 64, d]
        k, v = (torch.full((blocks, hkv, 64, d), math.nan, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2))
    elif layout == "joined":   # one allocation [blocks, 2, 64, heads, d + 8]
        both = torch.full((blocks, 2, 64, hkv, d + 8), math.nan, dtype=dtype, device=DEV)
        k, v = both[:, 0, :, :, 8:], both[:, 1, :, :, :d]
    else:
        k, v = (torch.full((blocks, 64, hkv, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    return k, v


class Step:
    """Decode requests of given key counts and query lengths over shuffled pages;
    every slot that holds no key is NaN."""

    def __init__(self, seed, keys, qlens, hq, hkv, d, dtype, layout="pages", max_seq_len=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        need = [(n + 63) // 64 for n in keys]
        blocks = sum(need) + 2
        perm = torch.randperm(blocks, generator=g, device=DEV).tolist()
        width = max(need + [1])
        bt = [[-7] * width for _ in keys]   # entries behind a row's pages are never read
        self.k, self.v = caches(g, blocks, hkv, d, dtype, layout)
        self.kf, self.vf = [], []
        at = 0
        for r, n in enumerate(keys):
            ids = perm[at:at + need[r]]
            at += need[r]
            bt[r][:need[r]] = ids
            k, v = (torch.randn((n, hkv, d), generator=g, device=DEV).to(dtype) for _ in range(2))
            for j, p in enumerate(ids):
                m = min(64, n - 64 * j)
                self.k[p, :m], self.v[p, :m] = k[64 * j:64 * j + m], v[64 * j:64 * j + m]
            self.kf.append(k)
            self.vf.append(v)
        qsl = [0]
        for n in qlens:
            qsl.append(qsl[-1] + n)
        req = [r for r, n in enumerate(qlens) for _ in range(n)]
        self.batch = dsa.Batch(i32(qsl), i32(keys), i32(bt), i32(req), len(keys), blocks,
                               max_seq_len=max_seq_len or max(max(keys), 1), num_decode_tokens=qsl[-1])
        self.rows = [(r, max(0, keys[r] - qlens[r] + i + 1)) for r in range(len(keys)) for i in range(qlens[r])]
        self.q = torch.randn((qsl[-1], hq, d), generator=g, device=DEV).to(dtype)
        self.g, self.scale, self.dtype = hq // hkv, d ** -0.5, dtype

    def check(self, out, lse, scale=None):
        for t, (r, n) in enumerate(self.rows):
            for e in range(self.q.shape[1]):
                h = e // self.g
                ref = attend(self.q[t, e], self.kf[r][:n, h], self.vf[r][:n, h], scale or self.scale, self.dtype)
                check(out[t, e], lse[t, e], ref, f"token {t} ({n} keys) head {e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (7, 1), (32, 2), (20, 1), (40, 1)])
def test_decode_lengths_and_groups(dtype, d, hq, hkv):
    s = Step(hq + d, [1, 0, 63, 64, 65, 130, 300], [1] * 7, hq, hkv, d, dtype)
    err = i32([0])
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v, dev_err=err)
    s.check(out, lse)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (16, 2), (24, 1)])
def test_decode_split_over_the_length(dtype, d, hq, hkv):
    s = Step(7 * hq + d, [5000, 1, 0, 777, 64, 2049], [1] * 6, hq, hkv, d, dtype)
    err = i32([0])
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v, dev_err=err)
    s.check(out, lse)
    assert int(err.item()) == 0
    # the same bits again, and with scratch full of NaN
    ws = torch.full((dsa.attn_decode_workspace_size(s.batch, hq, hkv, d),), 255, dtype=torch.uint8, device=DEV)
    out2, lse2 = dsa.attn_decode(s.batch, s.q, s.k, s.v, ws=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", ["heads", "joined"])
@pytest.mark.parametrize("keys", [[300, 64, 129], [3000, 64, 129]])
def test_decode_cache_layouts_and_strided_rows(layout, keys):
    s = Step(3, keys, [1, 1, 1], 8, 2, 128, torch.bfloat16, layout)
    # q and out as views of wider tensors
    wide = torch.zeros((3, 9, 200), dtype=torch.bfloat16, device=DEV)
    q = wide[:, 1:, 8:136]
    q.copy_(s.q)
    obuf = torch.full((3, 8, 160), 5.0, dtype=torch.bfloat16, device=DEV)
    out, lse = dsa.attn_decode(s.batch, q, s.k, s.v, out=obuf[:, :, 16:144])
    s.check(out, lse)
    assert bool((obuf[:, :, :16] == 5).all()) and bool((obuf[:, :, 144:] == 5).all())


def test_decode_several_tokens_per_request_and_padding():
    # query lengths above one; a request shorter than its query (its first rows see nothing)
    s = Step(11, [700, 2, 65, 0], [3, 4, 2, 1], 8, 4, 64, torch.bfloat16)
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    s.check(out, lse)


def test_decode_many_short_requests():
    keys = [(37 * i) % 200 for i in range(300)]
    s = Step(12, keys, [1] * 300, 4, 2, 64, torch.float16, max_seq_len=3000)
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    s.check(out, lse)


def test_batch_elsewhere_is_refused():
    s = Step(25, [100], [1], 2, 1, 64, torch.bfloat16)
    s.batch.seq_lens = s.batch.seq_lens.cpu()
    for call in (dsa.attn_decode, dsa.attn_prompt):
        with pytest.raises(dsa.DsaError, match="the batch"):
            call(s.batch, s.q, s.k, s.v)


def test_decode_more_tokens_than_one_count():
    # tokens are counted 512 at a time: long rows among short and empty ones
    keys = [(53 * i) % 170 for i in range(900)]
    keys[17], keys[450], keys[899] = 5000, 0, 2100
    s = Step(22, keys, [1 + i % 3 for i in range(900)], 2, 1, 64, torch.bfloat16)
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    s.check(out, lse)


def test_decode_half_a_million_rows():
    # more than 1024 counts of 512; the last three rows of a request see a key
    s = Step(23, [3] * 540, [1000] * 540, 1, 1, 64, torch.bfloat16)
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    out, lse = out.reshape(540, 1000, 64), lse.reshape(540, 1000)
    assert bool((out[:, :997] == 0).all()) and bool((lse[:, :997] == -math.inf).all())
    q, k, v = s.q.reshape(540, 1000, 64)[:, 997:].double(), torch.stack(s.kf)[:, :, 0].double(), \
        torch.stack(s.vf)[:, :, 0].double()
    score = (q @ k.transpose(1, 2) / 8).masked_fill(torch.ones(3, 3, device=DEV).triu(1).bool(), -math.inf)
    want = score.softmax(-1) @ v
    # weights and result in bf16: 2^-8 of max |v| each, and little else
    assert bool(((out[:, 997:].double() - want).abs() <= 2.1 * 2.0 ** -8 * v.abs().max()).all())
    assert bool(((lse[:, 997:].double() - score.logsumexp(-1)).abs() <= 1e-4).all())


def test_decode_rows_behind_stay_and_scale():
    s = Step(13, [100, 600], [1, 1], 4, 1, 128, torch.float16)
    q = torch.cat([s.q, s.q])
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 3.0, device=DEV)
    dsa.attn_decode(s.batch, q, s.k, s.v, scale=0.25, out=out, lse=lse)
    s.check(out[:2], lse[:2], 0.25)
    assert bool((out[2:] == 3).all()) and bool((lse[2:] == 3).all())


def test_decode_large_scores():
    # scores of several hundred: the running maximum moves, weights underflow
    s = Step(14, [900, 70], [1, 1], 4, 2, 128, torch.bfloat16)
    q = s.q * 16
    s.q = q
    out, lse = dsa.attn_decode(s.batch, q, s.k, s.v)
    s.check(out, lse)


def test_decode_growing_scores_rescale():
    # later keys score ever higher, so the reference moves in most tiles
    for dtype in (torch.bfloat16, torch.float16):
        s = Step(15, [1500], [1], 2, 1, 64, dtype)
        s.q = torch.ones_like(s.q)
        k = (torch.arange(1500, device=DEV)[:, None, None] / 64).expand(1500, 1, 64).to(dtype)
        s.kf[0] = k
        bt = s.batch.block_table[0].tolist()
        for j in range(0, 1500, 64):
            m = min(64, 1500 - j)
            s.k[bt[j // 64], :m] = k[j:j + m]
        out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
        s.check(out, lse)


def test_decode_visible_nan_stays_in_its_rows():
    s = Step(16, [300, 300], [1, 1], 4, 2, 64, torch.bfloat16)
    page = int(s.batch.block_table[0, 1])
    s.v[page, 3, 0, 5] = math.nan
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    bad = torch.isnan(out)
    assert bool(bad[0, :2, 5].all()) and int(bad.sum()) == 2
    s.k[page, 3, 0, 5] = math.nan
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v)
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isnan(lse[0, :2]).all())
    assert not bool(torch.isnan(out[0, 2:]).any()) and not bool(torch.isnan(out[1]).any())


@pytest.mark.parametrize("keys", [40, 3000])
def test_rows_of_nothing_but_nan_or_infinity(keys):
    s = Step(18, [keys, keys, keys, 5], [1] * 4, 4, 2, 64, torch.bfloat16)
    bt = s.batch.block_table.long()
    pages = [bt[r, :(keys + 63) // 64] for r in range(3)]
    s.k[pages[0], :, 0, 3] = math.nan       # request 0, KV head 0: every score NaN
    s.q[1].abs_()
    s.k[pages[1], :, 1, :] = -math.inf      # request 1, KV head 1: every score -infinity
    s.q[2].abs_()
    s.k[pages[2][0], 7, 1, :] = math.inf    # request 2, KV head 1: one score +infinity
    phys = torch.full((4, keys), -1, dtype=torch.int32, device=DEV)
    for r in range(3):
        j = torch.arange(keys, device=DEV)
        phys[r] = (bt[r][j // 64] * 64 + j % 64).to(torch.int32)
    for out, lse in (dsa.attn_decode(s.batch, s.q, s.k, s.v), dsa.attn_selected(s.q, s.k, s.v, phys)):
        assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isnan(lse[0, :2]).all())
        assert bool(torch.isfinite(out[0, 2:]).all()) and bool(torch.isfinite(out[1, :2]).all())
        assert bool((out[1, 2:] == 0).all()) and bool((lse[1, 2:] == -math.inf).all())
        assert bool(torch.isnan(out[2, 2:]).all()) and bool(torch.isfinite(out[2, :2]).all())


def test_decode_bad_metadata_is_flagged():
    s = Step(17, [100, 200, 300], [1, 1, 1], 4, 2, 64, torch.bfloat16)
    err = i32([0])
    s.batch.block_table[1, 2] = 10 ** 6   # outside the cache: the page's keys are left out
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v, dev_err=err)
    assert int(err.item()) == 2
    keep = [i for i in range(200) if not 128 <= i < 192]
    for e in range(4):
        check(out[1, e], lse[1, e], attend(s.q[1, e], s.kf[1][keep, e // 2], s.vf[1][keep, e // 2], s.scale, s.dtype))
    for bad in (-1, 301):
        err.zero_()
        s.batch.seq_lens[0] = bad
        out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v, dev_err=err)
        assert int(err.item()) & 16
        assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    s.batch.seq_lens[0] = 100
    err.zero_()
    s.batch.req_id_per_token[2] = 9
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v, dev_err=err)
    assert int(err.item()) & 16 and bool((lse[2] == -math.inf).all())


# ------------------------------------------------------------------- selected

def selected_case(seed, tokens, topk, hq, hkv, d, dtype, blocks=40, none=0.2, layout="pages"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k, v = caches(g, blocks, hkv, d, dtype, layout)
    n = blocks * 64
    used = torch.rand(n, generator=g, device=DEV) < 0.7   # the other slots are NaN
    ids = used.nonzero()[:, 0]
    kk, vv = (torch.randn((ids.numel(), hkv, d), generator=g, device=DEV).to(dtype) for _ in range(2))
    k[ids // 64, ids % 64], v[ids // 64, ids % 64] = kk, vv
    pick = torch.randint(0, ids.numel(), (tokens, topk), generator=g, device=DEV)
    phys = ids[pick].to(torch.int32)
    phys[torch.rand((tokens, topk), generator=g, device=DEV) < none] = -1
    q = torch.randn((tokens, hq, d), generator=g, device=DEV).to(dtype)
    return q, k, v, phys


def check_selected(q, k, v, phys, out, lse, dtype):
    hkv, d = k.shape[2], k.shape[3]
    grp = q.shape[1] // hkv
    for t in range(q.shape[0]):
        ids = phys[t][phys[t] >= 0].long()
        kk, vv = k[ids // 64, ids % 64], v[ids // 64, ids % 64]
        for e in range(q.shape[1]):
            check(out[t, e], lse[t, e], attend(q[t, e], kk[:, e // grp], vv[:, e // grp], d ** -0.5, dtype),
                  f"token {t} head {e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,topk,hq,hkv", [(3, 1, 4, 2), (2, 37, 8, 8), (5, 512, 16, 2), (3, 1030, 33, 1),
                                                (70, 600, 6, 2)])
def test_selected_shapes(dtype, d, tokens, topk, hq, hkv):
    q, k, v, phys = selected_case(tokens + topk, tokens, topk, hq, hkv, d, dtype)
    phys[1] = -1                       # a token with nothing selected
    if topk > 100:
        phys[0, 50:] = -1              # a short row's tail
    err = i32([0])
    out, lse = dsa.attn_selected(q, k, v, phys, dev_err=err)
    check_selected(q, k, v, phys, out, lse, dtype)
    assert int(err.item()) == 0


@pytest.mark.parametrize("layout", ["heads", "joined"])
def test_selected_layouts_and_bad_slots(layout):
    q, k, v, phys = selected_case(5, 4, 900, 8, 4, 128, torch.bfloat16, layout=layout)
    bad = phys.clone()
    bad[2, 10], bad[2, 11], bad[3, 899] = 40 * 64, -2, 2 ** 31 - 1
    err = i32([0])
    out, lse = dsa.attn_selected(q, k, v, bad, dev_err=err)
    assert int(err.item()) == 4
    bad[2, 10] = bad[2, 11] = bad[3, 899] = -1
    check_selected(q, k, v, bad, out, lse, torch.bfloat16)


def test_selected_all_slots_equals_decode():
    s = Step(21, [700, 90], [1, 1], 8, 2, 128, torch.bfloat16)
    phys = torch.full((2, 704), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate([700, 90]):
        j = torch.arange(n, device=DEV)
        phys[r, :n] = (s.batch.block_table[r].long()[j // 64] * 64 + j % 64).to(torch.int32)
    out, lse = dsa.attn_selected(s.q, s.k, s.v, phys)
    s.check(out, lse)


def test_slots_past_32_bit_offsets():
    # a cache of more than 2^31 elements: its last page is read and written there
    blocks, hkv, d = (1 << 31) // (64 * 8 * 128) + 3, 8, 128
    k, v = dsa.new_kv_cache(blocks, hkv, d)
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = [torch.randn((64, hkv, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    slots = torch.arange((blocks - 1) * 64, blocks * 64, device=DEV)
    dsa.kv_write(rows[0], rows[1], slots, k, v)
    q = torch.randn((1, 8, d), generator=g, device=DEV).to(torch.bfloat16)
    out, lse = dsa.attn_selected(q, k, v, slots.to(torch.int32)[None])
    batch = dsa.Batch(i32([0, 1]), i32([64]), i32([[blocks - 1]]), i32([0]), 1, blocks)
    out2, lse2 = dsa.attn_decode(batch, q, k, v)
    for e in range(8):
        ref = attend(q[0, e], rows[0][:, e], rows[1][:, e], d ** -0.5, torch.bfloat16)
        check(out[0, e], lse[0, e], ref)
        check(out2[0, e], lse2[0, e], ref)


# ---------------------------------------------------------- graphs and streams

def test_rows_captured_and_replayed_on_a_side_stream():
    s = Step(31, [2000, 100], [1, 1], 8, 2, 128, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = dsa.attn_decode(s.batch, s.q, s.k, s.v, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    s.check(out, lse)
    want = out.clone()
    ws = torch.empty(dsa.attn_decode_workspace_size(s.batch, 8, 2, 128), dtype=torch.uint8, device=DEV)
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (g1, g2):   # two graphs that share the scratch, replayed one after the other
        with torch.cuda.graph(g):
            dsa.attn_decode(s.batch, s.q, s.k, s.v, out=o, lse=l, ws=ws)
    for g in (g1, g2, g1):
        o.zero_()
        g.replay()
        assert torch.equal(o, want)
    s.batch.seq_lens[0] = 1500   # new lengths within the captured bounds
    g2.replay()
    s.rows[0] = (0, 1500)
    s.check(o, l)
