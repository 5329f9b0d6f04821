"""Causal attention over prompts, against plain attention in 64 bits: keys in
pages and packed, head groups, lengths, chunks, and what may not leak."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import attend_rows, check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Prompts:
    """Requests of given query and key counts; with ``paged`` the keys lie in
    shuffled pages whose other slots are NaN, else packed with NaN rows between."""

    def __init__(self, seed, qlens, klens, hq, hkv, d, dtype, paged, decodes=(), layout="pages", gap=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        nd = len(decodes)   # decode requests in front, one token each; the prompts' rows come behind
        qlens, klens = [1] * nd + list(qlens), list(decodes) + list(klens)
        self.nd, self.qlens, self.klens, self.paged = nd, qlens, klens, paged
        need = [(n + 63) // 64 for n in klens]
        blocks = sum(need) + 2
        perm = torch.randperm(blocks, generator=g, device=DEV).tolist()
        bt = [[-3] * max(need + [1]) for _ in klens]
        at = 0
        for r, m in enumerate(need):
            bt[r][:m] = perm[at:at + m]
            at += m
        self.kf, self.vf = ([torch.randn((n, hkv, d), generator=g, device=DEV).to(dtype) for n in klens]
                            for _ in range(2))
        self.starts = None
        if paged:
            shape = (blocks, hkv, 64, d) if layout == "heads" else (blocks, 64, hkv, d)
            self.k, self.v = (torch.full(shape, math.nan, dtype=dtype, device=DEV) for _ in range(2))
            if layout == "heads":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        else:
            self.starts = []
            at = gap
            for n in klens:
                self.starts.append(at)
                at += n + gap
            self.k, self.v = (torch.full((at, hkv, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
        self.bt = bt
        for r, n in enumerate(klens):
            for c, f in ((self.k, self.kf[r]), (self.v, self.vf[r])):
                if paged:
                    for j in range(0, n, 64):
                        c[bt[r][j // 64], :min(64, n - j)] = f[j:j + 64]
                else:
                    c[self.starts[r]:self.starts[r] + n] = f
        qsl = [0]
        for n in qlens:
            qsl.append(qsl[-1] + n)
        req = [r for r, n in enumerate(qlens) for _ in range(n)]
        self.qsl = qsl
        self.batch = dsa.Batch(i32(qsl), i32(klens), i32(bt), i32(req), nd, blocks, max_seq_len=max(klens + [1]),
                               num_decode_tokens=qsl[nd])
        self.q = torch.randn((qsl[-1], hq, d), generator=g, device=DEV).to(dtype)
        self.g, self.d, self.dtype = hq // hkv, d, dtype

    def run(self, **kw):
        return dsa.attn_prompt(self.batch, self.q, self.k, self.v,
                               kv_start=None if self.paged else i32(self.starts), **kw)

    def check(self, out, lse, scale=None, only=None):
        for r in range(self.nd, len(self.qlens)):
            n, m, a = self.qlens[r], self.klens[r], self.qsl[r]
            if n == 0 or (only is not None and r not in only):
                continue
            vis = [min(max(m - n + i + 1, 0), m) for i in range(n)]
            for e in range(self.q.shape[1]):
                ref = attend_rows(self.q[a:a + n, e], self.kf[r][:, e // self.g], self.vf[r][:, e // self.g], vis,
                                  scale or self.d ** -0.5, self.dtype)
                check(out[a:a + n, e], lse[a:a + n, e], ref, f"request {r} ({n} of {m}) head {e}")


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (3, 3), (8, 2), (5, 1)])
def test_prompt_lengths_and_groups(paged, dtype, d, hq, hkv):
    n = [1, 300, 64, 0, 127, 128, 129, 256, 513]
    p = Prompts(hq * d, n, n, hq, hkv, d, dtype, paged)
    err = i32([0])
    out, lse = p.run(dev_err=err)
    p.check(out, lse)
    assert int(err.item()) == 0


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (3, 1)])
def test_prompt_chunks_and_short_keys(paged, hq, hkv):
    # chunks behind a context; a request with fewer keys than queries; none at all
    p = Prompts(5, [200, 1, 130, 64, 70, 3], [1000, 700, 131, 20, 0, 3], hq, hkv, 128, torch.bfloat16, paged)
    out, lse = p.run()
    p.check(out, lse)


def test_prompt_long_one():
    p = Prompts(6, [5000], [5000], 2, 1, 128, torch.bfloat16, True)
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_growing_scores_rescale(dtype):
    p = Prompts(7, [1000], [1000], 2, 2, 64, dtype, False, gap=0)
    p.q = torch.ones_like(p.q)
    k = (torch.arange(1000, device=DEV)[:, None, None] / 40).expand(1000, 2, 64).to(dtype)
    p.k.copy_(k)
    p.kf[0] = k
    out, lse = p.run()
    p.check(out, lse)


def test_prompt_large_scores_and_scale():
    p = Prompts(8, [400], [400], 4, 1, 128, torch.bfloat16, True)
    out, lse = p.run(scale=1.5)
    p.check(out, lse, 1.5)


def test_prompt_heads_layout_and_views():
    p = Prompts(9, [150, 260], [150, 300], 4, 2, 64, torch.float16, True, layout="heads")
    wide = torch.zeros((410, 6, 96), dtype=torch.float16, device=DEV)
    q = wide[:, 2:, 16:80]
    q.copy_(p.q)
    obuf = torch.full((410, 4, 72), 2.0, dtype=torch.float16, device=DEV)
    out, lse = dsa.attn_prompt(p.batch, q, p.k, p.v, out=obuf[:, :, :64])
    p.check(out, lse)
    assert bool((obuf[:, :, 64:] == 2).all())
    # packed keys as column views of one projection
    n = 333
    qkv = torch.randn((n, 8, 128), device=DEV).to(torch.bfloat16)
    b = dsa.Batch(i32([0, n]), i32([n]), i32([[0]]), i32([0] * n), 0, 1, max_seq_len=n, num_decode_tokens=0)
    out, lse = dsa.attn_prompt(b, qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], kv_start=i32([0]))
    for e in range(4):
        check(out[:, e], lse[:, e], attend_rows(qkv[:, e], qkv[:, 4 + e // 2], qkv[:, 6 + e // 2],
                                                list(range(1, n + 1)), 128 ** -0.5, torch.bfloat16))


def test_mixed_step_decode_and_prompt_share_buffers():
    # decode rows in front, prompts behind: each call writes its own rows only
    p = Prompts(10, [300, 65], [300, 400], 8, 2, 128, torch.bfloat16, True, decodes=[1, 700, 64])
    out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=DEV)
    dsa.attn_prompt(p.batch, p.q, p.k, p.v, out=out, lse=lse)
    assert bool((out[:3] == 7).all()) and bool((lse[:3] == 7).all())
    p.check(out, lse)
    mine = out.clone()
    dsa.attn_decode(p.batch, p.q, p.k, p.v, out=out, lse=lse)
    assert torch.equal(out[3:], mine[3:])
    for t, n in enumerate([1, 700, 64]):
        for e in range(8):
            check(out[t:t + 1, e], lse[t:t + 1, e],
                  attend_rows(p.q[t:t + 1, e], p.kf[t][:, e // 4], p.vf[t][:, e // 4], [n], 128 ** -0.5, p.dtype))


@pytest.mark.parametrize("hq,hkv", [(2, 1), (3, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_non_finite_rows_reach_only_those_that_see_them(hq, hkv, dtype):
    n = 400
    p = Prompts(11, [n], [n], hq, hkv, 64, dtype, False, gap=0)
    clean, clean_lse = p.run()
    p.v[200, 0, 7] = math.inf
    p.v[330, 0, 9] = math.nan
    p.k[350, 0, 3] = math.nan
    out, lse = p.run()
    bad = torch.zeros((n, 64), dtype=torch.bool, device=DEV)
    bad[200:, 7] = True
    bad[330:, 9] = True
    bad[350:, :] = True
    for e in range(hq):
        assert torch.equal(torch.isfinite(out[:, e]), ~bad), f"head {e}"
        assert torch.equal(out[:, e][~bad], clean[:, e][~bad])
        assert bool((out[200:350, e, 7] == math.inf).all())
    assert torch.equal(lse[:350], clean_lse[:350]) and bool(torch.isnan(lse[350:]).all())


@pytest.mark.parametrize("hq,hkv", [(2, 1), (3, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_rows_of_nothing_but_nan_or_infinity(hq, hkv, dtype):
    n = 300
    p = Prompts(16, [n, n], [n, n], hq, hkv, 128, dtype, False, gap=0)
    clean, _ = p.run()
    p.k[:, 0, 5] = torch.where(torch.arange(2 * n, device=DEV) < 140, math.nan, p.k[:, 0, 5].float()).to(dtype)
    out, lse = p.run()
    # rows that see NaN scores, or nothing else
    assert bool(torch.isnan(out[:n]).all()) and bool(torch.isnan(lse[:n]).all())
    assert torch.equal(out[n:], clean[n:])
    p.q.abs_()
    p.k[:140] = -math.inf        # the first rows' scores are all -infinity: as if they saw no key
    out, lse = p.run()
    assert bool((out[:140] == 0).all()) and bool((lse[:140] == -math.inf).all())
    assert bool(torch.isfinite(out[140:]).all()) and bool(torch.isfinite(lse[140:]).all())
    for e in range(hq):          # the later ones see the finite keys alone
        k, v = p.k[140:n, 0], p.v[140:n, 0]
        check(out[140:n, e], lse[140:n, e], attend_rows(p.q[140:n, e], k, v, range(1, n - 139), 128 ** -0.5, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_first_columns_say_little_of_the_others(d, dtype):
    # a first reference far below the maximum, at it, or none: -infinity in the first columns
    n = 500
    p = Prompts(21, [n] * 3, [n] * 3, 4, 1, d, dtype, False, gap=0)
    p.q.abs_()
    p.k[40:n] *= 20.0
    p.k[n:n + 50] = 4.0
    p.k[2 * n:2 * n + 60] = -math.inf
    p.kf = list(p.k.split(n))
    out, lse = p.run()
    p.check(out, lse, only=(0, 1))
    assert bool((out[2 * n:2 * n + 60] == 0).all()) and bool((lse[2 * n:2 * n + 60] == -math.inf).all())
    k, v = p.k[2 * n + 60:, 0], p.v[2 * n + 60:, 0]
    for e in range(4):
        check(out[2 * n + 60:, e], lse[2 * n + 60:, e],
              attend_rows(p.q[2 * n + 60:, e], k, v, range(1, n - 59), d ** -0.5, dtype))


def test_prompt_bad_metadata_is_flagged():
    p = Prompts(12, [100, 200, 90], [100, 200, 90], 4, 2, 64, torch.bfloat16, True)
    err = i32([0])
    p.batch.seq_lens[1] = 10 ** 6
    out, lse = p.run(dev_err=err)
    assert int(err.item()) == 16
    p.check(out, lse, only=(0, 2))
    assert bool((out[100:300] == 0).all()) and bool((lse[100:300] == -math.inf).all())
    p.batch.seq_lens[1] = 200
    err.zero_()
    p.batch.block_table[2, 1] = p.batch.num_blocks
    out, lse = p.run(dev_err=err)
    assert int(err.item()) == 2
    p.check(out, lse, only=(0, 1))
    p.batch.query_start_loc[2] = 10 ** 6   # tokens outside the batch: nothing is written for them
    err.zero_()
    keep = torch.full_like(p.q, 4.0)
    p.run(out=keep, dev_err=err)
    assert int(err.item()) & 16
    packed = Prompts(13, [100, 200], [100, 200], 4, 2, 64, torch.bfloat16, False)
    packed.starts[1] = packed.k.shape[0] - 199
    err.zero_()
    out, lse = packed.run(dev_err=err)
    assert int(err.item()) == 16 and bool((lse[100:] == -math.inf).all())
    packed.check(out, lse, only=(0,))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_rows_bits_are_their_own(d, dtype):
    # some rows' weights come out too large in a later tile: the other rows' bits stay
    p = Prompts(24, [900], [900], 2, 1, d, dtype, False, gap=0)
    want, wlse = p.run()
    rows = [500, 577, 700, 899]
    p.q[rows] *= 60
    out, lse = p.run()
    rest = [r for r in range(900) if r not in rows]
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], wlse[rest])
    assert not torch.equal(out[rows], want[rows])
    p.check(out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_uneven_pairs_of_tiles(d, dtype):
    # token tiles in pairs of 2, 1 and unequal numbers of key tiles, several pairs
    # a CTA; scores that rise over the keys, so that references move in any of them
    q = [100, 300, 256, 1, 129, 640, 128, 257, 31, 511] * 4
    k = [m + c for m, c in zip(q, [3000, 0, 700, 1500, 127, 0, 0, 1, 900, 130] * 4)]
    p = Prompts(19, q, k, 7, 7, d, dtype, False, gap=0)
    up = torch.cat([torch.arange(n, device=DEV) / 100 for n in k])[:, None, None]
    p.q[:, 1:4] = p.q[:, 1:4].abs()
    p.k[:, 1:4] = (p.k[:, 1:4].float() / 4 + up).to(dtype)
    p.kf = list(p.k.split(k))
    out, lse = p.run()
    p.check(out, lse)


def test_prompt_many_requests_and_same_bits():
    n = [(17 * i) % 90 for i in range(80)]
    p = Prompts(14, n, n, 2, 1, 64, torch.bfloat16, False)
    out, lse = p.run()
    p.check(out, lse)
    again, _ = p.run()
    assert torch.equal(out, again)


def test_prompt_requests_beyond_one_search_step_with_bad_ones_between():
    # 32 requests are searched at a time: units far apart, empty requests and bad ones in between
    n = [0 if i % 7 == 3 else 1 + (37 * i) % 150 for i in range(1200)]
    p = Prompts(20, n, n, 2, 1, 64, torch.bfloat16, False)
    seq = p.batch.seq_lens.clone()
    bad = list(range(5, 1200, 97))
    seq[bad] = -1
    p.batch = dsa.Batch(p.batch.query_start_loc, seq, p.batch.block_table, p.batch.req_id_per_token, 0,
                        p.batch.num_blocks, max_seq_len=max(n), num_decode_tokens=0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = p.run(dev_err=err)
    assert int(err.item()) == 16
    for r in bad:
        a = p.qsl[r]
        assert bool((out[a:a + n[r]] == 0).all()) and bool((lse[a:a + n[r]] == -math.inf).all())
    p.check(out, lse, only=[r for r in range(1200) if r not in bad])


def test_prompt_captured_and_replayed():
    p = Prompts(15, [300, 100], [500, 100], 4, 2, 128, torch.bfloat16, True)
    want, _ = p.run()
    o, l = torch.zeros_like(want), torch.zeros(p.q.shape[:2], device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.attn_prompt(p.batch, p.q, p.k, p.v, out=o, lse=l)
    for _ in range(2):
        o.zero_()
        g.replay()
        assert torch.equal(o, want)
