"""The 8-bit cache's writer and its reading back, against a plain writer in 64 bits:
codes and scales are equal, and what a call does not own keeps its bits."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests import kv8_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cache8(gen, blocks, hkv, d, layout="pages", filled=True):
    """An 8-bit cache in one of several memory layouts, its codes and scales random
    (what slots may hold that were written before), or as it is made."""
    if layout == "heads":       # [blocks, heads, 64, d], scales [blocks, heads, 4, 2]
        k, v = (torch.zeros((blocks, hkv, 64, d), dtype=torch.uint8, device=DEV).view(F8).transpose(1, 2)
                for _ in range(2))
        sc = torch.zeros((blocks, hkv, 4, 2), device=DEV).transpose(1, 2)
    elif layout == "joined":    # K and V in one allocation with room between the rows, scales in wider rows
        both = torch.zeros((blocks, 2, 64, hkv, d + 16), dtype=torch.uint8, device=DEV).view(F8)
        k, v = both[:, 0, :, :, 16:], both[:, 1, :, :, :d]
        sc = torch.zeros((blocks, 5, hkv + 1, 4), device=DEV)[:, :4, :hkv, :2]
    elif layout == "loose":     # pages that are no whole number of slots apart
        k, v = (torch.zeros((blocks, 64 * hkv * d + 48), dtype=torch.uint8, device=DEV).view(F8)[:, 16:16 + 64 * hkv * d]
                .unflatten(1, (64, hkv, d)) for _ in range(2))
        sc = torch.zeros((blocks, 4, hkv, 2), device=DEV)
    else:
        k, v, sc = dsa.new_kv_cache8(blocks, hkv, d)
    if filled:
        for c in (k, v):
            c.copy_((100 * torch.randn(c.shape, generator=gen, device=DEV)).clamp(-448, 448).to(F8))
        sc.copy_(2.0 ** torch.randint(-9, -3, sc.shape, generator=gen, device=DEV).float())
    return k, v, sc


def bits(c):
    return c.contiguous().view(torch.uint8).clone()


class Mirror:
    """A cache and its plain double."""

    def __init__(self, k, v, sc):
        self.k, self.v, self.sc = k, v, sc
        self.codes = [c.float().double().cpu() for c in (k, v)]
        self.scales = [sc[..., i].double().cpu() for i in range(2)]

    def write(self, k, v, slots, **kw):
        dsa.kv_write8(k, v, torch.tensor(slots, dtype=torch.int64, device=DEV), self.k, self.v, self.sc, **kw)
        for i, x in enumerate((k, v)):
            kv8_ref.write(self.codes[i], self.scales[i], x.double().cpu(), slots)

    def check(self):
        for i, c in enumerate((self.k, self.v)):
            assert torch.equal(self.sc[..., i].double().cpu(), self.scales[i])
            got, want = c.float().double().cpu(), self.codes[i]
            assert bool((torch.isnan(got) == torch.isnan(want)).all())
            assert bool((got == want).logical_or(torch.isnan(want)).all())


def rows(gen, n, hkv, d, dtype, spread=1.0):
    """K and V rows of uneven magnitudes, as column views of a wider tensor."""
    wide = torch.randn((n, 2 * hkv * d + 64), generator=gen, device=DEV)
    wide *= torch.exp(spread * torch.randn((n, 1), generator=gen, device=DEV))
    wide = wide.to(dtype)
    return wide[:, 32:32 + hkv * d].unflatten(1, (hkv, d)), wide[:, 64 + hkv * d:].unflatten(1, (hkv, d))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,layout", [(1, "pages"), (3, "heads"), (8, "joined")])
def test_write_lists_of_slots(dtype, d, hkv, layout):
    g = torch.Generator(device=DEV).manual_seed(d + hkv)
    m = Mirror(*cache8(g, 6, hkv, d, layout))
    err = i32([0])
    for slots in ([5],                                         # joins a block
                  [16],                                        # opens one
                  list(range(60, 70)) + [-1] + list(range(30, 36)) + [70, 71, -1],  # a page's end, a block twice
                  [383, 0, 382, 15, 7]):                       # in no order
        m.write(*rows(g, len(slots), hkv, d, dtype), slots, dev_err=err)
        m.check()
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1023, 1024, 1025, 2049])
def test_write_many_tokens(dtype, n):
    # both ways of finding a block's tokens; padding, blocks in several runs
    g = torch.Generator(device=DEV).manual_seed(n)
    m = Mirror(*cache8(g, 40, 2, 64))
    slots = torch.randperm(40 * 64, generator=g, device=DEV)[:n].tolist() if n % 2 else list(range(37, 37 + n))
    slots[n // 2] = -1
    ws = torch.randint(0, 256, (dsa.kv_write8_workspace_size(n, 40),), dtype=torch.uint8, device=DEV)
    m.write(*rows(g, n, 2, 64, dtype), slots, ws=ws)
    m.check()
    m.write(*rows(g, n, 2, 64, dtype), slots[::-1], ws=ws)   # scratch full of the last call's entries
    m.check()


@pytest.mark.parametrize("n", [40, 1700])
def test_write_one_slot_twice(n):
    # the last of the list stands, whole
    g = torch.Generator(device=DEV).manual_seed(n)
    m = Mirror(*cache8(g, 4, 2, 128))
    slots = [(7 * i) % 90 + 20 for i in range(n)]
    m.write(*rows(g, n, 2, 128, torch.bfloat16), slots)
    m.check()


def test_write_token_by_token():
    # a sequence grows by ever larger rows: scales rise, rows there move with them
    g = torch.Generator(device=DEV).manual_seed(3)
    m = Mirror(*cache8(g, 3, 2, 64))
    for s in range(20, 150):
        k, v = rows(g, 1, 2, 64, torch.bfloat16, 2.0)
        m.write(k * 2.0 ** (s % 11 - 4), v, [s])
    m.check()


def test_write_scales_at_their_borders():
    # 448 * 2^e and its neighbours; zeros; the type's least and largest values
    vals = [448.0, 450.0, 446.0, 1.75, 1.7578125, 1.7421875, 0.0, -0.0, 2.0 ** -70, 2.0 ** -133, 3.38953139e38,
            -3.38953139e38, 2.0 ** -55.2, 7.0 * 2 ** -60]
    g = torch.Generator(device=DEV).manual_seed(4)
    m = Mirror(*cache8(g, len(vals), 1, 64))
    k = torch.zeros((len(vals), 1, 64), dtype=torch.bfloat16, device=DEV)
    k[:, 0, 3] = torch.tensor(vals, device=DEV).to(torch.bfloat16)
    m.write(k, -k, [64 * i + 16 for i in range(len(vals))])
    m.check()
    assert m.sc[:3, 1, 0, 0].tolist() == [1.0, 2.0, 1.0]
    assert m.sc[6, 1, 0, 0].item() == 2.0 ** -64 and m.sc[10, 1, 0, 0].item() == 2.0 ** 120
    k = k.clamp(-60000, 60000).to(torch.float16)
    k[0, 0, 3], k[1, 0, 3] = 65504.0, 2.0 ** -24
    m.write(k, -k, [64 * i + 32 for i in range(len(vals))])
    m.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_write_values_that_are_not_finite(dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    m = Mirror(*cache8(g, 3, 2, 64))
    k, v = (x.clone() for x in rows(g, 20, 2, 64, dtype))
    k[2, 0, 5], k[3, 1, 7], k[4, 0, 8] = math.nan, math.inf, -math.inf
    v[:, 1] = math.nan      # nothing finite: the least scale
    v[17, 0] = math.inf
    m.write(k, v, list(range(16, 36)))
    m.check()
    assert int(torch.isnan(m.k.float()).sum()) == 3
    m.write(*rows(g, 1, 2, 64, dtype, 0.0), [36])   # joins them, their NaN stays
    m.check()
    assert int(torch.isnan(m.k.float()).sum()) == 3


def test_write_into_blocks_whose_scale_is_none():
    g = torch.Generator(device=DEV).manual_seed(6)
    k, v, sc = cache8(g, 5, 2, 64)
    bad = [0.0, -1.0, math.nan, math.inf, -math.inf]
    for i, x in enumerate(bad):
        sc[i, 1] = x
    m = Mirror(k, v, sc)
    m.write(*rows(g, 5, 2, 64, torch.bfloat16), [64 * i + 20 for i in range(5)])
    m.check()


@pytest.mark.parametrize("n", [6, 1600])
def test_write_bad_slots_are_flagged(n):
    g = torch.Generator(device=DEV).manual_seed(7)
    m = Mirror(*cache8(g, 30, 2, 64))
    slots = list(range(20, 20 + n))
    slots[1], slots[3], slots[5] = 30 * 64, -5, 2 ** 40
    err = i32([0])
    m.write(*rows(g, n, 2, 64, torch.bfloat16), slots, dev_err=err)
    m.check()
    assert int(err.item()) == 1
    m.write(*rows(g, n, 2, 64, torch.bfloat16), [-1] * n)   # nothing but padding
    m.check()


# ------------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,layout,past", [(1, "pages", False), (3, "heads", True), (8, "joined", False)])
def test_read(dtype, d, hkv, layout, past):
    g = torch.Generator(device=DEV).manual_seed(d + hkv)
    lens, qlens, starts = [1, 0, 15, 64, 17, 300, 90], [1, 0, 3, 64, 2, 11, 1], [700, 0, 3, 100, 20, 200, -1]
    k, v, sc = cache8(g, 14, hkv, d, layout)
    perm = torch.randperm(14, generator=g, device=DEV).tolist()
    bt = [[-7] * 5 for _ in lens]
    for r, n in enumerate(lens):
        for j in range((n + 63) // 64):
            bt[r][j] = perm.pop()
    qsl = [0]
    for n in qlens:
        qsl.append(qsl[-1] + n)
    batch = dsa.Batch(i32(qsl), i32(lens), i32(bt), i32([0] * qsl[-1]), 0, 14)
    wide = torch.full((2, 701, hkv, d + 8), 9.0, dtype=dtype, device=DEV)
    ko, vo = wide[0, :, :, 8:], wide[1, :, :, :d]
    err = i32([0])
    got = dsa.kv_read8(batch, k, v, sc, i32(starts), ko, vo, past=past, dev_err=err)
    assert int(err.item()) == 0
    assert got[0] is ko and got[1] is vo
    for i, (c, o) in enumerate(((k, ko), (v, vo))):
        val = kv8_ref.value(c, sc[..., i])
        left = torch.ones(701, dtype=torch.bool)
        for r, n in enumerate(lens):
            n -= qlens[r] if past else 0
            if starts[r] < 0:
                continue
            for s in range(n):
                want = val[bt[r][s // 64], s % 64].to(dtype)   # powers of two: nothing is rounded
                assert torch.equal(o[starts[r] + s], want)
                left[starts[r] + s] = False
        assert bool((o[left.to(DEV)] == 9).all())
    assert bool((wide[0, :, :, :8] == 9).all()) and bool((wide[1, :, :, d:] == 9).all())


def test_read_many_requests():
    # lengths are counted 256 requests at a time
    g = torch.Generator(device=DEV).manual_seed(9)
    n = 700
    lens = [(37 * i) % 70 for i in range(n)]
    k, v, sc = cache8(g, 2 * n, 1, 64)
    bt = torch.randperm(2 * n, generator=g, device=DEV).to(torch.int32).view(n, 2)
    starts = [sum(lens[:i]) for i in range(n)]
    batch = dsa.Batch(i32([0] * (n + 1)), i32(lens), bt, i32([]), 0, 2 * n)
    ko, vo = (torch.zeros((sum(lens), 1, 64), dtype=torch.float16, device=DEV) for _ in range(2))
    dsa.kv_read8(batch, k, v, sc, i32(starts), ko, vo)
    row = torch.arange(sum(lens), device=DEV)
    r = torch.searchsorted(i32(starts), row.to(torch.int32), right=True) - 1
    # an empty request's start is its neighbour's: the last of them has the row
    j = row - i32(starts)[r]
    for i, (c, o) in enumerate(((k, ko), (v, vo))):
        assert torch.equal(o, kv8_ref.value(c, sc[..., i])[bt[r, j // 64].long(), j % 64].to(torch.float16))


def test_read_bad_metadata_is_flagged():
    g = torch.Generator(device=DEV).manual_seed(10)
    k, v, sc = cache8(g, 8, 2, 64)
    bt = i32([[0, 1], [2, 3], [4, 99], [6, 7], [5, 5]])

    def read(lens, qlens, starts, past=False):
        qsl = [3]
        for n in qlens:
            qsl.append(qsl[-1] + n)
        batch = dsa.Batch(i32(qsl), i32(lens), bt, i32([]), 0, 8, max_seq_len=128)
        ko, vo = (torch.full((400, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        err = i32([0])
        dsa.kv_read8(batch, k, v, sc, i32(starts), ko, vo, past=past, dev_err=err)
        return ko, vo, int(err.item())

    val = kv8_ref.value(k, sc[..., 0])
    ko, vo, err = read([100, 129, 128, -1, 100], [0] * 5, [0, 100, 230, 0, 301])
    assert err == 2 | 16
    assert torch.equal(ko[:64], val[0].to(torch.bfloat16)) and torch.equal(ko[64:100], val[1, :36].to(torch.bfloat16))
    assert bool((ko[100:230] == 9).all())                       # longer than the row: not read
    # page 99; beyond the rows
    assert torch.equal(ko[230:294], val[4].to(torch.bfloat16)) and bool((ko[294:] == 9).all())
    ko, vo, err = read([10, 10, 0, 0, 0], [11, 10, 0, 0, 0], [0, 20, 50, 60, 2 ** 31 - 1], past=True)
    assert err == 16 and bool((ko == 9).all())                  # shorter than the query; nothing but the query
    ko, vo, err = read([10, 20, 0, 0, 0], [-2, 4, 0, 0, 0], [0, 100, 0, 0, 0], past=True)
    assert err == 16 and bool((ko[:100] == 9).all()) and bool((ko[116:] == 9).all())
    assert torch.equal(ko[100:116], val[2, :16].to(torch.bfloat16))


def test_read_and_write_beyond_32_bit_offsets():
    blocks, hkv, d = (1 << 32) // (64 * 8 * 128) + 3, 8, 128
    k, v, sc = dsa.new_kv_cache8(blocks, hkv, d)
    g = torch.Generator(device=DEV).manual_seed(2)
    x = [torch.randn((80, hkv, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    slots = torch.arange((blocks - 2) * 64 + 48, blocks * 64, device=DEV)
    dsa.kv_write8(x[0], x[1], slots, k, v, sc)
    ko, vo = torch.zeros_like(x[0]), torch.zeros_like(x[1])
    batch = dsa.Batch(i32([0, 0]), i32([64]), i32([[blocks - 1]]), i32([]), 0, blocks)
    dsa.kv_read8(batch, k, v, sc, i32([16]), ko, vo)
    for a, b in ((x[0], ko), (x[1], vo)):
        amax = a[16:].float().view(4, 16, hkv, d).abs().amax((1, 3)).repeat_interleave(16, 0)[..., None]
        # a code of at most 448 is off by half a step, 2^-4 of it; the block's largest is above 224
        assert bool(((b[16:].float() - a[16:].float()).abs() <= 2.0 ** -4 * amax).all())
    assert bool((k[:2].view(torch.uint8) == 0).all()) and bool((sc[:2] == 0).all())


# ----------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("n", [64, 1200])
def test_write_and_read_on_a_stream_and_in_a_graph(n):
    g = torch.Generator(device=DEV).manual_seed(n)
    m = Mirror(*cache8(g, 20, 2, 128))
    k, v = rows(g, n, 2, 128, torch.bfloat16)
    slots = torch.arange(10, 10 + n, device=DEV)
    batch = dsa.Batch(i32([0, 0]), i32([n + 10]), torch.arange(20, dtype=torch.int32, device=DEV)[None], i32([]), 0, 20)
    ko, vo = (torch.zeros((n + 10, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    start = i32([0])
    ws = torch.empty(dsa.kv_write8_workspace_size(n, 20), dtype=torch.uint8, device=DEV)

    def calls(stream=None):
        dsa.kv_write8(k, v, slots, m.k, m.v, m.sc, ws=ws, stream=stream)
        dsa.kv_read8(batch, m.k, m.v, m.sc, start, ko, vo, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)
    side.synchronize()
    for i, x in enumerate((k, v)):
        kv8_ref.write(m.codes[i], m.scales[i], x.double().cpu(), slots.tolist())
    m.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in range(2):
        a, b = rows(torch.Generator(device=DEV).manual_seed(seed), n, 2, 128, torch.bfloat16)
        k.copy_(a)
        v.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, x in enumerate((k, v)):
            kv8_ref.write(m.codes[i], m.scales[i], x.double().cpu(), slots.tolist())
        m.check()
        assert torch.equal(ko, kv8_ref.value(m.k, m.sc[..., 0]).view(-1, 2, 128)[:n + 10].to(torch.bfloat16))
