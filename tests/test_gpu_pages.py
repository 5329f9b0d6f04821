"""The KV cache's writer and the page calls, against the same steps on the CPU,
entry by entry."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLOT, BLOCK, SEQ, STATE, NOPAGE = 1, 2, 16, 64, 128


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(t):
    return t.contiguous().view(torch.int16)


# ------------------------------------------------------------------- kv_write

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,hkv,d,layout", [(1, 1, 64, "pages"), (7, 8, 128, "pages"), (333, 3, 64, "heads"),
                                            (65, 5, 128, "joined")])
def test_kv_write(dtype, n, hkv, d, layout):
    g = torch.Generator(device=DEV).manual_seed(n)
    blocks = 9
    if layout == "heads":
        k, v = (torch.zeros((blocks, hkv, 64, d), dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2))
    elif layout == "joined":
        both = torch.zeros((blocks, 64, hkv, 2 * d), dtype=dtype, device=DEV)
        k, v = both[..., :d], both[..., d:]
    else:
        k, v = dsa.new_kv_cache(blocks, hkv, d, dtype)
    new = torch.randn((n, 2 * hkv + 1, d), generator=g, device=DEV).to(dtype)   # views of one projection
    kn, vn = new[:, :hkv], new[:, hkv + 1:]
    slots = torch.randperm(blocks * 64, generator=g, device=DEV)[:n]
    slots[n // 2] = -1
    err = i32([0])
    dsa.kv_write(kn, vn, slots, k, v, dev_err=err)
    for c, src in ((k, kn), (v, vn)):
        want = torch.zeros((blocks * 64, hkv, d), dtype=dtype, device=DEV)
        want[slots[slots >= 0]] = src[slots >= 0]
        assert torch.equal(bits(c.reshape(-1, hkv, d)), bits(want))
    assert int(err.item()) == 0
    bad = slots.clone()
    bad[0] = blocks * 64
    before = k.clone()
    dsa.kv_write(kn[:1], vn[:1], bad[:1], k, v, dev_err=err)
    assert int(err.item()) == SLOT and torch.equal(bits(k), bits(before))


# ----------------------------------------------------------------- pool model

class Pool:
    """A pool of pages on the GPU with caches of several formats, and its model in numpy."""

    def __init__(self, seed, blocks, rows, lens, width=None, n_caches=3):
        rng = np.random.default_rng(seed)
        self.width = width or max([(n + 63) // 64 for n in lens] + [1]) + 1
        self.refs = np.zeros(blocks, np.int32)
        self.bt = np.full((rows, self.width), -1, np.int32)
        self.seq = np.zeros(rows, np.int32)
        perm, at = rng.permutation(blocks), 0
        for r, n in enumerate(lens):
            m = (n + 63) // 64
            self.bt[r, :m] = perm[at:at + m]
            self.refs[perm[at:at + m]] += 1
            self.seq[r] = n
            at += m
        sizes = [8448, 64 * 2 * 64 * 2, 16, 4352, 70000, 32768][:n_caches]
        self.caches = [rng.integers(0, 256, (blocks, s), dtype=np.uint8) for s in sizes]
        # one cache whose pages lie further apart than they are long
        self.dev = [torch.from_numpy(c).to(DEV) for c in self.caches]
        if n_caches > 1:
            wide = torch.zeros((blocks, sizes[1] + 48), dtype=torch.uint8, device=DEV)
            self.dev[1] = wide[:, :sizes[1]]
            self.dev[1].copy_(torch.from_numpy(self.caches[1]))
        self.err = i32([0])
        self.up()

    def up(self):
        self.d_refs, self.d_bt, self.d_seq = (torch.from_numpy(x.copy()).to(DEV)
                                              for x in (self.refs, self.bt, self.seq))

    def same(self, err=0):
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        assert np.array_equal(self.d_bt.cpu().numpy(), self.bt)
        assert np.array_equal(self.d_seq.cpu().numpy(), self.seq)
        for d, c in zip(self.dev, self.caches):
            assert np.array_equal(d.cpu().numpy(), c)
        assert int(self.err.item()) == err
        self.err.zero_()

    def fork(self, parents, children, run=True):
        if run:
            dsa.pages_fork(self.d_refs, self.d_bt, self.d_seq, i32(parents), i32(children), self.dev, dev_err=self.err)
        err, seq0 = 0, self.seq.copy()
        free = list(np.nonzero(self.refs == 0)[0])
        taken, ok = set(), []
        for p, c in zip(parents, children):
            good = 0 <= p < len(seq0) and 0 <= c < len(seq0) and 0 <= seq0[p] <= self.width * 64
            if not good:
                err |= SEQ
            elif seq0[c] != 0 or c in taken:
                err |= STATE
            else:
                taken.add(c)
                ok.append((p, c))
        for p, c in ok:
            n = int(seq0[p])
            if n % 64 and not free:
                err |= NOPAGE
                continue
            self.bt[c, :n // 64] = self.bt[p, :n // 64]
            for b in self.bt[p, :n // 64]:
                self.refs[b] += 1
            if n % 64:
                new = free.pop(0)
                self.refs[new] = 1
                for x in self.caches:
                    x[new] = x[self.bt[p, n // 64]]
                self.bt[c, n // 64] = new
            self.seq[c] = n
        return err

    def free(self, rows):
        dsa.pages_free(self.d_refs, self.d_bt, self.d_seq, i32(rows), dev_err=self.err)
        err = 0
        for r in rows:
            if not 0 <= r < len(self.seq):
                err |= SEQ
                continue
            for j in range((int(self.seq[r]) + 63) // 64):
                b, self.bt[r, j] = self.bt[r, j], -1
                if b < 0:
                    continue
                if self.refs[b] <= 0:
                    err |= STATE
                else:
                    self.refs[b] -= 1
            self.seq[r] = 0
        return err

    def compact(self, caches=None):
        dsa.pages_compact(self.d_refs, self.d_bt, self.dev if caches is None else caches, dev_err=self.err)
        live = self.refs > 0
        n = int(live.sum())
        holes = [i for i in range(n) if not live[i]]
        moved = [i for i in range(n, len(live)) if live[i]]
        new = {s: h for s, h in zip(moved, holes)}
        for s, h in new.items():
            self.refs[h], self.refs[s] = self.refs[s], 0
            for x in self.caches:
                x[h] = x[s]
        self.bt = np.array([[new.get(b, b) for b in row] for row in self.bt.tolist()], np.int32)


@pytest.mark.parametrize("seed,blocks,lens", [(1, 40, [130, 64, 1, 0, 700]), (2, 3000, [64 * 40, 5, 2000, 63]),
                                              (3, 9000, [1000] * 20)])
def test_fork_free_compact_sequence(seed, blocks, lens):
    p = Pool(seed, blocks, 2 * len(lens) + 4, lens)
    k = len(lens)
    assert p.fork([0, 1, 2, 0, 3], [k, k + 1, k + 2, k + 3, len(p.seq) - 1]) == 0
    p.same()
    assert p.free([0, k + 1, 2]) == 0
    p.same()
    p.compact()
    p.same()
    assert p.fork([k, 1], [0, 2]) == 0     # of a fork, into freed rows
    p.same()
    assert p.free(list(range(len(p.seq)))) == 0
    p.same()
    assert int(p.refs.sum()) == 0
    p.compact()
    p.same()


def test_fork_refuses_entry_by_entry():
    p = Pool(4, 30, 8, [100, 128, 70])
    # outside the table; a child in use; one child twice; a parent that is empty
    want = p.fork([0, -1, 0, 8, 1, 2, 0, 4, 2], [3, 4, 1, 5, 3, 3, 99, 5, 6])
    assert want == SEQ | STATE
    p.same(want)
    p.seq[1] = p.width * 64 + 1
    p.up()
    assert p.fork([1], [7]) == SEQ
    p.same(SEQ)


def test_fork_without_pages():
    p = Pool(5, 8, 9, [100, 130, 1])     # 6 pages used
    want = p.fork([0, 1, 2, 0], [3, 4, 5, 6])
    assert want == NOPAGE
    p.same(want)
    assert p.seq[3] == 100 and p.seq[4] == 130 and p.seq[5] == 0


def test_fork_many_entries_of_one_parent():
    p = Pool(6, 5000, 2600, [64 * 3 + 9, 640])
    assert p.fork([0, 1] * 1200, list(range(100, 2500))) == 0
    p.same()


def test_fork_with_a_bad_table_entry():
    p = Pool(7, 30, 6, [200, 200])
    p.d_bt[0, 3] = 30                       # the part-filled page: the child's page is taken, nothing is copied
    dsa.pages_fork(p.d_refs, p.d_bt, p.d_seq, i32([0]), i32([3]), p.dev, dev_err=p.err)
    assert int(p.err.item()) == BLOCK
    for d, c in zip(p.dev, p.caches):
        assert np.array_equal(d.cpu().numpy(), c)


def test_free_twice_and_bad_rows():
    p = Pool(8, 40, 6, [300, 64, 1])
    assert p.free([0, 0, 2, -1, 6, 2]) == SEQ
    p.same(SEQ)
    p.bt[3, :2] = [p.bt[1, 0], 39 if p.refs[39] == 0 else int(np.nonzero(p.refs == 0)[0][0])]
    p.seq[3] = 128
    p.up()
    assert p.free([3]) == STATE            # its second page has count 0 already
    p.same(STATE)


@pytest.mark.parametrize("blocks", [1, 5, 2047, 2048, 2049, 10000])
@pytest.mark.parametrize("fill", [0.0, 0.1, 0.5, 1.0])
def test_compact_densities(blocks, fill):
    rng = np.random.default_rng(blocks)
    p = Pool(9, blocks, 3, [], width=4, n_caches=2 if blocks < 3000 else 1)
    p.refs = (rng.random(blocks) < fill).astype(np.int32) * rng.integers(1, 4, blocks).astype(np.int32)
    p.bt = rng.integers(-1, blocks + 2, (3, 4)).astype(np.int32)
    p.up()
    p.compact()
    p.same()


def test_compact_without_caches_and_with_many():
    p = Pool(10, 100, 4, [500, 900], n_caches=1)
    keep = [c.copy() for c in p.caches]
    p.compact(caches=[])
    p.caches = keep
    p.same()
    # more caches than one launch takes
    p = Pool(11, 60, 4, [500, 900], n_caches=1)
    rng = np.random.default_rng(0)
    p.caches = [rng.integers(0, 256, (60, 32 * (1 + i % 3)), dtype=np.uint8) for i in range(150)]
    p.dev = [torch.from_numpy(c).to(DEV) for c in p.caches]
    p.compact()
    p.same()
    assert p.fork([0, 1], [2, 3]) == 0
    p.same()


# ----------------------------------------------------------------- pages_copy

def test_copy_pairs():
    rng = np.random.default_rng(12)
    caches = [rng.integers(0, 256, (50, s), dtype=np.uint8) for s in (8448, 33000 // 16 * 16)]
    dev = [torch.from_numpy(c).to(DEV) for c in caches]
    err = i32([0])
    src, dst = [1, 1, 2, -1, 3, 7], [10, 11, 12, 13, -1, 7]
    dsa.pages_copy(dev, i32(src), i32(dst), dev_err=err)
    for c, d in zip(caches, dev):
        for a, b in ((1, 10), (1, 11), (2, 12)):
            c[b] = c[a]
        assert np.array_equal(d.cpu().numpy(), c)
    assert int(err.item()) == 0
    # two pairs with one destination: the first; a destination that is a source: not copied; outside: not copied
    dsa.pages_copy(dev, i32([4, 5, 6, 20, 50, 1]), i32([30, 30, 20, 21, 31, -2]), dev_err=err)
    for c, d in zip(caches, dev):
        for a, b in ((4, 30), (20, 21)):
            c[b] = c[a]
        assert np.array_equal(d.cpu().numpy(), c)
    assert int(err.item()) == STATE | BLOCK
    dsa.pages_copy(dev, i32([]), i32([]))


def test_copy_all_of_a_pool():
    dev = torch.arange(4000 * 4224, device=DEV).to(torch.int16).view(4000, 4224)
    want = dev.clone()
    src = torch.randperm(2000, device=DEV).to(torch.int32)
    dst = (torch.randperm(2000, device=DEV) + 2000).to(torch.int32)
    want[dst.long()] = want[src.long()]
    dsa.pages_copy([dev], src, dst)
    assert torch.equal(dev, want)


def test_pages_captured_and_replayed():
    p = Pool(13, 200, 8, [300, 700, 64])
    start = [t.clone() for t in (p.d_refs, p.d_bt, p.d_seq)]
    ws = torch.empty(dsa.pages_workspace_size(200, 2), dtype=torch.uint8, device=DEV)
    a, b = i32([0, 1]), i32([4, 5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.pages_fork(p.d_refs, p.d_bt, p.d_seq, a, b, p.dev, ws=ws)
        dsa.pages_free(p.d_refs, p.d_bt, p.d_seq, a)
        dsa.pages_compact(p.d_refs, p.d_bt, p.dev, ws=ws)
    for t, s in zip((p.d_refs, p.d_bt, p.d_seq), start):
        assert torch.equal(t, s)
    g.replay()
    model = Pool(13, 200, 8, [300, 700, 64])
    model.dev = [d.clone() for d in model.dev]
    model.fork([0, 1], [4, 5])
    model.free([0, 1])
    model.compact()
    model.same()
    for t, s in zip((p.d_refs, p.d_bt, p.d_seq), (model.refs, model.bt, model.seq)):
        assert np.array_equal(t.cpu().numpy(), s)
    for d, c in zip(p.dev, model.caches):
        assert np.array_equal(d.cpu().numpy(), c)
