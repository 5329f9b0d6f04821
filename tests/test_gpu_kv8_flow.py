"""The 8-bit cache's writer, its reading back, the attention over it, the page calls and
the indexer's layer runner together, as a serving loop uses them: prompts in chunks,
forked sequences, decode steps over selected and over all keys, a compacted pool."""
import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests import kv8_ref
from tests.attn_ref import attend_rows, check
from tests.test_gpu_attention_flow import i32, rand, slots_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, BLOCKS, WIDTH = 8, 2, 128, 64, 10


class Loop8:
    """Two layers' 8-bit caches and one indexer cache over one pool of pages."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv = [dsa.new_kv_cache8(BLOCKS, HKV, D) for _ in range(2)]
        self.index = dsa.new_k_cache(BLOCKS)
        self.refs = torch.zeros(BLOCKS, dtype=torch.int32, device=DEV)
        self.bt = torch.full((8, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.seq = torch.zeros(8, dtype=torch.int32, device=DEV)
        self.err = i32([0])
        self.keys = [[([], []) for _ in range(8)] for _ in range(2)]   # [layer][row]: K's and V's rows as given

    @property
    def caches(self):
        return [c for three in self.kv for c in three] + [self.index]

    def take_pages(self, row, length):
        free = (self.refs == 0).nonzero()[:, 0].tolist()
        for j in range((length + 63) // 64):
            if self.bt[row, j] < 0:
                self.bt[row, j] = free.pop()
                self.refs[self.bt[row, j].long()] = 1

    def stored(self, layer, row):
        """K and V of a row's keys as the cache has them, in 64 bits, and V's scales;
        checked against what was given: a value is off by half a step, 2^-4 of it, or
        half of the least step, 2^-10 of the scale, which moves to higher scales (each
        at least twice the one before) add at most once more."""
        n = int(self.seq[row])
        at = slots_of(self.bt, row, 0, n)
        kc, vc, sc = self.kv[layer]
        both = []
        for i, c in enumerate((kc, vc)):
            x = kv8_ref.value(c, sc[..., i]).flatten(0, 1)[at]
            want = torch.cat(self.keys[layer][row][i]).double()
            s = sc[..., i].repeat_interleave(16, 1).flatten(0, 1)[at].double()[..., None]
            assert want.shape == x.shape
            assert bool(((x - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * s).all())
            both.append(x)
        return (*both, sc[..., 1].repeat_interleave(16, 1).flatten(0, 1)[at])

    def chunk(self, rows, lens):
        """The next lens[i] tokens of the prompts in rows: written, and attended to
        with the earlier ones read back."""
        past = self.seq[rows].tolist()
        total = [p + n for p, n in zip(past, lens)]
        for r, n in zip(rows, total):
            self.take_pages(r, n)
            self.seq[r] = n
        qsl = [0]
        for n in lens:
            qsl.append(qsl[-1] + n)
        batch = dsa.Batch(i32(qsl), i32(total), self.bt[rows].contiguous(),
                          i32([i for i, n in enumerate(lens) for _ in range(n)]), 0, BLOCKS)
        slots = torch.cat([slots_of(self.bt, r, p, n) for r, p, n in zip(rows, past, total)])
        dsa.indexer_k_quant_write(rand(self.g, qsl[-1], 128), slots, self.index, self.err)
        start = i32([sum(total[:i]) for i in range(len(rows))])
        for layer, (kc, vc, sc) in enumerate(self.kv):
            q, k, v = rand(self.g, qsl[-1], HQ, D), rand(self.g, qsl[-1], HKV, D), rand(self.g, qsl[-1], HKV, D)
            packed = [torch.full((sum(total), HKV, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            dsa.kv_write8(k, v, slots, kc, vc, sc, dev_err=self.err)
            dsa.kv_read8(batch, kc, vc, sc, start, *packed, past=True, dev_err=self.err)
            for i, r in enumerate(rows):
                a, b = int(start[i]), qsl[i]
                for p, x, keep in zip(packed, (k, v), self.keys[layer][r]):
                    assert bool((p[a + past[i]:a + total[i]] == 9).all())   # its own rows are not read back
                    p[a + past[i]:a + total[i]] = x[b:b + lens[i]]
                    keep.append(x[b:b + lens[i]])
            out, lse = dsa.attn_prompt(batch, q, *packed, kv_start=start, dev_err=self.err)
            for i, r in enumerate(rows):
                a, b = int(start[i]), qsl[i]
                stored = self.stored(layer, r)
                for p, x in zip(packed, stored):
                    assert torch.equal(p[a:a + past[i]].double(), x[:past[i]])
                for e in range(HQ):
                    kk, vv = (p[a:a + total[i], e // 4] for p in packed)
                    check(out[b:b + lens[i], e], lse[b:b + lens[i], e],
                          attend_rows(q[b:b + lens[i], e], kk, vv, range(past[i] + 1, total[i] + 1), D ** -0.5,
                                      torch.bfloat16))

    def fork(self, parents, children):
        dsa.pages_fork(self.refs, self.bt, self.seq, i32(parents), i32(children), self.caches, dev_err=self.err)
        for layer in range(2):
            for p, c in zip(parents, children):
                self.keys[layer][c] = tuple(list(x) for x in self.keys[layer][p])

    def step(self, rows):
        """One new token per row through a stack of an F and an S layer, whose
        consumer runs the sparse attention with every key selected."""
        lens = (self.seq[rows] + 1).tolist()
        for r, n in zip(rows, lens):
            self.take_pages(r, n)
        self.seq[rows] += 1
        n = len(rows)
        bt = self.bt[rows].contiguous()
        batch = dsa.Batch(i32(list(range(n + 1))), i32(lens), bt, i32(list(range(n))), n, BLOCKS)
        slots = torch.cat([slots_of(bt, i, lens[i] - 1, lens[i]) for i in range(n)])
        q = [rand(self.g, n, HQ, D) for _ in range(2)]
        for layer, cache in enumerate(self.kv):
            k, v = (rand(self.g, n, HKV, D) * 2 ** (lens[0] % 3) for _ in range(2))   # larger rows: scales rise
            dsa.kv_write8(k, v, slots, *cache, dev_err=self.err)
            for i, r in enumerate(rows):
                self.keys[layer][r][0].append(k[i:i + 1])
                self.keys[layer][r][1].append(v[i:i + 1])
        fs, _ = dsa.schedule_build(2, pattern="FS")
        layers = [dict(q=rand(self.g, n, 64, 128), w=torch.rand((n, 64), generator=self.g, device=DEV),
                       k_new=rand(self.g, n, 128), k_cache=self.index), None]
        got = {}

        def consumer(layer, producer, phys, valid):
            got[layer] = dsa.attn_selected8(q[layer], *self.kv[layer], stack.phys_buf, dev_err=self.err)

        stack = dsa.LayerStack(batch, fs, layers, 1024, slot_mapping=slots, consumer=consumer, dev_err=self.err)
        stack.run()
        assert stack.valid_buf.tolist() == lens
        for layer in range(2):
            dense = dsa.attn_decode8(batch, q[layer], *self.kv[layer], dev_err=self.err)
            for i, r in enumerate(rows):
                k, v, sv = self.stored(layer, r)
                assert k.shape[0] == lens[i]
                for e in range(HQ):
                    h = e // 4
                    ref = kv8_ref.attend(q[layer][i, e], k[:, h], v[:, h], sv[:, h], D ** -0.5, torch.bfloat16)
                    for out, lse in (got[layer], dense):
                        check(out[i, e], lse[i, e], ref, f"layer {layer} row {r} head {e}")
        assert dsa.check_device_error(self.err) == 0


def test_serving_loop():
    s = Loop8(1)
    s.chunk([0, 1], [200, 37])
    s.chunk([0, 1], [101, 93])         # the second chunks end inside blocks of the scales
    s.step([0, 1])
    s.fork([0, 0, 1], [2, 3, 4])       # parallel samples: shared full pages, their own last page and its scales
    assert s.refs.max() == 3
    for _ in range(4):
        s.step([0, 1, 2, 3, 4])        # every sequence grows on its own
    dsa.pages_free(s.refs, s.bt, s.seq, i32([0, 2]), dev_err=s.err)
    s.keys = [[k if r not in (0, 2) else ([], []) for r, k in enumerate(layer)] for layer in s.keys]
    s.step([1, 3, 4])
    used = int((s.refs > 0).sum())
    dsa.pages_compact(s.refs, s.bt, s.caches, dev_err=s.err)
    assert int((s.refs[:used] > 0).sum()) == used and int(s.bt.max()) < used
    s.step([1, 3, 4])                  # the same contexts at new places
    s.chunk([2], [130])                # a new sequence in pages that others have used
    s.step([2, 4])
    dsa.pages_free(s.refs, s.bt, s.seq, i32([1, 2, 3, 4]), dev_err=s.err)
    assert int(s.refs.abs().sum()) == 0 and dsa.check_device_error(s.err) == 0


def test_python_calls_refuse_what_does_not_fit():
    k, v, sc = dsa.new_kv_cache8(4, 2, 128)
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((3, 8), dtype=torch.int32, device=DEV)
    slots = torch.arange(3, device=DEV)
    start = i32([0, 1, 2])
    b = dsa.Batch(i32([0, 1, 2, 3]), i32([5, 6, 7]), i32([[0], [1], [2]]), i32([0, 1, 2]), 3, 4)
    shifted = torch.zeros(3 * 512 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(3, 4, 128)
    odd = torch.zeros(4 * 64 * 2 * 128 + 8, dtype=torch.uint8, device=DEV)[8:].view(k.dtype).view(k.shape)
    wrong = [
        lambda: dsa.attn_selected8(q.float(), k, v, sc, ids),                     # no fp32
        lambda: dsa.attn_selected8(q, k.view(torch.uint8), v, sc, ids),           # codes are E4M3
        lambda: dsa.attn_selected8(q, k, v[:3], sc, ids),                         # shapes differ
        lambda: dsa.attn_selected8(q, k, v, sc[:3], ids),
        lambda: dsa.attn_selected8(q, k, v, sc.half(), ids),
        lambda: dsa.attn_selected8(q, k, v, sc.transpose(2, 3), ids),
        lambda: dsa.attn_selected8(q, k, v, torch.zeros((4, 4, 2, 4), device=DEV)[..., ::2], ids),
        lambda: dsa.attn_selected8(q[:, :3], k, v, sc, ids),                      # heads do not divide
        lambda: dsa.attn_selected8(q[..., :64], k, v, sc, ids),                   # head sizes differ
        lambda: dsa.attn_selected8(q, k, v, sc, ids[:2]),                         # rows differ
        lambda: dsa.attn_selected8(q, k, v, sc, ids.long()),
        lambda: dsa.attn_selected8(q, k, v, sc, ids[:, ::2]),                     # not contiguous
        lambda: dsa.attn_selected8(q, k, v, sc, ids, out=q[:2]),
        lambda: dsa.attn_selected8(q, k, v, sc, ids, lse=torch.zeros((3, 5), device=DEV)),
        lambda: dsa.attn_selected8(q, k[:, :32], v[:, :32], sc, ids),             # pages of 32
        lambda: dsa.attn_selected8(q, odd, v, sc, ids),                           # 8 bytes off a 16-byte boundary
        lambda: dsa.attn_decode8(b, q[:2], k, v, sc),                             # too few rows
        lambda: dsa.attn_decode8(b, q, k[:3], v[:3], sc[:3]),                     # another pool than the batch's
        lambda: dsa.attn_decode8(b, shifted, k, v, sc),
        lambda: dsa.attn_decode8(b, q, k, v, sc, ws=torch.zeros(64, device=DEV)), # scratch is bytes
        lambda: dsa.kv_write8(q, q, slots, k, v, sc),                             # 4 heads into 2
        lambda: dsa.kv_write8(x, x.half(), slots, k, v, sc),
        lambda: dsa.kv_write8(x, x, start, k, v, sc),                             # int32 slots
        lambda: dsa.kv_write8(x, x[:2], slots, k, v, sc),
        lambda: dsa.kv_write8(x.repeat(700, 1, 1), x.repeat(700, 1, 1), slots.repeat(700), k, v, sc,
                              ws=torch.zeros(16, dtype=torch.uint8, device=DEV)),  # too little scratch
        lambda: dsa.kv_read8(b, k, v, sc, start, q, q),
        lambda: dsa.kv_read8(b, k, v, sc, start[:2], x, x),                       # an entry per request
        lambda: dsa.kv_read8(b, k, v, sc, slots, x, x),
        lambda: dsa.kv_read8(b, k, v, sc, start, x, x.cpu()),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(dsa.DsaError):
            call()
            print("accepted:", i)
    torch.cuda.synchronize()


def test_results_are_made_on_the_given_stream():
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v, sc = dsa.new_kv_cache8(40, HKV, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = [rand(g, 2000, HKV, D) for _ in range(2)]
    slots = torch.arange(2000, device=DEV)
    q = rand(g, 1, HQ, D)
    b = dsa.Batch(i32([0, 1]), i32([2000]), torch.arange(40, dtype=torch.int32, device=DEV)[None], i32([0]), 1, 40)
    phys = torch.arange(2000, dtype=torch.int32, device=DEV)[None]
    side.wait_stream(torch.cuda.current_stream())
    dsa.kv_write8(*x, slots, k, v, sc, stream=side)     # its scratch is made there too
    got = dsa.attn_decode8(b, q, k, v, sc, stream=side), dsa.attn_selected8(q, k, v, sc, phys, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    kk, vv = (kv8_ref.value(c, sc[..., i]).flatten(0, 1)[:2000] for i, c in enumerate((k, v)))
    sv = sc[..., 1].repeat_interleave(16, 1).flatten(0, 1)[:2000]
    for out, lse in got:
        for e in range(HQ):
            check(out[0, e], lse[0, e], kv8_ref.attend(q[0, e], kk[:, e // 4], vv[:, e // 4], sv[:, e // 4], D ** -0.5,
                                                       torch.bfloat16))
