"""The attention, the cache's writer, the page calls and the indexer's layer
runner together, as a serving loop uses them: prompts, forked sequences, decode
steps over selected and over all keys, ended sequences, a compacted pool."""
import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests.attn_ref import attend, attend_rows, check

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, BLOCKS, WIDTH = 8, 2, 128, 64, 10


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def slots_of(bt, row, first, last):
    j = torch.arange(first, last, device=DEV)
    return bt[row].long()[j // 64] * 64 + j % 64


class Loop:
    """Two layers' KV caches and one indexer cache over one pool of pages."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv = [dsa.new_kv_cache(BLOCKS, HKV, D) for _ in range(2)]
        self.index = dsa.new_k_cache(BLOCKS)
        self.refs = torch.zeros(BLOCKS, dtype=torch.int32, device=DEV)
        self.bt = torch.full((8, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.seq = torch.zeros(8, dtype=torch.int32, device=DEV)
        self.err = i32([0])
        self.keys = [[[] for _ in range(8)] for _ in range(2)]  # [layer][row]: (k, v) as written

    @property
    def caches(self):
        return [c for pair in self.kv for c in pair] + [self.index]

    def prompt(self, rows, lens):
        """Whole prompts into rows; checks the attention of both layers."""
        perm = torch.randperm(BLOCKS, generator=self.g, device=DEV).tolist()
        for r, n in zip(rows, lens):
            for j in range((n + 63) // 64):
                self.bt[r, j] = perm.pop()
                self.refs[self.bt[r, j].long()] = 1
            self.seq[r] = n
        qsl = [0]
        for n in lens:
            qsl.append(qsl[-1] + n)
        batch = dsa.Batch(i32(qsl), i32(lens), self.bt[rows].contiguous(), i32([i for i, n in enumerate(lens)
                                                                               for _ in range(n)]), 0, BLOCKS)
        slots = torch.cat([slots_of(self.bt, r, 0, n) for r, n in zip(rows, lens)])
        dsa.indexer_k_quant_write(rand(self.g, qsl[-1], 128), slots, self.index, self.err)
        for layer, (kc, vc) in enumerate(self.kv):
            q, k, v = rand(self.g, qsl[-1], HQ, D), rand(self.g, qsl[-1], HKV, D), rand(self.g, qsl[-1], HKV, D)
            dsa.kv_write(k, v, slots, kc, vc, dev_err=self.err)
            out, lse = dsa.attn_prompt(batch, q, kc, vc, dev_err=self.err)
            packed, plse = dsa.attn_prompt(batch, q, k, v, kv_start=i32(qsl[:-1]))
            assert torch.equal(out, packed) and torch.equal(lse, plse)  # the same keys, paged or packed
            for i, (r, n) in enumerate(zip(rows, lens)):
                a, b = qsl[i], qsl[i + 1]
                self.keys[layer][r] = [(k[a:b], v[a:b])]
                for e in range(HQ):
                    check(out[a:b, e], lse[a:b, e], attend_rows(q[a:b, e], k[a:b, e // 4], v[a:b, e // 4],
                                                                range(1, n + 1), D ** -0.5, torch.bfloat16))

    def fork(self, parents, children):
        dsa.pages_fork(self.refs, self.bt, self.seq, i32(parents), i32(children), self.caches, dev_err=self.err)
        for layer in range(2):
            for p, c in zip(parents, children):
                self.keys[layer][c] = list(self.keys[layer][p])

    def step(self, rows):
        """One new token per row through a stack of an F and an S layer, whose
        consumer runs the sparse attention; every key is selected, so the dense
        decode attention must agree, and the plain one."""
        self.seq[rows] += 1
        lens = self.seq[rows].tolist()
        n = len(rows)
        bt = self.bt[rows].contiguous()
        batch = dsa.Batch(i32(list(range(n + 1))), i32(lens), bt, i32(list(range(n))), n, BLOCKS)
        slots = torch.cat([slots_of(bt, i, lens[i] - 1, lens[i]) for i in range(n)])
        q = [rand(self.g, n, HQ, D) for _ in range(2)]
        for layer, (kc, vc) in enumerate(self.kv):
            k, v = rand(self.g, n, HKV, D), rand(self.g, n, HKV, D)
            dsa.kv_write(k, v, slots, kc, vc, dev_err=self.err)
            for i, r in enumerate(rows):
                self.keys[layer][r].append((k[i:i + 1], v[i:i + 1]))
        fs, _ = dsa.schedule_build(2, pattern="FS")
        layers = [dict(q=rand(self.g, n, 64, 128), w=torch.rand((n, 64), generator=self.g, device=DEV),
                       k_new=rand(self.g, n, 128), k_cache=self.index), None]
        got = {}

        def consumer(layer, producer, phys, valid):
            got[layer] = dsa.attn_selected(q[layer], *self.kv[layer], stack.phys_buf, dev_err=self.err)

        stack = dsa.LayerStack(batch, fs, layers, 1024, slot_mapping=slots, consumer=consumer, dev_err=self.err)
        stack.run()
        assert sorted(got) == [0, 1]
        assert stack.valid_buf.tolist() == lens
        for layer in range(2):
            dense = dsa.attn_decode(batch, q[layer], *self.kv[layer], dev_err=self.err)
            for i, r in enumerate(rows):
                k, v = (torch.cat([x[j] for x in self.keys[layer][r]]) for j in (0, 1))
                assert k.shape[0] == lens[i]
                for e in range(HQ):
                    ref = attend(q[layer][i, e], k[:, e // 4], v[:, e // 4], D ** -0.5, torch.bfloat16)
                    for out, lse in (got[layer], dense):
                        check(out[i, e], lse[i, e], ref, f"layer {layer} row {r} head {e}")
        assert dsa.check_device_error(self.err) == 0


def test_serving_loop():
    s = Loop(1)
    s.prompt([0, 1], [300, 130])
    s.step([0, 1])
    s.fork([0, 0, 1], [2, 3, 4])       # parallel samples: shared full pages, their own last page
    assert s.refs.max() == 3
    s.step([0, 1, 2, 3, 4])            # every sequence grows on its own
    s.step([3, 4, 1, 2, 0])
    dsa.pages_free(s.refs, s.bt, s.seq, i32([0, 2]), dev_err=s.err)
    s.step([1, 3, 4])
    used = int((s.refs > 0).sum())
    dsa.pages_compact(s.refs, s.bt, s.caches, dev_err=s.err)
    assert int((s.refs[:used] > 0).sum()) == used and int(s.bt.max()) < used
    s.step([1, 3, 4])                  # the same contexts at new places
    dsa.pages_free(s.refs, s.bt, s.seq, i32([1, 3, 4]), dev_err=s.err)
    assert int(s.refs.abs().sum()) == 0 and dsa.check_device_error(s.err) == 0


def test_python_calls_refuse_what_does_not_fit():
    k, v = dsa.new_kv_cache(4, 2, 128)
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((3, 8), dtype=torch.int32, device=DEV)
    b = dsa.Batch(i32([0, 1, 2, 3]), i32([5, 6, 7]), i32([[0], [1], [2]]), i32([0, 1, 2]), 3, 4)
    shifted = torch.zeros(3 * 512 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(3, 4, 128)
    wrong = [
        lambda: dsa.attn_selected(q.half(), k, v, ids),                       # types differ
        lambda: dsa.attn_selected(q.float(), k.float(), v.float(), ids),      # no fp32
        lambda: dsa.attn_selected(q, k, v[:3], ids),                          # shapes differ
        lambda: dsa.attn_selected(q, k, v.half(), ids),
        lambda: dsa.attn_selected(q[:, :3], k, v, ids),                       # heads do not divide
        lambda: dsa.attn_selected(q[..., :64], k, v, ids),                    # head sizes differ
        lambda: dsa.attn_selected(q, k, v, ids[:2]),                          # rows differ
        lambda: dsa.attn_selected(q, k, v, ids.long()),
        lambda: dsa.attn_selected(q, k, v, ids[:, ::2]),                      # not contiguous
        lambda: dsa.attn_selected(q, k, v, ids, out=q[:2]),
        lambda: dsa.attn_selected(q, k, v, ids, lse=torch.zeros((3, 5), device=DEV)),
        lambda: dsa.attn_selected(q.transpose(0, 1).contiguous().transpose(0, 1)[..., ::2], k[..., ::2], v[..., ::2], ids),
        lambda: dsa.attn_selected(q, k[:, :32], v[:, :32], ids),              # pages of 32
        lambda: dsa.attn_decode(b, q[:2], k, v),                              # too few rows
        lambda: dsa.attn_decode(b, q, k[:3], v[:3]),                          # another pool than the batch's
        lambda: dsa.attn_decode(b, shifted, k, v),                            # 8 bytes off a 16-byte boundary
        lambda: dsa.attn_prompt(b, q, k, v, kv_start=i32([0, 1, 2])),         # packed rows are 3-D
        lambda: dsa.attn_prompt(b, q, k[0], v[0], kv_start=i32([0, 1])),      # an entry per request
        lambda: dsa.kv_write(q, q, torch.arange(3, device=DEV), k, v),        # 4 heads into 2
        lambda: dsa.kv_write(q[:, :2], q[:, :2], i32([0, 1, 2]), k, v),       # int32 slots
        lambda: dsa.pages_copy([k, v[:3]], i32([0]), i32([1])),
        lambda: dsa.pages_copy([k.transpose(1, 2)[:, :, ::2]], i32([0]), i32([1])),
        lambda: dsa.pages_copy([k], i32([0]), i32([1, 2])),
        lambda: dsa.pages_fork(i32([0] * 4), i32([[0]]), i32([1, 2]), i32([0]), i32([0])),
        lambda: dsa.pages_free(i32([0] * 4), i32([[0]]), None, i32([0])),
        lambda: dsa.pages_compact(i32([[0] * 4]), i32([[0]])),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(dsa.DsaError):
            call()
            print("accepted:", i)
    torch.cuda.synchronize()


def test_results_are_made_on_the_given_stream():
    s = Loop(2)
    s.prompt([0], [200])
    g = torch.Generator(device=DEV).manual_seed(3)
    q = rand(g, 1, HQ, D)
    b = dsa.Batch(i32([0, 1]), i32([200]), s.bt[:1].contiguous(), i32([0]), 1, BLOCKS)
    want = dsa.attn_decode(b, q, *s.kv[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    phys = slots_of(s.bt, 0, 0, 200).to(torch.int32)[None].contiguous()
    side.wait_stream(torch.cuda.current_stream())
    a = dsa.attn_decode(b, q, *s.kv[0], stream=side)
    c = dsa.attn_selected(q, *s.kv[0], phys, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    for e in range(HQ):
        k, v = s.keys[0][0][0]
        check(c[0][0, e], c[1][0, e], attend(q[0, e], k[:, e // 4], v[:, e // 4], D ** -0.5, torch.bfloat16))
