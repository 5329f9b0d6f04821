"""The attention and page entry points without a GPU: their host checks refuse
bad arguments before anything is launched, empty calls succeed, valid ones
report that there is no device; and the Python calls refuse what they cannot pass
on."""
import ctypes

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from dsa_sparse_attention_quant_gb300 import attention, binding

P = ctypes.c_void_p
OK, EINVAL, ENOSPACE, ENODEV = binding.DSA_OK, binding.DSA_EINVAL, binding.DSA_ENOSPACE, binding.DSA_ENODEV
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers would reach the kernels")


def batch(**kw):
    b = dict(num_reqs=3, num_decodes=2, num_decode_tokens=2, num_tokens=12, max_seq_len=900, bt_stride=20,
             num_blocks=50, query_start_loc=256, seq_lens=256, block_table=256, req_id_per_token=256)
    b.update(kw)
    return binding.DsaBatchC(**b)


def kv(**kw):
    d = kw.get("head_dim", 128)
    c = dict(k=4096, v=8192, dtype=0, num_kv_heads=2, head_dim=d, num_blocks=50, k_page_stride=64 * 2 * d,
             k_slot_stride=2 * d, k_head_stride=d, v_page_stride=64 * 2 * d, v_slot_stride=2 * d, v_head_stride=d)
    c.update(kw)
    return binding.DsaKvC(**c)


def attn(**kw):
    a = dict(q=4096, q_row_stride=1024, q_head_stride=128, out=8192, out_row_stride=1024, out_head_stride=128,
             lse=None, num_heads=8, scale=0.0)
    a.update(kw)
    return binding.DsaAttnC(**a)


def decode(b=None, c=None, a=None, ws=4096, size=1 << 30):
    lib = binding.load()
    b, c, a = b or batch(), c or kv(), a or attn()
    return lib.dsa_attn_decode(ctypes.byref(b), ctypes.byref(c), ctypes.byref(a), P(ws), size, None, None)


def prompt(b=None, c=None, a=None, start=None):
    lib = binding.load()
    b, c, a = b or batch(), c or kv(), a or attn()
    return lib.dsa_attn_prompt(ctypes.byref(b), ctypes.byref(c), start, ctypes.byref(a), None, None)


def selected(c=None, a=None, phys=4096, n=4, topk=700, ws=4096, size=1 << 30):
    lib = binding.load()
    c, a = c or kv(), a or attn()
    return lib.dsa_attn_selected(ctypes.byref(c), ctypes.byref(a), P(phys), n, topk, P(ws), size, None, None)


BAD_KV = [dict(dtype=2), dict(dtype=-1), dict(num_kv_heads=0), dict(head_dim=96), dict(head_dim=256),
          dict(num_blocks=0), dict(num_blocks=2 ** 31), dict(k=None), dict(v=None), dict(k=4104), dict(v=8200),
          dict(k_slot_stride=0), dict(v_head_stride=4), dict(k_head_stride=132), dict(k_page_stride=-8),
          dict(v_page_stride=1 << 39), dict(num_kv_heads=3)]
BAD_ATTN = [dict(q=None), dict(out=None), dict(q=4104), dict(out=8200), dict(lse=4098), dict(num_heads=0),
            dict(num_heads=7), dict(num_heads=65536), dict(q_row_stride=1020), dict(q_head_stride=64),
            dict(out_row_stride=0), dict(out_head_stride=-128), dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_KV, ids=str)
def test_cache_descriptions_refused(bad):
    for call in (decode, prompt, selected):
        assert call(c=kv(**bad)) == EINVAL


@pytest.mark.parametrize("bad", BAD_ATTN, ids=str)
def test_attention_descriptions_refused(bad):
    for call in (decode, prompt, selected):
        assert call(a=attn(**bad)) == EINVAL


@pytest.mark.parametrize("scale", [float("nan"), 3e38])
def test_scales_refused(scale):
    for call in (decode, prompt, selected):
        assert call(a=attn(scale=scale)) == EINVAL


def test_batches_refused():
    for bad in (dict(num_reqs=-1), dict(num_decodes=4), dict(num_decode_tokens=13), dict(num_tokens=-1),
                dict(num_reqs=0, num_decodes=0), dict(max_seq_len=-1), dict(query_start_loc=None), dict(seq_lens=None),
                dict(block_table=None), dict(bt_stride=0), dict(req_id_per_token=None), dict(num_blocks=49)):
        assert decode(b=batch(**bad)) == EINVAL, bad
        assert prompt(b=batch(**bad)) == EINVAL, bad
    assert decode(b=batch(num_decodes=0)) == EINVAL   # decode tokens of no request
    assert prompt(b=batch(num_decodes=3)) == EINVAL   # prefill tokens of no request
    assert binding.load().dsa_attn_decode(None, None, None, None, 0, None, None) == EINVAL


def test_selected_refused():
    assert selected(phys=None) == EINVAL
    assert selected(topk=0) == EINVAL
    assert selected(n=-1) == EINVAL
    assert selected(n=1 << 31) == EINVAL


def test_scratch_checked_and_sized():
    lib = binding.load()
    b = batch()
    need = lib.dsa_attn_decode_workspace_size(ctypes.byref(b), 8, 2, 128)
    assert need > 0
    assert decode(size=need - 1) == ENOSPACE
    assert decode(ws=None) == EINVAL
    assert decode(ws=4104) == EINVAL
    need = lib.dsa_attn_selected_workspace_size(4, 700, 8, 2, 128)
    assert need > 0 and selected(size=need - 1) == ENOSPACE
    # short rows are not cut and need none
    assert lib.dsa_attn_selected_workspace_size(4, 64, 8, 2, 128) == 0
    assert lib.dsa_attn_decode_workspace_size(ctypes.byref(batch(max_seq_len=100)), 8, 2, 128) == 0
    for bad in ((4, 700, 7, 2, 128), (4, 700, 8, 2, 100), (-1, 700, 8, 2, 128), (4, 0, 8, 2, 128), (4, 700, 8, 0, 128)):
        assert lib.dsa_attn_selected_workspace_size(*bad) == 0
    assert lib.dsa_attn_decode_workspace_size(ctypes.byref(batch(num_reqs=-1)), 8, 2, 128) == 0
    # the scratch does not grow with the batch's length, but with the heads of a group
    assert lib.dsa_attn_selected_workspace_size(4096, 2048, 64, 8, 128) <= 16 << 20


def test_empty_calls_succeed_without_a_device():
    lib = binding.load()
    empty = binding.DsaBatchC(0, 0, 0, 0, 0, 1, 50, None, None, None, None)
    assert decode(b=empty) == OK and prompt(b=empty) == OK
    assert selected(n=0) == OK
    assert decode(b=batch(num_decodes=0, num_decode_tokens=0)) == OK   # no decode rows
    assert prompt(b=batch(num_decodes=3, num_decode_tokens=12)) == OK  # no prefill rows
    c = kv()
    assert lib.dsa_kv_write(None, 256, 128, None, 256, 128, 0, None, ctypes.byref(c), None, None) == OK


@no_gpu
def test_valid_calls_report_no_device():
    lib = binding.load()
    assert decode() == ENODEV
    assert selected() == ENODEV
    assert prompt() == ENODEV
    assert prompt(start=P(256)) == ENODEV
    # strides of one-element axes are not looked at
    assert decode(c=kv(num_kv_heads=1, k_head_stride=3, v_head_stride=0, num_blocks=1, k_page_stride=1),
                  b=batch(num_blocks=1)) == ENODEV
    c = kv()
    assert lib.dsa_kv_write(P(4096), 256, 128, P(4096), 256, 128, 5, P(256), ctypes.byref(c), None, None) == ENODEV
    g = binding.DsaPagesC(4096, 50, 4096, 20, 8, 4096)
    d = (binding.DsaCacheDescC * 1)(binding.DsaCacheDescC(4096, 8448, 8448))
    big = 1 << 30
    assert lib.dsa_pages_copy(d, 1, 50, P(256), P(256), 3, P(256), big, None, None) == ENODEV
    assert lib.dsa_pages_fork(ctypes.byref(g), P(256), P(256), 3, d, 1, P(256), big, None, None) == ENODEV
    assert lib.dsa_pages_free(ctypes.byref(g), P(256), 3, None, None) == ENODEV
    assert lib.dsa_pages_compact(ctypes.byref(g), d, 1, P(256), big, None, None) == ENODEV


def test_kv_write_refused():
    lib = binding.load()
    c = kv()

    def write(k=4096, kr=256, kh=128, v=4096, vr=256, vh=128, n=5, slots=256, c=c):
        return lib.dsa_kv_write(P(k), kr, kh, P(v), vr, vh, n, P(slots), ctypes.byref(c), None, None)
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(k=4104), dict(n=-1), dict(kr=100), dict(kh=64),
                dict(vr=0), dict(vh=130)):
        assert write(**bad) == EINVAL, bad
    for bad in BAD_KV:
        if bad != dict(num_kv_heads=3):
            assert write(c=kv(**bad)) == EINVAL, bad


def test_pages_refused():
    lib = binding.load()
    big = 1 << 30

    def pool(**kw):
        g = dict(refs=4096, num_blocks=50, block_table=4096, bt_stride=20, n_rows=8, seq_lens=4096)
        g.update(kw)
        return binding.DsaPagesC(**g)

    def caches(**kw):
        d = dict(base=4096, page_bytes=8448, page_stride=8448)
        d.update(kw)
        return (binding.DsaCacheDescC * 1)(binding.DsaCacheDescC(**d))

    def fork(g=None, n=3, d=None, m=1, ws=256, size=big, a=256, b=256):
        g = g or pool()
        return lib.dsa_pages_fork(ctypes.byref(g), P(a), P(b), n, d or caches(), m, P(ws), size, None, None)

    def compact(g=None, d=None, m=1, ws=256, size=big):
        g = g or pool()
        return lib.dsa_pages_compact(ctypes.byref(g), d or caches(), m, P(ws), size, None, None)

    def copy(d=None, m=1, blocks=50, n=3, ws=256, size=big, a=256, b=256):
        return lib.dsa_pages_copy(d or caches(), m, blocks, P(a), P(b), n, P(ws), size, None, None)

    def free(g=None, n=3, a=256):
        g = g or pool()
        return lib.dsa_pages_free(ctypes.byref(g), P(a), n, None, None)

    for bad in (dict(refs=None), dict(refs=4100), dict(num_blocks=0), dict(num_blocks=2 ** 26), dict(block_table=None),
                dict(bt_stride=0), dict(bt_stride=2 ** 26), dict(n_rows=-1), dict(seq_lens=None)):
        assert fork(g=pool(**bad)) == EINVAL, bad
        assert free(g=pool(**bad)) == EINVAL, bad
        if bad != dict(seq_lens=None):   # compaction does not use the lengths
            assert compact(g=pool(**bad)) == EINVAL, bad
    for bad in (dict(base=None), dict(base=4104), dict(page_bytes=0), dict(page_bytes=100), dict(page_stride=8440),
                dict(page_stride=8432), dict(page_bytes=2 << 30, page_stride=2 << 30)):
        for call in (fork, compact, copy):
            assert call(d=caches(**bad)) == EINVAL, bad
    for call in (fork, compact, copy):
        assert call(ws=None) == EINVAL and call(ws=264) == EINVAL and call(size=16) == ENOSPACE and call(m=-1) == EINVAL
    many = (binding.DsaCacheDescC * 1025)(*[binding.DsaCacheDescC(4096, 8448, 8448) for _ in range(1025)])
    for bad in (dict(a=None), dict(b=None), dict(n=-1)):
        assert fork(**bad) == EINVAL and copy(**bad) == EINVAL
    assert free(n=-1) == EINVAL and free(a=None) == EINVAL
    assert copy(blocks=0) == EINVAL
    assert fork(n=0) == OK and copy(n=0) == OK and free(n=0) == OK
    for call in (fork, compact, copy):
        assert call(d=many, m=1025) == EINVAL
    assert lib.dsa_pages_workspace_size(0, 1) == 0 and lib.dsa_pages_workspace_size(10, -1) == 0
    assert lib.dsa_pages_workspace_size(1000, 10) >= 3 * 4000 + 10 * 20


def test_struct_layouts_match_the_header():
    # the packed forms that the calls pass are the C structs, field by field
    raw = attention._KV.pack(1, 2, 1, 3, 64, 5, 6, 7, 8, 9, 10, 11)
    c = binding.DsaKvC.from_buffer_copy(raw)
    assert [getattr(c, f) for f, _ in c._fields_] == [1, 2, 1, 3, 64, 5, 6, 7, 8, 9, 10, 11]
    c = binding.DsaAttnC.from_buffer_copy(attention._ATTN.pack(1, 2, 3, 4, 5, 6, 7, 8, 0.5))
    assert [getattr(c, f) for f, _ in c._fields_] == [1, 2, 3, 4, 5, 6, 7, 8, 0.5]
    c = binding.DsaPagesC.from_buffer_copy(attention._PAGES.pack(1, 2, 3, 4, 5, 6))
    assert [getattr(c, f) for f, _ in c._fields_] == [1, 2, 3, 4, 5, 6]


def test_python_calls_refuse_cpu_tensors():
    k = torch.zeros((4, 64, 2, 128), dtype=torch.bfloat16)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    ids = torch.zeros((1, 8), dtype=torch.int32)
    for call in (lambda: dsa.attn_selected(q, k, k, ids), lambda: dsa.attn_decode(None, q, k, k),
                 lambda: dsa.attn_prompt(None, q, k, k), lambda: dsa.kv_write(q, q, ids, k, k),
                 lambda: dsa.pages_copy([k], ids[0], ids[0]), lambda: dsa.pages_compact(ids[0], ids, [k]),
                 lambda: dsa.pages_free(ids[0], ids, ids[0], ids[0]),
                 lambda: dsa.pages_fork(ids[0], ids, ids[0], ids[0], ids[0])):
        with pytest.raises(dsa.DsaError, match="CUDA tensor"):
            call()
    with pytest.raises(dsa.DsaError):
        dsa.new_kv_cache(4, 2, 96)
    with pytest.raises(dsa.DsaError):
        dsa.new_kv_cache(4, 2, 128, torch.float32)
    with pytest.raises(dsa.DsaError):
        dsa.pages_copy([], ids[0], ids[0])
