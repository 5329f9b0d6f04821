"""The 8-bit cache's entry points without a GPU: host checks refuse bad arguments
before anything is launched, empty calls succeed, valid ones report that there is no
device; the kernels' sources keep the rules of launches that overlap."""
import ctypes

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from dsa_sparse_attention_quant_gb300 import attention, binding
from tests.test_attention_cpu import BAD_ATTN, attn, batch, kv, no_gpu
from tests.test_overlapped_launches_cpu import bodies, source

P = ctypes.c_void_p
OK, EINVAL, ENOSPACE, ENODEV = binding.DSA_OK, binding.DSA_EINVAL, binding.DSA_ENOSPACE, binding.DSA_ENODEV


def kv8(**kw):
    d = kw.get("head_dim", 128)
    c = dict(k=4096, v=8192, scale=12288, dtype=0, num_kv_heads=2, head_dim=d, num_blocks=50, k_page_stride=64 * 2 * d,
             k_slot_stride=2 * d, k_head_stride=d, v_page_stride=64 * 2 * d, v_slot_stride=2 * d, v_head_stride=d,
             s_page_stride=16, s_block_stride=4, s_head_stride=2)
    c.update(kw)
    return binding.DsaKv8C(**c)


def decode(b=None, c=None, a=None, ws=4096, size=1 << 30):
    return binding.load().dsa_attn_decode8(ctypes.byref(b or batch()), ctypes.byref(c or kv8()), ctypes.byref(a or attn()),
                                           P(ws), size, None, None)


def selected(c=None, a=None, phys=4096, n=4, topk=700, ws=4096, size=1 << 30):
    return binding.load().dsa_attn_selected8(ctypes.byref(c or kv8()), ctypes.byref(a or attn()), P(phys), n, topk, P(ws),
                                             size, None, None)


def write(k=4096, kr=256, kh=128, v=4096, vr=256, vh=128, n=5, slots=256, c=None, ws=None, size=0):
    return binding.load().dsa_kv_write8(P(k), kr, kh, P(v), vr, vh, n, P(slots), ctypes.byref(c or kv8()), P(ws), size,
                                        None, None)


def read(b=None, c=None, start=256, rows=None, past=0):
    return binding.load().dsa_kv_read8(ctypes.byref(b or batch()), ctypes.byref(c or kv8()), P(start),
                                       ctypes.byref(rows or kv(num_blocks=2000)), past, None, None)


BAD = [dict(dtype=2), dict(dtype=-1), dict(num_kv_heads=0), dict(num_kv_heads=65536), dict(head_dim=96),
       dict(num_blocks=0), dict(num_blocks=2 ** 25), dict(k=None), dict(v=None), dict(scale=None), dict(k=4104),
       dict(v=8200), dict(scale=12296), dict(k_slot_stride=0), dict(v_head_stride=8), dict(k_head_stride=136),
       dict(k_page_stride=-16), dict(v_page_stride=1 << 39), dict(s_page_stride=0), dict(s_block_stride=3),
       dict(s_head_stride=-2), dict(s_page_stride=1 << 39)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_cache_descriptions_refused(bad):
    for call in (decode, selected, write, read):
        assert call(c=kv8(**bad)) == EINVAL, call


@pytest.mark.parametrize("bad", BAD_ATTN + [dict(scale=float("nan")), dict(scale=3e38)], ids=str)
def test_attention_descriptions_refused(bad):
    assert decode(a=attn(**bad)) == EINVAL and selected(a=attn(**bad)) == EINVAL


def test_batches_refused():
    for bad in (dict(num_reqs=-1), dict(num_decodes=4), dict(num_decode_tokens=13), dict(num_tokens=-1),
                dict(num_reqs=0, num_decodes=0), dict(max_seq_len=-1), dict(query_start_loc=None), dict(seq_lens=None),
                dict(block_table=None), dict(bt_stride=0), dict(req_id_per_token=None), dict(num_blocks=49)):
        assert decode(b=batch(**bad)) == EINVAL, bad
    assert decode(b=batch(num_decodes=0)) == EINVAL   # decode tokens of no request
    assert binding.load().dsa_attn_decode8(None, None, None, None, 0, None, None) == EINVAL
    for bad in (dict(num_reqs=-1), dict(max_seq_len=-1), dict(seq_lens=None), dict(block_table=None), dict(bt_stride=0),
                dict(num_blocks=49), dict(max_seq_len=1 << 30, bt_stride=1 << 24)):
        assert read(b=batch(**bad)) == EINVAL, bad
    assert read(b=batch(query_start_loc=None), past=1) == EINVAL
    assert binding.load().dsa_kv_read8(None, None, None, None, 0, None, None) == EINVAL


def test_selected_refused():
    assert selected(phys=None) == EINVAL and selected(topk=0) == EINVAL
    assert selected(n=-1) == EINVAL and selected(n=1 << 31) == EINVAL


def test_write_refused():
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(k=4104), dict(n=-1), dict(n=1 << 31), dict(kr=100),
                dict(kh=64), dict(vr=0), dict(vh=130)):
        assert write(**bad) == EINVAL, bad


def test_read_refused():
    assert read(start=None) == EINVAL
    for bad in (dict(dtype=1), dict(num_kv_heads=1), dict(head_dim=64), dict(num_blocks=0), dict(k=None), dict(v=8200),
                dict(k_slot_stride=8), dict(v_head_stride=12)):
        assert read(rows=kv(**bad)) == EINVAL, bad


def test_scratch_checked_and_sized():
    lib = binding.load()
    b = batch(max_seq_len=50000, bt_stride=800)
    need = lib.dsa_attn_decode8_workspace_size(ctypes.byref(b), 8, 2, 128)
    assert need > 0 and decode(b=b, size=need - 1) == ENOSPACE
    assert decode(b=b, ws=None) == EINVAL and decode(b=b, ws=4104) == EINVAL
    need = lib.dsa_attn_selected8_workspace_size(4, 20000, 8, 2, 128)
    assert need > 0 and selected(topk=20000, size=need - 1) == ENOSPACE
    # short rows are not cut, or among CTAs that join them without scratch
    assert lib.dsa_attn_selected8_workspace_size(4, 64, 8, 2, 128) == 0
    assert lib.dsa_attn_selected8_workspace_size(4, 700, 8, 2, 128) == 0
    # what suffices for more tokens or longer rows suffices for fewer and shorter ones
    for hq, hkv in ((8, 8), (8, 1), (32, 8), (40, 2)):
        size = [[lib.dsa_attn_selected8_workspace_size(n, 64 * t, hq, hkv, 128) for t in (1, 3, 8, 9, 16, 33, 64, 65, 300)]
                for n in (1, 2, 5, 9, 20, 60, 150, 500, 4000)]
        assert all(a <= b for row in size for a, b in zip(row, row[1:]))
        assert all(a <= b for col in zip(*size) for a, b in zip(col, col[1:]))
    for bad in ((4, 700, 7, 2, 128), (4, 700, 8, 2, 100), (-1, 700, 8, 2, 128), (4, 0, 8, 2, 128), (4, 700, 8, 0, 128)):
        assert lib.dsa_attn_selected8_workspace_size(*bad) == 0
    assert lib.dsa_attn_decode8_workspace_size(ctypes.byref(batch(num_reqs=-1)), 8, 2, 128) == 0
    size = lib.dsa_kv_write8_workspace_size
    assert size(5, 50) == 0 and size(5000, 50) == 4 * 64 * 50 and size(5000, 0) == 0 and size(1 << 31, 50) == 0
    assert write(n=5000, ws=4096, size=4 * 64 * 50 - 1) == ENOSPACE
    assert write(n=5000, ws=None, size=1 << 30) == EINVAL and write(n=5000, ws=4104, size=1 << 30) == EINVAL


def test_empty_calls_succeed_without_a_device():
    empty = binding.DsaBatchC(0, 0, 0, 0, 0, 1, 50, None, None, None, None)
    assert decode(b=empty) == OK and read(b=empty) == OK
    assert decode(b=batch(num_decodes=0, num_decode_tokens=0)) == OK
    assert selected(n=0) == OK
    assert write(k=None, v=None, slots=None, n=0) == OK


@no_gpu
def test_valid_calls_report_no_device():
    assert decode() == ENODEV and selected() == ENODEV and write() == ENODEV and read() == ENODEV
    assert read(past=1) == ENODEV and read(b=batch(query_start_loc=None, req_id_per_token=None)) == ENODEV
    assert write(n=5000, ws=4096, size=1 << 20) == ENODEV
    # strides of one-element axes are not looked at
    one = kv8(num_kv_heads=1, k_head_stride=3, v_head_stride=0, s_head_stride=0, num_blocks=1, k_page_stride=1,
              s_page_stride=1)
    assert decode(c=one, b=batch(num_blocks=1)) == ENODEV
    assert write(c=one, n=1, kr=1, kh=1, vr=1, vh=1) == ENODEV


def test_struct_layout_matches_the_header():
    c = binding.DsaKv8C.from_buffer_copy(attention._KV8.pack(*range(1, 17)))
    assert [getattr(c, f) for f, _ in c._fields_] == list(range(1, 17))


def test_python_calls_refuse_what_they_cannot_pass_on():
    k, v, sc = dsa.new_kv_cache8(4, 2, 128, device="cpu")
    assert k.shape == v.shape == (4, 64, 2, 128) and sc.shape == (4, 4, 2, 2) and k.dtype == torch.float8_e4m3fn
    q, ids = torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.zeros((1, 8), dtype=torch.int32)
    for call in (lambda: dsa.attn_selected8(q, k, v, sc, ids), lambda: dsa.attn_decode8(None, q, k, v, sc),
                 lambda: dsa.kv_write8(q, q, ids, k, v, sc), lambda: dsa.kv_read8(None, k, v, sc, ids, q, q)):
        with pytest.raises(dsa.DsaError, match="CUDA tensor"):
            call()
    for bad in ((4, 2, 96), (0, 2, 64), (4, 0, 64)):
        with pytest.raises(dsa.DsaError):
            dsa.new_kv_cache8(*bad, device="cpu")


@pytest.mark.parametrize("name", ["attn_rows8.cu", "attn_rows.cuh", "kv8.cu"])
def test_nothing_is_read_as_read_only(name):
    text = source(name)
    for word in ("__ldg", "__restrict__", "ld.global.nc"):
        assert word not in text, word


KERNELS = {"attn_rows8_kernel", "write8_claim_kernel", "write8_few_kernel", "write8_many_kernel", "read8_kernel"}


def test_kernels_wait_whatever_they_have_to_do():
    # at the kernel's outermost level, before any return
    seen = set()
    for name, body in bodies():
        if name not in KERNELS:
            continue
        seen.add(name)
        head = body[:body.index("pdl_wait();")]
        assert head.count("{") == head.count("}") and "return" not in head, name
    assert seen == KERNELS
