"""The 8-bit cache where a scale is not a power of two, or a V scale less than 2^-64:
what the header says of them, against 64 bits."""
import math

import pytest
import torch

import dsa_sparse_attention_quant_gb300 as dsa
from tests import kv8_ref
from tests.test_gpu_kv8_cache import Mirror, cache8, i32, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def halfway(gen, n, bits):
    """n numbers in [1, 2) of `bits` bits that end in a one: half-way between two of one bit less."""
    return 1 + (2 * torch.randint(0, 1 << (bits - 2), (n,), generator=gen) + 1).double() * 2.0 ** (1 - bits)


def round_to(x, dtype):
    """x (64 bits, finite, within the range) to the type's nearest value, ties to even, in one step."""
    info = torch.finfo(dtype)
    e = torch.clamp(torch.frexp(x)[1].double() - 1, min=math.log2(info.tiny))
    step = torch.exp2(e) * info.eps
    return torch.round(x / step) * step


# ----------------------------------------------------------------------- write

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_write_joins_blocks_of_any_scale(dtype, d):
    # some scales stay, some are raised
    g = torch.Generator(device=DEV).manual_seed(d)
    k, v, sc = cache8(g, 40, 3, d)
    sc *= 1 + torch.rand(sc.shape, generator=g, device=DEV)
    m = Mirror(k, v, sc)
    m.write(*rows(g, 40, 3, d, dtype, 3.0), [64 * i + 20 for i in range(40)])
    m.check()
    m.write(*rows(g, 40, 3, d, dtype, 3.0), [64 * i + 21 for i in range(40)])
    m.check()


@pytest.mark.parametrize("n", [160, 1200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_write_quotients_beside_a_tie(dtype, n):
    # x / scale is half-way between two codes but for the scale's own rounding: less than 32 bits tell apart
    g = torch.Generator().manual_seed(n)
    blocks, hkv, d = n // 4, 4, 64
    k, v, sc = cache8(torch.Generator(device=DEV).manual_seed(n), blocks, hkv, d)
    new = []
    for i in range(2):
        x = torch.zeros((blocks * 4, hkv, d), dtype=dtype)
        mag = (1 + torch.rand(blocks * 4 * hkv, generator=g)).to(dtype)
        x[:, :, 7] = mag.view(-1, hkv) * (1 - 2 * torch.randint(0, 2, (blocks * 4, hkv), generator=g)).to(dtype)
        tie = halfway(g, mag.numel(), 5) * 2.0 ** torch.randint(-5, 7, (mag.numel(),), generator=g).double()
        sc[..., i] = (mag.double() / tie).float().view(blocks, 4, hkv).to(DEV)
        new.append(x.to(DEV))
    m = Mirror(k, v, sc)
    m.write(*new, [16 * i + 5 for i in range(4 * blocks)])
    m.check()


@pytest.mark.parametrize("raise_by", [1, 3, 8])
def test_write_raises_a_scale_beside_a_tie(raise_by):
    # the codes that are there, times the old scale over the raised one, as above
    g = torch.Generator().manual_seed(raise_by)
    blocks, hkv, d = 60, 4, 64
    k, v, sc = cache8(torch.Generator(device=DEV).manual_seed(1), blocks, hkv, d)
    for i, c in enumerate((k, v)):
        m = torch.randint(9, 16, (blocks * 4 * hkv,), generator=g)           # significand of the code, in eighths
        code = (m.double() / 8 * 16).view(blocks, 4, hkv)
        old = halfway(g, m.numel(), 5).view(blocks, 4, hkv) / code * 16      # in (0.5, 2)
        old = torch.where(old >= 1, old / 2, old).float()
        sc[..., i] = old.to(DEV)
        at = code.float().to(DEV).to(F8)
        for b in range(4):
            c[:, 16 * b + 9, :, 3] = at[:, b]
    m = Mirror(k, v, sc)
    x = torch.full((blocks * 4, hkv, d), 0.25, dtype=torch.bfloat16, device=DEV)
    x[:, :, 0] = 440.0 * 2.0 ** (raise_by - 1)
    m.write(x, -x, [16 * i + 5 for i in range(4 * blocks)])
    assert bool((m.sc == 2.0 ** (raise_by - 1)).all())
    m.check()


# ------------------------------------------------------------------------ read

def read_all(k, v, sc, dtype):
    blocks, _, hkv, d = k.shape
    batch = dsa.Batch(i32([0, 0]), i32([64 * blocks]), torch.arange(blocks, dtype=torch.int32, device=DEV)[None],
                      i32([]), 0, blocks)
    out = [torch.zeros((64 * blocks, hkv, d), dtype=dtype, device=DEV) for _ in range(2)]
    err = i32([0])
    dsa.kv_read8(batch, k, v, sc, i32([0]), *out, dev_err=err)
    assert int(err.item()) == 0
    return [o.view(blocks, 64, hkv, d) for o in out]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_read_rounds_once(dtype, d):
    # products half-way between two values of the type but for the scale's own rounding, and others
    g = torch.Generator().manual_seed(d)
    blocks, hkv = 50, 3
    k, v, sc = cache8(torch.Generator(device=DEV).manual_seed(d), blocks, hkv, d)
    bits = round(1 - math.log2(torch.finfo(dtype).eps))
    for i, c in enumerate((k, v)):
        n = blocks * 4 * hkv
        code = (torch.randint(9, 16, (n,), generator=g).double() / 8).view(blocks, 4, hkv)
        tie = halfway(g, n, bits + 1).view(blocks, 4, hkv)
        sc[..., i] = (tie / code).float().to(DEV)
        c[:, ::16, :, 3] = code.float().to(DEV).to(F8)
    for c, s, out in zip((k, v), (sc[..., 0], sc[..., 1]), read_all(k, v, sc, dtype)):
        want = round_to(kv8_ref.value(c, s).cpu(), dtype)
        assert torch.equal(out.double().cpu(), want)


@pytest.mark.parametrize("d", [64, 128])
def test_read_small_scales_of_values_as_attention_does(d):
    # V's scales below 2^-64 count as 2^-64, as in the attention over the same cache
    k, v, sc = cache8(torch.Generator(device=DEV).manual_seed(d), 3, 2, d)
    small = [0.0, 2.0 ** -65, 1.5 * 2.0 ** -65, 2.0 ** -100, 2.0 ** -64, 1.25 * 2.0 ** -64]
    for i, x in enumerate(small):
        sc[i // 4, i % 4, :, 1] = x
    ko, vo = read_all(k, v, sc, torch.bfloat16)
    assert torch.equal(ko.double().cpu(), round_to(kv8_ref.value(k, sc[..., 0]).cpu(), torch.bfloat16))
    want = round_to(kv8_ref.value(v, sc[..., 1].clamp(min=2.0 ** -64)).cpu(), torch.bfloat16)
    assert torch.equal(vo.double().cpu(), want)
    # one key: its weight is 1, so attention gives its V row (in fp32, rounded to the type)
    q = torch.randn((1, 2, d), device=DEV).to(torch.bfloat16)
    for i in range(len(small)):
        slot = 16 * i + 3
        out, _ = dsa.attn_selected8(q, k, v, sc, i32([[slot]]))
        got, row = out[0].double().cpu(), want[slot // 64, slot % 64]
        assert bool(((got - row).abs() <= 2.0 ** -7 * row.abs()).all()), small[i]
