"""The 8-bit cache in 64 bits: a plain writer, and how far attention over it may be
from plain attention over the values that codes and scales stand for.

Error of a row of attention, from the arithmetic (u = half a step of the result's
type; p_j the weights of the softmax; sv_j, cv_j V's scales and codes, v_j their
product; A = sum_j p_j |v_j|):
  * a score is a sum of D products in fp32, two roundings by the scales and one when
    log2(sv_j) is added, whose own error is two steps of fp32 or 2^-22: es <= (D + 8) *
    2^-23 * (sum_d |q_d k_d| * scale + |s|) + 2^-21 * (1 + |log2 sv_j|), where 2^-23
    allows for truncating adders; bf16 rows of q are moved to fp16, where an element
    is off by 2^-39 of the row's largest at most: D * 2^-39 * max |q| * max |k| * scale
    more; a weight e^s is off by es plus the exponential's 2^-21, relative;
  * the weights p_j sv_j are rounded to fp16 for the product with the codes: 2^-11 *
    A; below 2^-14 to multiples of 2^-24, an error of 2^-25 at most, where the largest
    is 2^6 or more: n * 2^-31 of the largest p_j sv_j times 448;
  * fp32 sums over n keys: n * 2^-24 * A in the numerator, n * 2^-24 of the sum;
  * the result is rounded to the type: u * |out| (fp16: or half its least step).
"""
import math

import torch

F8 = torch.float8_e4m3fn


def round_e4m3(x):
    """x (64 bits) to the nearest E4M3 value, ties to even; magnitudes of 448 at most."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.where(x == 0, x, torch.round(x / step) * step)


def need(amax):
    """The least power of two with amax <= 448 * it, at least 2^-64."""
    e = -64
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def write(codes, scale, rows, slots):
    """One call's rows [tokens, heads, d] (64 bits) into codes [blocks, 64, heads, d]
    and scale [blocks, 4, heads] (64 bits, on the CPU), in place."""
    blocks = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * 64:
            blocks.setdefault(s // 16, {})[s % 16] = t   # the last of several
    for b, at in blocks.items():
        page, part = b // 4, b % 4
        there = codes[page, 16 * part:16 * part + 16]
        new = torch.stack([rows[t] for t in at.values()])
        for h in range(codes.shape[2]):
            x = new[:, h]
            fine = x[torch.isfinite(x)]
            s = need(float(fine.abs().max()) if fine.numel() else 0.0)
            old = float(scale[page, part, h])
            if 0 not in at and 0 < old < math.inf:
                if old < s:
                    there[:, h] = round_e4m3(there[:, h] * old / s)
                s = max(s, old)
            scale[page, part, h] = s
            there[list(at), h] = round_e4m3(torch.where(torch.isfinite(x), x, math.nan) / s)


def value(codes, scale):
    """Values [blocks, 64, heads, d] in 64 bits of an 8-bit cache's K or V (its half of
    the scales)."""
    return codes.to(torch.float32).double() * scale.double().repeat_interleave(16, 1)[..., None]


def attend(q, k, v, sv, scale, dtype):
    """One query head over the keys it sees: q [D], values k, v [n, D] and V's scales
    sv [n]; returns (out, lse, out tolerance, lse tolerance) in 64 bits."""
    q, k, v, sv = q.double(), k.double(), v.double(), sv.double()
    n, d = k.shape
    if n == 0:
        return torch.zeros_like(q), -math.inf, torch.zeros_like(q), 0.0
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    out = p @ v
    a = p @ v.abs()
    u = torch.finfo(dtype).eps / 2
    es = (d + 8) * 2.0 ** -23 * float(((k.abs() @ q.abs()) * scale + s.abs()).max())
    es += d * 2.0 ** -39 * float(q.abs().max() * k.abs().max()) * scale
    es += 2.0 ** -21 * (2 + float(torch.log2(sv).abs().max()))
    sums = n * 2.0 ** -24
    low = n * 2.0 ** -31 * float((p * sv).max()) * 448
    tol = (2.0 ** -11 + 2 * es + 2 * sums) * a + u * out.abs() + low + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    return out, float(lse), tol, es + sums + 2.0 ** -22 * (1 + abs(float(lse)))
