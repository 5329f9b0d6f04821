"""Plain attention in 64 bits, and how far the kernels may be from it.

Error of a kernel's row, from the arithmetic (u = half a step of the inputs'
type, ``torch.finfo(t).eps / 2``; A = sum_j p_j |v_j| / sum_j p_j):
  * a score is a sum of D products in fp32 and two roundings by the scale and
    the reference M: es <= (D + 8) * 2^-23 * (sum_d |q_d k_d| * scale + |s|),
    where 2^-23 allows for truncating adders; a weight e^s is off by es plus
    the exponential's 2^-21, relative;
  * weights are rounded to the type for the product with V: u * A;
  * fp32 sums over n keys: n * 2^-24 * A in the numerator, n * 2^-24 of the sum;
  * fp16 weights below 2^-24 are rounded to a multiple of it, an error of 2^-25
    at most, where the row's largest weight is 2^4 or more: n * 2^-29 of it,
    times max |v|;
  * the result is rounded to the type: u * |out| (fp16: or half its least step).
"""
import math

import torch


def attend(q, k, v, scale, dtype):
    """One query head over the keys it sees: q [D], k, v [n, D]; returns (out,
    lse, out tolerance, lse tolerance) in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    n, d = k.shape
    if n == 0:
        return torch.zeros_like(q), -math.inf, torch.zeros_like(q), 0.0
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    out = p @ v
    a = p @ v.abs()
    u = torch.finfo(dtype).eps / 2
    es = (d + 8) * 2.0 ** -23 * float(((k.abs() @ q.abs()) * scale + s.abs()).max()) + 2.0 ** -21
    sums = n * 2.0 ** -24
    low = n * 2.0 ** -29 * float(v.abs().max()) if dtype == torch.float16 else 0.0
    tol = (u + 2 * es + 2 * sums) * a + u * out.abs() + low + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    return out, float(lse), tol, es + sums + 2.0 ** -22 * (1 + abs(float(lse)))


def attend_rows(q, k, v, visible, scale, dtype):
    """As attend() for rows q [n, D] of one head over k, v [m, D]; row i sees
    the first visible[i] keys. Vectorised."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:   # a key that no row sees
        k, v = torch.zeros((2, 1, q.shape[1]), dtype=q.dtype, device=q.device)
    m, d = k.shape
    vis = torch.as_tensor(visible, device=q.device)
    seen = torch.arange(m, device=q.device)[None, :] < vis[:, None]
    raw = (q @ k.T) * scale
    s = torch.where(seen, raw, torch.full_like(raw, -math.inf))
    lse = torch.logsumexp(s, 1)
    p = torch.where(seen, torch.exp(s - torch.where(vis > 0, lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(s))
    out, a = p @ v, p @ v.abs()
    u = torch.finfo(dtype).eps / 2
    mag = torch.where(seen, (q.abs() @ k.abs().T) * scale + raw.abs(), torch.zeros_like(raw))
    es = (d + 8) * 2.0 ** -23 * mag.amax(1) + 2.0 ** -21
    sums = vis.double() * 2.0 ** -24
    low = vis.double() * 2.0 ** -29 * v.abs().max() if dtype == torch.float16 else sums * 0
    tol = (u + 2 * es + 2 * sums)[:, None] * a + u * out.abs() + low[:, None]
    tol = tol + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    return out, lse, tol, es + sums + 2.0 ** -22 * (1 + torch.where(vis > 0, lse, torch.zeros_like(lse)).abs())


def check(got, lse, ref, what=""):
    """got [..., D] and lse [...] of a kernel against attend()/attend_rows()."""
    out, want, tol, ltol = ref
    off = (got.double() - out).abs()
    worst = (off - tol).max()
    assert bool((off <= tol).all()), f"{what}: out off by {float(off.max()):.3g}, {float(worst):.3g} over the bound"
    want = torch.as_tensor(want, dtype=torch.float64, device=got.device)
    ltol = torch.as_tensor(ltol, dtype=torch.float64, device=got.device)
    lse = lse.double()
    empty = torch.isinf(want)
    assert bool((lse[empty] == -math.inf).all()), f"{what}: lse of an empty row"
    far = (lse - want).abs()[~empty]
    assert bool((far <= ltol.expand_as(want)[~empty]).all()), f"{what}: lse off by {float(far.max()):.3g}"
