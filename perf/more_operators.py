"""Timed cases of the operators around a K/V cache held in 8 bits: what a pass is,
its plain form in elementary torch operations, and its floor in bytes and
operations.

The cache has E4M3 codes [pages, 64, heads, d] for K and for V, and scales [pages,
4, heads, 2] (K's, V's): one power of two for each block of 16 slots and head. A
row's values are codes times scale.

  write     a step's K and V rows quantised into the cache at their slots
  read      sequences' rows back in 16 bits, packed, as prompt attention takes them
  decode    one new token per request over the request's pages
  selected  attention over the slots that the indexer selected for each token

Writing a block's first slot opens it: its scale is then the least power of two
that brings its new rows' largest magnitude to 448 at most, 2^-64 at least. Rows
that join a block may raise its scale, and the rows that are there are rounded to
the raised one.

``own`` chooses between the plain form and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 64   # slots of a page
GROUP = 16   # slots that share a scale
PARTS = BLOCK // GROUP
F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step: a token of each of 64 requests joins its block
        dict(name="write_64", op="write", reqs=64, lo=1, hi=1, past=3000, hkv=8, d=128, dtype="bf16"),
        # a few drafted tokens of three requests, small heads
        dict(name="write_3x7", op="write", reqs=3, lo=2, hi=7, past=500, hkv=2, d=64, dtype="fp16"),
        # a prefill step: eight chunks of prompts of uneven lengths, column views of a fused projection
        dict(name="write_prefill", op="write", reqs=8, lo=3500, hi=4096, past=37, hkv=8, d=128, dtype="bf16"),
        # one short cached prefix in front of a prompt
        dict(name="read_1x301", op="read", reqs=1, lo=301, hi=301, hkv=2, d=64, dtype="fp16"),
        # the cached prefixes of a prefill step's eight requests
        dict(name="read_8x16k", op="read", reqs=8, lo=12001, hi=16384, hkv=8, d=128, dtype="bf16"),
        # a single short conversation: one launch's latency
        dict(name="decode_1x300", op="decode", reqs=1, lo=300, hi=300, hq=32, hkv=8, d=128, dtype="bf16"),
        # a serving batch of 32 requests of 4K to 8K keys
        dict(name="decode_32x8k", op="decode", reqs=32, lo=4096, hi=8192, hq=64, hkv=8, d=128, dtype="bf16"),
        # long contexts, few requests: the length has to be split; odd lengths
        dict(name="decode_8x128k", op="decode", reqs=8, lo=130001, hi=131072, hq=64, hkv=8, d=128, dtype="fp16"),
        # a head of keys for each query head, small heads, ragged lengths
        dict(name="decode_24_ragged", op="decode", reqs=24, lo=1, hi=4001, hq=16, hkv=16, d=64, dtype="fp16"),
        # the sparse attention of 64 decode tokens at 32K keys, 2048 selected
        dict(name="selected_64x2048", op="selected", tokens=64, topk=2048, ctx=32768, reqs=64, hq=64, hkv=8, d=128,
             dtype="bf16"),
        # a few tokens whose context is shorter than the list: -1 tails, small heads
        dict(name="selected_3x512", op="selected", tokens=3, topk=512, ctx=301, reqs=3, hq=16, hkv=2, d=64,
             dtype="fp16"),
        # one long conversation's token with many query heads
        dict(name="selected_1x2048", op="selected", tokens=1, topk=2048, ctx=131001, reqs=1, hq=40, hkv=2, d=128,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "selected"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128])
    dt = rng.choice(["bf16", "fp16"])
    if op == "write":
        reqs = _log(rng, 1, 96)
        hi = _log(rng, 1, 32768 // reqs)
        return dict(op=op, reqs=reqs, lo=rng.randint(1, hi), hi=hi, past=rng.choice([0, _log(rng, 1, 3000)]), hkv=hkv,
                    d=d, dtype=dt)
    if op == "read":
        reqs = _log(rng, 1, 64)
        hi = _log(rng, 1, 131072 // reqs)
        return dict(op=op, reqs=reqs, lo=rng.randint(1, hi), hi=hi, hkv=hkv, d=d, dtype=dt)
    if op == "decode":
        reqs = _log(rng, 1, 96)
        hi = min(_log(rng, 1, 131072), (8 * 131072) // reqs)
        return dict(op=op, reqs=reqs, lo=max(1, int(hi * rng.uniform(0.2, 1.0))), hi=hi, hq=hq, hkv=hkv, d=d, dtype=dt)
    return dict(op=op, tokens=_log(rng, 1, 64), topk=4 * _log(rng, 1, 512), ctx=_log(rng, 1, 32768),
                reqs=rng.randint(1, 16), hq=hq, hkv=hkv, d=d, dtype=dt)


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi] in no order, the last one hi: a case's lengths
    are the same for every seed."""
    return [lo + int((0.618034 * (i + 1)) % 1.0 * (hi - lo + 1)) for i in range(n - 1)] + [hi]


def _lens(case):
    return _spread(case["lo"], case["hi"], case["reqs"])


def _paged(g, lens, extra=3):
    """Shuffled pages for sequences of these lengths: (block table, pages)."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    blocks = sum(need) + extra
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    bt = torch.zeros((len(lens), max(need + [1])), dtype=torch.int32, device=DEV)
    at = 0
    for r, m in enumerate(need):
        bt[r, :m] = perm[at:at + m]
        at += m
    return bt, blocks


def _rows(g, shape):
    """K or V rows [..., heads, d] as models have them: some tokens and some
    channels larger than others."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.4 * torch.randn(shape[:-2], generator=g, device=DEV))[..., None, None]
    return x * torch.exp(0.3 * torch.randn(shape[-2:], generator=g, device=DEV))


def _pow2(e):
    """2^e in 32 bits for whole e."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _scale_of(amax):
    """The least power of two with amax / scale <= 448 = 0.875 * 2^9, at least 2^-64."""
    m, e = torch.frexp(amax)
    return _pow2((e - 9 + (m > 0.875)).clamp(min=-64))


def _cache(g, blocks, hkv, d):
    """A filled cache: (K codes, V codes, scales), made in slices of pages."""
    kc, vc = (torch.empty((blocks, BLOCK, hkv, d), dtype=F8, device=DEV) for _ in range(2))
    sc = torch.empty((blocks, PARTS, hkv, 2), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (BLOCK * hkv * d))
    for a in range(0, blocks, step):
        n = min(step, blocks - a)
        for i, c in enumerate((kc, vc)):
            x = _rows(g, (n, PARTS, GROUP, hkv, d))
            s = _scale_of(x.abs().amax(dim=(2, 4)))
            sc[a:a + n, :, :, i] = s
            c[a:a + n] = (x / s[:, :, None, :, None]).flatten(1, 2).to(F8)
    return kc, vc, sc


def _batch(lens, bt, blocks, decodes):
    """The library's step metadata: a new token per request."""
    import dsa_sparse_attention_quant_gb300 as dsa
    n = len(lens)
    return dsa.Batch(_i32(list(range(n + 1))), _i32(lens), bt, _i32(list(range(n))), decodes, blocks,
                     max_seq_len=max(lens), num_decode_tokens=decodes)


def prepare(case, seed):
    g = _gen(seed)
    op, hkv, d, dt = case["op"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if op == "write":
        new = _lens(case)
        past = _spread(0, case["past"], case["reqs"] + 1)[:0:-1]
        bt, blocks = _paged(g, [p + n for p, n in zip(past, new)])
        req = torch.tensor([r for r, n in enumerate(new) for _ in range(n)], device=DEV)
        pos = torch.tensor([p + i for p, n in zip(past, new) for i in range(n)], device=DEV)
        s["slots"] = bt[req, pos // BLOCK].long() * BLOCK + pos % BLOCK
        n = req.numel()
        if n > 8:
            s["slots"][n // 3] = -1  # a padding token
        # k and v are column views of one projection's output
        s["qkv"] = torch.randn((n, 2 * hkv * d + 3 * d), generator=g, device=DEV).to(dt)
        s["k"] = s["qkv"][:, 2 * d:2 * d + hkv * d].unflatten(1, (hkv, d))
        s["v"] = s["qkv"][:, 3 * d + hkv * d:].unflatten(1, (hkv, d))
        s["k"].copy_(_rows(g, (n, hkv, d)))
        s["v"].copy_(_rows(g, (n, hkv, d)))
        s["kc"], s["vc"], s["sc"] = _cache(g, blocks, hkv, d)
        if own:
            import dsa_sparse_attention_quant_gb300 as dsa
            s["ws"] = torch.empty(dsa.kv_write8_workspace_size(n, blocks), dtype=torch.uint8, device=DEV)
        return s
    if op == "selected":
        t, k, ctx, reqs = case["tokens"], case["topk"], case["ctx"], case["reqs"]
        bt, blocks = _paged(g, [ctx] * reqs)
        n = min(k, ctx)
        ids = torch.rand((t, ctx), generator=g, device=DEV).topk(n, dim=1).indices
        rows = (torch.arange(t, device=DEV) % reqs)[:, None]
        s["phys"] = torch.full((t, k), -1, dtype=torch.int32, device=DEV)
        s["phys"][:, :n] = (bt.long()[rows, ids // BLOCK] * BLOCK + ids % BLOCK).to(torch.int32)
        s["q"] = torch.randn((t, case["hq"], d), generator=g, device=DEV).to(dt)
    else:
        lens = _lens(case)
        s["lens"] = lens
        s["bt"], blocks = _paged(g, lens)
        if op == "decode":
            s["q"] = torch.randn((len(lens), case["hq"], d), generator=g, device=DEV).to(dt)
        else:
            s["starts"] = _i32([sum(lens[:r]) for r in range(len(lens))])
            s["k"], s["v"] = (torch.empty((sum(lens), hkv, d), dtype=dt, device=DEV) for _ in range(2))
        s["klens"] = _i32(lens)
        if own:
            s["batch"] = _batch(lens, s["bt"], blocks, len(lens) if op == "decode" else 0)
    s["kc"], s["vc"], s["sc"] = _cache(g, blocks, hkv, d)
    if op != "read":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        if own:
            import dsa_sparse_attention_quant_gb300 as dsa
            heads = case["hq"], hkv, d
            size = (dsa.attn_decode8_workspace_size(s["batch"], *heads) if op == "decode" else
                    dsa.attn_selected8_workspace_size(case["tokens"], case["topk"], *heads))
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------- one pass, both forms

def run(s):
    return _RUN_OWN[s["case"]["op"]](s) if own else _RUN_PLAIN[s["case"]["op"]](s)


def _own_write(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    dsa.kv_write8(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["sc"], ws=s["ws"])
    return s["kc"], s["vc"], s["sc"]


def _own_read(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    return dsa.kv_read8(s["batch"], s["kc"], s["vc"], s["sc"], s["starts"], s["k"], s["v"])


def _own_decode(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    return dsa.attn_decode8(s["batch"], s["q"], s["kc"], s["vc"], s["sc"], out=s["out"], lse=s["lse"], ws=s["ws"])


def _own_selected(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    return dsa.attn_selected8(s["q"], s["kc"], s["vc"], s["sc"], s["phys"], out=s["out"], lse=s["lse"], ws=s["ws"])


def _bytes_at(c, at):
    """c[at] of 8-bit codes."""
    return c.view(torch.uint8)[at].view(F8)


def _plain_write(s):
    kc, vc, sc = s["kc"], s["vc"], s["sc"]
    hkv, d = kc.shape[2:]
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    blocks, which = torch.unique(slots // GROUP, return_inverse=True)
    first = torch.full_like(blocks, GROUP).scatter_reduce(0, which, slots % GROUP, "amin")
    flat = sc.view(-1, hkv, 2)
    old = torch.where((first == 0)[:, None, None], 0.0, flat[blocks])
    x = torch.stack((s["k"][keep], s["v"][keep]), -1).float()  # [rows, heads, d, 2]
    most = x.abs().amax(dim=2)
    amax = torch.zeros((blocks.numel(), hkv, 2), device=DEV).scatter_reduce(
        0, which[:, None, None].expand_as(most), most, "amax")
    new = torch.maximum(_scale_of(amax), old)
    ratio = torch.where(old > 0, old / new, 1.0)
    flat[blocks] = new
    x = (x / new[which][:, :, None, :]).to(F8).view(torch.uint8)
    at = blocks[:, None] * GROUP + torch.arange(GROUP, device=DEV)
    for i, c in enumerate((kc, vc)):
        rows = c.view(torch.uint8).view(-1, hkv, d)
        there = rows[at].view(F8).float() * ratio[:, None, :, None, i]
        rows[at] = there.to(F8).view(torch.uint8)
        rows[slots] = x[..., i]
    return kc, vc, sc


def _values(s, slots):
    """K and V rows in 32 bits, [..., heads, d], of these slots."""
    hkv, d = s["kc"].shape[2:]
    scale = s["sc"].view(-1, hkv, 2)[slots // GROUP]
    return tuple(_bytes_at(c.view(-1, hkv, d), slots).float() * scale[..., i, None]
                 for i, c in enumerate((s["kc"], s["vc"])))


def _plain_read(s):
    row = torch.arange(s["k"].shape[0], device=DEV)
    r = torch.searchsorted(s["starts"], row.to(torch.int32), right=True) - 1
    j = row - s["starts"][r]
    k, v = _values(s, s["bt"][r, j // BLOCK].long() * BLOCK + j % BLOCK)
    s["k"].copy_(k)
    s["v"].copy_(v)
    return s["k"], s["v"]


def _attend(s, slots, seen):
    """softmax(q k^T / sqrt(d)) v and the log of the sum over the slots [rows, n]
    that are seen, in 32 bits."""
    hkv = s["case"]["hkv"]
    k, v = _values(s, slots)
    q = s["q"].float().unflatten(1, (hkv, -1))  # [rows, kv heads, group, d]
    w = torch.matmul(q, k.permute(0, 2, 3, 1)) * (q.shape[-1] ** -0.5)
    w = torch.where(seen[:, None, None, :], w, -math.inf)
    m = w.amax(dim=-1, keepdim=True)
    p = torch.exp(w - m)
    t = p.sum(dim=-1, keepdim=True)
    s["out"].copy_((torch.matmul(p, v.transpose(1, 2)) / t).flatten(1, 2))
    s["lse"].copy_((m + torch.log(t)).flatten(1))
    return s["out"], s["lse"]


def _plain_decode(s):
    j = torch.arange(s["bt"].shape[1] * BLOCK, device=DEV)
    slots = s["bt"][:, j // BLOCK].long() * BLOCK + j % BLOCK
    return _attend(s, slots, j < s["klens"][:, None])


def _plain_selected(s):
    return _attend(s, s["phys"].clamp(min=0).long(), s["phys"] >= 0)


_RUN_OWN = dict(write=_own_write, read=_own_read, decode=_own_decode, selected=_own_selected)
_RUN_PLAIN = dict(write=_plain_write, read=_plain_read, decode=_plain_decode, selected=_plain_selected)


# -------------------------------------------------- floors and exact results

def work(case):
    """Bytes read and written once (codes, scales, rows in 16 bits, indices) and
    multiply-adds (two operations each)."""
    op, hkv, d = case["op"], case["hkv"], case["d"]
    key = 2 * hkv * (d + 4 / GROUP)  # a cached key: codes and its share of the scales
    if op == "selected":
        n = min(case["topk"], case["ctx"])
        # slots read once each, however many tokens share them; a scale for each slot where they stand alone
        keys = case["reqs"] * case["ctx"] * (1 - (1 - n / case["ctx"]) ** (case["tokens"] / case["reqs"]))
        rows, pairs, index = case["tokens"], case["tokens"] * n, 4 * case["tokens"] * case["topk"]
    else:
        keys = sum(_lens(case))
        rows, pairs, index = case["reqs"], keys, keys / BLOCK * 4
    if op == "write":
        return dict(bytes=keys * (4 * hkv * d + key + 8), flops=0)
    if op == "read":
        return dict(bytes=keys * (4 * hkv * d + key) + index, flops=0)
    return dict(bytes=keys * key + rows * case["hq"] * (4 * d + 4) + index, flops=4 * case["hq"] * d * pairs)


def exact(case, seed):
    """The outputs in 64 bits from the definition. Attention: every query head on
    its own, out = sum_j e^(s_j) v_j / sum_j e^(s_j), lse = log sum_j e^(s_j).
    Written codes: a row's values over its block's scale, not rounded to 8 bits."""
    op, hkv, d = case["op"], case["hkv"], case["d"]
    s = prepare(case, seed)
    if op == "write":
        return _exact_write(s)
    codes = [c.reshape(-1, hkv, d) for c in (s["kc"], s["vc"])]
    scales = [s["sc"][..., i].reshape(-1, hkv) for i in range(2)]

    def rows_of(i, at, h):
        """K's (i = 0) or V's rows of head h at these slots."""
        c = codes[i][:, h].contiguous().view(torch.uint8)[at].view(F8).to(torch.float64)
        return c * scales[i][at // GROUP, h].double()[:, None]

    def keys_of(r):
        if op == "selected":
            return s["phys"][r][s["phys"][r] >= 0].long()
        pages = s["bt"][r, :(s["lens"][r] + BLOCK - 1) // BLOCK].long()
        return (pages[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten()[:s["lens"][r]]

    if op == "read":
        at = torch.cat([keys_of(r) for r in range(case["reqs"])])
        return tuple(torch.stack([rows_of(i, at, h) for h in range(hkv)], 1) for i in range(2))
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
    group = case["hq"] // hkv
    heads = [(h, slice(h * group, (h + 1) * group)) for h in range(hkv)]
    for r in range(q.shape[0]):
        at = keys_of(r)
        for h, e in heads:
            w = (q[r, e] @ rows_of(0, at, h).T) / math.sqrt(d)
            lse[r, e] = torch.logsumexp(w, dim=1)
            out[r, e] = torch.softmax(w, dim=1) @ rows_of(1, at, h)
    return out, lse


def _exact_write(s):
    """Block by block of the whole cache, from what each slot stands for."""
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    slots = s["slots"]
    n = s["kc"].shape[0] * BLOCK
    token = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    token[slots[slots >= 0]] = torch.arange(slots.numel(), device=DEV)[slots >= 0]
    fresh = (token >= 0).view(-1, GROUP)
    touched, opened = fresh.any(1), fresh[:, 0]
    outs, scales = [], []
    for i, (c, x) in enumerate(((s["kc"], s["k"]), (s["vc"], s["v"]))):
        was = s["sc"][..., i].reshape(-1, hkv)
        there = c.view(-1, GROUP, hkv, d).to(torch.float64)
        value = x[token.clamp(min=0)].double().view(-1, GROUP, hkv, d)
        value = torch.where(fresh[:, :, None, None], value, torch.zeros_like(value))
        most = value.abs().amax(dim=(1, 3))
        up = torch.round(torch.log2((most / 448).clamp(min=2.0 ** -64)))  # the nearest power, then the next if it is too small
        scale = torch.ldexp(torch.ones_like(up), up)
        scale = torch.where(scale * 448 < most, 2 * scale, scale)
        scale = torch.where(opened[:, None], scale, torch.maximum(scale, was.double()))
        scale = torch.where(touched[:, None], scale, was.double())
        # slots of an opened block that were not written keep their codes, whatever those stand for
        kept = torch.where(opened[:, None], torch.ones_like(scale), was.double() / scale)
        codes = torch.where(fresh[:, :, None, None], value / scale[:, None, :, None], there * kept[:, None, :, None])
        outs.append(codes.view(c.shape))
        scales.append(scale.view(s["sc"].shape[:3]))
    return outs[0], outs[1], torch.stack(scales, -1)
