"""Timed cases of the attention and page operators: what a pass is, its plain
form in elementary torch operations, and its floor in bytes and operations.

Five operators around the paged cache:

  decode    one new token per request over the request's pages
  selected  attention over the slots that the indexer selected for each token
  prompt    causal attention over prompts, keys in pages or packed
  write     the step's K and V rows into the cache at their slots
  pages     forking and compacting sequences' pages over several caches

``own`` chooses between the plain form and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a single short conversation: one launch's latency
        dict(name="decode_1x300", op="decode", reqs=1, lo=300, hi=300, hq=32, hkv=8, d=128, dtype="bf16"),
        # a serving batch of 32 requests of 4K to 8K keys
        dict(name="decode_32x8k", op="decode", reqs=32, lo=4096, hi=8192, hq=64, hkv=8, d=128, dtype="bf16"),
        # long contexts, few requests: the length has to be split; odd lengths
        dict(name="decode_8x128k", op="decode", reqs=8, lo=130001, hi=131072, hq=64, hkv=8, d=128, dtype="fp16"),
        # the sparse attention of 64 decode tokens at 32K keys, 2048 selected
        dict(name="selected_64x2048", op="selected", tokens=64, topk=2048, ctx=32768, reqs=64, hq=64, hkv=8, d=128,
             dtype="bf16"),
        # a few tokens whose context is shorter than the list: -1 tails, small heads
        dict(name="selected_3x512", op="selected", tokens=3, topk=512, ctx=301, reqs=3, hq=16, hkv=2, d=64,
             dtype="fp16"),
        # a short single prompt, odd length, keys packed beside the queries
        dict(name="prompt_1x509", op="prompt", lens="509", past=0, paged=False, hq=16, hkv=2, d=128, dtype="bf16"),
        # prompts of very different lengths in one packed batch
        dict(name="prompt_ragged", op="prompt", lens="1 2047 130 777 64 1500 333 4001", past=0, paged=False,
             hq=32, hkv=32, d=64, dtype="fp16"),
        # four 8K prompts whose keys are in the pages already
        dict(name="prompt_4x8k", op="prompt", lens="8192 8192 8192 8192", past=0, paged=True, hq=64, hkv=8, d=128,
             dtype="bf16"),
        # one decode step's rows into the cache
        dict(name="write_64", op="write", tokens=64, hkv=8, d=128, dtype="bf16"),
        # a prefill step's rows, column views of a fused projection's output
        dict(name="write_32768", op="write", tokens=32768, hkv=8, d=128, dtype="bf16"),
        # 64 sequences forked for parallel sampling, eight layers' K and V
        dict(name="pages_fork_64", op="pages", kind="fork", rows=64, forks=64, lo=1000, hi=3000, layers=8, hkv=2,
             d=128, blocks=4096),
        # half of the sequences gone: the others' pages move to the front
        dict(name="pages_compact_4k", op="pages", kind="compact", rows=96, forks=0, lo=1000, hi=3000, layers=4, hkv=4,
             d=128, blocks=4096),
    ]


def _lens(case):
    return [int(n) for n in case["lens"].split()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "selected", "prompt", "prompt", "write", "pages"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 8, 16])
    d = rng.choice([64, 128])
    dt = rng.choice(["bf16", "fp16"])
    if op == "decode":
        reqs = _log(rng, 1, 96)
        hi = min(_log(rng, 1, 131072), (8 * 131072) // reqs)
        return dict(op=op, reqs=reqs, lo=max(1, int(hi * rng.uniform(0.2, 1.0))), hi=hi, hq=hkv * min(g, 8), hkv=hkv,
                    d=d, dtype=dt)
    if op == "selected":
        return dict(op=op, tokens=_log(rng, 1, 64), topk=4 * _log(rng, 1, 512), ctx=_log(rng, 1, 32768),
                    reqs=rng.randint(1, 16), hq=hkv * min(g, 8), hkv=hkv, d=d, dtype=dt)
    if op == "prompt":
        n = rng.randint(1, 8)
        return dict(op=op, lens=" ".join(str(_log(rng, 1, 4096)) for _ in range(n)), past=rng.choice([0, 0, _log(rng, 1, 2048)]),
                    paged=rng.random() < 0.5, hq=hkv * g if g < 16 else hkv * 4, hkv=hkv, d=d, dtype=dt)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 32768), hkv=hkv, d=d, dtype=dt)
    kind = rng.choice(["fork", "compact"])
    rows = _log(rng, 2, 96)
    return dict(op=op, kind=kind, rows=rows, forks=rng.randint(1, rows), lo=rng.randint(1, 500),
                hi=rng.randint(500, 2500), layers=rng.randint(1, 4), hkv=hkv if hkv < 8 else 4, d=d, blocks=4096)


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _normal_big(g, shape, dtype):
    """As _normal, filled in slices: a large cache is not held in 32 bits."""
    t = torch.empty(shape, dtype=dtype, device=DEV)
    flat = t.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV, dtype=torch.float32).to(dtype)
    return t


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _spread(lo, hi, n, seed):
    """n lengths in [lo, hi], the last one hi; from the seed."""
    c = torch.Generator().manual_seed(seed * 31 + 7)
    lens = torch.randint(lo, hi + 1, (n,), generator=c).tolist()
    lens[-1] = hi
    return lens


def _paged(g, lens, extra=3):
    """Shuffled pages for sequences of these lengths: (block table, pages)."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    width = max(max(need), 1)
    blocks = sum(need) + extra
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    bt = torch.zeros((len(lens), width), dtype=torch.int32, device=DEV)
    at = 0
    for r, m in enumerate(need):
        bt[r, :m] = perm[at:at + m]
        at += m
    return bt, blocks


def _batch(qlens, klens, bt, blocks, decodes):
    """The library's step metadata for these requests."""
    import dsa_sparse_attention_quant_gb300 as dsa
    qsl = [0]
    for n in qlens:
        qsl.append(qsl[-1] + n)
    req = [r for r, n in enumerate(qlens) for _ in range(n)]
    return dsa.Batch(_i32(qsl), _i32(klens), bt, _i32(req), decodes, blocks, max_seq_len=max(klens),
                     num_decode_tokens=qsl[decodes])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "pages":
        return _prepare_pages(case, seed, g, s)
    dt = DTYPES[case["dtype"]]
    hkv, d = case["hkv"], case["d"]
    if op == "write":
        n = case["tokens"]
        blocks = (n + BLOCK - 1) // BLOCK + 9
        # k and v are column views of one projection's output
        s["qkv"] = _normal(g, (n, 2 * hkv * d + 3 * d), dt)
        s["k"] = s["qkv"][:, 2 * d:2 * d + hkv * d].unflatten(1, (hkv, d))
        s["v"] = s["qkv"][:, 3 * d + hkv * d:].unflatten(1, (hkv, d))
        s["slots"] = torch.randperm(blocks * BLOCK, generator=g, device=DEV)[:n].contiguous()
        if n > 8:
            s["slots"][n // 3] = -1  # a padding token
        s["kc"] = torch.zeros((blocks, BLOCK, hkv, d), dtype=dt, device=DEV)
        s["vc"] = torch.zeros((blocks, BLOCK, hkv, d), dtype=dt, device=DEV)
        return s
    hq = case["hq"]
    if op == "decode":
        lens = _spread(case["lo"], case["hi"], case["reqs"], seed)
        s["lens"] = lens
        s["bt"], blocks = _paged(g, lens)
        s["q"] = _normal(g, (len(lens), hq, d), dt)
        s["kc"] = _normal_big(g, (blocks, BLOCK, hkv, d), dt)
        s["vc"] = _normal_big(g, (blocks, BLOCK, hkv, d), dt)
        if own:
            import dsa_sparse_attention_quant_gb300 as dsa
            s["batch"] = _batch([1] * len(lens), lens, s["bt"], blocks, len(lens))
            s["ws"] = torch.empty(dsa.attn_decode_workspace_size(s["batch"], hq, hkv, d), dtype=torch.uint8,
                                  device=DEV)
    elif op == "selected":
        t, k, ctx, reqs = case["tokens"], case["topk"], case["ctx"], case["reqs"]
        bt, blocks = _paged(g, [ctx] * reqs)
        n = min(k, ctx)
        ids = torch.rand((t, ctx), generator=g, device=DEV).topk(n, dim=1).indices
        rows = (torch.arange(t, device=DEV) % reqs)[:, None]
        phys = bt.long()[rows, ids // BLOCK] * BLOCK + ids % BLOCK
        s["phys"] = torch.full((t, k), -1, dtype=torch.int32, device=DEV)
        s["phys"][:, :n] = phys.to(torch.int32)
        s["q"] = _normal(g, (t, hq, d), dt)
        s["kc"] = _normal_big(g, (blocks, BLOCK, hkv, d), dt)
        s["vc"] = _normal_big(g, (blocks, BLOCK, hkv, d), dt)
        if own:
            import dsa_sparse_attention_quant_gb300 as dsa
            s["ws"] = torch.empty(dsa.attn_selected_workspace_size(t, k, hq, hkv, d), dtype=torch.uint8, device=DEV)
    else:
        qlens = _lens(case)
        klens = [n + case["past"] for n in qlens]
        s["lens"], s["klens"] = qlens, klens
        s["q"] = _normal(g, (sum(qlens), hq, d), dt)
        if case["paged"]:
            s["bt"], blocks = _paged(g, klens)
            shape = (blocks, BLOCK, hkv, d)
        else:
            s["bt"], blocks = _i32([[0]] * len(qlens)), 1
            shape = (sum(klens), hkv, d)
        s["kc"] = _normal_big(g, shape, dt)
        s["vc"] = _normal_big(g, shape, dt)
        starts = [sum(klens[:r]) for r in range(len(klens))]
        s["starts"] = starts
        if own:
            s["batch"] = _batch(qlens, klens, s["bt"], blocks, 0)
            s["kv_start"] = None if case["paged"] else _i32(starts)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    return s


def _prepare_pages(case, seed, g, s):
    rows, blocks = case["rows"], case["blocks"]
    lens = _spread(case["lo"], case["hi"], rows, seed)
    width = (max(lens) + BLOCK - 1) // BLOCK + 1
    total = rows + case["forks"]
    bt = torch.full((total, width), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    at = 0
    for r, n in enumerate(lens):
        m = (n + BLOCK - 1) // BLOCK
        ids = perm[at:at + m]
        at += m
        if case["kind"] == "compact" and r % 2 and r:
            continue  # this sequence has ended: its pages are free
        bt[r, :m] = ids
        refs[ids.long()] += 1
    if case["kind"] == "compact":
        lens = [0 if r % 2 else n for r, n in enumerate(lens)]
    s["refs0"], s["bt0"] = refs, bt
    s["lens0"] = _i32(lens + [0] * case["forks"])
    s["refs"], s["bt"], s["seq"] = refs.clone(), bt.clone(), s["lens0"].clone()
    s["lens"] = lens
    c = torch.Generator().manual_seed(seed * 17 + 3)
    s["par"] = torch.randint(0, rows, (case["forks"],), generator=c).tolist()
    s["parents"] = _i32(s["par"])
    s["children"] = _i32(list(range(rows, total)))
    shape = (blocks, BLOCK, case["hkv"], case["d"])
    s["caches"] = [_normal_big(g, shape, torch.bfloat16) for _ in range(2 * case["layers"])]
    if own:
        import dsa_sparse_attention_quant_gb300 as dsa
        s["ws"] = torch.empty(dsa.pages_workspace_size(blocks, case["forks"]), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------- one pass, both forms

def run(s):
    return _RUN_OWN[s["case"]["op"]](s) if own else _RUN_PLAIN[s["case"]["op"]](s)


def _own_decode(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    return dsa.attn_decode(s["batch"], s["q"], s["kc"], s["vc"], out=s["out"], lse=s["lse"], ws=s["ws"])


def _own_selected(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    return dsa.attn_selected(s["q"], s["kc"], s["vc"], s["phys"], out=s["out"], lse=s["lse"], ws=s["ws"])


def _own_prompt(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    return dsa.attn_prompt(s["batch"], s["q"], s["kc"], s["vc"], kv_start=s["kv_start"], out=s["out"], lse=s["lse"])


def _own_write(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    dsa.kv_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
    return s["kc"], s["vc"]


def _reset_pages(s):
    """The bookkeeping as it was before the pass (the pages' bytes need no reset:
    a pass writes the same bytes again)."""
    s["refs"].copy_(s["refs0"])
    s["bt"].copy_(s["bt0"])
    s["seq"].copy_(s["lens0"])


def _own_pages(s):
    import dsa_sparse_attention_quant_gb300 as dsa
    _reset_pages(s)
    if s["case"]["kind"] == "fork":
        dsa.pages_fork(s["refs"], s["bt"], s["seq"], s["parents"], s["children"], s["caches"], ws=s["ws"])
    else:
        dsa.pages_compact(s["refs"], s["bt"], s["caches"], ws=s["ws"])
    return s["refs"], s["bt"], s["seq"], s["caches"]


def _attend(q, k, v, visible=None):
    """softmax(q k^T / sqrt(d)) v and the log of the sum, in q's precision.
    q [H, n, d], k and v [H, m, d] (heads already shared out), visible [n, m]."""
    sc = torch.matmul(q, k.transpose(1, 2)) * (q.shape[-1] ** -0.5)
    if visible is not None:
        sc = torch.where(visible, sc, -math.inf)
    m = sc.amax(dim=-1, keepdim=True)
    p = torch.exp(sc - m)
    t = p.sum(dim=-1, keepdim=True)
    return torch.matmul(p, v) / t, (m + torch.log(t))[..., 0]


def _causal(n, m):
    """Row i of the last n of m positions sees keys up to its own."""
    return torch.arange(m, device=DEV)[None, :] <= torch.arange(m - n, m, device=DEV)[:, None]


def _pages_of(s, r, n):
    """K and V rows of request r's first n keys, [n, Hkv, d], from its pages."""
    ids = s["bt"][r, :(n + BLOCK - 1) // BLOCK].long()
    return tuple(c[ids].flatten(0, 1)[:n] for c in (s["kc"], s["vc"]))


def _plain_decode(s):
    hkv = s["case"]["hkv"]
    for r, n in enumerate(s["lens"]):
        k, v = _pages_of(s, r, n)
        q = s["q"][r].float().unflatten(0, (hkv, -1))
        o, l = _attend(q, k.float().transpose(0, 1), v.float().transpose(0, 1))
        s["out"][r] = o.flatten(0, 1).to(s["out"].dtype)
        s["lse"][r] = l.flatten()
    return s["out"], s["lse"]


def _plain_selected(s):
    hkv = s["case"]["hkv"]
    kf, vf = s["kc"].flatten(0, 1), s["vc"].flatten(0, 1)
    for t in range(s["q"].shape[0]):
        ids = s["phys"][t]
        at = ids.clamp(min=0).long()
        q = s["q"][t].float().unflatten(0, (hkv, -1))
        o, l = _attend(q, kf[at].float().transpose(0, 1), vf[at].float().transpose(0, 1), (ids >= 0)[None, :])
        s["out"][t] = o.flatten(0, 1).to(s["out"].dtype)
        s["lse"][t] = l.flatten()
    return s["out"], s["lse"]


def _rows_of(s, r):
    """K and V rows [m, Hkv, d] of prompt r."""
    m = s["klens"][r]
    if s["case"]["paged"]:
        return _pages_of(s, r, m)
    a = s["starts"][r]
    return s["kc"][a:a + m], s["vc"][a:a + m]


def _plain_prompt(s):
    hq, hkv = s["case"]["hq"], s["case"]["hkv"]
    g = hq // hkv
    at = 0
    for r, n in enumerate(s["lens"]):
        k, v = _rows_of(s, r)
        seen = _causal(n, s["klens"][r])
        for h in range(hkv):
            q = s["q"][at:at + n, h * g:(h + 1) * g].float().transpose(0, 1)
            o, l = _attend(q, k[:, h].float()[None], v[:, h].float()[None], seen)
            s["out"][at:at + n, h * g:(h + 1) * g] = o.transpose(0, 1).to(s["out"].dtype)
            s["lse"][at:at + n, h * g:(h + 1) * g] = l.transpose(0, 1)
        at += n
    return s["out"], s["lse"]


def _plain_write(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    s["kc"].flatten(0, 1)[at] = s["k"][keep]
    s["vc"].flatten(0, 1)[at] = s["v"][keep]
    return s["kc"], s["vc"]


def _plain_pages(s):
    _reset_pages(s)
    refs, bt, seq = s["refs"], s["bt"], s["seq"]
    if s["case"]["kind"] == "fork":
        free = (refs == 0).nonzero()[:, 0]
        src, used = [], 0
        for i, p in enumerate(s["par"]):
            n = s["lens"][p]
            child = s["case"]["rows"] + i
            full, part = n // BLOCK, n % BLOCK
            bt[child, :full] = bt[p, :full]
            refs.index_add_(0, bt[p, :full].long(), torch.ones(full, dtype=torch.int32, device=DEV))
            if part:
                bt[child, full] = free[used].to(torch.int32)
                src.append(bt[p, full])
                used += 1
            seq[child] = seq[p]
        dst = free[:used]
        refs[dst] = 1
        if used:
            at = torch.stack(src).long()
            for c in s["caches"]:
                c[dst] = c[at]
    else:
        live = refs > 0
        n = live.sum()
        place = torch.arange(refs.shape[0], device=DEV)
        holes = (~live & (place < n)).nonzero()[:, 0]
        moved = (live & (place >= n)).nonzero()[:, 0]
        new = place.clone()
        new[moved] = holes
        bt.copy_(torch.where(bt >= 0, new[bt.clamp(min=0).long()].to(torch.int32), bt))
        refs[holes] = refs[moved]
        refs[moved] = 0
        for c in s["caches"]:
            c[holes] = c[moved]
    return refs, bt, seq, s["caches"]


_RUN_OWN = dict(decode=_own_decode, selected=_own_selected, prompt=_own_prompt, write=_own_write, pages=_own_pages)
_RUN_PLAIN = dict(decode=_plain_decode, selected=_plain_selected, prompt=_plain_prompt, write=_plain_write,
                  pages=_plain_pages)


# -------------------------------------------------- floors and exact results

def work(case):
    """Bytes read and written once and multiply-adds (two operations each)."""
    op = case["op"]
    if op == "write":
        row = case["hkv"] * case["d"] * 2
        return dict(bytes=case["tokens"] * (4 * row + 8), flops=0)
    if op == "pages":
        page = BLOCK * case["hkv"] * case["d"] * 2
        mean = (case["lo"] + case["hi"]) / 2 / BLOCK
        # fork: nearly every parent has a part-filled page; compact: live pages above the live count
        n = case["forks"] if case["kind"] == "fork" else (case["rows"] / 2 * mean) * (1 - case["rows"] / 2 * mean
                                                                                     / case["blocks"])
        return dict(bytes=2 * n * page * 2 * case["layers"] + 8 * case["blocks"], flops=0)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "decode":
        rows, keys = case["reqs"], (case["reqs"] - 1) * (case["lo"] + case["hi"]) / 2 + case["hi"]
        pairs, index = keys, keys / BLOCK * 4
    elif op == "selected":
        n = min(case["topk"], case["ctx"])
        rows, pairs, index = case["tokens"], case["tokens"] * n, 4 * case["tokens"] * case["topk"]
        # slots read once each, however many tokens share them
        slots = case["reqs"] * case["ctx"]
        keys = slots * (1 - (1 - n / case["ctx"]) ** (case["tokens"] / case["reqs"]))
    else:
        lens, past = _lens(case), case["past"]
        rows = sum(lens)
        keys = rows + past * len(lens)
        pairs = sum(n * past + n * (n + 1) / 2 for n in lens)
        index = keys / BLOCK * 4 if case["paged"] else 0
    return dict(bytes=keys * hkv * d * 4 + rows * hq * (4 * d + 4) + index, flops=4 * hq * d * pairs)


def exact(case, seed):
    """The outputs in 64 bits from the definition: every query head on its own,
    out = sum_j e^(s_j) v_j / sum_j e^(s_j), lse = log sum_j e^(s_j)."""
    op = case["op"]
    if op in ("write", "pages"):
        return None  # bytes are moved, nothing is computed
    if work(case)["flops"] > 4e11:
        return None
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)

    def keys_of(i):
        """(rows of q, index of the keys in the flattened cache, first key a row may not see)"""
        if op == "decode":
            n = s["lens"][i]
            j = torch.arange(n, device=DEV)
            return slice(i, i + 1), s["bt"][i].long()[j // BLOCK] * BLOCK + j % BLOCK, torch.tensor([n], device=DEV)
        if op == "selected":
            ids = s["phys"][i].long()
            ids = ids[ids >= 0]
            return slice(i, i + 1), ids, torch.tensor([ids.numel()], device=DEV)
        n, m = s["lens"][i], s["klens"][i]
        a = sum(s["lens"][:i])
        j = torch.arange(m, device=DEV)
        at = s["bt"][i].long()[j // BLOCK] * BLOCK + j % BLOCK if case["paged"] else s["starts"][i] + j
        return slice(a, a + n), at, torch.arange(m - n + 1, m + 1, device=DEV)

    flat = [c.reshape(-1, hkv, d) for c in (s["kc"], s["vc"])]
    for i in range(len(s["lens"]) if op != "selected" else case["tokens"]):
        rows, at, limit = keys_of(i)
        for h in range(hkv):
            k, v = (c[at, h].double() for c in flat)
            for e in range(h * group, (h + 1) * group):
                w = (q[rows, e] @ k.T) / math.sqrt(d)
                w.masked_fill_(torch.arange(at.numel(), device=DEV) >= limit[:, None], -math.inf)
                total = torch.logsumexp(w, dim=1)
                lse[rows, e] = total
                out[rows, e] = torch.exp(w - total[:, None]) @ v
    return out, lse
