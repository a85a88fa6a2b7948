"""Cases of the operators that a decode step of many continuations of one prompt needs beside the paged cache:
attention of sequences that share the first pages of their tables, the sharing itself (fork, growth with a copy of
shared last pages, compaction), and the verification of drafted tokens.

``run`` computes a case in its plain form (elementary torch operations, 32-bit arithmetic rounded once at the end,
64 bits for the long sums whose borders decide a token), or, where ``own`` is true, through the package's entry
points.  ``exact`` is the operator's definition in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
FORMATS = ("bf16", "e4m3", "e2m1")


# ---------------------------------------------------------------- cases

def _shared(name, groups, per, prefix, tail, draft, chain, hq, hkv, d, page, fmt):
    return {"name": name, "op": "shared", "groups": groups, "per": per, "prefix": prefix, "tail": tail, "draft": draft,
            "chain": chain, "hq": hq, "hkv": hkv, "d": d, "page": page, "fmt": fmt}


def _fork(name, batch, out, tokens, add, ranked, hkv, d, page, fmt):
    return {"name": name, "op": "fork", "batch": batch, "out": out, "tokens": tokens, "add": add, "ranked": ranked,
            "hkv": hkv, "d": d, "page": page, "fmt": fmt}


def _compact(name, batch, pages, live, hkv, d, page, fmt):
    return {"name": name, "op": "compact", "batch": batch, "pages": pages, "live": live, "hkv": hkv, "d": d,
            "page": page, "fmt": fmt}


def _verify(name, batch, draft, chain, drawn, vocab, dtype):
    return {"name": name, "op": "verify", "batch": batch, "draft": draft, "chain": chain, "drawn": drawn,
            "vocab": vocab, "dtype": dtype}


def listed():
    return [
        # the smallest step: three continuations of a short prompt, two drafted tokens each, 4 bits
        _shared("shared_short_e2m1", 1, 3, 11, 40, 2, False, 4, 2, 64, 64, "e2m1"),
        # 32 answers to one 128K prompt, a token each
        _shared("shared_step_bf16", 1, 32, 1024, 700, 1, True, 32, 4, 128, 128, "bf16"),
        # eight answers to one 128K prompt over the 8-bit cache
        _shared("shared_step_e4m3", 1, 8, 1024, 3000, 1, True, 32, 4, 128, 128, "e4m3"),
        # four prompts of different lengths, six continuations each, trees of five drafted tokens
        _shared("shared_groups_e4m3", 4, 6, 255, 501, 5, False, 32, 4, 128, 64, "e4m3"),
        # sixteen continuations of a 32K prompt verify sixteen drafted tokens each
        _shared("shared_drafts_bf16", 1, 16, 256, 1000, 16, False, 32, 4, 128, 128, "bf16"),
        # a prompt of odd length becomes nineteen sequences, which then grow by a token
        _fork("fork_prompt_e4m3", 1, 19, 32711, 1, False, 4, 128, 64, "e4m3"),
        # a beam step of 64 rows over 8K tokens each, every row keeping up to five accepted tokens
        _fork("fork_beam_bf16", 64, 64, 8191, 5, True, 4, 128, 128, "bf16"),
        # a small pool after some sequences have ended
        _compact("compact_small_e4m3", 3, 61, 0.5, 2, 64, 64, "e4m3"),
        # a pool of half a million tokens, two fifths of it free
        _compact("compact_pool_bf16", 32, 4096, 0.6, 4, 128, 128, "bf16"),
        # one sequence, a chain of four drafted tokens
        _verify("verify_chain", 1, 4, True, True, 32768, "fp32"),
        # drafts that were looked up, not drawn: chains of eight, an odd vocabulary
        _verify("verify_lookup", 19, 8, True, False, 50021, "fp32"),
        # trees of 32 drafted tokens for 32 sequences over a large vocabulary
        _verify("verify_tree", 32, 32, False, True, 131072, "fp32"),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("shared", "shared", "shared", "fork", "compact", "verify", "verify"))
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8))
    page = rng.choice((64, 128, 256))
    fmt = rng.choice(FORMATS)
    if op == "shared":
        group = rng.choice((1, 2, 4, 8, 16))
        groups = _spread(rng, 1, 6)
        per = _spread(rng, 1, 32)
        draft = _spread(rng, 1, max(1, min(16, 256 // (groups * per))))
        rows = groups * per * draft * hkv * group
        tokens = max(page, min(131072 * 4 // hkv // groups, 16 * 16 * 32 * 32768 // 2 // rows))
        prefix = _spread(rng, 1, max(1, tokens // page))
        tail = _spread(rng, 1, max(1, min(3000, 16 * 16 * 32 * 4000 // rows)))
        c = _shared("", groups, per, prefix, tail, draft, rng.random() < 0.4, hkv * group, hkv, d, page, fmt)
    elif op == "fork":
        batch = _spread(rng, 1, 64)
        out = _spread(rng, 1, 64)
        tokens = _spread(rng, 1, max(1, min(60000, 8191 * 64 * 2 // (max(batch, out) * hkv))))
        c = _fork("", batch, out, tokens, _spread(rng, 1, 300), rng.random() < 0.4, hkv, d, page, fmt)
    elif op == "compact":
        pages = _spread(rng, 2, 4096 * 128 * 2 // (page * hkv))
        c = _compact("", _spread(rng, 1, min(32, pages)), pages, rng.choice((0.1, 0.5, 0.9)), hkv, d, page, fmt)
    else:
        batch, draft = _spread(rng, 1, 32), _spread(rng, 1, 32)
        vocab = _spread(rng, 100, min(131072, 131072 * 32 * 32 // 2 // (batch * draft)))
        c = _verify("", batch, draft, rng.random() < 0.4, rng.random() < 0.7, vocab, rng.choice(("fp32", "bf16")))
    del c["name"]
    return c


def _prefixes(case):
    """Shared pages of every group, from `prefix` down to about half of it."""
    p, g = case["prefix"], case["groups"]
    return [max(1, p - (p * i) // (2 * g)) for i in range(g)]


def _shared_lengths(case):
    """Cached tokens of every sequence: its group's pages and a tail of its own, some without one."""
    batch = case["groups"] * case["per"]
    return [_prefixes(case)[b // case["per"]] * case["page"] + case["tail"] - (case["tail"] * b) // max(1, batch - 1)
            for b in range(batch)]


def _drafts(case):
    return [max(1, case["draft"] - b % 3) for b in range(case["groups"] * case["per"])]


def _fork_lengths(case):
    n, batch = case["tokens"], case["batch"]
    return [max(1, n - (n * b) // (2 * batch)) for b in range(batch)]


def _row_bytes(d, fmt):
    """Bytes of one token's keys of one head: codes and scales."""
    return {"bf16": 2 * d, "e4m3": d + 1, "e2m1": d // 2 + d // 16 + 1}[fmt]


def work(case):
    op = case["op"]
    if op == "verify":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = 2 if case["drawn"] else 1  # the row a token is drawn from, and what it is drawn against
        n = case["batch"] * case["vocab"]
        return {"bytes": n * rows * size + 20 * case["batch"] * case["draft"], "flops": 3 * n}
    d, hkv, page = case["d"], case["hkv"], case["page"]
    if op == "shared":
        bts = 2 * sum(_prefixes(case)) * page * hkv * _row_bytes(d, case["fmt"])
        flops = 0
        for b, (length, t) in enumerate(zip(_shared_lengths(case), _drafts(case))):
            tail = length - _prefixes(case)[b // case["per"]] * page
            bts += 2 * tail * hkv * _row_bytes(d, case["fmt"]) + t * d * (4 * case["hq"] + 4 * hkv) + 4 * t * case["hq"]
            flops += 4 * d * case["hq"] * t * (length + 1)
        return {"bytes": bts, "flops": flops}
    page_bytes = 2 * page * hkv * _row_bytes(d, case["fmt"])
    if op == "fork":
        # every sequence's table in and out; half a last page copied for every sequence but the last of each page
        # (of `out` sequences drawn from `batch`, this many pages on average)
        entries = sum(-(-n // page) for n in _fork_lengths(case)) + case["out"] * (-(-case["tokens"] // page))
        copies = case["out"] - case["batch"] * (1 - (1 - 1 / case["batch"]) ** case["out"])
        return {"bytes": int(4 * entries + copies * page_bytes), "flops": entries}
    moved = int(case["live"] * (1 - case["live"]) * case["pages"])
    return {"bytes": 2 * moved * page_bytes + 16 * case["pages"], "flops": case["pages"]}


# ---------------------------------------------------------------- the cache's rows

def _pow2(k):
    """2^k as fp32, k an integer tensor in [-126, 127]."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _row_exponent(amax, mantissa, bits):
    """The least k >= -126 with amax <= mantissa * 2^(bits + k), mantissa in [1, 2)."""
    m, e = torch.frexp(amax)
    return torch.where(2 * m <= mantissa, e - 1 - bits, e - bits).clamp_min(-126).masked_fill(amax == 0, -126)


def _e2m1_round(x):
    """The e2m1 code of x: nearest value, ties to the even code, saturated at 6."""
    a = x.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * (torch.signbit(x)).int()


def _e2m1_values(code):
    """The values of e2m1 codes 0..15."""
    m = code & 7
    v = torch.where(m < 2, m.float() * 0.5, (1.0 + 0.5 * (m & 1).float()) * _pow2((m >> 1) - 1))
    return torch.where(code >= 8, -v, v)


def _quantise(x, fmt):
    """Rows x [..., d] (fp32) as (codes uint8, exponents [...] uint8, group scales [..., d/16] uint8)."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), None, None
    amax = x.abs().amax(-1)
    if fmt == "e4m3":
        k = _row_exponent(amax, 1.75, 8)
        return (x * _pow2(-k)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (k + 127).to(torch.uint8), None
    k = _row_exponent(amax, 1.3125, 11)
    y = (x * _pow2(-k)[..., None]).unflatten(-1, (-1, 16))
    s8 = (y.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    s = s8.float()
    code = torch.where(s[..., None] > 0, _e2m1_round(y / s.clamp_min(2.0 ** -9)[..., None]), 0).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), (k + 127).to(torch.uint8), s8.view(torch.uint8)


def _dequantise(codes, exps, groups, fmt):
    """fp32 values of rows of codes."""
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).float()
    scale = _pow2(exps.int() - 127)[..., None]
    if fmt == "e4m3":
        return codes.contiguous().view(torch.float8_e4m3fn).float() * scale
    c = codes.int()
    v = _e2m1_values(torch.stack((c & 15, c >> 4), -1).flatten(-2)).unflatten(-1, (-1, 16))
    return (v * groups.contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * scale


def _split_scales(scales, page):
    """The planes of a page's scale bytes [..., page * (1 + d/16)]: exponents, then group scales."""
    return scales[..., :page], scales[..., page:].unflatten(-1, (page, -1)) if scales.shape[-1] > page else None


def _empty_cache(case, pages):
    """Pages [pages, hkv, page, row bytes] of zeros and their scales."""
    d, page, fmt = case["d"], case["page"], case["fmt"]
    rb, sb = {"bf16": (2 * d, 0), "e4m3": (d, page), "e2m1": (d // 2, page * (1 + d // 16))}[fmt]
    out = {}
    for name in ("k", "v"):
        out[name] = torch.zeros((pages, case["hkv"], page, rb), dtype=torch.uint8, device=DEV)
        out[name + "_scale"] = torch.zeros((pages, case["hkv"], sb), dtype=torch.uint8, device=DEV) if sb else None
    return out


def _put(cache, name, x, page_id, case):
    """Whole pages x [pages, page, hkv, d] (fp32) into the pages page_id."""
    codes, exps, groups = _quantise(x.transpose(1, 2), case["fmt"])
    cache[name][page_id] = codes
    if exps is not None:
        e, g = _split_scales(cache[name + "_scale"], case["page"])
        e[page_id] = exps
        if groups is not None:
            g[page_id] = groups


def _rows(cache, name, table, n, case):
    """fp32 rows [hkv, n, d] of the first n tokens of the pages `table`."""
    exps, groups = None, None
    if cache[name + "_scale"] is not None:
        exps, groups = _split_scales(cache[name + "_scale"][table], case["page"])
    return _dequantise(cache[name][table], exps, groups, case["fmt"]).transpose(0, 1).flatten(1, 2)[:, :n]


def _cache_values(cache, case, table, lengths, page_values):
    """The cache as the values it holds: its buffers, or for 4-bit codes the sequences' rows."""
    if case["fmt"] == "bf16":
        return {"k": cache["k"].view(torch.bfloat16), "v": cache["v"].view(torch.bfloat16)}
    if case["fmt"] == "e4m3":
        return {n: cache[n].view(torch.float8_e4m3fn if n in "kv" else torch.float8_e8m0fnu)
                for n in ("k", "v", "k_scale", "v_scale")}
    return page_values(table, lengths)


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _fill(cache, case, page_id, g):
    """Pages of keys clustered by block, as the framework's synthetic prompts have them, and of normal values."""
    for at in range(0, len(page_id), 256):
        ids = page_id[at:at + 256]
        n = len(ids)
        centre = 0.5 * _normal(g, n, 1, case["hkv"], case["d"])
        sigma = torch.exp(torch.empty(n, 1, case["hkv"], 1, device=DEV).uniform_(math.log(0.2), math.log(1.5), generator=g))
        k = centre + sigma * _normal(g, n, case["page"], case["hkv"], case["d"])
        _put(cache, "k", k.to(torch.bfloat16).float(), ids, case)
        _put(cache, "v", _normal(g, n, case["page"], case["hkv"], case["d"]).to(torch.bfloat16).float(), ids, case)


def _cu(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cache_shape(case, pages):
    import block_sparse_long_kv_gb300 as bsa
    fmt = {"bf16": bsa.CACHE_BF16, "e4m3": bsa.CACHE_E4M3, "e2m1": bsa.CACHE_E2M1}[case["fmt"]]
    return bsa.make_cache_shape(pages, case["page"], case["hkv"], case["d"], fmt)


def _tree(g, counts):
    """Each drafted token hangs on one of the few before it in its sequence; the first is the root."""
    i = torch.cat([torch.arange(t, device=DEV) for t in counts])
    back = torch.randint(1, 4, (len(i),), generator=g, device=DEV)
    return torch.where(i == 0, -1, (i - back).clamp_min(0)).int()


def prepare(case, seed):
    g = _generator(seed)
    return {"shared": _prepare_shared, "fork": _prepare_fork, "compact": _prepare_compact,
            "verify": _prepare_verify}[case["op"]](case, g)


def _prepare_shared(case, g):
    page, d, hkv, hq, per = case["page"], case["d"], case["hkv"], case["hq"], case["per"]
    lengths, prefixes, drafts = _shared_lengths(case), _prefixes(case), _drafts(case)
    batch, total = len(lengths), sum(drafts)
    own_pages = [-(-n // page) - prefixes[b // per] for b, n in enumerate(lengths)]
    pages = sum(prefixes) + sum(own_pages) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    stride = (max(-(-n // page) for n in lengths) + 3) // 4 * 4
    table = torch.full((batch, stride), -1, dtype=torch.int32, device=DEV)
    at = 0
    for x, p in enumerate(prefixes):
        table[x * per:(x + 1) * per, :p] = perm[at:at + p]
        at += p
    for b, n in enumerate(own_pages):
        table[b, prefixes[b // per]:prefixes[b // per] + n] = perm[at:at + n]
        at += n
    st = {"case": case, "cache": _empty_cache(case, pages), "pages": pages, "table": table, "lengths": _i32(lengths),
          "prefixes": _i32(prefixes), "cu_group": _i32([x * per for x in range(case["groups"] + 1)]), "cu": _cu(drafts)}
    _fill(st["cache"], case, perm[:at].long(), g)
    st["q"] = _normal(g, total, hq, d).to(torch.bfloat16)
    st["k_new"] = (0.7 * _normal(g, total, hkv, d)).to(torch.bfloat16)
    st["v_new"] = _normal(g, total, hkv, d).to(torch.bfloat16)
    st["parents"] = None if case["chain"] else _tree(g, drafts)
    st["o"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty(total, hq, dtype=torch.float32, device=DEV)
    if own:
        import block_sparse_long_kv_gb300 as bsa
        st["shape"] = bsa.make_shared_shape(case["groups"], batch, total, case["draft"], max(lengths), hq, stride)
        n = bsa.shared_workspace_bytes(st["shape"], _cache_shape(case, pages))
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return st


def _prepare_fork(case, g):
    page, batch, out = case["page"], case["batch"], case["out"]
    lengths = _fork_lengths(case)
    have = [-(-n // page) for n in lengths]
    stride = -(-(case["tokens"] + case["add"]) // page)
    pages = sum(have) + out * (1 + -(-case["add"] // page)) + 5
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((batch, stride), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    st = {"case": case, "cache": _empty_cache(case, pages), "pages": pages, "table": table, "cached": _i32(lengths)}
    st["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    st["refs"][perm[:at].long()] = 1
    last = [int(h) for h in table[torch.arange(batch), torch.tensor(have) - 1].tolist()]
    _fill(st["cache"], case, torch.tensor(last, device=DEV), g)   # the pages that may be copied
    st["source"] = torch.randint(0, batch, (out,), generator=g, device=DEV).int()
    if out > 3:
        st["source"][out // 2] = -1                               # one row of the batch stands empty
    # what each row gets: `add` tokens, or of `add` drafted tokens the accepted ones in their order
    n = out * case["add"]
    st["cu"] = _i32([case["add"] * b for b in range(out + 1)])
    st["rank"] = st["grow"] = None
    if case["ranked"]:
        taken = (torch.rand(out, case["add"], generator=g, device=DEV) < 0.6).int()
        st["rank"] = torch.where(taken > 0, taken.cumsum(1) - 1, -1).flatten().int()
        st["grow"] = taken.sum(1).int()
    st["cached_out"] = torch.empty(out, dtype=torch.int32, device=DEV)
    st["table_out"] = torch.empty(out, stride, dtype=torch.int32, device=DEV)
    st["slots"] = torch.empty(n, dtype=torch.int32, device=DEV)
    st["refs_out"] = torch.empty_like(st["refs"])
    if own:
        import block_sparse_long_kv_gb300 as bsa
        st["workspace"] = torch.empty(bsa.cache_grow_workspace_bytes(out), dtype=torch.uint8, device=DEV)
    if case["fmt"] == "e2m1":
        top = out * (case["tokens"] + case["add"])
        st["k_out"] = torch.zeros(top, case["hkv"], case["d"], dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.zeros_like(st["k_out"])
        st["most"] = case["tokens"] + case["add"]
    return st


def _prepare_compact(case, g):
    page, batch, pages = case["page"], case["batch"], case["pages"]
    live = min(pages, max(1, int(case["live"] * pages)))
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    cuts = [live * b // batch for b in range(batch + 1)]
    have = [cuts[b + 1] - cuts[b] for b in range(batch)]
    stride = (max(have) + 3) // 4 * 4 + 4
    table = torch.full((batch, stride), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(have):
        table[b, :n] = perm[cuts[b]:cuts[b + 1]]
    shared = min(have[0], have[-1], 2)                             # first and last sequence share some pages
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    if batch > 1 and shared:
        table[-1, :shared] = table[0, :shared]
    refs.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    lengths = [max(0, n * page - (b * 37) % page) for b, n in enumerate(have)]
    st = {"case": case, "cache": _empty_cache(case, pages), "table": table, "refs": refs, "cached": _i32(lengths),
          "pages": pages}
    _fill(st["cache"], case, perm[:live].long(), g)
    st["table_out"], st["refs_out"] = torch.empty_like(table), torch.empty_like(refs)
    st["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    if own:
        import block_sparse_long_kv_gb300 as bsa
        n = bsa.cache_compact_workspace_bytes(_cache_shape(case, pages))
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    if case["fmt"] == "e2m1":
        st["most"] = max(1, max(lengths))
        top = max(1, sum(lengths))
        st["k_out"] = torch.zeros(max(top, st["most"]), case["hkv"], case["d"], dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.zeros_like(st["k_out"])
    return st


def _prepare_verify(case, g):
    batch, vocab = case["batch"], case["vocab"]
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    counts = [max(1, case["draft"] - b % 3) for b in range(batch)]
    total, cu = sum(counts), _cu(counts)
    parents = None if case["chain"] else _tree(g, counts)
    start = torch.cat([torch.full((t,), int(s), device=DEV) for t, s in zip(counts, cu.tolist())])
    i = torch.arange(total, device=DEV)
    above = torch.where(i == start, i, i - 1 if parents is None else start + parents.long())  # the token's parent
    logits = 2.5 * _normal(g, total, vocab)                        # of the target, behind every token
    guess = logits + 0.8 * _normal(g, total, vocab)                # of the drafting model, there too
    st = {"case": case, "cu": cu, "parents": parents, "p": torch.softmax(logits, -1).to(dtype)}
    from_row = torch.softmax(guess, -1)
    if case["drawn"]:
        drawn = torch.multinomial(from_row, case["draft"], replacement=True, generator=g)
        tokens = drawn[above, i - start]
        st["q"] = from_row[above].to(dtype)
    else:
        tokens = from_row.argmax(-1)[above]
        st["q"] = None
    st["tokens"] = tokens.int()
    st["u_accept"] = torch.rand(total, generator=g, device=DEV)
    st["u_sample"] = torch.rand(batch, generator=g, device=DEV)
    st["count"] = torch.empty(batch, dtype=torch.int32, device=DEV)
    st["rank"] = torch.empty(total, dtype=torch.int32, device=DEV)
    st["next"] = torch.empty(batch, dtype=torch.int32, device=DEV)
    if own:
        import block_sparse_long_kv_gb300 as bsa
        st["shape"] = bsa.make_verify_shape(batch, total, case["draft"], vocab)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return _run_own(st) if own else {"shared": _plain_shared, "fork": _plain_fork, "compact": _plain_compact,
                                     "verify": _plain_verify}[st["case"]["op"]](st)


def _run_own(st):
    import block_sparse_long_kv_gb300 as bsa
    case = st["case"]
    op = case["op"]
    if op == "verify":
        bsa.verify(st["shape"], st["cu"], st["parents"], st["tokens"], st["p"], st["q"], st["u_accept"], st["u_sample"],
                   st["count"], st["rank"], st["next"])
        return {"count": st["count"], "rank": st["rank"], "next": st["next"]}
    cs = _cache_shape(case, st["pages"])
    if op == "shared":
        bsa.shared_fwd(st["shape"], cs, st["cu_group"], st["prefixes"], st["cu"], st["lengths"], st["table"],
                       st["parents"], st["q"], st["k_new"], st["v_new"], st["cache"], case["d"] ** -0.5, st["o"],
                       st["lse"], st["workspace"])
        return {"o": st["o"], "lse": st["lse"]}

    def values(table, lengths):
        cu = torch.nn.functional.pad(lengths.cumsum(0), (1, 0)).int()
        bsa.cache_read(cs, cu, table, st["most"], st["cache"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}

    st["refs_out"].copy_(st["refs"])
    if op == "fork":
        bsa.cache_fork(cs, st["source"], st["cached"], st["table"], st["refs_out"], st["cached_out"], st["table_out"])
        bsa.cache_grow(cs, st["cu"], st["rank"], st["grow"], st["cached_out"], st["table_out"], st["refs_out"],
                       st["cache"], st["slots"], st["workspace"])
        out = {"table": st["table_out"], "cached": st["cached_out"], "refs": st["refs_out"], "slots": st["slots"]}
        return out | _cache_values(st["cache"], case, st["table_out"], st["cached_out"], values)
    st["table_out"].copy_(st["table"])
    bsa.cache_compact(cs, st["cached"], st["table_out"], st["refs_out"], st["cache"], st["live"], st["workspace"])
    out = {"table": st["table_out"], "refs": st["refs_out"], "live": st["live"]}
    return out | _cache_values(st["cache"], case, st["table_out"], st["cached"], values)


def _plain_values(st):
    """For 4-bit codes: every sequence's rows, packed, as bf16."""
    def values(table, lengths):
        out = {"k": torch.zeros_like(st["k_out"]), "v": torch.zeros_like(st["v_out"])}
        at = 0
        for b, n in enumerate(lengths.tolist()):
            ids = table[b, :-(-n // st["case"]["page"])].long()
            for name in ("k", "v"):
                out[name][at:at + n] = _rows(st["cache"], name, ids, n, st["case"]).transpose(0, 1).to(torch.bfloat16)
            at += n
        return out
    return values


def _plain_shared(st):
    case = st["case"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    group, scale = hq // hkv, case["d"] ** -0.5
    at = 0
    for b, (n, t) in enumerate(zip(_shared_lengths(case), _drafts(case))):
        ids = st["table"][b, :-(-n // page)].long()
        k = torch.cat((_rows(st["cache"], "k", ids, n, case), st["k_new"][at:at + t].float().transpose(0, 1)), 1)
        v = torch.cat((_rows(st["cache"], "v", ids, n, case), st["v_new"][at:at + t].float().transpose(0, 1)), 1)
        # who sees whom among the drafted tokens: itself and the tokens on its path to the root
        i = torch.arange(t, device=DEV)
        parent = i - 1 if st["parents"] is None else st["parents"][at:at + t].long()
        see = (torch.eye(t, device=DEV) + (parent[:, None] == i).float()).clamp_max(1.0)
        for _ in range(max(1, (t - 1).bit_length())):
            see = (see @ see).clamp_max(1.0)
        q = st["q"][at:at + t].float().view(t, hkv, group, -1).permute(1, 2, 0, 3).flatten(1, 2)   # [hkv, group * t, d]
        s = (q @ k.transpose(1, 2)) * scale
        s.unflatten(1, (group, t))[..., n:].masked_fill_(see == 0, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        z = p.sum(-1, keepdim=True)
        o = (p @ v / z).unflatten(1, (group, t)).permute(2, 0, 1, 3).flatten(1, 2)
        st["o"][at:at + t] = o.to(torch.bfloat16)
        st["lse"][at:at + t] = (m + z.log()).unflatten(1, (group, t)).permute(2, 0, 1, 3).reshape(t, hq)
        at += t
    return {"o": st["o"], "lse": st["lse"]}


def _plain_fork(st):
    case = st["case"]
    page, cache, source = case["page"], st["cache"], st["source"].long()
    batch, stride = st["table"].shape
    out, add = case["out"], case["add"]
    col = torch.arange(stride, device=DEV)
    # fork: rows of the new table, and how often every page is named now
    there = source >= 0
    cached = torch.where(there, st["cached"][source.clamp_min(0)], 0)
    have = (cached + page - 1) // page
    table = torch.where(col < have[:, None], st["table"][source.clamp_min(0)], -1)
    uses = torch.zeros(batch, dtype=torch.int32, device=DEV).index_add_(0, source.clamp_min(0), there.int())
    old = col < ((st["cached"] + page - 1) // page)[:, None]
    refs = st["refs_out"].copy_(st["refs"])
    refs.index_add_(0, st["table"].clamp_min(0).flatten().long(), torch.where(old, uses[:, None] - 1, 0).flatten().int())
    # growth: a shared last page that gets tokens is copied, but for the last sequence that holds it
    grow = torch.full_like(cached, add) if st["grow"] is None else st["grow"]
    last = torch.gather(table, 1, (have - 1).clamp_min(0)[:, None].long())[:, 0].clamp_min(0).long()
    fill = cached % page
    part = (grow > 0) & (fill > 0)
    b = torch.arange(out, device=DEV)
    earlier = ((last[:, None] == last) & part[:, None] & part & (b < b[:, None])).sum(1)
    copy = part & (refs[last] - earlier > 1)
    need = torch.where(grow > 0, (cached + grow + page - 1) // page - have + copy.int(), 0)
    first = need.cumsum(0) - need
    free = torch.argsort((refs != 0).int(), stable=True)
    for k in range(1 + -(-add // page)):
        mine = k < need
        at = (have - copy.int() + k).clamp_max(stride - 1).long()
        page_id = free[(first + k).clamp_max(len(free) - 1)]
        old_id = torch.gather(table, 1, at[:, None])[:, 0]
        table.scatter_(1, at[:, None], torch.where(mine, page_id.int(), old_id)[:, None])
        refs.index_add_(0, page_id, mine.int())
        if k == 0:
            refs.index_add_(0, last, -copy.int())
            src, dst = last[copy], page_id[copy]
            row = torch.arange(page, device=DEV) < fill[copy][:, None]
            for name in ("k", "v"):
                planes = (cache[name],)
                if cache[name + "_scale"] is not None:
                    planes += _split_scales(cache[name + "_scale"], page)
                for plane in planes:
                    if plane is not None:
                        live = row[:, None, :, None] if plane.dim() == 4 else row[:, None]
                        plane[dst] = torch.where(live, plane[src], plane[dst])
    seq = torch.arange(out * add, device=DEV) // add
    rank = torch.arange(out * add, device=DEV) % add if st["rank"] is None else st["rank"]
    pos = cached[seq] + rank
    slot = torch.gather(table[seq], 1, (pos // page).clamp(0, stride - 1)[:, None].long())[:, 0] * page + pos % page
    slots = torch.where((rank >= 0) & (rank < grow[seq]), slot, -1).int()
    cached = (cached + grow).int()
    out = {"table": table, "cached": cached, "refs": refs, "slots": slots}
    return out | _cache_values(cache, case, table, cached, _plain_values(st))


def _plain_compact(st):
    case, cache = st["case"], st["cache"]
    used = st["refs"] > 0
    live = used.sum()
    page = torch.arange(case["pages"], device=DEV)
    moved, hole = page[used & (page >= live)], page[~used & (page < live)]
    for t in cache.values():
        if t is not None:
            t[hole] = t[moved]
    to = page.clone()
    to[moved] = hole
    table = torch.where(st["table"] >= 0, to[st["table"].clamp_min(0).long()].int(), -1)
    refs = st["refs"].clone()
    refs[hole] = st["refs"][moved]
    refs[moved] = 0
    out = {"table": table, "refs": refs, "live": live.int()[None]}
    return out | _cache_values(cache, case, table, st["cached"], _plain_values(st))


def _plain_verify(st):
    case = st["case"]
    batch, vocab, most = case["batch"], case["vocab"], case["draft"]
    cu = st["cu"].long()
    count, b = cu[1:] - cu[:-1], torch.arange(batch, device=DEV)
    at = cu[:-1].clone()                                   # the token reached, its row of p
    rest = st["p"][at].double()                            # what is left of that row after the tokens turned down
    mass = torch.ones(batch, dtype=torch.float64, device=DEV)
    took = torch.zeros(len(st["tokens"]), dtype=torch.int32, device=DEV)
    took[at] = 1
    for i in range(1, most):
        t = (cu[:-1] + i).clamp_max(len(took) - 1)
        parent = cu[:-1] + (i - 1 if st["parents"] is None else st["parents"][t].long())
        tested = (i < count) & (parent == at)
        x = st["tokens"][t].long()
        if st["q"] is None:
            q = torch.zeros(batch, vocab, dtype=torch.float64, device=DEV).scatter_(1, x[:, None], 1.0)
        else:
            q = st["q"][t].double()
        taken = tested & (st["u_accept"][t].double() * mass * q[b, x] < rest[b, x])
        turned = tested & ~taken
        less = (rest - mass[:, None] * q).clamp_min(0)
        rest = torch.where(turned[:, None], less, torch.where(taken[:, None], st["p"][t].double(), rest))
        mass = torch.where(turned, less.sum(1), torch.where(taken, 1.0, mass))
        at = torch.where(taken, t, at)
        took.index_add_(0, t, taken.int())
    rest = torch.where((mass > 0)[:, None], rest, st["p"][at].double())
    run = rest.cumsum(1)
    nxt = (run <= st["u_sample"].double()[:, None] * run[:, -1:]).sum(1)
    index = torch.arange(vocab, device=DEV)
    nxt = torch.minimum(nxt, torch.where(rest > 0, index, 0).amax(1))
    seq = torch.repeat_interleave(b, count, output_size=len(took))
    before = took.cumsum(0).int()
    rank = torch.where(took > 0, before - before[cu[:-1]][seq], -1).int()
    return {"count": (before[cu[1:] - 1] - before[cu[:-1]] + 1).int(), "rank": rank, "next": nxt.int()}


# ---------------------------------------------------------------- 64 bits

_E4M3 = [(1 - 2 * (c >> 7)) * (float("nan") if c & 127 == 127 else
                               (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else
                               (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)]
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _two(k):
    """2^k in 64 bits, k an integer tensor: the exponent field itself, since a power function may round."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _values64(cache, name, page_id, head, case):
    """64-bit rows of one page list of one head: [pages * page, d]."""
    page, fmt = case["page"], case["fmt"]
    raw = cache[name][page_id, head]
    if fmt == "bf16":
        return raw.contiguous().view(torch.bfloat16).double().flatten(0, 1)
    sc = cache[name + "_scale"][page_id, head].long()
    power = _two(sc[:, :page] - 127)
    e4m3 = torch.tensor(_E4M3, dtype=torch.float64, device=DEV)
    if fmt == "e4m3":
        return (e4m3[raw.long()] * power[..., None]).flatten(0, 1)
    codes = torch.stack((raw.long() % 16, raw.long() // 16), -1).flatten(-2)
    groups = e4m3[sc[:, page:]].view(len(page_id), page, -1)
    v = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)[codes] * groups.repeat_interleave(16, -1)
    return (v * power[..., None]).flatten(0, 1)


def exact(case, seed):
    st = prepare(case, seed)
    return {"shared": _exact_shared, "fork": _exact_fork, "compact": _exact_compact,
            "verify": _exact_verify}[case["op"]](st)


def _exact_shared(st):
    case = st["case"]
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    group, cu, lengths = hq // hkv, st["cu"].tolist(), st["lengths"].tolist()
    o = torch.empty(cu[-1], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(cu[-1], hq, dtype=torch.float64, device=DEV)
    parents = None if st["parents"] is None else st["parents"].tolist()
    for g in range(hkv):
        for b, n in enumerate(lengths):
            t0, t = cu[b], cu[b + 1] - cu[b]
            seen = []
            for i in range(t):  # a token sees itself and what its parent sees
                p = i - 1 if parents is None else parents[t0 + i]
                seen.append((set() if p < 0 else seen[p]) | {i})
            hidden = torch.tensor([[j not in s for j in range(t)] for s in seen], device=DEV)
            ids = st["table"][b, :(n + page - 1) // page].long()
            keys = torch.cat((_values64(st["cache"], "k", ids, g, case)[:n], st["k_new"][t0:t0 + t, g].double()))
            vals = torch.cat((_values64(st["cache"], "v", ids, g, case)[:n], st["v_new"][t0:t0 + t, g].double()))
            for h in range(g * group, (g + 1) * group):
                logit = st["q"][t0:t0 + t, h].double() @ keys.T / math.sqrt(d)
                logit[:, n:][hidden] = float("-inf")
                lse[t0:t0 + t, h] = torch.logsumexp(logit, -1)
                o[t0:t0 + t, h] = torch.exp(logit - lse[t0:t0 + t, h, None]) @ vals
    return {"o": o, "lse": lse}


def _wide(values):
    return {k: v if v.dtype == torch.float64 else v.to(torch.float32).double() for k, v in values.items()}


def _packed64(st, table, lengths):
    """For 4-bit codes: the sequences' rows in 64 bits, packed."""
    case = st["case"]
    out = {}
    for name in ("k", "v"):
        rows = [torch.stack([_values64(st["cache"], name, torch.tensor(table[b][:-(-n // case["page"])], device=DEV), h,
                                       case)[:n] for h in range(case["hkv"])], 1)
                for b, n in enumerate(lengths) if n]
        rows.append(torch.zeros(len(st["k_out"]) - sum(lengths), case["hkv"], case["d"], dtype=torch.float64, device=DEV))
        out[name] = torch.cat(rows)
    return out


def _exact_values(st, table, lengths):
    return _wide(_cache_values(st["cache"], st["case"], None, None, lambda *_: _packed64(st, table, lengths)))


def _exact_fork(st):
    # one sequence after the other, on the host
    case = st["case"]
    page, add = case["page"], case["add"]
    old, cached = st["table"].tolist(), st["cached"].tolist()
    refs = st["refs"].tolist()
    stride = len(old[0])
    table, lengths = [], []
    for s in st["source"].tolist():
        n = cached[s] if s >= 0 else 0
        lengths.append(n)
        table.append([old[s][j] if j * page < n else -1 for j in range(stride)])
    for row, n in zip(old, cached):
        for j in range(-(-n // page)):
            refs[row[j]] -= 1
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    grow = [add] * len(table) if st["grow"] is None else st["grow"].tolist()
    free = [p for p, r in enumerate(refs) if r == 0][::-1]
    slots = []
    for b, row in enumerate(table):
        n, want = lengths[b], grow[b]
        at = n // page
        if want and n % page and refs[row[at]] > 1:
            new = free.pop()
            rows = n % page
            for name in ("k", "v"):
                st["cache"][name][new, :, :rows] = st["cache"][name][row[at], :, :rows]
                if st["cache"][name + "_scale"] is not None:
                    sc = st["cache"][name + "_scale"]
                    sc[new, :, :rows] = sc[row[at], :, :rows]
                    if sc.shape[-1] > page:
                        width = rows * case["d"] // 16
                        sc[new, :, page:page + width] = sc[row[at], :, page:page + width]
            refs[row[at]] -= 1
            refs[new] = 1
            row[at] = new
        for j in range(-(-n // page), -(-(n + want) // page)):
            row[j] = free.pop()
            refs[row[j]] = 1
        rank = range(add) if st["rank"] is None else st["rank"][b * add:(b + 1) * add].tolist()
        slots += [row[(n + r) // page] * page + (n + r) % page if 0 <= r < want else -1 for r in rank]
        lengths[b] = n + want
    return {"table": _i32(table), "cached": _i32(lengths), "refs": _i32(refs), "slots": _i32(slots)} | \
        _exact_values(st, table, lengths)


def _exact_compact(st):
    refs, table = st["refs"].tolist(), st["table"].tolist()
    live = sum(r > 0 for r in refs)
    holes = iter([p for p in range(live) if refs[p] == 0])
    to = {}
    for p in range(live, len(refs)):
        if refs[p] > 0:
            to[p] = next(holes)
    for src, dst in to.items():
        refs[dst], refs[src] = refs[src], 0
    src, dst = torch.tensor(list(to), device=DEV).long(), torch.tensor(list(to.values()), device=DEV).long()
    for t in st["cache"].values():
        if t is not None:
            t.index_copy_(0, dst, t.index_select(0, src))
    table = [[to.get(p, p) for p in row] for row in table]
    return {"table": _i32(table), "refs": _i32(refs), "live": _i32([live])} | \
        _exact_values(st, table, st["cached"].tolist())


def _exact_verify(st):
    cu, tokens = st["cu"].tolist(), st["tokens"].tolist()
    u, us = st["u_accept"].tolist(), st["u_sample"].tolist()
    parents = None if st["parents"] is None else st["parents"].tolist()
    rank, count, nxt = [-1] * len(tokens), [], []
    for b in range(len(us)):
        t0, n = cu[b], cu[b + 1] - cu[b]
        above = [i - 1 if parents is None else parents[t0 + i] for i in range(n)]
        node, depth = 0, 1
        rank[t0] = 0
        while True:
            row = st["p"][t0 + node].double()
            left, mass, step = row, 1.0, None
            for c in (i for i in range(1, n) if above[i] == node):
                x = tokens[t0 + c]
                q = torch.zeros_like(row) if st["q"] is None else st["q"][t0 + c].double()
                if st["q"] is None:
                    q[x] = 1.0
                if u[t0 + c] * mass * float(q[x]) < float(left[x]):
                    step = c
                    break
                left = torch.relu(left - mass * q)
                mass = float(left.sum())
            if step is None:
                break
            rank[t0 + step], node, depth = depth, step, depth + 1
        w = left if mass > 0 else row
        run = torch.cumsum(w, 0)
        j = int(torch.searchsorted(run, us[b] * float(run[-1]), right=True))
        nxt.append(min(j, int(torch.nonzero(w > 0)[-1])))
        count.append(depth)
    return {"count": _i32(count), "rank": _i32(rank), "next": _i32(nxt)}
