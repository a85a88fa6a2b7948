"""Cases of the operators around the paged cache: query / key norm with rotation, cache write, cache read
and the attention of drafted tokens.

``run`` computes a case in its plain form (elementary torch operations, 32-bit arithmetic rounded once at the
end), or, where ``own`` is true, through the package's entry points.  ``exact`` is the operator's definition in
64 bits, written apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
FORMATS = ("bf16", "e4m3", "e2m1")


# ---------------------------------------------------------------- cases

def _rope(name, tokens, hq, hkv, d, rotary, pairs, norm, fused):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rotary": rotary,
            "pairs": pairs, "norm": norm, "fused": fused}


def _write(name, tokens, hkv, d, page, fmt):
    return {"name": name, "op": "write", "tokens": tokens, "hkv": hkv, "d": d, "page": page, "fmt": fmt}


def _read(name, batch, cached, hkv, d, page, fmt):
    return {"name": name, "op": "read", "batch": batch, "cached": cached, "hkv": hkv, "d": d, "page": page, "fmt": fmt}


def _tree(name, batch, cached, draft, chain, hq, hkv, d, page, fmt, keep):
    return {"name": name, "op": "tree", "batch": batch, "cached": cached, "draft": draft, "chain": chain, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "fmt": fmt, "keep": keep}


def listed():
    return [
        # one new token of one sequence: the latency of a decode step's first kernel
        _rope("rope_step", 1, 32, 4, 128, 128, False, True, True),
        # a whole 128K prompt, read in place from the rows of a fused projection
        _rope("rope_prompt", 131072, 32, 4, 128, 128, False, True, True),
        # an odd number of tokens, half of each head rotated in adjacent pairs
        _rope("rope_partial", 10007, 4, 2, 64, 32, True, True, False),
        # a decode step of 19 sequences appends one token each
        _write("write_step_e4m3", 19, 4, 128, 128, "e4m3"),
        # a 128K prompt goes into the 8-bit cache
        _write("write_prompt_e4m3", 131072, 4, 128, 128, "e4m3"),
        # a prompt of odd length goes into the 4-bit cache and is read back
        _write("write_read_e2m1", 30011, 4, 128, 64, "e2m1"),
        # a 128K sequence comes back for its block summaries and the next prefill
        _read("read_prompt_e4m3", 1, 131072, 4, 128, 128, "e4m3"),
        # 19 sequences of mixed lengths come back from the 4-bit cache
        _read("read_mixed_e2m1", 19, 9001, 4, 128, 128, "e2m1"),
        # the smallest step: five drafted tokens over a short cache
        _tree("tree_short_e2m1", 1, 777, 5, False, 4, 2, 64, 64, "e2m1", 0.0),
        # one new token over a 128K cache in bf16, every page
        _tree("tree_step_bf16", 1, 131072, 1, True, 32, 4, 128, 128, "bf16", 0.0),
        # sixteen drafted tokens over the pages a 128K sequence keeps, 8 bits
        _tree("tree_kept_e4m3", 1, 131072, 16, False, 32, 4, 128, 128, "e4m3", 0.12),
        # a batch of eight ragged sequences verifies 64 drafted tokens each
        _tree("tree_batch_e4m3", 8, 32768, 64, False, 32, 4, 128, 128, "e4m3", 0.0),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "write", "read", "tree", "tree"))
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8))
    page = rng.choice((64, 128, 256))
    if op == "rope":
        hq = hkv * rng.choice((1, 2, 4, 8))
        top = max(1, 131072 * 36 * 128 // ((hq + hkv) * d) // 2)
        rotary = rng.choice((d, d, d // 2, 16))
        c = _rope("", _spread(rng, 1, min(131072, top)), hq, hkv, d, rotary, rng.random() < 0.4, rng.random() < 0.8,
                  rng.random() < 0.5)
    elif op == "write":
        c = _write("", _spread(rng, 1, 131072 * 4 // hkv // 2), hkv, d, page, rng.choice(FORMATS))
    elif op == "read":
        batch = _spread(rng, 1, 19)
        c = _read("", batch, _spread(rng, 1, 131072 * 4 // hkv // batch // 2), hkv, d, page, rng.choice(FORMATS))
    else:
        group = rng.choice((1, 2, 4, 8, 16))
        batch = _spread(rng, 1, 8)
        draft = _spread(rng, 1, 64)
        top = 8 * 32768 * 64 * 32 // 2 // (batch * draft * hkv * group)
        cached = _spread(rng, 1, max(1, min(top, 131072 * 4 // hkv // batch)))
        c = _tree("", batch, cached, draft, rng.random() < 0.3, hkv * group, hkv, d, page, rng.choice(FORMATS),
                  rng.choice((0.0, 0.0, 0.1, 0.3)))
    del c["name"]
    return c


def _lengths(top, batch):
    """Ragged lengths of a batch, from `top` down to about half of it."""
    return [max(1, top - (top * b) // (2 * batch)) for b in range(batch)]


def _drafts(top, batch):
    return [max(1, top - b % 3) for b in range(batch)]


def _kept_pages(pages, keep):
    """How many of a row's pages are kept: all, or a share of them with the first and the last."""
    if keep == 0.0:
        return pages
    return min(pages, max(2, math.ceil(keep * pages)))


def _row_bytes(d, fmt):
    """Bytes of one token's keys of one head: codes and scales."""
    return {"bf16": 2 * d, "e4m3": d + 1, "e2m1": d // 2 + d // 16 + 1}[fmt]


def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * d
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 10 * n}
    if op == "write":
        n = case["tokens"] * case["hkv"]
        rows = 2 * n * (2 * d + _row_bytes(d, case["fmt"])) + 4 * case["tokens"]
        if case["fmt"] == "e2m1":
            rows += 2 * n * (2 * d + _row_bytes(d, case["fmt"]))
        return {"bytes": rows, "flops": 6 * n * d}
    if op == "read":
        n = sum(_lengths(case["cached"], case["batch"])) * case["hkv"]
        return {"bytes": 2 * n * (2 * d + _row_bytes(d, case["fmt"])), "flops": 2 * n * d}
    bts = flops = 0
    for length, t in zip(_lengths(case["cached"], case["batch"]), _drafts(case["draft"], case["batch"])):
        pages = -(-length // case["page"])
        kept = _kept_pages(pages, case["keep"]) * case["page"] - (pages * case["page"] - length)
        bts += 2 * kept * case["hkv"] * _row_bytes(d, case["fmt"])
        bts += t * d * (4 * case["hq"] + 4 * case["hkv"]) + 4 * t * case["hq"]
        flops += 4 * d * case["hq"] * t * (kept + 1)
    return {"bytes": bts, "flops": flops}


# ---------------------------------------------------------------- the plain codecs

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
    """Rows x [..., d] (fp32) as (codes [..., row bytes] uint8, exponents [...] uint8, group scales [..., d/16] uint8)."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), None, None
    amax = x.abs().amax(-1)
    if fmt == "e4m3":
        k = _row_exponent(amax, 1.75, 8)
        codes = (x * _pow2(-k)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes, (k + 127).to(torch.uint8), None
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


def _page_bytes(case):
    """(row bytes, scale bytes of one page and head)."""
    d, page, fmt = case["d"], case["page"], case["fmt"]
    return {"bf16": (2 * d, 0), "e4m3": (d, page), "e2m1": (d // 2, page * (1 + d // 16))}[fmt]


def _empty_cache(case, pages):
    """Pages [pages, hkv, page, row bytes] and their scales, of bytes that nobody has written."""
    rb, sb = _page_bytes(case)
    out = {}
    for name in ("k", "v"):
        out[name] = torch.full((pages, case["hkv"], case["page"], rb), 255, dtype=torch.uint8, device=DEV)
        out[name + "_scale"] = torch.full((pages, case["hkv"], sb), 255, dtype=torch.uint8, device=DEV) if sb else None
    return out


def _plain_write(cache, name, x, slots, case):
    """Rows x [tokens, hkv, d] into their slots."""
    page = case["page"]
    codes, exps, groups = _quantise(x.float(), case["fmt"])
    pg, off = torch.div(slots, page, rounding_mode="floor").long(), (slots % page).long()
    live = slots >= 0
    pg, off = pg[live], off[live]
    cache[name][pg, :, off] = codes[live]
    if exps is not None:
        e, g = _split_scales(cache[name + "_scale"], page)
        e[pg, :, off] = exps[live]
        if groups is not None:
            g[pg, :, off] = groups[live]


def _gather(cache, name, table, case, heads=None):
    """fp32 rows of the pages `table`: [..., hkv, page, d], or, with a head for each page, [..., page, d]."""
    page = case["page"]
    pick = (lambda t: t[table]) if heads is None else (lambda t: t[table, heads])
    codes, exps, groups = pick(cache[name]), None, None
    if cache[name + "_scale"] is not None:
        exps, groups = _split_scales(pick(cache[name + "_scale"]), page)
    return _dequantise(codes, exps, groups, case["fmt"])


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _keys(g, tokens, hkv, d, page):
    """Keys clustered by block, as the framework's synthetic prompts have them."""
    blocks = -(-tokens // page)
    centre = 0.5 * _normal(g, blocks, hkv, d)
    sigma = torch.exp(torch.empty(blocks, hkv, 1, device=DEV).uniform_(math.log(0.2), math.log(1.5), generator=g))
    of = torch.arange(tokens, device=DEV) // page
    return (centre[of] + sigma[of] * _normal(g, tokens, hkv, d)).to(torch.bfloat16)


def _filled(case, g, lengths):
    """A cache that holds the sequences, and their page table."""
    page, batch = case["page"], len(lengths)
    blocks = [-(-n // page) for n in lengths]
    stride = (max(blocks) + 3) // 4 * 4
    pages = sum(blocks) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((batch, stride), -1, dtype=torch.int32, device=DEV)
    cache = _empty_cache(case, pages)
    at = 0
    for b, n in enumerate(lengths):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
        pos = torch.arange(n, device=DEV)
        slots = table[b, pos // page] * page + (pos % page).int()
        _plain_write(cache, "k", _keys(g, n, case["hkv"], case["d"], page), slots, case)
        _plain_write(cache, "v", _normal(g, n, case["hkv"], case["d"]).to(torch.bfloat16), slots, case)
    return cache, table, pages


def _cache_shape(case, pages):
    import block_sparse_long_kv_gb300 as bsa
    fmt = {"bf16": bsa.CACHE_BF16, "e4m3": bsa.CACHE_E4M3, "e2m1": bsa.CACHE_E2M1}[case["fmt"]]
    return bsa.make_cache_shape(pages, case["page"], case["hkv"], case["d"], fmt)


def _cu(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    op, d = case["op"], case["d"]
    st = {"case": case}
    if op == "rope":
        n, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        if case["fused"]:  # q and k are columns of the rows [q | k | v] of one projection
            row = _normal(g, n, (hq + 2 * hkv) * d).to(torch.bfloat16)
            st["q"] = row[:, :hq * d].view(n, hq, d)
            st["k"] = row[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        else:
            st["q"] = _normal(g, n, hq, d).to(torch.bfloat16)
            st["k"] = _normal(g, n, hkv, d).to(torch.bfloat16)
        st["q_weight"] = (1 + 0.2 * _normal(g, d)).to(torch.bfloat16) if case["norm"] else None
        st["k_weight"] = (1 + 0.2 * _normal(g, d)).to(torch.bfloat16) if case["norm"] else None
        first = int(torch.randint(0, 131072, (1,), generator=g, device=DEV))
        st["positions"] = first + torch.arange(n, dtype=torch.int32, device=DEV)
        half = case["rotary"] // 2
        st["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)).float()
        st["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        st["k_out"] = torch.empty(n, hkv, d, dtype=torch.bfloat16, device=DEV)
        return st
    if op == "write":
        n, hkv, page = case["tokens"], case["hkv"], case["page"]
        pages = -(-n // page) + 1
        st["k"] = _keys(g, n, hkv, d, page)
        st["v"] = _normal(g, n, hkv, d).to(torch.bfloat16)
        perm = torch.randperm(pages, generator=g, device=DEV).int()
        pos = torch.arange(n, device=DEV)
        st["slots"] = perm[pos // page] * page + (pos % page).int()
        st["pages"] = pages
        st["cache"] = _empty_cache(case, pages)
        st["table"] = perm[None].contiguous()
        st["cu"] = _cu([n])
        st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        return st
    lengths = _lengths(case["cached"], case["batch"])
    st["cache"], st["table"], st["pages"] = _filled(case, g, lengths)
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    if op == "read":
        st["cu"] = _cu(lengths)
        total = sum(lengths)
        st["k_out"] = torch.empty(total, case["hkv"], d, dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.empty(total, case["hkv"], d, dtype=torch.bfloat16, device=DEV)
        return st
    batch, hq, hkv = case["batch"], case["hq"], case["hkv"]
    drafts = _drafts(case["draft"], batch)
    total = sum(drafts)
    st["cu"] = _cu(drafts)
    st["q"] = _normal(g, total, hq, d).to(torch.bfloat16)
    st["k_new"] = _keys(g, total, hkv, d, case["page"])
    st["v_new"] = _normal(g, total, hkv, d).to(torch.bfloat16)
    st["parents"] = None
    if not case["chain"]:  # each drafted token hangs on one of the few before it, or starts anew
        i = torch.cat([torch.arange(t, device=DEV) for t in drafts])
        back = torch.randint(1, 5, (total,), generator=g, device=DEV)
        st["parents"] = (i - back).clamp_min(-1).int()
    st["kv_idx"] = st["kv_cnt"] = None
    if case["keep"]:
        stride = st["table"].shape[1]
        counts = torch.tensor([-(-n // case["page"]) for n in lengths], device=DEV)
        kept = torch.tensor([_kept_pages(-(-n // case["page"]), case["keep"]) for n in lengths], device=DEV)
        j = torch.arange(stride, device=DEV)
        rank = torch.rand(batch, hkv, stride, generator=g, device=DEV)
        rank = rank.masked_fill((j == 0) | (j == counts[:, None, None] - 1), -1.0)
        rank = rank.masked_fill(j >= counts[:, None, None], 2.0)
        order = rank.argsort(-1)
        chosen = torch.zeros(batch, hkv, stride, dtype=torch.bool, device=DEV)
        chosen.scatter_(-1, order, (j < kept[:, None, None]).expand(batch, hkv, stride))
        st["kv_idx"] = (~chosen).int().argsort(dim=-1, stable=True).int().contiguous()
        st["kv_cnt"] = kept[:, None].expand(batch, hkv).int().contiguous()
    st["o"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty(total, hq, dtype=torch.float32, device=DEV)
    if own:
        import block_sparse_long_kv_gb300 as bsa
        ts = bsa.make_tree_shape(batch, total, case["draft"], case["cached"], hq, st["table"].shape[1])
        n = bsa.tree_workspace_bytes(ts, _cache_shape(case, st["pages"]))
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import block_sparse_long_kv_gb300 as bsa
    case = st["case"]
    op, d = case["op"], case["d"]
    if op == "rope":
        rs = bsa.make_rope_shape(case["tokens"], case["hq"], case["hkv"], d, case["rotary"], 1e-6,
                                 (bsa.ROPE_PAIRS if case["pairs"] else 0) | (0 if case["norm"] else bsa.ROPE_NO_NORM))
        bsa.qk_norm_rope(rs, st["q"], st["k"], st["q_weight"], st["k_weight"], st["positions"], st["inv_freq"],
                         st["q_out"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    cs = _cache_shape(case, st["pages"])
    if op == "write":
        bsa.cache_write(cs, st["k"], st["v"], st["slots"], st["cache"])
        if case["fmt"] == "e2m1":
            bsa.cache_read(cs, st["cu"], st["table"], case["tokens"], st["cache"], st["k_out"], st["v_out"])
            return {"k": st["k_out"], "v": st["v_out"]}
        return _cache_values(st["cache"], case["fmt"])
    if op == "read":
        bsa.cache_read(cs, st["cu"], st["table"], case["cached"], st["cache"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    ts = bsa.make_tree_shape(case["batch"], st["q"].shape[0], case["draft"], case["cached"], case["hq"],
                             st["table"].shape[1])
    bsa.tree_fwd(ts, cs, st["cu"], st["lengths"], st["table"], st["parents"], st["q"], st["k_new"], st["v_new"],
                 st["cache"], st["kv_idx"], st["kv_cnt"], d ** -0.5, st["o"], st["lse"], st["workspace"])
    return {"o": st["o"], "lse": st["lse"]}


def _cache_values(cache, fmt):
    """The cache's buffers as the values they hold."""
    if fmt == "bf16":
        return {"k": cache["k"].view(torch.bfloat16), "v": cache["v"].view(torch.bfloat16)}
    out = {}
    for name in ("k", "v"):
        out[name] = cache[name].view(torch.float8_e4m3fn)
        out[name + "_scale"] = cache[name + "_scale"].view(torch.float8_e8m0fnu)
    return out


def _run_plain(st):
    return {"rope": _plain_rope, "write": _plain_write_case, "read": _plain_read, "tree": _plain_tree}[st["case"]["op"]](st)


def _plain_rope(st):
    case = st["case"]
    r = case["rotary"]
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def head(x, w):
        x = x.float()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        rot, rest = x[..., :r], x[..., r:]
        if case["pairs"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = rot[..., :r // 2], rot[..., r // 2:]
            rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((rot, rest), -1).to(torch.bfloat16)

    return {"q": head(st["q"], st["q_weight"]), "k": head(st["k"], st["k_weight"])}


def _plain_write_case(st):
    case = st["case"]
    _plain_write(st["cache"], "k", st["k"], st["slots"], case)
    _plain_write(st["cache"], "v", st["v"], st["slots"], case)
    if case["fmt"] == "e2m1":
        n = case["tokens"]
        return {name: _gather(st["cache"], name, st["table"][0].long(), case).transpose(1, 2).flatten(0, 1)[:n]
                .to(torch.bfloat16) for name in ("k", "v")}
    return _cache_values(st["cache"], case["fmt"])


def _plain_read(st):
    case = st["case"]
    page = case["page"]
    table = st["table"].long().clamp_min(0)
    live = torch.arange(table.shape[1] * page, device=DEV) < st["lengths"][:, None]
    return {name: _gather(st["cache"], name, table, case).transpose(2, 3).flatten(1, 2)[live].to(torch.bfloat16)
            for name in ("k", "v")}


def _plain_tree(st):
    case = st["case"]
    batch, hq, hkv, d, page = case["batch"], case["hq"], case["hkv"], case["d"], case["page"]
    group, t = hq // hkv, case["draft"]
    cu = st["cu"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(t, device=DEV)
    there = i < count[:, None]                                        # [b, t]
    at = (cu[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)          # the packed row of (b, t)
    q = st["q"][at].float().view(batch, t, hkv, group, d)
    k_new, v_new = st["k_new"][at].float(), st["v_new"][at].float()   # [b, t, hkv, d]
    # who sees whom among the drafted tokens: itself and the tokens on its path to the root
    parent = (i - 1).expand(batch, t) if st["parents"] is None else st["parents"][at].long()
    see = (torch.eye(t, device=DEV) + (parent[..., None] == i).float()).clamp_max(1.0)
    for _ in range(max(1, (t - 1).bit_length())):
        see = (see @ see).clamp_max(1.0)
    see = (see > 0) & there[:, None]                                  # [b, t, t]
    # the kept pages of every (sequence, KV head)
    stride = st["table"].shape[1]
    pages = (st["lengths"].long() + page - 1) // page
    if st["kv_idx"] is None:
        most = stride
        idx = torch.arange(stride, device=DEV).expand(batch, hkv, stride)
        cnt = pages[:, None].expand(batch, hkv)
    else:
        most = _kept_pages(-(-case["cached"] // page), case["keep"])
        idx, cnt = st["kv_idx"][..., :most].long(), st["kv_cnt"].long()
    entry = torch.arange(most, device=DEV) < cnt[..., None]
    idx = torch.where(entry, idx, 0)
    pos = idx[..., None] * page + torch.arange(page, device=DEV)
    live = (entry[..., None] & (pos < st["lengths"][:, None, None, None])).flatten(2)   # [b, hkv, keys]
    rows = torch.gather(st["table"].long()[:, None].expand(batch, hkv, stride), 2, idx).clamp_min(0)
    heads = torch.arange(hkv, device=DEV)[None, :, None].expand_as(rows)
    k = _gather(st["cache"], "k", rows, case, heads).flatten(2, 3)    # [b, hkv, keys, d]
    v = torch.where(live[..., None], _gather(st["cache"], "v", rows, case, heads).flatten(2, 3), 0.0)
    scale = d ** -0.5
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                        # [b, hkv, group * t, d]
    s = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~live[:, :, None], float("-inf"))
    s_new = (q @ k_new.permute(0, 2, 3, 1)) * scale                   # [b, hkv, group * t, t]
    s_new = s_new.unflatten(2, (group, t)).masked_fill(~see[:, None, None], float("-inf")).flatten(2, 3)
    m = torch.maximum(s.amax(-1), s_new.amax(-1)).clamp_min(-1e30)[..., None]
    p, p_new = s.sub_(m).exp_(), (s_new - m).exp()
    z = p.sum(-1) + p_new.sum(-1)
    o = (p @ v + p_new @ v_new.transpose(1, 2)) / z[..., None]
    lse = m[..., 0] + z.log()
    o = o.unflatten(2, (group, t)).permute(0, 3, 1, 2, 4).flatten(2, 3)   # [b, t, hq, d]
    lse = lse.unflatten(2, (group, t)).permute(0, 3, 1, 2).flatten(2, 3)
    return {"o": o[there].to(torch.bfloat16), "lse": lse[there]}


# ---------------------------------------------------------------- 64 bits

_E4M3 = [(1 - 2 * (c >> 7)) * (float("nan") if c & 127 == 127 else
                               (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else
                               (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)]
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _two(k):
    """2^k in 64 bits, k an integer tensor: the exponent field itself, since a power function may round."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _round_grid(x, bits, low):
    """x to the nearest multiple (ties to even) of a float's step: `bits` fraction bits, exponents from `low`."""
    step = _two((torch.frexp(x)[1] - 1).clamp_min(low) - bits)
    return torch.round(x / step) * step


def _exponent64(amax, most):
    k = torch.full(amax.shape, -126, dtype=torch.int64, device=amax.device)
    e = torch.frexp(amax / most)[1]                       # amax / most in [2^(e-1), 2^e)
    exact_power = most * _two(e - 1) == amax
    return torch.maximum(k, torch.where(amax > 0, torch.where(exact_power, e - 1, e), -126).long())


def _held(x, fmt):
    """(the values the codes of rows x stand for, before the row's power of two; that power), in 64 bits."""
    if fmt == "bf16":
        return x, torch.zeros(x.shape[:-1], dtype=torch.int64, device=x.device)
    amax = x.abs().amax(-1)
    k = _exponent64(amax, 448.0 if fmt == "e4m3" else 2688.0)
    y = x * _two(-k)[..., None]
    if fmt == "e4m3":
        return _round_grid(y, 3, -6), k
    y = y.unflatten(-1, (-1, 16))
    s = _round_grid(y.abs().amax(-1, keepdim=True) / 6, 3, -6)
    c = torch.where(s > 0, _round_grid(y / torch.where(s > 0, s, 1.0), 1, 0).clamp(-6, 6), 0.0)
    return (c * s).flatten(-2), k


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
    op, d = case["op"], case["d"]
    if op == "rope":
        turns = torch.outer(st["positions"].double(), st["inv_freq"].double())
        phase = torch.polar(torch.ones_like(turns), turns)[:, None]
        half = case["rotary"] // 2
        first = 2 * torch.arange(half, device=DEV) if case["pairs"] else torch.arange(half, device=DEV)
        second = first + 1 if case["pairs"] else first + half
        out = {}
        for name in ("q", "k"):
            x = st[name].double()
            if case["norm"]:
                x = x / (x.square().sum(-1, keepdim=True) / d + 1e-6).sqrt() * st[name + "_weight"].double()
            z = torch.complex(x[..., first], x[..., second]) * phase
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
        return out
    if op == "write":
        out = {}
        for name in ("k", "v"):
            val, power = _held(st[name].double(), case["fmt"])
            if case["fmt"] == "e2m1":
                out[name] = val * _two(power)[..., None]
                continue
            buf = _cache_values(st["cache"], case["fmt"])
            slots, page = st["slots"].long(), case["page"]
            held = buf[name].to(torch.float32).double()
            held[slots // page, :, slots % page] = val
            out[name] = held
            if case["fmt"] == "e4m3":
                sc = buf[name + "_scale"].to(torch.float32).double()
                sc[slots // page, :, slots % page] = _two(power)
                out[name + "_scale"] = sc
        return out
    lengths, page = st["lengths"].tolist(), case["page"]
    if op == "read":
        out = {}
        for name in ("k", "v"):
            seqs = []
            for b, n in enumerate(lengths):
                ids = st["table"][b, :-(-n // page)].long()
                seqs.append(torch.stack([_values64(st["cache"], name, ids, h, case)[:n] for h in range(case["hkv"])], 1))
            out[name] = torch.cat(seqs)
        return out
    cu, hq, hkv = st["cu"].tolist(), case["hq"], case["hkv"]
    group = hq // hkv
    o = torch.empty(cu[-1], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(cu[-1], hq, dtype=torch.float64, device=DEV)
    parents = None if st["parents"] is None else st["parents"].tolist()
    for b, n in enumerate(lengths):
        t0, t = cu[b], cu[b + 1] - cu[b]
        seen = []
        for i in range(t):  # a token sees itself and what its parent sees
            p = i - 1 if parents is None else parents[t0 + i]
            seen.append((set() if p < 0 else seen[p]) | {i})
        mask = torch.tensor([[j in s for j in range(t)] for s in seen], device=DEV)
        for g in range(hkv):
            blocks = torch.arange(-(-n // page), device=DEV)
            if st["kv_idx"] is not None:
                blocks = st["kv_idx"][b, g, :int(st["kv_cnt"][b, g])].long()
            ids = st["table"][b].long()[blocks]
            inside = (blocks[:, None] * page + torch.arange(page, device=DEV) < n).flatten()
            keys = torch.cat((_values64(st["cache"], "k", ids, g, case)[inside], st["k_new"][t0:t0 + t, g].double()))
            vals = torch.cat((_values64(st["cache"], "v", ids, g, case)[inside], st["v_new"][t0:t0 + t, g].double()))
            hidden = torch.cat((torch.zeros(t, len(keys) - t, dtype=torch.bool, device=DEV), ~mask), 1)
            for h in range(g * group, (g + 1) * group):
                logit = (st["q"][t0:t0 + t, h].double() @ keys.T / math.sqrt(d)).masked_fill(hidden, float("-inf"))
                lse[t0:t0 + t, h] = torch.logsumexp(logit, -1)
                o[t0:t0 + t, h] = torch.exp(logit - lse[t0:t0 + t, h, None]) @ vals
    return {"o": o, "lse": lse}
