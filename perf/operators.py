"""Cases of the cache-side operators of a verify step: what is measured, and their plain forms.

A verify step runs the target model over each request's k_b + 1 new tokens.  In every layer it
normalises and rotates their queries and keys and appends keys and values to a paged cache
(spec_append), then attends over that cache (spec_attention); once per step it takes, shares,
moves and gives back the pages themselves (spec_page_*).  A case is one call of these on inputs
as such a server holds them: a pool of pages in random order, requests of very different
lengths, pages that left a sliding window already given back.

The plain forms use elementary torch operations in 32 bits (64 for angles); `own` selects the
library's calls instead.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
BASE = 500000.0                # rotation base; inv_freq_j = BASE^(-2j / rotary_dim)
WORKSPACE = 64 << 20           # more than every call's workspace
TAIL = 256                     # append cases: tokens of context whose pages are still held


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _append(name, requests, drafts, ragged, q_heads, kv_heads, head_dim, rotary, dtype, page, context, norm=True,
            interleaved=False, layout="nhd"):
    return dict(name=name, op="append", requests=requests, drafts=drafts, ragged=ragged, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, rotary=rotary, dtype=dtype, page=page, context=context,
                norm=norm, interleaved=interleaved, layout=layout)


def _attention(name, requests, drafts, ragged, q_heads, kv_heads, head_dim, dtype, page, context, window=0, sinks=0,
               lse=False, layout="nhd"):
    return dict(name=name, op="attention", requests=requests, drafts=drafts, ragged=ragged, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page=page, context=context, window=window,
                sinks=sinks, lse=lse, layout=layout)


def _step(name, requests, forks, drafts, page, context, max_pages, pages, layers, page_values, window=0, sinks=0):
    return dict(name=name, op="step", requests=requests, forks=forks, drafts=drafts, page=page, context=context,
                max_pages=max_pages, pages=pages, layers=layers, page_values=page_values, window=window, sinks=sinks)


def _compact(name, requests, page, max_pages, pages, used, layers, page_values, capacity):
    return dict(name=name, op="compact", requests=requests, page=page, max_pages=max_pages, pages=pages, used=used,
                layers=layers, page_values=page_values, capacity=capacity)


def listed():
    return [
        # one chat user, one new token and no drafts: pure latency
        _append("append_single", 1, 0, False, 32, 8, 128, 128, "bf16", 16, 777),
        # the verify batch of the benchmark (256 requests, 4 drafts) at far positions
        _append("append_verify", 256, 4, False, 32, 8, 128, 128, "bf16", 16, 131072),
        # a ragged batch, half precision, interleaved rotation of a part of each head, no norm
        _append("append_ragged", 512, 8, True, 24, 4, 96, 48, "fp16", 32, 20011, norm=False, interleaved=True,
                layout="hnd"),
        # one chat user decoding: latency, one row per head group
        _attention("attention_single", 1, 0, False, 32, 8, 128, "bf16", 16, 2049),
        # one request with a very long context: the length has to be split over the chip
        _attention("attention_long", 1, 7, False, 32, 8, 128, "bf16", 64, 131071, lse=True),
        # the verify batch of the benchmark over ordinary contexts: the cache's bytes
        _attention("attention_verify", 256, 4, False, 32, 8, 128, "bf16", 16, 4096),
        # mixed traffic: lengths from one token to long ones, ragged drafts, narrow heads
        _attention("attention_ragged", 96, 8, True, 28, 4, 64, "fp16", 32, 32768, lse=True, layout="hnd"),
        # long contexts under a sliding window with a few first tokens kept; odd head width
        _attention("attention_window", 64, 4, True, 40, 8, 80, "bf16", 16, 50000, window=4096, sinks=4),
        # long draft chains on shared heads: many rows per key, bound by the products
        _attention("attention_chain", 16, 64, False, 32, 4, 128, "bf16", 64, 8192),
        # a small server's step: fork two requests, reserve, roll back, release
        _step("pages_small", 8, 2, 4, 16, 1000, 128, 1024, 2, 4096),
        # a large server's step: every fourth request forks, windowed pages are given back
        _step("pages_step", 512, 128, 4, 16, 16384, 1024, 81920, 3, 8192, window=4096, sinks=4),
        # a fragmented pool pulled together so that its upper part can be given back
        _compact("pages_compact", 256, 16, 1024, 32768, 0.45, 2, 8192, 16384),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "attention", "step", "compact"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    head_dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128])
    dtype, page, layout = rng.choice(["bf16", "bf16", "fp16"]), rng.choice([8, 16, 32, 64, 128, 256]), rng.choice(["nhd", "hnd"])
    drafts = rng.choice([0, 1, 2, 3, 4, 5, 6, 8, 8, 15, 16, 31, 64])
    ragged = rng.random() < 0.6
    if op == "append":
        rows = 1280 * 48 * 128 // ((q_heads + 2 * kv_heads) * head_dim)
        requests = _log(rng, 1, max(1, min(512, rows // (drafts + 1))))
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, 16])
        return {k: v for k, v in _append("", requests, drafts, ragged, q_heads, kv_heads, head_dim, rotary, dtype,
                                         page, _log(rng, drafts + 1, 400000), rng.random() < 0.7, rng.random() < 0.3,
                                         layout).items() if k != "name"}
    if op == "attention":
        # keys and values within 4 GB, the plain form's scores within 4 GB, 120 GFLOP
        requests = _log(rng, 1, 256)
        scores = requests * q_heads * (drafts + 1)
        most = min(4e9 / (requests * kv_heads * head_dim * 4), 1e9 / scores, 3e10 / (scores * head_dim), 131072)
        context = _log(rng, drafts + 1, max(drafts + 1, int(most)))
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        return {k: v for k, v in _attention("", requests, drafts, ragged, q_heads, kv_heads, head_dim, dtype, page,
                                            context, window, rng.choice([0, 1, 4, 100]) if window else 0,
                                            rng.random() < 0.5, layout).items() if k != "name"}
    page = rng.choice([8, 16, 32])
    values = page * rng.choice([64, 128, 256, 384])
    requests = _log(rng, 2, 512)
    if op == "step":
        max_pages = _log(rng, 8, 1024)
        window = rng.choice([0, _log(rng, 1, 4096)])
        forks, context = rng.randint(0, requests // 4), rng.randint(1, max(1, (max_pages - 5) * page // 2))
        return {k: v for k, v in _step("", requests, forks, rng.randint(0, 16), page, context, max_pages,
                                       requests * (max_pages // 2 + 5) // 2 * 2 + _log(rng, 64, 20000), rng.randint(1, 2), min(values, 4096),
                                       window, rng.choice([0, 4, 33]) if window else 0).items() if k != "name"}
    pages = _log(rng, 100, 32768)
    return {k: v for k, v in _compact("", requests, page, max(1, -(-pages // requests)), pages, rng.uniform(0.05, 0.95),
                                      rng.randint(1, 2), min(values, 8192), _log(rng, 16, 16384)).items() if k != "name"}


# ---------------------------------------------------------------------------------------------
# sizes (from the case alone) and inputs (from the seed)
# ---------------------------------------------------------------------------------------------

def _plan(c):
    """Host lists: drafts per request, and lengths after the new tokens."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    B = c["requests"]
    drafts = [r.randint(0, c["drafts"]) if c["ragged"] else c["drafts"] for _ in range(B)]
    if c["op"] == "append":
        lens = [max(n + 1, r.randint(c["context"] // 2, c["context"]) if B > 1 else c["context"]) for n in drafts]
    elif c["ragged"]:
        lens = [max(n + 1, _log(r, 1, c["context"])) for n in drafts]
    else:
        lens = [c["context"]] * B
    return drafts, lens


def _visible(c, n, L):
    """Keys that the n rows of a request of length L see in all, and keys that any of them sees."""
    W, s = c["window"], c["sinks"]
    if not W:
        return n * L - n * (n - 1) // 2, L
    pairs = 0
    for i in range(n):
        end = L - n + i + 1
        first = max(0, end - W)
        pairs += end - first + min(s, first)
    first = max(0, L - n + 1 - W)
    return pairs, L - first + min(s, first)


def _table(keep, num_pages, gen):
    """Page ids in random order where `keep`, -1 elsewhere."""
    t = torch.full(keep.shape, -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(num_pages, device="cuda", generator=gen)[:int(keep.sum())]
    t[keep] = ids.to(torch.int32)
    return t


def _cache(c, pages, gen):
    shape = (pages, c["page"], c["kv_heads"], c["head_dim"])
    dt = DTYPES[c["dtype"]]
    if c["layout"] == "nhd":
        return [torch.randn(shape, device="cuda", generator=gen, dtype=dt) for _ in range(2)]
    return [torch.randn((pages, shape[2], shape[1], shape[3]), device="cuda", generator=gen, dtype=dt).transpose(1, 2)
            for _ in range(2)]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c, "workspace": torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")}
    if c["op"] == "step":
        return _prepare_step(s, c, gen)
    if c["op"] == "compact":
        return _prepare_compact(s, c, gen)
    drafts, lens = _plan(c)
    P, dt, Hq, Hk, D = c["page"], DTYPES[c["dtype"]], c["q_heads"], c["kv_heads"], c["head_dim"]
    off = [0]
    for n in drafts:
        off.append(off[-1] + n + 1)
    R = off[-1]
    s.update(num_drafts=_ints(drafts), lens=_ints(lens), k_max=c["drafts"], off=_ints(off),
             row_offsets=_ints(off) if c["ragged"] else None)
    max_pages = -(-max(lens) // P)
    j = torch.arange(max_pages, device="cuda")[None]
    L, n = s["lens"].long()[:, None], s["num_drafts"].long()[:, None] + 1
    keep = j * P < L
    if c["op"] == "append":
        keep &= (j + 1) * P > L - n - TAIL
    elif c["window"]:
        keep &= ((j + 1) * P > L - n + 1 - c["window"]) | (j * P < c["sinks"])
    pages = int(keep.sum()) * 11 // 10 + 3
    s["block_table"] = _table(keep, pages, gen)
    s["k_cache"], s["v_cache"] = _cache(c, pages, gen)
    if c["op"] == "append":
        # the three projections of one product's output, as a layer hands them over
        qkv = torch.randn((R, (Hq + 2 * Hk) * D), device="cuda", generator=gen, dtype=dt)
        s["q"] = qkv[:, :Hq * D].view(R, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(R, Hk, D)
        s["v"] = qkv[:, (Hq + Hk) * D:].view(R, Hk, D)
        s["q_weight"] = s["k_weight"] = None
        if c["norm"]:
            s["q_weight"], s["k_weight"] = (torch.rand(2, D, device="cuda", generator=gen) + 0.5).to(dt)
        half = torch.arange(c["rotary"] // 2, dtype=torch.float64)
        s["inv_freq"] = (BASE ** (-2 * half / c["rotary"])).float().cuda()
        s["out"] = torch.empty((R, Hq, D), dtype=dt, device="cuda")
    else:
        s["q"] = torch.randn((R, Hq, D), device="cuda", generator=gen, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((R, Hq), device="cuda") if c["lse"] else None
        s["scale"] = 1 / math.sqrt(D)
    return s


def _bytes_of_pages(c, gen):
    shape = (c["layers"], c["pages"], c["page"], 1, c["page_values"] // c["page"])
    return [torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16) for _ in range(2)]


def _small(s, **parts):
    """The cache's small state in one buffer, and a saved copy that every pass starts from."""
    s["saved"] = torch.cat([t.reshape(-1) for t in parts.values()])
    s["live"] = s["saved"].clone()
    at = 0
    for name, t in parts.items():
        s[name] = s["live"][at:at + t.numel()].view(t.shape)
        at += t.numel()


def _step_plan(c):
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    B, F = c["requests"], c["forks"]
    most = min(c["context"], c["max_pages"] * c["page"] - c["drafts"] - 1)
    # the first F slots are empty (the forks' children), the others run
    lens = [0] * F + [_log(r, 1, most) for _ in range(B - F)]
    if F:
        lens[F] = most
    parents = [r.randrange(F, B) for _ in range(F)]
    fork_len = [r.randint(max(1, lens[p] - 64), lens[p]) for p in parents]
    drafts = [r.randint(0, c["drafts"]) for _ in range(B)]
    accept = [r.randint(0, n) for n in drafts]
    return lens, parents, fork_len, drafts, accept


def _prepare_step(s, c, gen):
    lens, parents, fork_len, drafts, accept = _step_plan(c)
    L = _ints(lens)
    j = torch.arange(c["max_pages"], device="cuda")[None]
    table = _table(j * c["page"] < L[:, None], c["pages"], gen)
    ref = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    _small(s, lens=L, block_table=table, ref_count=ref)
    s.update(parents=_ints(parents), children=_ints(range(c["forks"])), fork_len=_ints(fork_len),
             num_drafts=_ints(drafts), accept=_ints(accept))
    s["copy_src"], s["copy_dst"] = torch.full((2, c["forks"]), -1, dtype=torch.int32, device="cuda")
    s["k_cache"], s["v_cache"] = _bytes_of_pages(c, gen)
    return s


def _prepare_compact(s, c, gen):
    B, M = c["requests"], c["max_pages"]
    used = min(int(c["used"] * c["pages"]), B * M)
    keep = torch.zeros(B * M, dtype=torch.bool, device="cuda")
    keep[:used] = True
    table = _table(keep.view(B, M), c["pages"], gen)
    ref = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    # every eighth request shares its pages with the one before it
    if B > 1:
        table[7::8] = table[6::8][:table[7::8].shape[0]]
        ref.zero_().index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    _small(s, block_table=table, ref_count=ref)
    s["copy_src"], s["copy_dst"] = torch.full((2, c["capacity"]), -1, dtype=torch.int32, device="cuda")
    s["k_cache"], s["v_cache"] = _bytes_of_pages(c, gen)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if op in ("step", "compact"):
        s["live"].copy_(s["saved"])
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_append(s):
    from speculative_decoding_verification_12_gb300 import spec_append
    spec_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["inv_freq"], s["k_cache"], s["v_cache"],
                s["block_table"], s["lens"], s["num_drafts"], s["row_offsets"], s["k_max"], s["out"], s["workspace"],
                interleaved=s["case"]["interleaved"])
    return {"q": s["out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_attention(s):
    from speculative_decoding_verification_12_gb300 import spec_attention
    c = s["case"]
    spec_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["num_drafts"], s["row_offsets"],
                   s["k_max"], s["scale"], c["window"], c["sinks"], s["out"], s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}


def _own_step(s):
    from speculative_decoding_verification_12_gb300 import (spec_page_copy, spec_page_fork, spec_page_release,
                                                            spec_page_reserve, spec_rollback)
    c, ws = s["case"], s["workspace"]
    small = s["lens"], s["block_table"], s["ref_count"], c["page"]
    if c["forks"]:
        spec_page_fork(s["parents"], s["children"], s["fork_len"], *small, s["copy_src"], s["copy_dst"], ws)
        spec_page_copy(s["k_cache"], s["v_cache"], s["copy_src"], s["copy_dst"], ws)
    spec_page_reserve(s["num_drafts"], *small, ws)
    spec_rollback(s["lens"], s["accept"], s["num_drafts"], ws)
    spec_page_release(*small, c["window"], c["sinks"], ws)
    return _step_outputs(s)


def _own_compact(s):
    from speculative_decoding_verification_12_gb300 import spec_page_compact, spec_page_copy
    spec_page_compact(s["block_table"], s["ref_count"], s["copy_src"], s["copy_dst"], s["workspace"])
    spec_page_copy(s["k_cache"], s["v_cache"], s["copy_src"], s["copy_dst"], s["workspace"])
    return _compact_outputs(s)


def _step_outputs(s):
    out = {n: s[n] for n in ("lens", "block_table", "ref_count")}
    if s["case"]["forks"]:
        out.update({n: s[n] for n in ("copy_src", "copy_dst", "k_cache", "v_cache")})
    return out


def _compact_outputs(s):
    return {n: s[n] for n in ("block_table", "ref_count", "copy_src", "copy_dst", "k_cache", "v_cache")}


def _rows(s):
    """For each row: its request, and its position in the request's sequence."""
    rows = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["off"].long(), rows, right=True) - 1
    return b, s["lens"].long()[b] - 1 - s["num_drafts"].long()[b] + rows - s["off"].long()[b]


def _plain_append(s):
    c = s["case"]
    b, pos = _rows(s)
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
        r = c["rotary"]
        a, z = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        both = (a * cos - z * sin, a * sin + z * cos)
        y = torch.stack(both, -1).flatten(-2) if c["interleaved"] else torch.cat(both, -1)
        return torch.cat((y, x[..., r:]), -1).to(DTYPES[c["dtype"]])

    s["out"].copy_(turned(s["q"], s["q_weight"]))
    page = s["block_table"][b, pos // c["page"]].long()
    s["k_cache"][page, pos % c["page"]] = turned(s["k"], s["k_weight"])
    s["v_cache"][page, pos % c["page"]] = s["v"]
    return {"q": s["out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    Hk, D, G = c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    B, n = c["requests"], c["drafts"] + 1
    L, m = s["lens"].long(), s["num_drafts"].long() + 1
    at = s["block_table"].long().clamp(min=0)
    T = at.shape[1] * c["page"]
    k = s["k_cache"][at].reshape(B, T, Hk, D).permute(0, 2, 3, 1).float()
    v = s["v_cache"][at].reshape(B, T, Hk, D).transpose(1, 2).float()
    i = torch.arange(n, device="cuda")
    row = s["off"].long()[:-1, None] + torch.minimum(i, m[:, None] - 1)
    q = s["q"][row].float().reshape(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    z = (q @ k).view(B, Hk, n, G, T) * s["scale"]
    pos = (L - m)[:, None, None] + torch.minimum(i, m[:, None] - 1)[:, :, None]
    j = torch.arange(T, device="cuda")
    seen = j <= pos
    if c["window"]:
        seen &= (j > pos - c["window"]) | (j < c["sinks"])
    z = z.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = z.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(B, Hk, n * G, T) @ v).view(B, Hk, n, G, D) / total
    used = (i < m[:, None]).flatten().nonzero()[:, 0] if c["ragged"] else slice(None)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, c["q_heads"], D)[used].to(DTYPES[c["dtype"]])
    if not c["lse"]:
        return {"out": o}
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B * n, c["q_heads"])[used]
    return {"out": o, "lse": lse}


def _plain_free(ref):
    """Free page ids in ascending order, then the others."""
    return torch.argsort((ref != 0).int(), stable=True).to(torch.int32)


def _plain_copy(s):
    src, dst = s["copy_src"].long(), s["copy_dst"].long()
    some = (dst >= 0).nonzero()[:, 0]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, dst[some]] = cache[:, src[some]]


def _plain_step(s):
    c = s["case"]
    P, M, N = c["page"], c["max_pages"], c["pages"]
    table, ref, lens = s["block_table"], s["ref_count"], s["lens"]
    j = torch.arange(M, device="cuda")
    if c["forks"]:
        # children share the parents' full pages; a partly filled last page is copied
        par, ch, fl = s["parents"].long(), s["children"].long(), s["fork_len"].long()
        free = _plain_free(ref)
        tail = fl % P != 0
        rank = torch.cumsum(tail, 0) - 1
        fresh = torch.where(tail, free[rank.clamp(min=0)], -1)
        shared = torch.where(j < (fl // P)[:, None], table[par], -1)
        ref.index_add_(0, shared.clamp(min=0).flatten().long(), (shared >= 0).flatten().int())
        ref.index_add_(0, fresh.clamp(min=0).long(), tail.int())
        last = table[par, (fl // P).clamp(max=M - 1)]
        table[ch] = torch.where((j == (fl // P)[:, None]) & tail[:, None], fresh[:, None], shared)
        lens[ch] = fl.int()
        s["copy_src"].copy_(torch.where(tail, last, -1))
        s["copy_dst"].copy_(fresh)
        _plain_copy(s)
    # reserve: the lowest free pages, in request order
    have, grown = -(-lens // P), lens + s["num_drafts"] + 1
    need = -(-grown // P) - have
    first = torch.cumsum(need, 0) - need
    free = _plain_free(ref)
    new = (j >= have[:, None]) & (j < (have + need)[:, None])
    rank = (first[:, None] + j - have[:, None]).clamp(0, N - 1)
    ids = torch.where(new, free[rank], -1)
    table.copy_(torch.where(new, ids, table))
    ref.index_add_(0, ids.clamp(min=0).flatten().long(), new.flatten().int())
    # rolled back to the accepted drafts, then pages past the end or out of the window go
    lens.copy_(grown - s["num_drafts"] + s["accept"])
    drop = j >= (-(-lens // P))[:, None]
    if c["window"]:
        drop |= ((j + 1) * P <= (lens + 1 - c["window"])[:, None]) & (j * P >= c["sinks"])
    drop &= table >= 0
    ref.index_add_(0, table.clamp(min=0).flatten().long(), -drop.flatten().int())
    table.masked_fill_(drop, -1)
    return _step_outputs(s)


def _plain_compact(s):
    table, ref = s["block_table"], s["ref_count"]
    N, cap = ref.numel(), s["copy_src"].numel()
    ids = torch.arange(N, device="cuda")
    used = ref > 0
    U = used.sum()
    above, hole = used & (ids >= U), ~used & (ids < U)
    up, down = (torch.argsort((~m).int(), stable=True) for m in (above, hole))
    moves = torch.clamp(above.sum(), max=cap)
    r = torch.arange(min(N, cap), device="cuda")
    src, dst = (torch.where(r < moves, x[:r.numel()], -1) for x in (up, down))
    s["copy_src"].fill_(-1)
    s["copy_dst"].fill_(-1)
    s["copy_src"][:r.numel()] = src.int()
    s["copy_dst"][:r.numel()] = dst.int()
    goes = ids.clone()
    goes = torch.where(above & (torch.cumsum(above, 0) - 1 < moves), down[(torch.cumsum(above, 0) - 1).clamp(min=0)], goes)
    count = torch.zeros_like(ref).index_add_(0, goes, ref)
    ref.copy_(count)
    table.copy_(torch.where(table >= 0, goes[table.clamp(min=0).long()].int(), -1))
    _plain_copy(s)
    return _compact_outputs(s)


_OWN = {"append": _own_append, "attention": _own_attention, "step": _own_step, "compact": _own_compact}
_PLAIN = {"append": _plain_append, "attention": _plain_attention, "step": _plain_step, "compact": _plain_compact}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "step":
        lens, parents, fork_len, drafts, accept = _step_plan(c)
        P = c["page"]
        tails = sum(1 for f in fork_len if f % P)
        shared = sum(f // P for f in fork_len)
        for ch, f in enumerate(fork_len):
            lens[ch] = f
        new = sum(-(-(n + d + 1) // P) - -(-n // P) for n, d in zip(lens, drafts))
        # page contents once in and once out; a table entry read and written and a count updated
        # for a shared page, the same for a taken one; the counts looked through once for free ones
        return {"bytes": tails * c["page_values"] * 2 * 2 * 2 * c["layers"] + 16 * (shared + new) + 4 * c["pages"] + 16 * c["requests"],
                "flops": 0}
    if c["op"] == "compact":
        used = min(int(c["used"] * c["pages"]), c["requests"] * c["max_pages"])
        moves = min(c["capacity"], used * (c["pages"] - used) // c["pages"])   # expected, pages in random order
        return {"bytes": moves * (c["page_values"] * 2 * 2 * 2 * c["layers"] + 16) + 4 * c["pages"] + 8 * used, "flops": 0}
    drafts, lens = _plan(c)
    R, D, Hq, Hk = sum(drafts) + len(drafts), c["head_dim"], c["q_heads"], c["kv_heads"]
    if c["op"] == "append":
        return {"bytes": 2 * R * (Hq + 2 * Hk) * D * 2 + 12 * len(drafts) + 4 * R + 2 * c["rotary"] + 4 * D,
                "flops": R * (Hq + Hk) * (4 * D * c["norm"] + 3 * c["rotary"])}
    pairs = keys = 0
    for n, L in zip(drafts, lens):
        p, k = _visible(c, n + 1, L)
        pairs, keys = pairs + p, keys + k
    return {"bytes": keys * Hk * D * 2 * 2 + 2 * R * Hq * D * 2 + 4 * keys // c["page"] + 4 * R * Hq * c["lse"],
            "flops": pairs * Hq * D * 4}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "step": _exact_step,
            "compact": _exact_compact}[c["op"]](c, s)


def _exact_append(c, s):
    r, dt = c["rotary"], torch.float64
    k_cache, v_cache = s["k_cache"].to(dt), s["v_cache"].to(dt)
    out = torch.zeros(s["q"].shape, dtype=dt, device="cuda")
    drafts, lens = _plan(c)
    freq = s["inv_freq"].to(dt)
    row = 0
    for b, (n, L) in enumerate(zip(drafts, lens)):
        rows = slice(row, row + n + 1)
        row += n + 1
        pos = torch.arange(L - n - 1, L, device="cuda")
        phase = torch.polar(torch.ones((), dtype=dt, device="cuda"), pos[:, None] * freq)[:, None]
        at = s["block_table"][b][pos // c["page"]].long(), pos % c["page"]
        for x, w, to in ((s["q"], s["q_weight"], None), (s["k"], s["k_weight"], k_cache)):
            x = x[rows].to(dt)
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / c["head_dim"] + EPS).sqrt() * w.to(dt)
            pairs = x[..., :r].unflatten(-1, (-1, 2)) if c["interleaved"] else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
            x[..., :r] = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
            if to is None:
                out[rows] = x
            else:
                to[at] = x
        v_cache[at] = s["v"][rows].to(dt)
    return {"q": out, "k": k_cache, "v": v_cache}


def _exact_attention(c, s):
    dt, Hk, D = torch.float64, c["kv_heads"], c["head_dim"]
    drafts, lens = _plan(c)
    outs, lses = [], []
    row = 0
    for b, (n, L) in enumerate(zip(drafts, lens)):
        m = n + 1
        q = s["q"][row:row + m].to(dt)
        row += m
        first = max(0, L - m + 1 - c["window"]) if c["window"] else 0
        j = torch.cat([torch.arange(min(c["sinks"], first), device="cuda"), torch.arange(first, L, device="cuda")])
        page = s["block_table"][b][j // c["page"]].long()
        k, v = (x[page, j % c["page"]].to(dt) for x in (s["k_cache"], s["v_cache"]))
        p = torch.arange(L - m, L, device="cuda")[:, None]
        hidden = j > p
        if c["window"]:
            hidden |= (p - j >= c["window"]) & (j >= c["sinks"])
        z = torch.einsum("mhgd,jhd->hgmj", q.view(m, Hk, -1, D), k) / math.sqrt(D)
        z = torch.where(hidden, -math.inf, z)
        lse = torch.logsumexp(z, -1)
        o = torch.einsum("hgmj,jhd->mhgd", torch.exp(z - lse[..., None]), v)
        outs.append(o.reshape(m, -1, D))
        lses.append(lse.permute(2, 0, 1).reshape(m, -1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)} if c["lse"] else {"out": torch.cat(outs)}


def _moved(s, src, dst):
    """Copies of the two caches with pages moved."""
    out = []
    for x in (s["k_cache"], s["v_cache"]):
        y = x.clone()
        if src:
            y[:, torch.tensor(dst, device="cuda")] = x[:, torch.tensor(src, device="cuda")]
        out.append(y)
    return out


def _exact_step(c, s):
    lens, parents, fork_len, drafts, accept = _step_plan(c)
    P, M, W = c["page"], c["max_pages"], c["window"]
    table, ref = s["block_table"].tolist(), s["ref_count"].tolist()
    copies = []

    def take(start):
        while ref[start]:
            start += 1
        ref[start] = 1
        return start

    at = 0
    for ch, (p, f) in enumerate(zip(parents, fork_len)):
        for x in range(f // P):
            table[ch][x] = table[p][x]
            if table[p][x] >= 0:
                ref[table[p][x]] += 1
        if f % P:
            at = take(at)
            table[ch][f // P] = at
            copies.append((table[p][f // P], at))
        else:
            copies.append((-1, -1))
        lens[ch] = f
    at = 0
    for b in range(c["requests"]):
        have, new = -(-lens[b] // P), lens[b] + drafts[b] + 1
        for x in range(have, -(-new // P)):
            at = take(at)
            table[b][x] = at
        lens[b] = new - drafts[b] + accept[b]
    for b in range(c["requests"]):
        for x in range(M):
            gone = x * P >= lens[b] or (W and (x + 1) * P <= lens[b] + 1 - W and x * P >= c["sinks"])
            if gone and table[b][x] >= 0:
                ref[table[b][x]] -= 1
                table[b][x] = -1
    out = {"lens": _ints(lens), "block_table": _ints(table), "ref_count": _ints(ref)}
    if c["forks"]:
        real = [(a, d) for a, d in copies if d >= 0]
        k, v = _moved(s, [a for a, _ in real], [d for _, d in real])
        out.update(copy_src=_ints([a for a, _ in copies]), copy_dst=_ints([d for _, d in copies]), k_cache=k, v_cache=v)
    return out


def _exact_compact(c, s):
    table, ref, cap = s["block_table"].tolist(), s["ref_count"].tolist(), c["capacity"]
    used = sum(1 for r in ref if r > 0)
    src = [i for i in range(used, len(ref)) if ref[i] > 0][:cap]
    dst = [i for i in range(used) if ref[i] == 0][:cap]
    dst = dst[:len(src)]
    to = dict(zip(src, dst))
    for a, d in to.items():
        ref[d], ref[a] = ref[a], 0
    table = [[to.get(x, x) for x in row] for row in table]
    k, v = _moved(s, src, dst)
    pad = [-1] * (cap - len(src))
    return {"block_table": _ints(table), "ref_count": _ints(ref), "copy_src": _ints(src + pad),
            "copy_dst": _ints(dst + pad), "k_cache": k, "v_cache": v}
