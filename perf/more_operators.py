"""Cases of the 8-bit cache and of the constrained logits of a verify step: what is measured, and their plain forms.

A server that is short of memory holds keys and values as e4m3 numbers, with one scale for each
block of tokens and head.  The new tokens of a verify step are normalised, rotated and appended in
that form (spec_append8), and their rows attend over it (spec_attention8).  Between the model and
spec_verify stand the requests' own rules about tokens: penalties for repeated ones, biases, and the
masks of a grammar (spec_logits).  A case is one call of these on inputs as such a server holds them.

The plain forms use elementary torch operations in 32 bits (64 for angles); `own` selects the
library's calls instead.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0                    # the largest e4m3 number
LEAST, MOST = 2.0 ** -40, 2.0 ** 40   # of a scale
EPS = 1e-6
BASE = 500000.0                # rotation base; inv_freq_j = BASE^(-2j / rotary_dim)
WORKSPACE = 64 << 20           # more than every call's workspace
TAIL = 256                     # append cases: tokens of context whose pages are still held


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _append(name, requests, drafts, ragged, q_heads, kv_heads, head_dim, rotary, dtype, page, block, context, norm=True,
            interleaved=False, layout="nhd"):
    return dict(name=name, op="append", requests=requests, drafts=drafts, ragged=ragged, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, rotary=rotary, dtype=dtype, page=page, block=block,
                context=context, norm=norm, interleaved=interleaved, layout=layout)


def _attention(name, requests, drafts, ragged, q_heads, kv_heads, head_dim, dtype, page, block, context, window=0,
               sinks=0, lse=False, layout="nhd"):
    return dict(name=name, op="attention", requests=requests, drafts=drafts, ragged=ragged, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page=page, block=block, context=context,
                window=window, sinks=sinks, lse=lse, layout=layout)


def _logits(name, requests, drafts, ragged, vocab, dtype, history, bias, masks, penalties=True, in_place=False):
    """masks: share of the rows under a grammar; history, bias: most entries of a request."""
    return dict(name=name, op="logits", requests=requests, drafts=drafts, ragged=ragged, vocab=vocab, dtype=dtype,
                history=history, bias=bias, masks=masks, penalties=penalties, in_place=in_place)


def listed():
    return [
        # one chat user, one new token and no drafts: pure latency
        _append("append8_single", 1, 0, False, 32, 8, 128, 128, "bf16", 16, 16, 777),
        # the verify batch of the benchmark (256 requests, 4 drafts) at far positions
        _append("append8_verify", 256, 4, False, 32, 8, 128, 128, "bf16", 16, 16, 131072),
        # a ragged batch, half precision, interleaved rotation of a part of each head, no norm
        _append("append8_ragged", 512, 8, True, 24, 4, 96, 48, "fp16", 64, 32, 20011, norm=False, interleaved=True,
                layout="hnd"),
        # one chat user decoding: latency, one row per head group
        _attention("attention8_single", 1, 0, False, 32, 8, 128, "bf16", 16, 16, 2049),
        # one request with a very long context: the length has to be split over the chip
        _attention("attention8_long", 1, 7, False, 32, 8, 128, "bf16", 64, 64, 131071, lse=True),
        # the verify batch of the benchmark over ordinary contexts: the cache's bytes
        _attention("attention8_verify", 256, 4, False, 32, 8, 128, "bf16", 16, 16, 4096),
        # mixed traffic: lengths from one token to long ones, ragged drafts, narrow heads, a window
        _attention("attention8_ragged", 96, 8, True, 28, 4, 64, "fp16", 32, 8, 32768, window=8000, sinks=4, lse=True,
                   layout="hnd"),
        # long draft chains on shared heads: many rows per key, bound by the products
        _attention("attention8_chain", 16, 64, False, 32, 4, 128, "bf16", 64, 32, 8192),
        # one user's next token under a grammar
        _logits("logits_single", 1, 0, False, 32000, "bf16", 500, 8, 1.0),
        # the verify batch of the benchmark: penalties, biases, half of the rows under a grammar
        _logits("logits_verify", 256, 4, False, 128256, "bf16", 1000, 16, 0.5),
        # ragged drafts, penalties alone, a vocabulary whose rows are not whole 16 bytes
        _logits("logits_ragged", 512, 8, True, 151937, "bf16", 2000, 0, 0.0),
        # grammar masks alone, written over the logits
        _logits("logits_masks", 256, 7, False, 128256, "fp32", 0, 0, 1.0, penalties=False, in_place=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "attention", "logits", "logits"])
    drafts, ragged = rng.choice([0, 1, 2, 3, 4, 5, 6, 8, 8, 15, 16, 31, 64]), rng.random() < 0.6
    if op == "logits":
        vocab = rng.choice([_log(rng, 100, 260000), 32000, 50257, 128256, 151936])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        rows = int(2.5e8 / vocab) // (2 if dtype == "fp32" else 1)
        requests = _log(rng, 1, max(1, min(512, rows // (drafts + 1))))
        in_place = rng.random() < 0.3    # (masks alone: what is written over itself stays the same)
        c = _logits("", requests, drafts, ragged, vocab, dtype, 0 if in_place else min(rng.choice([0, 10, 300, 5000]), vocab),
                    0 if in_place else min(rng.choice([0, 1, 30, 300]), vocab), 1.0 if in_place else rng.choice([0.0, 0.3, 1.0]),
                    not in_place, in_place)
        return {k: v for k, v in c.items() if k != "name"}
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    head_dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128])
    dtype, page, layout = rng.choice(["bf16", "bf16", "fp16"]), rng.choice([8, 16, 32, 64, 128, 256]), rng.choice(["nhd", "hnd"])
    block = min(page, rng.choice([8, 16, 32, 64, 256]))
    if op == "append":
        rows = 1280 * 48 * 128 // ((q_heads + 2 * kv_heads) * head_dim)
        requests = _log(rng, 1, max(1, min(512, rows // (drafts + 1))))
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, 16])
        c = _append("", requests, drafts, ragged, q_heads, kv_heads, head_dim, rotary, dtype, page, block,
                    _log(rng, drafts + 1, 400000), rng.random() < 0.7, rng.random() < 0.3, layout)
        return {k: v for k, v in c.items() if k != "name"}
    # keys and values within 2 GB, the plain form's scores within 4 GB, 120 GFLOP
    requests = _log(rng, 1, 256)
    scores = requests * q_heads * (drafts + 1)
    most = min(4e9 / (requests * kv_heads * head_dim * 4), 1e9 / scores, 3e10 / (scores * head_dim), 131072)
    context = _log(rng, drafts + 1, max(drafts + 1, int(most)))
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    c = _attention("", requests, drafts, ragged, q_heads, kv_heads, head_dim, dtype, page, block, context, window,
                   rng.choice([0, 1, 4, 100]) if window else 0, rng.random() < 0.5, layout)
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------------------------------------
# sizes (from the case alone) and inputs (from the seed)
# ---------------------------------------------------------------------------------------------

def _plan(c):
    """Host lists: drafts per request, and (but for logits) lengths after the new tokens."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    B = c["requests"]
    drafts = [r.randint(0, c["drafts"]) if c["ragged"] else c["drafts"] for _ in range(B)]
    if c["op"] == "logits":
        return drafts, None
    if c["op"] == "append":
        lens = [max(n + 1, r.randint(c["context"] // 2, c["context"]) if B > 1 else c["context"]) for n in drafts]
    elif c["ragged"]:
        lens = [max(n + 1, _log(r, 1, c["context"])) for n in drafts]
    else:
        lens = [c["context"]] * B
    return drafts, lens


def _entries(c):
    """Host lists of a logits case: each request's history and bias lengths, and each row's mask (-1: none)."""
    r = random.Random(repr(sorted((k, str(v)) for k, v in c.items() if k != "name")) + "entries")
    drafts, _ = _plan(c)
    history = [r.randint(c["history"] // 2, c["history"]) for _ in drafts]
    bias = [r.randint(0, c["bias"]) for _ in drafts]
    rows, masks = [], 0
    for n in drafts:
        under = r.random() < c["masks"]
        for _ in range(n + 1):
            rows.append(masks if under else -1)
            masks += under
    return history, bias, rows, masks


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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(c, pages, gen):
    """Bytes [pages, slots, heads, head_dim] and scales [pages, blocks, heads] of standard normal values."""
    P, T, Hk, D = c["page"], c["block"], c["kv_heads"], c["head_dim"]
    data = torch.empty((pages, P, Hk, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, P // T, Hk), device="cuda")
    step = max(1, (1 << 27) // (P * Hk * D))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn((n, P // T, T, Hk, D), device="cuda", generator=gen, dtype=torch.bfloat16)
        s = _scale_of(x.abs().amax((2, 4)).float())
        scales[i:i + n] = s
        data[i:i + n] = (x / s[:, :, None, :, None].bfloat16()).to(E4M3).view(torch.uint8).view(n, P, Hk, D)
    if c["layout"] == "hnd":
        data = data.transpose(1, 2).contiguous().transpose(1, 2)
    return data.view(E4M3), scales


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c, "workspace": torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")}
    drafts, lens = _plan(c)
    off = [0]
    for n in drafts:
        off.append(off[-1] + n + 1)
    R, dt = off[-1], DTYPES[c["dtype"]]
    s.update(num_drafts=_ints(drafts), k_max=c["drafts"], off=_ints(off), row_offsets=_ints(off) if c["ragged"] else None)
    if c["op"] == "logits":
        return _prepare_logits(s, c, gen, R, dt)
    P, Hq, Hk, D = c["page"], c["q_heads"], c["kv_heads"], c["head_dim"]
    s["lens"] = _ints(lens)
    max_pages = -(-max(lens) // P)
    j = torch.arange(max_pages, device="cuda")[None]
    L, n = s["lens"].long()[:, None], s["num_drafts"].long()[:, None] + 1
    keep = j * P < L
    if c["op"] == "append":
        keep &= (j + 1) * P > L - n - TAIL
    elif c["window"]:
        keep &= ((j + 1) * P > L - n + 1 - c["window"]) | (j * P < c["sinks"])
    used = int(keep.sum())
    pages = used * 11 // 10 + 3
    s["block_table"] = torch.full(keep.shape, -1, dtype=torch.int32, device="cuda")
    s["block_table"][keep] = torch.randperm(pages, device="cuda", generator=gen)[:used].to(torch.int32)
    s["k_cache"], s["k_scale"] = _cache(c, pages, gen)
    s["v_cache"], s["v_scale"] = _cache(c, pages, gen)
    if c["op"] == "append":
        # the three projections of one product's output, as a layer hands them over; heads and requests differ in size
        qkv = torch.randn((R, Hq + 2 * Hk, D), device="cuda", generator=gen)
        qkv = (qkv * torch.exp(torch.randn((R, Hq + 2 * Hk, 1), device="cuda", generator=gen))).to(dt).view(R, -1)
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
        s["q"] = torch.randn((R, Hq, D), device="cuda", generator=gen).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((R, Hq), device="cuda") if c["lse"] else None
        s["scale"] = 1 / math.sqrt(D)
    return s


def _distinct(counts, vocab, gen):
    """Offsets, and for each request that many distinct token ids in ascending order."""
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    n = _ints(counts).long()
    b = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n)
    i = torch.arange(off[-1], device="cuda") - _ints(off).long()[b]
    # one id out of each of n equal ranges of the vocabulary
    lo, hi = i * vocab // n[b], (i + 1) * vocab // n[b]
    u = torch.rand(off[-1], device="cuda", generator=gen, dtype=torch.float64)
    ids = lo + torch.minimum((u * (hi - lo)).long(), hi - lo - 1)
    return _ints(off), ids.to(torch.int32)


def _prepare_logits(s, c, gen, R, dt):
    V, B = c["vocab"], c["requests"]
    history, bias, rows, masks = _entries(c)
    s["logits"] = torch.randn((R, V), device="cuda", generator=gen, dtype=dt) * 3
    s["out"] = s["logits"] if c["in_place"] else torch.empty_like(s["logits"])
    s["draft_tokens"] = torch.randint(0, V, (R - B,), device="cuda", generator=gen, dtype=torch.int32)
    s["repetition"] = s["presence"] = s["frequency"] = s["prior"] = s["bias"] = s["mask"] = s["mask_rows"] = None
    if c["penalties"]:
        s["repetition"] = 1 + 0.5 * torch.rand(B, device="cuda", generator=gen)
        s["presence"], s["frequency"] = torch.rand((2, B), device="cuda", generator=gen)
    if c["history"]:
        off, ids = _distinct(history, V, gen)
        # (0: a token of the prompt, which only the repetition penalty looks at)
        s["prior"] = off, ids, torch.randint(0, 4, ids.shape, device="cuda", generator=gen, dtype=torch.int32)
    if c["bias"]:
        off, ids = _distinct(bias, V, gen)
        s["bias"] = off, ids, 4 * torch.randn(ids.shape, device="cuda", generator=gen)
    if masks:
        # a grammar's state allows a few tokens, about half of them, or nearly all
        share = torch.tensor([0.001, 0.5, 0.97], device="cuda")[torch.randint(0, 3, (masks,), device="cuda", generator=gen)]
        W = -(-V // 32)
        s["mask"] = torch.empty((masks, W), dtype=torch.int32, device="cuda")
        bit = 2 ** torch.arange(32, device="cuda")
        for i in range(0, masks, 256):
            allowed = torch.rand((min(256, masks - i), W, 32), device="cuda", generator=gen) < share[i:i + 256, None, None]
            s["mask"][i:i + 256] = (allowed * bit).sum(-1).to(torch.int32)
        s["mask_rows"] = _ints(rows)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_append(s):
    from speculative_decoding_verification_12_gb300 import spec_append8
    spec_append8(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["inv_freq"], s["k_cache"], s["v_cache"],
                 s["k_scale"], s["v_scale"], s["block_table"], s["lens"], s["num_drafts"], s["row_offsets"], s["k_max"],
                 s["out"], s["workspace"], interleaved=s["case"]["interleaved"])
    return _appended(s)


def _own_attention(s):
    from speculative_decoding_verification_12_gb300 import spec_attention8
    c = s["case"]
    spec_attention8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["lens"],
                    s["num_drafts"], s["row_offsets"], s["k_max"], s["scale"], c["window"], c["sinks"], s["out"], s["lse"],
                    s["workspace"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}


def _own_logits(s):
    from speculative_decoding_verification_12_gb300 import spec_logits
    spec_logits(s["logits"], s["draft_tokens"], s["num_drafts"], s["row_offsets"], s["k_max"], s["repetition"],
                s["presence"], s["frequency"], s["prior"], s["bias"], s["mask"], s["mask_rows"], s["out"], s["workspace"])
    return {"logits": s["out"]}


def _appended(s):
    return {n: s[m] for n, m in (("q", "out"), ("k", "k_cache"), ("v", "v_cache"), ("k_scale", "k_scale"), ("v_scale", "v_scale"))}


def _rows(s):
    """For each row: its request, and its position in the request's sequence."""
    rows = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["off"].long(), rows, right=True) - 1
    return b, s["lens"].long()[b] - 1 - s["num_drafts"].long()[b] + rows - s["off"].long()[b]


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, within [LEAST, MOST]."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int()), LEAST).clamp(LEAST, MOST)


def _plain_append(s):
    c = s["case"]
    P, T, Hk = c["page"], c["block"], c["kv_heads"]
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
        return torch.cat((y, x[..., r:]), -1)

    s["out"].copy_(turned(s["q"], s["q_weight"]))
    # the blocks that the rows touch: of each request, from its first new token's block on
    first = s["lens"].long() - 1 - s["num_drafts"].long()
    most = c["drafts"] // T + 2
    row_block = pos // T - first[b] // T                      # block of its request that each row lies in
    at = s["block_table"][b, pos // P].long()
    block = (first // T)[:, None] + torch.arange(most, device="cuda")
    touched = block * T < s["lens"].long()[:, None]
    page = s["block_table"].long().gather(1, (block * T // P).clamp(max=s["block_table"].shape[1] - 1))
    page, sub = page[touched], (block % (P // T))[touched]
    older = torch.where(block == (first // T)[:, None], first[:, None] % T, 0)[touched]   # tokens in it before
    slots = sub[:, None] * T + torch.arange(T, device="cuda")
    for x, data, scales in ((turned(s["k"], s["k_weight"]), s["k_cache"], s["k_scale"]), (s["v"].float(), s["v_cache"], s["v_scale"])):
        data = data.view(torch.uint8)
        amax = torch.zeros((c["requests"] * most, Hk), device="cuda")
        amax.index_reduce_(0, b * most + row_block, x.abs().amax(-1), "amax")
        new = _scale_of(amax.view(-1, most, Hk)[touched])
        had = scales[page, sub]
        scale = torch.where(older[:, None] > 0, torch.maximum(had, new), new)
        scales[page, sub] = scale
        # older tokens of a block whose scale grew
        was = data[page[:, None], slots]
        moved = (was.view(E4M3).float() * (had / scale)[:, None, :, None]).to(E4M3).view(torch.uint8)
        keep = (torch.arange(T, device="cuda") < older[:, None])[:, :, None, None]
        data[page[:, None], slots] = torch.where(keep, moved, was)
        mine = torch.zeros((c["requests"], most, Hk), device="cuda")
        mine[touched] = scale
        data[at, pos % P] = (x / mine[b, row_block][:, :, None]).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)
    return _appended(s)


def _plain_attention(s):
    c = s["case"]
    Hk, D, G, P, T = c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"], c["page"], c["block"]
    B, n = c["requests"], c["drafts"] + 1
    L, m = s["lens"].long(), s["num_drafts"].long() + 1
    at = s["block_table"].long().clamp(min=0)
    keys = at.shape[1] * P

    def held(data, scales):
        x = data.view(torch.uint8)[at].view(E4M3).float().contiguous().view(B, -1, P // T, T, Hk, D)
        return x.mul_(scales[at][:, :, :, None, :, None]).view(B, keys, Hk, D)

    k = held(s["k_cache"], s["k_scale"]).permute(0, 2, 3, 1)
    v = held(s["v_cache"], s["v_scale"]).transpose(1, 2)
    i = torch.arange(n, device="cuda")
    row = s["off"].long()[:-1, None] + torch.minimum(i, m[:, None] - 1)
    q = s["q"][row].float().reshape(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    z = (q @ k).view(B, Hk, n, G, keys) * s["scale"]
    pos = (L - m)[:, None, None] + torch.minimum(i, m[:, None] - 1)[:, :, None]
    j = torch.arange(keys, device="cuda")
    seen = j <= pos
    if c["window"]:
        seen &= (j > pos - c["window"]) | (j < c["sinks"])
    z = z.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = z.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(B, Hk, n * G, keys) @ v).view(B, Hk, n, G, D) / total
    used = (i < m[:, None]).flatten().nonzero()[:, 0] if c["ragged"] else slice(None)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, c["q_heads"], D)[used].to(DTYPES[c["dtype"]])
    if not c["lse"]:
        return {"out": o}
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B * n, c["q_heads"])[used]
    return {"out": o, "lse": lse}


def _owners(s, R):
    """For each row: its request, and its number in the request."""
    rows = torch.arange(R, device="cuda")
    b = torch.searchsorted(s["off"].long(), rows, right=True) - 1
    return b, rows - s["off"].long()[b]


def _to_rows(s, c, off, R):
    """(row, entry) of each entry of a request and each of its rows."""
    b, _ = _owners(s, R)
    n = (off[1:] - off[:-1]).long()[b]
    row = torch.repeat_interleave(torch.arange(R, device="cuda"), n)
    return row, torch.arange(row.numel(), device="cuda") - (torch.cumsum(n, 0) - n)[row] + off.long()[b][row]


def _earlier_drafts(s, c, R):
    """(row, token) of each row and each draft of its request before it."""
    b, i = _owners(s, R)
    j = torch.arange(c["drafts"], device="cuda")
    row, j = (j < i[:, None]).nonzero(as_tuple=True)
    return row, s["draft_tokens"][s["off"].long()[b][row] - b[row] + j].long()


def _plain_logits(s):
    c = s["case"]
    R, V = s["logits"].shape
    b, _ = _owners(s, R)
    z = s["logits"].float()
    if c["penalties"]:
        count = torch.zeros((R, V), dtype=torch.int32, device="cuda")
        seen = torch.zeros((R, V), dtype=torch.bool, device="cuda")
        if s["prior"] is not None:
            off, ids, counts = s["prior"]
            row, e = _to_rows(s, c, off, R)
            count[row, ids[e].long()] = counts[e]
            seen[row, ids[e].long()] = True
        row, token = _earlier_drafts(s, c, R)
        count.index_put_((row, token), torch.ones_like(row, dtype=torch.int32), accumulate=True)
        seen[row, token] = True
        rep = s["repetition"][b][:, None]
        z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
        z = z - (s["presence"][b][:, None] * (count > 0) + s["frequency"][b][:, None] * count)
    if s["bias"] is not None:
        off, ids, values = s["bias"]
        row, e = _to_rows(s, c, off, R)
        z[row, ids[e].long()] += values[e]
    if s["mask"] is not None:
        at = s["mask_rows"].long()
        word = s["mask"][at.clamp(min=0)]
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        allowed = (word[:, :, None] >> bit & 1).view(R, -1)[:, :V] != 0
        z = z.masked_fill_(~(allowed | (at < 0)[:, None]), -math.inf)
    s["out"].copy_(z)
    return {"logits": s["out"]}


_OWN = {"append": _own_append, "attention": _own_attention, "logits": _own_logits}
_PLAIN = {"append": _plain_append, "attention": _plain_attention, "logits": _plain_logits}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    c = case
    drafts, lens = _plan(c)
    R = sum(drafts) + len(drafts)
    if c["op"] == "logits":
        history, bias, rows, masks = _entries(c)
        size = 4 if c["dtype"] == "fp32" else 2
        # masks alone, in place: the masks in and the refused tokens' logits out (half of them, on average)
        all_ = R * c["vocab"] * size * 2 if not c["in_place"] else masks * c["vocab"] * size * (1 - (0.001 + 0.5 + 0.97) / 3)
        return {"bytes": all_ + masks * c["vocab"] / 8 + 8 * (sum(history) + sum(bias)) + 8 * R + 16 * len(drafts), "flops": 0}
    D, Hq, Hk, T = c["head_dim"], c["q_heads"], c["kv_heads"], c["block"]
    if c["op"] == "append":
        # inputs in 16 bits, queries out in 16, keys and values out in 8, a scale for each block out
        blocks = sum((L - 1) // T - (L - n - 1) // T + 1 for n, L in zip(drafts, lens))
        return {"bytes": R * D * (4 * Hq + 2 * Hk * 3) + 8 * Hk * blocks + 12 * len(drafts) + 4 * R + 2 * c["rotary"] + 4 * D,
                "flops": R * (Hq + Hk) * (4 * D * c["norm"] + 3 * c["rotary"])}
    pairs = keys = 0
    for n, L in zip(drafts, lens):
        p, k = _visible(c, n + 1, L)
        pairs, keys = pairs + p, keys + k
    return {"bytes": keys * Hk * (D + 4 / T) * 2 + 2 * R * Hq * D * 2 + 4 * keys // c["page"] + 4 * R * Hq * c["lse"],
            "flops": pairs * Hq * D * 4}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "logits": _exact_logits}[c["op"]](c, s)


def _exact_append(c, s):
    """The stored numbers before their rounding to 8 bits; scales."""
    r, dt, T, P = c["rotary"], torch.float64, c["block"], c["page"]
    drafts, lens = _plan(c)
    if sum(drafts) + len(drafts) > 4000:
        return None
    out = torch.zeros(s["q"].shape, dtype=dt, device="cuda")
    k_cache, v_cache = (s[n].view(torch.uint8).view(E4M3).to(dt) for n in ("k_cache", "v_cache"))
    freq, row = s["inv_freq"].to(dt), 0
    for b, (n, L) in enumerate(zip(drafts, lens)):
        rows = slice(row, row + n + 1)
        row += n + 1
        pos = torch.arange(L - n - 1, L, device="cuda")
        phase = torch.polar(torch.ones((), dtype=dt, device="cuda"), pos[:, None] * freq)[:, None]
        for x, w, data, scales in ((s["q"], s["q_weight"], None, None), (s["k"], s["k_weight"], k_cache, s["k_scale"]),
                                   (s["v"], None, v_cache, s["v_scale"])):
            x = x[rows].to(dt)
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / c["head_dim"] + EPS).sqrt() * w.to(dt)
            if data is not v_cache:
                pairs = x[..., :r].unflatten(-1, (-1, 2)) if c["interleaved"] else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
                turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
                x[..., :r] = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
            if data is None:
                out[rows] = x
                continue
            for block in range((L - n - 1) // T, (L - 1) // T + 1):
                page, sub = s["block_table"][b, block * T // P].long(), block % (P // T)
                lo, hi = max(block * T, L - n - 1), min((block + 1) * T, L)
                mine = x[lo - (L - n - 1):hi - (L - n - 1)]
                top = mine.abs().amax((0, 2))
                need = torch.exp2(torch.ceil(torch.log2(top / TOP) - 1e-9)).clamp(LEAST, MOST)
                need = torch.where(top > TOP * need, 2 * need, need).clamp(LEAST, MOST)
                if lo > block * T:
                    had = scales[page, sub].to(dt)
                    need = torch.maximum(need, had)
                    data[page, sub * T:lo % P] *= (had / need)[None, :, None]
                scales[page, sub] = need.float()
                data[page, lo % P:(hi - 1) % P + 1] = (mine / need[None, :, None]).clamp(-TOP, TOP)
    return {"q": out, "k": k_cache, "v": v_cache, "k_scale": s["k_scale"].to(dt), "v_scale": s["v_scale"].to(dt)}


def _exact_attention(c, s):
    dt, Hk, D, P, T = torch.float64, c["kv_heads"], c["head_dim"], c["page"], c["block"]
    drafts, lens = _plan(c)
    outs, lses = [], []
    row = 0
    for b, (n, L) in enumerate(zip(drafts, lens)):
        m = n + 1
        q = s["q"][row:row + m].to(dt)
        row += m
        first = max(0, L - m + 1 - c["window"]) if c["window"] else 0
        j = torch.cat([torch.arange(min(c["sinks"], first), device="cuda"), torch.arange(first, L, device="cuda")])
        page = s["block_table"][b][j // P].long()
        k, v = (x.view(torch.uint8)[page, j % P].view(E4M3).to(dt) * y[page, j % P // T].to(dt)[:, :, None]
                for x, y in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
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


def _exact_logits(c, s):
    drafts, _ = _plan(c)
    R, V = s["logits"].shape
    if R * V > 4e8:
        return None
    out = s["logits"].double()
    bits = 1 << torch.arange(32, device="cuda")
    host = {n: [x.tolist() for x in s[n][:1]] for n in ("prior", "bias") if s[n] is not None}
    row = 0
    for b, n in enumerate(drafts):
        times = torch.zeros(V, dtype=torch.int64, device="cuda")
        met = torch.zeros(V, dtype=torch.bool, device="cuda")
        if s["prior"] is not None:
            e = slice(*host["prior"][0][b:b + 2])
            times[s["prior"][1][e].long()] = s["prior"][2][e].long()
            met[s["prior"][1][e].long()] = True
        for i in range(n + 1):
            x = out[row]
            if i:
                token = s["draft_tokens"][row - b - 1].long()
                times[token] += 1
                met[token] = True
            if c["penalties"]:
                rep = s["repetition"][b].double()
                x = torch.where(met, torch.where(x < 0, x * rep, x / rep), x)
                x = x - s["presence"][b].double() * (times >= 1) - s["frequency"][b].double() * times
            if s["bias"] is not None:
                e = slice(*host["bias"][0][b:b + 2])
                x = x.index_add(0, s["bias"][1][e].long(), s["bias"][2][e].double())
            if s["mask"] is not None and int(s["mask_rows"][row]) >= 0:
                words = s["mask"][int(s["mask_rows"][row])].long()
                refused = (words[:, None] & bits == 0).flatten()[:V]
                x = torch.where(refused, -math.inf, x)
            out[row] = x
            row += 1
    return {"logits": out}
