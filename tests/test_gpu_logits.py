"""spec_logits on the GPU against the definition in float64 (`plain` below, a loop over rows and tokens).

Tolerance: the output is rounded once to its type (eps / 2 of its value; fp32: the last of the operations), and
before that come at most five fp32 operations, each off by 2^-24 of its result: the quotient or product, the
product and sum of the penalties, the difference, the bias.  In all eps / 2 |z| + 5 * 2^-24 times the sum of the
magnitudes that enter.  Logits that no rule touches, and refused ones, are exact.
"""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_12_gb300 as sv
    sv.lib()
    return sv


def lists(r, counts, V, near=()):
    """For each request that many distinct ids, ascending; some of them from `near`."""
    out = []
    for b, n in enumerate(counts):
        ids = set(list(near[b])[:n]) if near else set()
        while len(ids) < min(n, V):
            ids.add(r.randrange(V))
        out.append(sorted(ids))
    return out


def make(seed, drafts, k_max, V, dtype, history=50, bias=20, masks=True, ragged=True, own_extra=0):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    B = len(drafts)
    off = [0]
    for k in drafts:
        off.append(off[-1] + (k + 1 + own_extra if ragged else k_max + 1))
    R = off[-1]
    toks = torch.randint(0, V, (R - B,), generator=g, dtype=torch.int32)
    mine = [toks[off[b] - b:off[b] - b + k].tolist() for b, k in enumerate(drafts)]
    for b, k in enumerate(drafts):
        if k > 2:   # the same draft twice
            toks[off[b] - b + 2] = toks[off[b] - b]
    prior = lists(r, [r.randint(0, history) for _ in drafts], V, mine)
    rules = lists(r, [r.randint(0, bias) for _ in drafts], V, [m[1:] + p[:5] for m, p in zip(mine, prior)])
    cat = lambda x: (torch.tensor([0] + [sum(map(len, x[:i + 1])) for i in range(B)], dtype=torch.int32),
                     torch.tensor([v for ids in x for v in ids], dtype=torch.int32))
    po, pt = cat(prior)
    bo, bt = cat(rules)
    W = -(-V // 32) + seed % 2
    share = torch.tensor([0.0, 0.01, 0.5, 0.98, 1.0])[torch.arange(R) % 5]
    mask = ((torch.rand((R, W, 32), generator=g) < share[:, None, None]) * 2 ** torch.arange(32)).sum(-1).to(torch.int32)
    rows = torch.randperm(R, generator=g).to(torch.int32)
    rows[torch.rand(R, generator=g) < 0.3] = -1
    return dict(z=(torch.randn((R, V), generator=g) * 3).to(DT[dtype]), toks=toks, nd=torch.tensor(drafts, dtype=torch.int32),
                ro=torch.tensor(off, dtype=torch.int32) if ragged else None, k_max=k_max, rep=1 + torch.rand(B, generator=g),
                pres=torch.rand(B, generator=g) - 0.3, freq=torch.rand(B, generator=g) - 0.3,
                prior=(po, pt, torch.randint(0, 4, pt.shape, generator=g, dtype=torch.int32)) if history else None,
                bias=(bo, bt, 4 * torch.randn(bt.shape, generator=g)) if bias else None,
                mask=mask if masks else None, rows=rows if masks else None)


def plain(s):
    """(result in float64, which logits a rule changed, magnitudes that entered); rows of no request as they are."""
    z = s["z"].double()
    size, hit = z.abs(), torch.zeros(z.shape, dtype=torch.bool)
    refused = torch.zeros(z.shape, dtype=torch.bool)
    used = torch.zeros(z.shape[0], dtype=torch.bool)
    V, B = z.shape[1], len(s["nd"])
    one = lambda name, b, other: float(s[name][b]) if s[name] is not None else other
    for b, k in enumerate(s["nd"].tolist()):
        row0 = int(s["ro"][b]) if s["ro"] is not None else b * (s["k_max"] + 1)
        rep, pres, freq = one("rep", b, 1.0), one("pres", b, 0.0), one("freq", b, 0.0)
        some = any(s[n] is not None for n in ("rep", "pres", "freq"))
        count = {}
        if s["prior"] is not None:
            o, t, c = s["prior"]
            count = dict(zip(t[o[b]:o[b + 1]].tolist(), c[o[b]:o[b + 1]].tolist()))
        for i in range(k + 1):
            row = row0 + i
            used[row] = True
            if i and some:
                t = int(s["toks"][row0 - b + i - 1])
                count[t] = count.get(t, 0) + 1
            if some:
                for t, c in count.items():
                    x = float(z[row, t])
                    x = x / rep if x > 0 else x * rep
                    p = pres * (c > 0) + freq * c
                    size[row, t] += abs(x) + abs(pres) + 2 * abs(freq) * c
                    z[row, t], hit[row, t] = x - p, True
            if s["bias"] is not None:
                o, t, v = s["bias"]
                for t, v in zip(t[o[b]:o[b + 1]].tolist(), v[o[b]:o[b + 1]].tolist()):
                    z[row, t] += v
                    size[row, t] += abs(v)
                    hit[row, t] = True
            if s["mask"] is not None and int(s["rows"][row]) >= 0:
                words = s["mask"][int(s["rows"][row])].long() & 0xffffffff
                bits = (words[:, None] >> torch.arange(32) & 1).flatten()[:V] == 0
                refused[row] = bits
    z[refused] = -math.inf
    return z, hit, size, refused, used


def call(sv, s, in_place=False, stream=None):
    c = lambda t: None if t is None else tuple(x.cuda() for x in t) if isinstance(t, tuple) else t.cuda()
    z = s["z"].cuda()
    out = z if in_place else torch.full_like(z, 7.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = [z, c(s["toks"]), c(s["nd"]), c(s["ro"]), s["k_max"], c(s["rep"]), c(s["pres"]), c(s["freq"]), c(s["prior"]),
            c(s["bias"]), c(s["mask"]), c(s["rows"]), out, ws]
    torch.cuda.synchronize()
    sv.spec_logits(*args, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), sv.sv_read_device_error(ws)


def check(s, out, in_place=False, rows=None):
    z, hit, size, refused, used = plain(s)
    free = ~hit & ~refused & used[:, None]
    if rows is not None:
        keep = torch.zeros(len(used), dtype=torch.bool)
        keep[rows] = True
        used, free, refused, hit = used & keep, free & keep[:, None], refused & keep[:, None], hit & keep[:, None]
    assert torch.equal(out[free], s["z"][free])
    assert bool((out[refused] == -math.inf).all())
    changed = hit & ~refused
    eps = torch.finfo(out.dtype).eps
    tol = eps / 2 * z.abs() + 5 * 2.0 ** -24 * size + torch.finfo(out.dtype).tiny
    d = (out.double() - z).abs()
    assert bool((d <= tol)[changed].all()), float((d / tol)[changed].max())
    if rows is None:
        rest = s["z"][~used] if in_place else torch.full_like(s["z"][~used], 7.0)
        assert torch.equal(out[~used], rest)


def run_and_check(sv, s, err=(0, -1)):
    a, e = call(sv, s)
    assert e == err
    check(s, a)
    b, e = call(sv, s, in_place=True)
    assert e == err
    check(s, b, True)
    used = plain(s)[4]
    assert torch.equal(a[used], b[used])
    return a


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 7, 31, 32, 33, 255, 1000, 2048, 4099, 32000])
def test_vocabularies(sv, dtype, V):
    """Rows that begin anywhere in 16 bytes, that end inside a word of the mask, of one token and of several pieces."""
    run_and_check(sv, make(V, [3, 0, 5, 1], 5, V, dtype, history=min(V, 40), bias=min(V, 15)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_batches(sv, dtype):
    """More than one piece a row and enough rows for the long pieces."""
    r = random.Random(3)
    run_and_check(sv, make(3, [r.randint(0, 8) for _ in range(60)], 8, 50257, dtype, history=400, bias=60))


@pytest.mark.parametrize("ragged,extra", [(True, 0), (True, 2), (False, 0)])
def test_rows_that_no_request_uses(sv, ragged, extra):
    run_and_check(sv, make(4, [2, 0, 4, 3], 4, 700, "bf16", ragged=ragged, own_extra=extra))


def test_many_drafts(sv):
    run_and_check(sv, make(5, [64, 63, 0, 64], 64, 300, "bf16"))


def test_offsets_that_leave_rows_at_both_ends(sv):
    s = make(6, [2, 1], 4, 500, "fp32", own_extra=1)
    s["ro"] = torch.tensor([0, 4, 6], dtype=torch.int32)
    run_and_check(sv, s)


@pytest.mark.parametrize("off", ["rep", "pres", "freq", "prior", "bias", "mask", "all penalties", "all"])
def test_rules_that_are_not_given(sv, off):
    s = make(7, [3, 0, 2], 4, 900, "bf16")
    for n in {"all penalties": ("rep", "pres", "freq"), "mask": ("mask", "rows"),
              "all": ("rep", "pres", "freq", "prior", "bias", "mask", "rows")}.get(off, (off,)):
        s[n] = None
    run_and_check(sv, s)


def test_empty_lists_and_no_drafts(sv):
    s = make(8, [0, 0, 0], 0, 400, "bf16", history=0, bias=0)
    zero, none = torch.zeros(4, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    s["prior"], s["bias"] = (zero, none, none), (zero, none, torch.zeros(0))
    run_and_check(sv, s)
    s = make(9, [2, 1], 2, 400, "fp32")
    s["mask"], s["rows"] = torch.zeros((0, 13), dtype=torch.int32), torch.full((5,), -1, dtype=torch.int32)
    run_and_check(sv, s)


def test_lists_of_the_whole_vocabulary(sv):
    run_and_check(sv, make(10, [3, 2], 3, 3000, "fp32", history=3000, bias=3000))


def test_values_at_the_edges(sv):
    """-inf, NaN and infinite logits; -inf biases; a mask that refuses what a rule would change."""
    s = make(11, [2, 2], 2, 300, "fp32", masks=False)
    s["z"][:, ::7], s["z"][:, 1::11] = -math.inf, 0.0
    s["bias"][2][::3] = -math.inf
    out, e = call(sv, s)
    z = plain(s)[0]
    assert e == (0, -1)
    low = z == -math.inf
    assert bool((out[low] == -math.inf).all()) and bool(out[~low].isfinite().all())
    s["z"][0, 5], s["z"][1, 6] = math.nan, math.inf
    s["bias"] = None
    out, e = call(sv, s)
    assert bool(out[0, 5].isnan()) and float(out[1, 6]) == math.inf
    assert e == (0, -1)


def test_sums_wait_for_one_rounding(sv):
    """bf16: repetition, penalties and bias of one token are one rounding, not three."""
    s = make(12, [0], 0, 64, "bf16", history=0, bias=0, masks=False)
    s["z"][0, 9] = 100.0
    s["rep"][0], s["pres"][0], s["freq"][0] = 1.0, 0.3, 0.0
    s["prior"] = tuple(torch.tensor(x, dtype=torch.int32) for x in ([0, 1], [9], [1]))
    s["bias"] = (*(torch.tensor(x, dtype=torch.int32) for x in ([0, 1], [9])), torch.tensor([0.2]))
    out, _ = call(sv, s)
    assert float(out[0, 9]) == float(torch.tensor(99.9).bfloat16())


@pytest.mark.parametrize("in_place", [False, True])
def test_errors_stay_with_their_request(sv, in_place):
    for what, code in [("drafts", 1), ("idle", 1), ("token", 2), ("high token", 2), ("rep 0", 6), ("rep nan", 6), ("pres", 6),
                       ("freq", 6), ("prior offsets", 8), ("bias offsets", 12), ("mask", 13), ("high mask", 13)]:
        s = make(13, [2, 3, 1], 3, 600, "bf16", ragged=False)
        ref = {n: t.clone() if torch.is_tensor(t) else t for n, t in s.items()}
        if what in ("drafts", "idle"):
            s["nd"][1] = 4 if what == "drafts" else -1
        if "token" in what:
            s["toks"][3 + 1] = -1 if what == "token" else 600
        if what.startswith("rep"):
            s["rep"][1] = 0.0 if what == "rep 0" else math.nan
        if what in ("pres", "freq"):
            s[what][1] = math.inf
        if what.endswith("offsets"):   # past the end; the last request's are wrong with it
            n = what.split()[0]
            o = s[n][0].clone()
            o[1], o[2] = len(s[n][1]) + 2, len(s[n][1]) + 5
            s[n] = (o, *s[n][1:])
        if "mask" in what:
            s["rows"][4 + 2] = -2 if what == "mask" else len(s["mask"])
        out, e = call(sv, s, in_place)
        if what.endswith("offsets"):
            assert e[0] == code
            continue
        assert e == (code, 1), what
        assert bool(out[4:8].isnan().all()), what
        check(ref, out, in_place, rows=[0, 1, 2, 8, 9])


def test_lists_that_do_not_ascend_are_reported(sv):
    for n, code in (("prior", 8), ("bias", 12)):
        for bad in ("order", "twice", "low", "high", "count"):
            if bad == "count" and n == "bias":
                continue
            s = make(14, [2, 3, 1], 3, 600, "bf16", history=40, bias=40)
            o, t, v = s[n][0].clone(), s[n][1].clone(), s[n][2].clone()
            lo, hi = int(o[1]), int(o[2])
            assert hi - lo > 3
            if bad == "order":
                t[lo], t[hi - 1] = int(t[hi - 1]), int(t[lo])
            elif bad == "twice":
                t[lo + 1] = t[lo]
            elif bad == "low":
                t[lo] = -5
            elif bad == "high":
                t[hi - 1] = 600
            else:
                v[lo] = -1
            s[n] = (o, t, v)
            out, e = call(sv, s)
            assert e == (code, 1), (n, bad)
            ref = make(14, [2, 3, 1], 3, 600, "bf16", history=40, bias=40)
            check(ref, out, rows=[0, 1, 2, 7, 8])


def test_requests_without_rows(sv):
    """A request that owns no row is reported, and the drafts of those after it are not where they should be."""
    s = make(15, [2, 1, 2], 2, 100, "bf16")
    s["ro"] = torch.tensor([0, 3, 3, 8], dtype=torch.int32)
    out, e = call(sv, s)
    assert e == (1, 1)
    check({**s, "nd": s["nd"][:1], "ro": s["ro"][:2], "prior": (s["prior"][0][:2], *s["prior"][1:]),
           "bias": (s["bias"][0][:2], *s["bias"][1:])}, out, rows=[0, 1, 2])


def test_same_bits_in_a_graph_and_on_another_stream(sv):
    s = make(16, [3, 0, 5, 1], 5, 32000, "bf16")
    a, _ = call(sv, s)
    b, _ = call(sv, s, stream=torch.cuda.Stream())
    used = plain(s)[4]
    assert torch.equal(a[used], b[used])
    c = lambda t: None if t is None else tuple(x.cuda() for x in t) if isinstance(t, tuple) else t.cuda()
    z, ws = s["z"].cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = [z, c(s["toks"]), c(s["nd"]), c(s["ro"]), s["k_max"], c(s["rep"]), c(s["pres"]), c(s["freq"]), c(s["prior"]),
            c(s["bias"]), c(s["mask"]), c(s["rows"]), z, ws]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_logits(*args)
    z.copy_(s["z"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z.cpu()[used], a[used])


def test_verify_after_the_rules(sv):
    """spec_verify on ruled logits: greedy requests take the largest allowed, penalised token."""
    B, k, V = 6, 3, 5000
    s = make(17, [k] * B, k, V, "fp32", ragged=False)
    s["rows"][:] = torch.arange(B * (k + 1)) % 4 + 1        # (masks that allow something)
    out, e = call(sv, s)
    assert e == (0, -1)
    best = out.argmax(1).view(B, k + 1)
    full = lambda v, t: torch.full((B,), v, dtype=t, device="cuda")
    tokens = torch.empty(B, k + 1, dtype=torch.int32, device="cuda")
    accept = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(sv.sv_workspace_bytes(B, B * (k + 1), V), dtype=torch.uint8, device="cuda")
    sv.spec_verify(out.cuda(), torch.zeros(B * k, V, device="cuda"), s["toks"].cuda(), s["nd"].cuda(), None, k,
                   full(1, torch.float32), full(0, torch.int32), full(1, torch.float32), None, None, full(1, torch.uint8),
                   torch.zeros(B * (k + 1), 2, device="cuda"), tokens, accept, None, ws)
    drafts = s["toks"].view(B, k)
    for b in range(B):
        a = 0
        while a < k and drafts[b, a] == best[b, a]:
            a += 1
        assert int(accept[b]) == a and int(tokens[b, a]) == int(best[b, a])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_largest_vocabulary(sv, dtype):
    run_and_check(sv, make(18, [1, 0], 1, 1 << 21, dtype, history=300, bias=30, masks=dtype == "fp32"))


def test_the_largest_counts(sv):
    """A history count of 2^31 - 1, and drafts of the same token."""
    s = make(19, [3], 3, 64, "fp32", history=0, bias=0, masks=False)
    s["toks"][:] = 9
    s["freq"][0], s["pres"][0] = 1e-9, 0.5
    s["prior"] = tuple(torch.tensor(x, dtype=torch.int32) for x in ([0, 2], [9, 12], [2 ** 31 - 1, 0]))
    run_and_check(sv, s)


def test_a_row_that_allows_one_token_or_none(sv):
    """Whatever the other rules say of them."""
    s = make(20, [4, 4], 4, 1000, "bf16", history=1000, bias=1000)
    s["mask"][:] = 0
    s["mask"][:, 17] = 1 << 5
    s["mask"][3] = 0
    s["rows"][:] = torch.tensor([0, 1, 2, 3, 4, 3, 3, 5, 5, 5])
    out = run_and_check(sv, s)
    assert (out > -math.inf).sum(1).tolist() == [1, 1, 1, 0, 1, 0, 0, 1, 1, 1]


def test_two_graphs_at_once(sv):
    """Graphs of calls of different sizes, replayed on two streams at a time."""
    calls = []
    c = lambda t: None if t is None else tuple(x.cuda() for x in t) if isinstance(t, tuple) else t.cuda()
    for seed, V, dtype in ((21, 32000, "bf16"), (22, 9001, "fp32")):
        s = make(seed, [3, 0, 5, 1], 5, V, dtype)
        z, ws = s["z"].cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(z)
        args = [z, c(s["toks"]), c(s["nd"]), c(s["ro"]), s["k_max"], c(s["rep"]), c(s["pres"]), c(s["freq"]), c(s["prior"]),
                c(s["bias"]), c(s["mask"]), c(s["rows"]), out, ws]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                sv.spec_logits(*args)
        calls.append((s, out, graph, torch.cuda.Stream(), args))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, graph, stream, _ in calls:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for s, out, _, _, _ in calls:
        check(s, out.cpu(), rows=plain(s)[4])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lists_that_end_at_the_last_index(sv, dtype):
    """Entries up to number 2^31 - 2 of each list, with more biases in a piece than are kept beside it and histories of
    several passes of a CTA: the same bits as from lists that begin at 0.  The lists are views of one buffer of 9 GB, each
    a few thousand entries further on, so that their ends lie side by side."""
    s = make(24, [5, 3], 5, 4099, dtype, history=4000, bias=4000)
    n, apart = 2 ** 31 - 1, 8192
    assert min(s[x][0].diff().min() for x in ("prior", "bias")) > 1500 and max(len(s[x][1]) for x in ("prior", "bias")) < apart
    want, _ = call(sv, s)
    buffer = torch.empty(n + 4 * apart, dtype=torch.int32, device="cuda")
    at = 0
    for name in ("prior", "bias"):
        o, t, v = s[name]
        views = []
        for x in (t, v):
            view = buffer[at:at + n]
            view[n - len(x):] = x.view(torch.int32).cuda()
            views.append(view.view(x.dtype))
            at += apart
        s[name] = (o + (n - len(t)), *views)
    for in_place in (False, True):
        out, e = call(sv, s, in_place)
        assert e == (0, -1)
        used = torch.cat([torch.arange(int(a), int(b)) for a, b in zip(s["ro"], s["ro"][1:])])
        assert torch.equal(out[used], want[used])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name,code", [("prior", 8), ("bias", 12)])
def test_offsets_out_of_range_stay_with_their_requests(sv, name, code, in_place):
    """Past the end, below 0 and decreasing: rows of NaN for the requests whose offsets those are, the others' as ever."""
    rows = [[0, 1, 2], [3, 4, 5, 6], [7, 8]]
    for change, bad, sound in (({2: 5}, [1, 2], [0]), ({3: 1}, [2], [0, 1]), ({3: 2 ** 31 - 1}, [2], [0, 1]), ({0: -1}, [0], [1, 2]),
                               ({0: -2 ** 31}, [0], [1, 2]), ({2: -1}, [1, 2], [0]), ({2: "less"}, [1], [0])):
        s = make(13, [2, 3, 1], 3, 600, "bf16")
        o = s[name][0].clone()
        assert o[2] > o[1] > 0
        for i, x in change.items():
            o[i] = int(o[1]) - 1 if x == "less" else x if x < 0 or x == 2 ** 31 - 1 else len(s[name][1]) + x
        out, e = call(sv, {**s, name: (o, *s[name][1:])}, in_place)
        assert e == (code, bad[0]), change
        for b in bad:
            assert bool(out[rows[b]].isnan().all()), (change, b)
        check(s, out, in_place, rows=sum((rows[b] for b in sound), []))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_lists_in_any_order_stay_with_their_request(sv, dtype):
    """Shuffled lists of some thousand entries, over several pieces of a row: reported, and the other request's rows as ever."""
    for name, code in (("prior", 8), ("bias", 12)):
        for how in ("shuffled", "reversed"):
            s = make(24, [5, 3], 5, 4099, dtype, history=4000, bias=4000)
            o, t, v = s[name]
            lo, hi = int(o[1]), int(o[2])
            order = torch.arange(lo, hi).flip(0) if how == "reversed" else lo + torch.randperm(hi - lo, generator=torch.Generator().manual_seed(1))
            t = t.clone()
            t[lo:hi] = t[order]
            out, e = call(sv, {**s, name: (o, t, v)})
            assert e == (code, 1), (name, how)
            check(s, out, rows=[0, 1, 2, 3, 4, 5])
