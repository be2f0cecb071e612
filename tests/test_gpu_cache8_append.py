"""spec_append8 on the GPU against the 64-bit definition (cache8_plain.append).

Queries: as spec_append.  A stored number n with its scale s stands for n s, the nearest to x: off by at most
half a step, 2^-4 of x for normal numbers and 2^-10 s for subnormal ones, plus the fp32 arithmetic before
it (2^-20 of a pair's size, as in spec_append's test).  A scale is the least power of two that holds
its block, except that a maximum within that arithmetic's error of a bound may fall on either side.
Rewritten older tokens are the nearest numbers exactly.
"""
import pytest

import cache8_plain as plain8
import cache_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_12_gb300 as sv
    sv.lib()
    return sv


def make(seed, lens, drafts, k_max, Hq, Hk, D, page, block, dtype, rotary, ragged=True, norm=True, sizes=1.0, old=1.0):
    g = torch.Generator().manual_seed(seed)
    dt, B = DT[dtype], len(lens)
    off = [0]
    for k in drafts:
        off.append(off[-1] + (max(k, 0) + 1 if ragged else k_max + 1))
    R, M = off[-1], max(1, -(-max(max(lens), 1) // page))
    table = torch.full((B, M), -1, dtype=torch.int32)
    want = [(b, x) for b, (L, k) in enumerate(zip(lens, drafts)) if k >= 0
            for x in range(max(L - k - 1, 0) // page, -(-L // page))]
    ids = torch.randperm(len(want) + 3, generator=g)
    for (b, x), p in zip(want, ids.tolist()):
        table[b, x] = p
    shape = (len(ids), page, Hk, D)
    kc, vc = ((torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(E4M3) for _ in range(2))
    ks, vs = (old * 2.0 ** torch.randint(-9, -5, (len(ids), page // block, Hk), generator=g).float() for _ in range(2))
    # heads and tokens of very different sizes
    qkv = torch.randn((R, Hq + 2 * Hk, D), generator=g) * torch.exp(sizes * torch.randn((R, Hq + 2 * Hk, 1), generator=g))
    qkv = qkv.to(dt).flatten(1)
    q, k, v = (x.reshape(R, -1, D) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    w = (torch.rand(2, D, generator=g) + 0.5).to(dt) if norm else (None, None)
    inv = (10000.0 ** (-torch.arange(rotary // 2).double() * 2 / max(rotary, 1))).float() if rotary else None
    return dict(q=q, k=k, v=v, w=w, inv=inv, kc=kc, vc=vc, ks=ks, vs=vs, table=table,
                lens=torch.tensor(lens, dtype=torch.int32), nd=torch.tensor(drafts, dtype=torch.int32),
                ro=torch.tensor(off, dtype=torch.int32) if ragged else None, k_max=k_max, dt=dt)


def gpu(c, layout):
    c = c.view(torch.uint8)
    if layout == "nhd":
        out = c.cuda()
    elif layout == "hnd":
        out = c.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    else:
        both = torch.full((c.shape[0], 2) + tuple(c.shape[1:]), 255, dtype=torch.uint8, device="cuda")
        both[:, 0] = c.cuda()
        out = both[:, 0]
    return out.view(E4M3)


def call(sv, s, layout="nhd", interleaved=False, rope_scale=1.0, inplace=False, eps=1e-6, stream=None):
    R, Hq, D = s["q"].shape
    Hk = s["k"].shape[1]
    dev = torch.cat([s[n].flatten(1) for n in "qkv"], 1).cuda()
    q, k, v = (x.view(R, -1, D) for x in dev.split([Hq * D, Hk * D, Hk * D], 1))
    kc, vc = gpu(s["kc"], layout), gpu(s["vc"], layout)
    # scales [pages, heads, blocks] with room beside them, seen as [pages, blocks, heads]
    ks, vs = (torch.stack((x.transpose(1, 2), x.transpose(1, 2)), 3).cuda()[..., 0].transpose(1, 2) if layout != "nhd" else x.cuda()
              for x in (s["ks"], s["vs"]))
    out = q if inplace else torch.full((R, Hq, D), 7.0, dtype=s["dt"], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    c = lambda t: None if t is None else t.cuda()
    args = [q, k, v, c(s["w"][0]), c(s["w"][1]), eps, c(s["inv"]), kc, vc, ks, vs, c(s["table"]), c(s["lens"]), c(s["nd"]),
            c(s["ro"]), s["k_max"], out, ws]
    torch.cuda.synchronize()
    sv.spec_append8(*args, interleaved=interleaved, rope_scale=rope_scale, stream=stream)
    torch.cuda.synchronize()
    got = dict(q=out, kc=kc.view(torch.uint8), vc=vc.view(torch.uint8), ks=ks, vs=vs)
    return {n: t.cpu() for n, t in got.items()}, sv.sv_read_device_error(ws)


def check(s, got, interleaved=False, rope_scale=1.0, eps=1e-6, rows=slice(None)):
    ro, so, sides = plain8.append(s["q"], s["k"], s["v"], *s["w"], eps, s["inv"], s["kc"], s["vc"], s["ks"], s["vs"],
                                  s["table"], s["lens"], s["nd"], s["ro"], s["k_max"], interleaved, rope_scale)
    tol = torch.finfo(s["dt"]).eps / 2 * ro.abs() + 2.0 ** -20 * so + torch.finfo(s["dt"]).tiny
    assert bool(((got["q"].double() - ro).abs() <= tol)[rows].all())
    for blocks, data, scales in ((sides[0], "kc", "ks"), (sides[1], "vc", "vs")):
        was, now = s[data].view(torch.uint8), got[data]
        numbers = now.view(E4M3).double()
        rest = torch.ones(was.shape[:3], dtype=torch.bool)     # slots that nothing may touch
        rest_scales = torch.ones(s[scales].shape, dtype=torch.bool)
        T = was.shape[1] // s[scales].shape[1]
        for page, sub, h, may, had, older, slots, x, e in blocks:
            scale = float(got[scales][page, sub, h])
            assert scale in may, (data, page, sub, h, scale, may)
            n = older.shape[0]
            rest[page, slots, h] = False
            rest[page, sub * T:sub * T + n, h] = False
            rest_scales[page, sub, h] = False
            have = numbers[page, sub * T:sub * T + n, h]
            want = older if scale == had else torch.tensor(
                [[plain8.nearest(y * had / scale) for y in t] for t in older.tolist()], dtype=torch.float64).view(older.shape)
            assert torch.equal(have.nan_to_num(999.0), want.nan_to_num(999.0)), (data, page, sub, h)
            y = numbers[page, slots, h] * scale
            lost = ~(x.abs() < float("inf"))
            assert torch.equal(y.isnan(), lost)
            x = x.clamp(-448 * scale, 448 * scale)
            tol = 2.0 ** -4 * x.abs() + 2.0 ** -10 * scale + 1.07 * e
            assert bool(((y - x).abs() <= tol)[~lost].all()), (data, page, sub, h, float(((y - x).abs() - tol)[~lost].max()))
        assert torch.equal(now[rest], was[rest])
        assert torch.equal(got[scales][rest_scales].nan_to_num(-7.0), s[scales][rest_scales].nan_to_num(-7.0))


def run_and_check(sv, s, layout="nhd", interleaved=False, rope_scale=1.0, inplace=False, err=(0, -1)):
    got, e = call(sv, s, layout, interleaved, rope_scale, inplace)
    assert e == err
    check(s, got, interleaved, rope_scale)
    return got


CASES = [
    # D, rotary, Hq, Hk, page, block, dtype, interleaved, layout
    (128, 128, 32, 8, 16, 16, "bf16", False, "nhd"), (128, 64, 8, 8, 8, 8, "fp16", True, "hnd"),
    (64, 64, 7, 1, 256, 32, "bf16", True, "both"), (64, 20, 12, 4, 64, 64, "fp16", False, "nhd"),
    (80, 80, 10, 2, 32, 8, "bf16", False, "hnd"), (96, 48, 9, 3, 128, 128, "fp16", True, "nhd"),
    (16, 16, 3, 1, 8, 8, "fp16", False, "nhd"), (16, 2, 1, 1, 16, 8, "bf16", True, "hnd"),
    (16, 0, 2, 2, 8, 8, "bf16", False, "nhd"), (112, 112, 64, 8, 16, 8, "bf16", False, "nhd"),
    (112, 70, 4, 2, 32, 16, "fp16", False, "both"), (48, 6, 5, 5, 256, 256, "bf16", False, "nhd"),
]


@pytest.mark.parametrize("D,rotary,Hq,Hk,page,block,dtype,il,layout", CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_matches_definition(sv, D, rotary, Hq, Hk, page, block, dtype, il, layout, norm):
    s = make(D + rotary, [1, 5, page, page + 1, 3 * page + 2, 40], [0, 4, 2, 1, 3, 7], 7, Hq, Hk, D, page, block, dtype,
             rotary, norm=norm)
    run_and_check(sv, s, layout, il, rope_scale=1.0 if norm else 0.83)


@pytest.mark.parametrize("which", [0, 1])
def test_one_weight_alone(sv, which):
    s = make(2, [9, 30], [4, 2], 4, 6, 2, 64, 16, 8, "bf16", 64)
    s["w"] = tuple(w if i == which else None for i, w in enumerate(s["w"]))
    run_and_check(sv, s)


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("D,page,block", [(64, 16, 8), (128, 256, 256), (128, 64, 32)])
def test_many_rows_and_idle_requests(sv, ragged, D, page, block):
    """Up to 65 rows, several blocks a request, rows that no request uses, blocks of more tokens than a warp keeps."""
    s = make(3, [1, 70, 65, 300, 9, 40], [0, 64, 64, 17, -1, 30], 64, 4, 2, D, page, block, "bf16", D, ragged=ragged)
    run_and_check(sv, s)


def test_idle_requests_that_own_no_row(sv):
    drafts = [-1] * 40 + [2, -1, 0] + [-1] * 100 + [3] + [-1] * 33 + [1] + [-1] * 50
    lens = [9 + b % 40 for b in range(len(drafts))]
    s = make(12, lens, drafts, 3, 4, 2, 64, 16, 16, "bf16", 64)
    rows = [k + 1 for k in drafts]
    off = [sum(rows[:b]) for b in range(len(rows) + 1)]
    s["ro"] = torch.tensor([x + 1 for x in off], dtype=torch.int32)      # and a row before and two after them
    s.update({n: s[n][:off[-1] + 3] for n in "qkv"})
    run_and_check(sv, s)


def test_queries_in_place(sv):
    s = make(4, [60, 7, 33], [8, 2, 0], 8, 16, 4, 128, 16, 16, "bf16", 128)
    a, b = run_and_check(sv, s), run_and_check(sv, s, inplace=True)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("old", [2.0 ** -12, 1.0, 2.0 ** 14])
@pytest.mark.parametrize("sizes", [0.0, 4.0])
def test_scales_that_grow_and_that_stay(sv, old, sizes):
    """Blocks that hold tokens of smaller, similar and larger numbers than the new ones'."""
    s = make(5, [6, 13, 27, 40], [2, 4, 0, 7], 7, 4, 2, 64, 16, 16, "fp16" if sizes == 0 else "bf16", 64, sizes=sizes, old=old)
    run_and_check(sv, s)


def test_a_block_that_grows_token_by_token_is_as_exact_as_one_written_at_once(sv):
    """16 tokens of rising size, one call each: every number is off by one rounding to e4m3, no more (and by what
    falls below the grown scale's subnormal step)."""
    D, T = 64, 16
    g = torch.Generator().manual_seed(6)
    x = (torch.randn(T, 1, D, generator=g) * 2.0 ** torch.linspace(0, 6, T)[:, None, None]).bfloat16().cuda()
    kc, vc = (torch.full((1, T, 1, D), 255, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.full((1, 1, 1), float("nan"), device="cuda") for _ in range(2))
    table, nd = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, out = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.empty(1, 1, D, dtype=torch.bfloat16, device="cuda")
    for t in range(T):
        lens = torch.full((1,), t + 1, dtype=torch.int32, device="cuda")
        row = x[t:t + 1]
        sv.spec_append8(row, row, row, None, None, 0.0, None, kc, vc, ks, vs, table, lens, nd, None, 0, out, ws)
    assert sv.sv_read_device_error(ws) == (0, -1)
    for c, s in ((kc, ks), (vc, vs)):
        scale = float(s)
        assert scale == plain8.scale_for(float(x.float().abs().max()))
        y = plain8.held(c.cpu(), s.cpu())[0]
        ref = x.cpu().double()
        # a token is rounded when it is written, and once more where a growth takes it below 2^-6 of the scale
        assert bool(((y - ref).abs() <= 2.0 ** -4 * ref.abs() + 2 * 2.0 ** -10 * scale).all())
        late = ref.abs() > 2.0 ** -5 * scale
        assert bool(((y - ref).abs() <= 2.0 ** -4 * ref.abs())[late].all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite(sv, bad):
    """Becomes NaN, and neither the scale nor the block's other numbers know of it."""
    s = make(7, [20], [4], 4, 2, 2, 64, 16, 16, "bf16", 0, norm=False)
    ref = {n: t.clone() if torch.is_tensor(t) else t for n, t in s.items()}
    s["k"][1, 0, 5] = s["v"][2, 1, 60] = bad
    got, e = call(sv, s)
    want, _ = call(sv, ref)
    assert e == (0, -1)
    check(s, got)
    p = int(s["table"][0, 1])   # positions 16, 17 are rows 1, 2
    assert bool(got["kc"].view(E4M3)[p, 0, 0, 5].isnan()) and bool(got["vc"].view(E4M3)[p, 1, 1, 60].isnan())
    assert int((got["kc"] != want["kc"]).sum()) <= 64 * 16 and bool(got["ks"].isfinite().all())


def test_the_range_of_scales(sv):
    """Zeros, numbers below every scale and above it; stored scales that are no scales."""
    s = make(8, [20, 20, 20, 20], [3] * 4, 3, 2, 1, 64, 16, 8, "bf16", 0, norm=False)
    s["k"][0:4], s["k"][4:8], s["k"][8:12] = 0.0, 1e-30, 1e30
    s["v"][0:4] = 2.0 ** -45
    s["ks"][int(s["table"][3, 1])] = float("nan")
    s["vs"][int(s["table"][3, 1])] = -1.0
    got = run_and_check(sv, s)
    assert float(got["ks"][int(s["table"][2, 1]), 0]) == 2.0 ** 40
    assert float(plain8.held(got["kc"].view(E4M3), got["ks"])[int(s["table"][2, 1]), 1].abs().max()) == 448 * 2.0 ** 40


def test_errors_stay_with_their_request(sv):
    for what, code in [("short", 1), ("long", 1), ("drafts", 1), ("below", 1), ("page", 9), ("high page", 9)]:
        s = make(9, [40, 33, 20], [4, 4, 4], 4, 4, 2, 64, 16, 16, "bf16", 64, ragged=False)
        ref = {n: t.clone() if torch.is_tensor(t) else t for n, t in s.items()}
        ref["nd"][1] = -1
        if what == "short":
            s["lens"][1] = 3
        if what == "long":
            s["lens"][1] = s["table"].shape[1] * 16 + 1
        if what == "drafts":
            s["nd"][1] = 5
        if what == "below":
            s["nd"][1] = -2
        if what in ("page", "high page"):   # of position 32, the last row; the four before it are sound
            s["table"][1, 2] = -1 if what == "page" else s["kc"].shape[0]
            ref["nd"][1], ref["lens"][1] = 3, 32
        got, e = call(sv, s)
        assert e == (code, 1), what
        rows = [r for r in range(15) if not (r == 9 if code == 9 else 5 <= r < 10)]
        check(ref, got, rows=rows)
        assert bool(got["q"][[r for r in range(15) if r not in rows]].isnan().all())


def test_same_bits_in_a_graph_and_on_another_stream(sv):
    s = make(10, [50, 17, 100], [4, 0, 4], 4, 8, 2, 128, 16, 16, "bf16", 128)
    a, _ = call(sv, s)
    b, _ = call(sv, s, stream=torch.cuda.Stream())
    assert all(torch.equal(a[n], b[n]) for n in a)
    c = lambda t: None if t is None else t.cuda()
    q, k, v, kc, vc, ks, vs = (s[n].cuda() for n in ("q", "k", "v", "kc", "vc", "ks", "vs"))
    out, ws = torch.empty_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = [q, k, v, *map(c, s["w"]), 1e-6, c(s["inv"]), kc, vc, ks, vs, c(s["table"]), c(s["lens"]), c(s["nd"]), c(s["ro"]), 4, out, ws]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_append8(*args)
    for n, t in (("kc", kc), ("vc", vc), ("ks", ks), ("vs", vs)):
        t.view(torch.uint8).copy_(s[n].view(torch.uint8)) if t.dtype == E4M3 else t.copy_(s[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), a["q"]) and torch.equal(kc.view(torch.uint8).cpu(), a["kc"]) and torch.equal(ks.cpu(), a["ks"])


def test_far_positions_and_a_pool_past_32_bits(sv):
    """Offsets beyond 2^31, and a position near the largest."""
    pages, page, D = 70000, 256, 128
    s = make(11, [300], [3], 3, 2, 1, D, page, 64, "bf16", D)
    got, _ = call(sv, s)
    kc, vc = (torch.zeros((pages, page, 1, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros((pages, page // 64, 1), device="cuda") for _ in range(2))
    far, was = pages - 1, int(s["table"][0, 1])
    for t, n in ((kc, "kc"), (vc, "vc")):
        t.view(torch.uint8)[far] = s[n].view(torch.uint8)[was].cuda()
    ks[far], vs[far] = s["ks"][was].cuda(), s["vs"][was].cuda()
    table = torch.tensor([[-1, far]], dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(s["q"], device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    c = lambda t: None if t is None else t.cuda()
    sv.spec_append8(c(s["q"]), c(s["k"]), c(s["v"]), *map(c, s["w"]), 1e-6, c(s["inv"]), kc, vc, ks, vs, table, c(s["lens"]),
                    c(s["nd"]), c(s["ro"]), 3, out, ws)
    assert torch.equal(kc.view(torch.uint8)[far].cpu(), got["kc"][was]) and torch.equal(vs[far].cpu(), got["vs"][was])


@pytest.mark.parametrize("Hq,Hk", [(1024, 1), (1024, 1024)])
def test_the_most_heads(sv, Hq, Hk):
    s = make(13, [5, 40], [1, 2], 2, Hq, Hk, 16, 16, 8, "bf16", 16)
    run_and_check(sv, s)


def test_a_batch_of_idle_requests(sv):
    s = make(14, [30, 7], [1, 1], 1, 4, 2, 64, 16, 16, "bf16", 64, ragged=False)
    s["nd"] = torch.tensor([-1, -1], dtype=torch.int32)
    got, e = call(sv, s)
    assert e == (0, -1) and not bool(got["q"].any())
    assert all(torch.equal(got[n], s[n].view(torch.uint8) if n in ("kc", "vc") else s[n]) for n in ("kc", "vc", "ks", "vs"))


def test_two_graphs_at_once(sv):
    """Replayed over and over, an append writes what it wrote the first time."""
    calls = []
    c = lambda t: None if t is None else t.cuda()
    for seed, Hq, Hk, D, dtype in ((15, 8, 2, 128, "bf16"), (16, 6, 3, 64, "fp16")):
        s = make(seed, [50, 17, 100], [4, 0, 4], 4, Hq, Hk, D, 16, 16, dtype, D)
        want, _ = call(sv, s)
        q, k, v, kc, vc, ks, vs = (s[n].cuda() for n in ("q", "k", "v", "kc", "vc", "ks", "vs"))
        out, ws = torch.empty_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")
        args = [q, k, v, *map(c, s["w"]), 1e-6, c(s["inv"]), kc, vc, ks, vs, *map(c, (s["table"], s["lens"], s["nd"], s["ro"])), 4, out, ws]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                sv.spec_append8(*args)
        calls.append((want, dict(q=out, kc=kc.view(torch.uint8), vc=vc.view(torch.uint8), ks=ks, vs=vs), graph, torch.cuda.Stream(), args))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, graph, stream, _ in calls:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for want, got, _, _, _ in calls:
        assert all(torch.equal(got[n].cpu(), want[n]) for n in want)


def uneven_scales():
    """Scales that are no powers of two: simple ones, and fp32 neighbours of x / t for ties t of e4m3's, so that x / s (and
    older numbers in a grown scale, n s / s') is a tie once it is rounded to fp32 and none before."""
    some = [1.75, 1.25, 3.0, 1.1, 1 + 2.0 ** -23, 2 - 2.0 ** -23, 1.7]
    some += [x / t for x in (129, 167, 201, 251) for t in (17, 19, 25, 31)]
    some += [t / n for n in (9, 11, 13, 15) for t in (1.5, 2.5, 17, 25, 31)]
    return [float(torch.tensor(s, dtype=torch.float32)) / 64 for s in some]


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp16", 128)])
@pytest.mark.parametrize("grow", [False, True])
def test_kept_scales_that_are_no_powers_of_two(sv, dtype, D, grow):
    """Every new number is the nearest to x / s with the kept scale (ties of x / s to even, and no others), and every older one
    to n s / s' where the scale grows.  No norm and no rotation: the elements are known exactly."""
    had = uneven_scales()
    B = len(had)
    s = make(17, [23] * B, [2] * B, 2, 1, 1, D, 32, 32, dtype, 0, norm=False)
    g = torch.Generator().manual_seed(18)
    for b, h in enumerate(had):
        page = int(s["table"][b, 0])
        s["ks"][page] = s["vs"][page] = h
        codes = torch.randint(0, 256, (20, D), generator=g, dtype=torch.uint8)
        s["kc"].view(torch.uint8)[page, :20, 0] = s["vc"].view(torch.uint8)[page, :20, 0] = codes
    ties = torch.tensor([(n + 0.5) * 2.0 ** e for n in range(8, 16) for e in range(-9, 4)] + [(n + 0.5) * 2.0 ** -9 for n in range(8)])
    for n in "kv":
        x = torch.tensor([129.0, 167, 201, 251])[torch.randint(0, 4, s[n].shape, generator=g)] * torch.exp2(
            torch.randint(-15, 0, s[n].shape, generator=g).float())
        near = ties[torch.randint(0, len(ties), s[n].shape, generator=g)] * torch.tensor(had).repeat_interleave(3)[:, None, None]
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, x / 64, near)
        x = torch.minimum(x, 220 * torch.tensor(had).repeat_interleave(3)[:, None, None])    # (a power of two below it holds them)
        if grow:                           # past 448 of the scale, by powers of two up to where older numbers are ties below 2^-6
            x[:, :, 0] = 1000.0 * torch.exp2(torch.arange(len(x)).float() % 7)[:, None] * torch.tensor(had).repeat_interleave(3)[:, None]
        s[n] = (x * torch.sign(torch.randn(x.shape, generator=g))).to(s["dt"])
    got = run_and_check(sv, s)
    for n, data, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
        numbers = got[data].view(E4M3).double()
        for b, h in enumerate(had):
            page = int(s["table"][b, 0])
            scale = float(got[scales][page, 0, 0])
            assert (scale != h and scale == 2.0 ** round(plain8.math.log2(scale))) if grow else scale == h
            want = [[plain8.nearest(x / scale) for x in row] for row in s[n][3 * b:3 * b + 3, 0].double().tolist()]
            assert torch.equal(numbers[page, 20:23, 0], torch.tensor(want, dtype=torch.float64)), (n, h)
            was = s[data].view(torch.uint8)[page, :20, 0].view(E4M3).double().nan_to_num(999.0)
            now = numbers[page, :20, 0].nan_to_num(999.0)
            if not grow:
                assert torch.equal(was, now)
                continue
            want = [[x if x == 999.0 else plain8.nearest(x * h / scale) for x in row] for row in was.tolist()]
            assert torch.equal(now, torch.tensor(want, dtype=torch.float64)), (n, h)
