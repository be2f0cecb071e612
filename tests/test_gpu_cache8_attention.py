"""spec_attention8 on the GPU against the 64-bit definition over the numbers that the cache stands for.

Tolerances as for spec_attention (its test derives them): an output is off by eps / 2 of its value, by the
weights' rounding (at most eps / 2 of S = sum_j p_j |v_j|; 2^-9 in bf16, whose eps / 2 is 2^-8), by twice what a score
is off, and by (T + 16) 2^-23 of S for exponentials and sums.  A score is off by head_dim 2^-23 sum |q k| scale as there,
and by the parts of the queries, 2^-21 of the row's largest element times sum |k| scale.
A weight, times its value's scale, is held relative to the row's largest such product, which the kernel keeps at 2^12 or
more, as a sum of e5m2 numbers: whatever its size it is off by at most their smallest step, 2^-16, where it is cut off,
and so by 2^-28 of the largest.  (Beside the relative rounding above this matters only where an output's large weights
meet zeros.)
"""
import math
import random

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


def make(seed, lens, drafts, k_max, Hq, Hk, D, page, block, dtype, window=0, sinks=0, ragged=True, layout="nhd", spare=2,
         sharpen=1.0, spread=1.0):
    """Requests over pages in random order; slots and blocks past each length, and pages out of the window,
    hold NaN or nothing (-1).  spread: of the blocks' sizes, in powers of two."""
    g = torch.Generator().manual_seed(seed)
    dt, B = DT[dtype], len(lens)
    off = [0]
    for k in drafts:
        off.append(off[-1] + (max(k, 0) + 1 if ragged else k_max + 1))
    R, M = off[-1], max(1, -(-max(max(lens), 1) // page)) + spare
    table = torch.full((B, M), -1, dtype=torch.int32)
    want = []
    for b, (L, k) in enumerate(zip(lens, drafts)):
        first = max(0, L - k - window) if window else 0
        want += [(b, x) for x in range(-(-L // page)) if (x + 1) * page > first or x * page < sinks]
    ids = torch.randperm(len(want) + 3, generator=g).tolist()
    kc, vc = ((torch.randn((len(ids), page, Hk, D), generator=g) * 100).clamp(-448, 448).to(E4M3).view(torch.uint8) for _ in range(2))
    ks, vs = (torch.exp2(spread * torch.randn((len(ids), page // block, Hk), generator=g) - 7) for _ in range(2))
    for (b, x), p in zip(want, ids):
        table[b, x] = p
        end = lens[b] - x * page
        if end < page:
            kc[p, end:] = vc[p, end:] = 255
            ks[p, -(-end // block):] = vs[p, -(-end // block):] = float("nan")
    for p in ids[len(want):]:
        kc[p] = vc[p] = 127
        ks[p] = vs[p] = float("nan")
    return dict(q=(torch.randn((R, Hq, D), generator=g) * sharpen).to(dt), kc=kc.view(E4M3), vc=vc.view(E4M3), ks=ks, vs=vs,
                table=table, lens=torch.tensor(lens, dtype=torch.int32), nd=torch.tensor(drafts, dtype=torch.int32),
                ro=torch.tensor(off, dtype=torch.int32) if ragged else None, k_max=k_max, layout=layout, dt=dt,
                window=window, sinks=sinks, scale=1 / math.sqrt(D))


def gpu(c, layout):
    c = c.view(torch.uint8)
    if layout == "nhd":
        return c.cuda().view(E4M3)
    if layout == "hnd":
        return c.transpose(1, 2).contiguous().cuda().transpose(1, 2).view(E4M3)
    both = torch.full((c.shape[0], 2) + tuple(c.shape[1:]), 255, dtype=torch.uint8, device="cuda")
    both[:, 0] = c.cuda()
    return both[:, 0].view(E4M3)


class OnGpu:
    def __init__(self, sv, s):
        self.sv, self.s = sv, s
        c = lambda t: None if t is None else t.cuda()
        self.q, self.table, self.lens, self.nd, self.ro = (c(s[n]) for n in ("q", "table", "lens", "nd", "ro"))
        self.kc, self.vc = gpu(s["kc"], s["layout"]), gpu(s["vc"], s["layout"])
        self.ks, self.vs = s["ks"].cuda(), s["vs"].cuda()
        if s["layout"] == "hnd":
            self.ks, self.vs = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (self.ks, self.vs))
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        self.ws = torch.full((sv.sv_attention_workspace_bytes(self.q.shape[2]),), 255, dtype=torch.uint8, device="cuda")
        self.ws[:256] = 0

    def call(self, stream=None, lse=True):
        s = self.s
        self.sv.spec_attention8(self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, self.nd, self.ro,
                                s["k_max"], s["scale"], s["window"], s["sinks"], self.out, self.lse if lse else None,
                                self.ws, stream)

    def results(self):
        torch.cuda.synchronize()
        return self.out.cpu(), self.lse.cpu(), self.sv.sv_read_device_error(self.ws)


def reference(s):
    """plain.attention, what the queries' parts may move each row's scores by, and the weights' smallest step each output."""
    rest = s["table"], s["lens"], s["nd"], s["ro"], s["k_max"], s["scale"], s["window"], s["sinks"]
    k, v = plain8.held(s["kc"], s["ks"]), plain8.held(s["vc"], s["vs"])
    ref = plain.attention(s["q"], k, v, *rest)
    top = s["q"].float().abs().amax(-1, keepdim=True).expand(s["q"].shape)
    low = 2.0 ** -28 * plain8.smallest(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], *rest)
    return *ref, 2.0 ** -21 * plain.attention(top, k, v, *rest)[3], low


def check(s, out, lse, rows=None):
    ro, rl, size, score, parts, low = reference(s)
    D, T, eps = s["q"].shape[2], int(s["lens"].max()), torch.finfo(s["dt"]).eps
    off = D * 2.0 ** -23 * score.double() + parts
    tol = eps / 2 * ro.abs() + size * (eps / 2 + 2 * off + (T + 16) * 2.0 ** -23)[..., None] + low + torch.finfo(s["dt"]).tiny
    rows = slice(None) if rows is None else rows
    d = (out.double() - ro).abs()[rows]
    assert bool((d <= tol[rows]).all()), (float((d / tol[rows]).max()), int((~(d <= tol[rows])).sum()))
    dl = (lse.double() - rl).abs()[rows]
    tl = (off + (T + 16) * 2.0 ** -23 + 2.0 ** -22 * rl.abs())[rows]
    assert bool((dl <= tl).all()), float((dl / tl).max())


def run_and_check(sv, s, err=(0, -1)):
    x = OnGpu(sv, s)
    x.call()
    out, lse, e = x.results()
    assert e == err
    check(s, out, lse)


HEADS = [
    # Hq, Hk, D, page, block, dtype, layout
    (8, 2, 128, 16, 16, "bf16", "nhd"), (8, 1, 64, 64, 8, "fp16", "hnd"), (7, 1, 80, 8, 8, "bf16", "both"),
    (6, 3, 96, 32, 16, "fp16", "nhd"), (4, 4, 112, 256, 64, "bf16", "hnd"), (32, 2, 48, 128, 128, "fp16", "nhd"),
    (3, 1, 16, 8, 8, "bf16", "nhd"), (5, 5, 16, 16, 8, "fp16", "both"), (48, 1, 128, 16, 16, "fp16", "nhd"),
    (2, 2, 32, 16, 16, "bf16", "hnd"), (130, 1, 64, 16, 16, "bf16", "nhd"), (1, 1, 128, 8, 8, "bf16", "nhd"),
    (17, 1, 128, 256, 256, "bf16", "nhd"), (33, 1, 64, 16, 16, "fp16", "nhd"), (49, 1, 128, 16, 16, "bf16", "nhd"),
]
MASKS = [(0, 0), (1, 0), (7, 3), (100, 4), (128, 128), (200, 0), (1 << 30, 5), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("Hq,Hk,D,page,block,dtype,layout", HEADS)
def test_heads_types_and_layouts(sv, Hq, Hk, D, page, block, dtype, layout):
    """Lengths of one token, of just the new tokens, and around pages and multiples of 64 and 128."""
    lens = [1, 5, 63, 64, 65, 127, 128, 129, 130, 256, 385, 700]
    drafts = [0, 4, 2, 0, 1, 3, 4, 0, 4, 1, 4, 2]
    run_and_check(sv, make(D + Hq, lens, drafts, 4, Hq, Hk, D, page, block, dtype, layout=layout))


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("page,block", [(8, 8), (64, 16), (256, 128)])
def test_windows_and_sinks(sv, window, sinks, page, block):
    lens = [1, 6, 130, 257, 300, 511, 640, 1000]
    drafts = [0, 5, 5, 0, 3, 2, 5, 4]
    run_and_check(sv, make(window % 1000 + sinks, lens, drafts, 5, 8, 2, 64, page, block, "fp16", window, sinks))


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("Hq,Hk,dtype", [(8, 1, "bf16"), (4, 4, "fp16"), (6, 2, "bf16")])
def test_many_rows_per_request(sv, ragged, Hq, Hk, dtype):
    """Up to 65 rows: 65 x 8 rows share a key head; rows that no request uses are zero."""
    run_and_check(sv, make(21, [65, 400, 66, 190, 5, 70], [64, 64, 31, 17, -1, 40], 64, Hq, Hk, 128, 16, 16, dtype, ragged=ragged))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(8, 1), (8, 2), (10, 2)])
def test_last_row_tiles_of_any_height(sv, D, Hq, Hk):
    """520, 260 and 325 rows per key head, and all the smaller counts beside them, over one and many CTAs."""
    rng = random.Random(Hq * 10 + Hk)
    run_and_check(sv, make(31, [65], [64], 64, Hq, Hk, D, 16, 16, "bf16"))
    run_and_check(sv, make(32, [2900, 700], [64, 31], 64, Hq, Hk, D, 64, 32, "fp16"))
    drafts = [rng.choice([-1, 0, 1, 15, 25, 31, 32, 50, 63, 64]) for _ in range(21)]
    lens = [k + 1 + rng.choice([0, 1, 127, 600]) for k in drafts]
    run_and_check(sv, make(33, lens, drafts, 64, Hq, Hk, D, 32, 8, "bf16", ragged=False))


def test_many_rows_with_a_window(sv):
    run_and_check(sv, make(22, [300, 70, 513, 65], [64, 64, 40, 64], 64, 8, 1, 64, 32, 32, "fp16", window=50, sinks=20))


@pytest.mark.parametrize("L,dtype", [(4096, "bf16"), (20011, "fp16"), (70001, "bf16")])
def test_long_contexts(sv, L, dtype):
    run_and_check(sv, make(L, [L, 3], [3, 0], 3, 8, 2, 128 if L < 50000 else 64, 16, 16, dtype))


@pytest.mark.parametrize("D", [64, 128])
def test_many_short_requests(sv, D):
    """More requests than one look at the batch takes, of one to five key tiles."""
    r = random.Random(D)
    drafts = [r.randint(0, 3) for _ in range(450)]
    lens = [r.randint(k + 1, 600) for k in drafts]
    run_and_check(sv, make(37, lens, drafts, 3, 4, 2, D, 32, 16, "bf16"))


def test_uneven_batch(sv):
    r = random.Random(5)
    drafts = [r.randint(0, 8) for _ in range(70)]
    lens = [max(k + 1, int(math.exp(r.uniform(0, math.log(3000))))) for k in drafts]
    run_and_check(sv, make(23, lens, drafts, 8, 12, 4, 64, 16, 16, "fp16"))


@pytest.mark.parametrize("sharpen,scale", [(30.0, None), (1.0, 0.0), (1.0, -0.3), (0.001, None), (8.0, 3.0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_score_ranges(sv, sharpen, scale, dtype):
    """One-hot and flat softmaxes, scores of hundreds, a negative and a zero scale."""
    s = make(24, [300, 129, 33], [4, 1, 0], 4, 8, 2, 64, 16, 8, dtype, sharpen=sharpen)
    if scale is not None:
        s["scale"] = scale
    run_and_check(sv, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_blocks_of_very_different_sizes(sv, dtype):
    """Scales over 2^+-12: a row's weight may lie on keys whose values are far smaller than others'."""
    run_and_check(sv, make(25, [700, 300, 40], [4, 2, 0], 4, 8, 2, 64, 16, 8, dtype, spread=4.0))


def test_weights_on_tiny_values_beside_huge_ones(sv):
    """The last block's values are 2^30 times the others', and no row gives it weight worth the name: the
    others' share of the sum must not vanish."""
    s = make(26, [300], [0], 0, 4, 1, 64, 16, 16, "bf16", ragged=False)
    last = int(s["table"][0, 18])
    s["vs"][last] = 2.0 ** 23
    s["kc"].view(torch.uint8)[last] = 0
    s["q"] = s["q"].abs() * 2
    other = [int(p) for p in s["table"][0, :18]]
    s["kc"].view(torch.uint8)[other] &= 127        # (scores far above the last block's zeros)
    run_and_check(sv, s)


def test_queries_whose_elements_differ_by_powers_of_two(sv):
    s = make(27, [200, 90], [3, 1], 3, 8, 2, 128, 16, 16, "fp16", sharpen=0.01)
    s["q"] = (s["q"].float() * torch.exp2(torch.randint(-6, 7, s["q"].shape, generator=torch.Generator().manual_seed(1)).float())).half()
    run_and_check(sv, s)
    s["dt"], s["q"] = torch.bfloat16, s["q"].bfloat16()
    s["q"][0, 0, 3], s["q"][1, 5] = 3e30, 0.0
    s["scale"] = 1e-30
    run_and_check(sv, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_that_are_not_finite(sv, dtype):
    """NaN rows, and no other."""
    s = make(28, [200, 90], [3, 1], 3, 8, 2, 64, 16, 16, dtype)
    ref = dict(s, q=s["q"].clone())
    s["q"][1, 2, 5], s["q"][4, 7, 60] = float("inf"), float("nan")
    x = OnGpu(sv, s)
    x.call()
    out, lse, e = x.results()
    assert e == (0, -1) and bool(out[1, 2].isnan().all()) and bool(out[4, 7].isnan().all())
    assert bool(lse[1, 2].isnan()) and bool(lse[4, 7].isnan())
    ro, rl, *_ = reference(ref)
    out[1, 2], out[4, 7], lse[1, 2], lse[4, 7] = ro[1, 2].to(s["dt"]), ro[4, 7].to(s["dt"]), rl[1, 2], rl[4, 7]
    check(ref, out, lse)


@pytest.mark.parametrize("what", ["numbers", "scales"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 2)])
def test_masked_tokens_have_no_influence(sv, what, window, sinks):
    """A NaN key and value (or, where no row sees the block, scales of any kind) of a later draft, or of a token
    that left some rows' window, must not reach the rows that do not see it."""
    s = make(29, [200, 140], [4, 4], 4, 8, 2, 64, 16, 8, "bf16", window, sinks, ragged=False)
    seen = []
    for b, L in enumerate([200, 140]):
        j = L - 2 if not window else L - 5 - 60 + 2
        p, t = int(s["table"][b, j // 16]), j % 16
        if what == "numbers":
            s["kc"].view(torch.uint8)[p, t] = 127
            s["vc"].view(torch.uint8)[p, t] = 255
            seen += [5 * b + i for i in range(5) if j in plain.visible(L - 5 + i, window, sinks)]
        else:   # the block after the last token's
            p = int(s["table"][b, L // 16]) if L % 16 <= 8 else -1
            if p >= 0:
                s["ks"][p, 1:] = s["vs"][p, 1:] = float("inf")
    x = OnGpu(sv, s)
    x.call()
    out, lse, e = x.results()
    clean = [r for r in range(10) if r not in seen]
    check(s, out, lse, clean)
    if what == "numbers":
        assert clean and seen and not bool(out[seen].isfinite().all(-1).any())
    assert e == (0, -1)


def test_non_finite_value_reaches_only_its_elements(sv):
    s = make(30, [150], [4], 4, 4, 1, 64, 16, 16, "bf16", ragged=False)
    p = int(s["table"][0, 148 // 16])
    s["vc"].view(torch.uint8)[p, 148 % 16, 0, 5] = 127
    x = OnGpu(sv, s)
    x.call()
    out, lse, _ = x.results()
    hit = torch.zeros(5, 4, 64, dtype=torch.bool)
    hit[3:, :, 5] = True
    assert bool(out[hit].isnan().all()) and bool(out[~hit].isfinite().all())
    s["vc"].view(torch.uint8)[p, 148 % 16, 0, 5] = 0
    ro, _, size, *_ = reference(s)
    assert bool(((out.double() - ro).abs() <= 2.0 ** -7 * size + 1e-4)[~hit].all())


def test_errors_stay_with_their_request(sv):
    base = make(28, [200, 260, 150, 40], [4, 3, 4, 2], 4, 4, 2, 64, 16, 16, "bf16", ragged=False)
    for what, code in [("short", 1), ("long", 1), ("drafts", 1), ("below", 1), ("failed", 1), ("page", 9), ("high page", 9)]:
        s = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in base.items()}
        ref = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in base.items()}
        ref["nd"][1] = -1
        if what == "short":
            s["lens"][1] = 3
        if what == "long":
            s["lens"][1] = s["table"].shape[1] * 16 + 1
        if what == "drafts":
            s["nd"][1] = 5
        if what == "below":
            s["nd"][1] = -2
        if what == "failed":
            s["lens"][1] = -261
        if what == "page":
            s["table"][1, 3] = -1
        if what == "high page":
            s["table"][1, 16] = s["kc"].shape[0]
        x = OnGpu(sv, s)
        x.call()
        out, lse, e = x.results()
        assert e == (code, 1), what
        used = 4 if code == 9 else 5
        assert bool(out[5:5 + used].isnan().all()) and bool(lse[5:5 + used].isnan().all()), what
        check(ref, out, lse, [r for r in range(20) if not 5 <= r < 10])


def test_offsets_out_of_order(sv):
    s = make(29, [50, 60, 70], [2, 2, 2], 2, 2, 1, 64, 16, 16, "bf16")
    s["ro"] = torch.tensor([0, 6, 3, 9], dtype=torch.int32)
    x = OnGpu(sv, s)
    x.call()
    assert x.results()[2] == (1, 1)


def test_idle_requests_that_own_no_row(sv):
    drafts = [-1] * 40 + [2, -1, 0] + [-1] * 500 + [3] + [-1] * 33 + [1] + [-1] * 50
    lens = [9 + b % 300 for b in range(len(drafts))]
    s = make(36, lens, drafts, 3, 4, 2, 64, 16, 16, "bf16")
    rows = [k + 1 for k in drafts]
    off = [sum(rows[:b]) for b in range(len(rows) + 1)]
    s["ro"] = torch.tensor(off, dtype=torch.int32)
    s["q"] = s["q"][:off[-1] + 2]      # and two rows after the last request
    run_and_check(sv, s)


def test_page_table_of_pages_never_seen(sv):
    s = make(30, [300, 40], [4, 4], 4, 4, 2, 64, 16, 16, "bf16", window=40, sinks=2)
    s["table"][s["table"] == -1] = 1 << 30
    run_and_check(sv, s)


def test_same_bits_every_time_and_on_another_stream(sv):
    s = make(31, [5000, 1, 777, 64], [4, 0, 4, 3], 4, 16, 2, 128, 16, 16, "bf16")
    x = OnGpu(sv, s)
    x.call()
    ref = x.results()
    for stream in (None, torch.cuda.Stream(), None):
        x.out.fill_(3.0)
        x.lse.fill_(3.0)
        torch.cuda.synchronize()
        x.call(stream)
        got = x.results()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    x.out.fill_(3.0)
    x.call(lse=False)
    assert torch.equal(x.results()[0], ref[0])


def test_lengths_change_between_replays(sv):
    s = make(32, [300, 17, 1030], [2, 2, 2], 2, 8, 2, 64, 16, 16, "fp16")
    for c in ("kc", "vc"):
        b = s[c].view(torch.uint8)
        b[(b & 127) == 127] = 40
    s["ks"], s["vs"] = s["ks"].nan_to_num(0.01), s["vs"].nan_to_num(0.01)
    x = OnGpu(sv, s)
    x.lens.copy_(torch.tensor([3, 3, 3]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.call()
    for lens in ([3, 3, 3], [300, 17, 1030], [128, 16, 640]):
        x.lens.copy_(torch.tensor(lens))
        graph.replay()
        out, lse, e = x.results()
        assert e == (0, -1)
        check(dict(s, lens=torch.tensor(lens, dtype=torch.int32)), out, lse)


def test_strided_queries(sv):
    s = make(33, [90, 200], [3, 3], 3, 4, 2, 80, 16, 16, "bf16")
    x = OnGpu(sv, s)
    x.call()
    ref = x.results()
    wide = torch.full((x.q.shape[0], 4 * 80 + 24), float("nan"), dtype=s["dt"], device="cuda")
    wide[:, 8:328] = x.q.flatten(1)
    x.q = wide[:, 8:328].unflatten(1, (4, 80))
    x.call()
    got = x.results()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_pool_past_32_bits(sv):
    """Offsets beyond 2^31: the same tokens at both ends of a large pool."""
    pages, page, Hk, D = 70000, 256, 1, 128
    s = make(34, [500], [3], 3, 4, Hk, D, page, 64, "bf16", spare=0)
    x = OnGpu(sv, s)
    x.call()
    ref = x.results()
    big = [torch.zeros((pages, page, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, page // 64, Hk), device="cuda") for _ in range(2)]
    far = [pages - 1, 66001]
    for c, t, o, u in zip(big, scales, (x.kc, x.vc), (x.ks, x.vs)):
        for i, p in enumerate(far):
            c[p] = o.view(torch.uint8)[int(s["table"][0, i])]
            t[p] = u[int(s["table"][0, i])]
    x.kc, x.vc = (c.view(E4M3) for c in big)
    (x.ks, x.vs), x.table = scales, torch.tensor([far], dtype=torch.int32, device="cuda")
    x.call()
    got = x.results()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_first_call_of_a_host_thread(sv):
    import threading

    s = make(48, [300], [2], 2, 4, 2, 64, 16, 16, "bf16", ragged=False)
    x = OnGpu(sv, s)
    x.call()
    want = x.results()
    x.out.fill_(7.0)
    stream, failed = torch.cuda.Stream(), []
    torch.cuda.synchronize()

    def run():
        try:
            x.call(stream.cuda_stream)
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not failed
    assert torch.equal(x.results()[0], want[0])


def test_calls_of_two_streams_at_once(sv):
    """A workspace each, row counts that need different amounts of shared memory."""
    calls = []
    for G, k_max, D, dtype in ((1, 0, 128, "bf16"), (8, 64, 128, "bf16"), (5, 3, 64, "fp16")):
        x = OnGpu(sv, make(50 + G, [k_max + 900], [k_max], k_max, G, 1, D, 16, 16, dtype, ragged=False))
        x.call()
        calls.append((x, x.results()[0], torch.cuda.Stream()))
        x.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(200):
        for x, _, stream in calls:
            x.call(stream)
    for x, want, _ in calls:
        assert torch.equal(x.results()[0], want)


@pytest.mark.parametrize("G,k_max", [(4, 4), (8, 3), (1, 0), (7, 6)])
@pytest.mark.parametrize("tiles", [1, 2, 3, 5, 6])
def test_segments_follow_each_other(sv, tiles, G, k_max):
    """Many segments a CTA.  One whose scores are far above the next one's would show in it."""
    B = 160
    r = random.Random(tiles)
    lens = [tiles * 128 - r.randint(0, 50) for _ in range(B)]
    s = make(70 + tiles, lens, [k_max] * B, k_max, 4 * G, 4, 64, 32, 16, "bf16", ragged=False)
    s["q"] *= torch.tensor([30.0, 0.02])[torch.arange(s["q"].shape[0]) // (k_max + 1) % 2][:, None, None].to(s["q"].dtype)
    x = OnGpu(sv, s)
    x.call()
    out, lse, e = x.results()
    assert e == (0, -1)
    check(s, out, lse)
    for _ in range(20):
        x.call()
        assert torch.equal(x.results()[0], out)


def test_a_batch_of_idle_requests(sv):
    """Nothing to do but to set the rows to zero; and between two replays nothing is left of the calls before."""
    s = make(81, [40, 300, 7], [2, 2, 2], 2, 8, 2, 64, 16, 16, "bf16", ragged=False)
    x = OnGpu(sv, s)
    for drafts in ([-1, -1, -1], [2, -1, 0], [-1, -1, -1]):
        x.nd.copy_(torch.tensor(drafts))
        x.out.fill_(3.0)
        x.lse.fill_(3.0)
        x.call()
        out, lse, e = x.results()
        assert e == (0, -1)
        if max(drafts) < 0:
            assert not bool(out.any()) and not bool(lse.any())
        else:
            check(dict(s, nd=torch.tensor(drafts, dtype=torch.int32)), out, lse)


@pytest.mark.parametrize("lse", [True, False])
def test_more_requests_than_threads(sv, lse):
    """Two passes over the batch find where a range begins."""
    r = random.Random(82)
    drafts = [r.choice([-1, 0, 1]) for _ in range(1500)]
    lens = [r.randint(max(k + 1, 1), 200) for k in drafts]
    s = make(82, lens, drafts, 1, 2, 1, 16, 32, 16, "fp16")
    x = OnGpu(sv, s)
    x.call(lse=lse)
    out, got, e = x.results()
    assert e == (0, -1)
    if lse:
        check(s, out, got)
    else:
        assert bool((got == 7.0).all())
        x.call()
        assert torch.equal(x.results()[0], out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_most_heads_of_a_key_head(sv, dtype):
    run_and_check(sv, make(83, [9, 300], [2, 0], 2, 1024, 1, 64, 16, 16, dtype))


def test_two_graphs_at_once(sv):
    calls = []
    for G, k_max, D, dtype in ((4, 4, 128, "bf16"), (7, 3, 64, "fp16")):
        x = OnGpu(sv, make(84 + G, [k_max + 900, 30, 513], [k_max, 0, k_max], k_max, G, 1, D, 16, 16, dtype))
        x.call()
        want = x.results()[0]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                x.call()
        x.out.fill_(7.0)
        calls.append((x, want, graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, graph, stream in calls:
            with torch.cuda.stream(stream):
                graph.replay()
    for x, want, _, _ in calls:
        out, _, e = x.results()
        assert e == (0, -1) and torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outputs_are_not_larger_or_smaller_on_average(sv, dtype):
    """Weights are rounded to 9 or 11 bits before their product with the values, and not in the sum that divides it: a
    rounding with a mean would move every output.  Values of one sign, so that nothing cancels.  The mean of the outputs'
    relative errors: their own rounding, rms eps / (2 sqrt 3), over 10^5 of them, and the weights', rms 8.5e-4 in bf16, over some
    50 keys that count in each of 1000 rows, are below 5e-6 each; five times both, and sums in 32 bits of up to
    400 terms, (400 + 16) 2^-23, are 1e-4 together."""
    r = random.Random(91)
    drafts = [r.randint(0, 4) for _ in range(64)]
    lens = [r.randint(250, 400) for _ in drafts]
    s = make(91, lens, drafts, 4, 8, 2, 128, 16, 16, dtype)
    s["vc"].view(torch.uint8).bitwise_and_(127)
    x = OnGpu(sv, s)
    x.call()
    out, _, e = x.results()
    ro, *_ = reference(s)
    assert e == (0, -1) and bool((ro > 0).all()) and ro.numel() > 10 ** 5
    assert abs(float(((out.double() - ro) / ro).mean())) < 1e-4


@pytest.mark.parametrize("size,scale", [(127, -128), (127, -129), (120, -121), (-127, 125), (-126, 124), (-120, 120)])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_every_finite_size(sv, D, size, scale):
    """Rows around 2^size, up to bf16's largest numbers and down into its subnormal ones, with a scale that makes scores
    of a few of them; beside them rows of zeros, and of ones, whose scores are next to nothing."""
    s = make(92, [200, 90, 40], [3, 1, 0], 3, 8, 2, D, 16, 16, "bf16")
    q = s["q"].double().clamp(-1.9, 1.9) * 2.0 ** size
    q[0, 0, 3], q[1, 1, 5], q[2, 3] = 1.98 * 2.0 ** size, -1.98 * 2.0 ** size, 0.0
    if size > 0:
        q[4, 1] = 1.0
    s["q"], s["scale"] = q.bfloat16(), 2.0 ** scale
    assert bool(s["q"].isfinite().all())
    run_and_check(sv, s)


# what spec_cache.h states of a query's parts: exact from this share of a row's largest element on, and off by that share below
EXACT_FROM, PARTS_OFF = 2.0 ** -13.8, {"bf16": 2.0 ** -21.8, "fp16": 2.0 ** -24.8}


@pytest.mark.parametrize("top", [226.0, 448.0, 337.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_query_element_keeps_its_bits(sv, dtype, top):
    """All numbers of the type up to the row's largest.  One key, 1 at the element in question and 0 at the largest, so that
    the lse is the score: the element times 2^20, and off by 2^-21 of itself and of the kernel's largest exponent, 12,
    in fp32."""
    dt, G, scale = DT[dtype], 1024, 2.0 ** 20
    x = torch.arange(0, 1 << 15).to(torch.int16).view(dt)
    x = x[x.double() <= top]
    R = -(-len(x) // G)
    q = torch.zeros(R * G, 1, 64, dtype=dt)
    q[:len(x), 0, 1], q[:, 0, 0] = x, top
    one = torch.zeros(1, 8, 1, 64)
    one[0, 0, 0, 1] = 1.0
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kc, ks = one.to(E4M3).cuda(), torch.ones(1, 1, 1, device="cuda")
    out, lse = torch.empty(R, G, 64, dtype=dt, device="cuda"), torch.empty(R, G, device="cuda")
    ws = torch.zeros(sv.sv_attention_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    sv.spec_attention8(q.view(R, G, 64).cuda(), kc, kc, ks, ks, ints(*[0] * R).view(R, 1), ints(*[1] * R), ints(*[0] * R), None,
                       0, scale, 0, 0, out, lse, ws)
    assert sv.sv_read_device_error(ws) == (0, -1)
    want = x.double() * scale
    off = (lse.cpu().double().flatten()[:len(x)] - want).abs()
    fp32 = 2.0 ** -21 * (want + 12)
    assert bool((off <= fp32)[x.double() >= EXACT_FROM * top].all())
    assert bool((off <= fp32 + PARTS_OFF[dtype] * top * scale).all())
