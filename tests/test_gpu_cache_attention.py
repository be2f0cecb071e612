"""spec_attention on the GPU against the 64-bit definition (cache_plain.attention).

Tolerances, from the arithmetic.  With S = sum_j p_j |v_j| of an output and eps the type's:
  - the output is rounded once: eps / 2 of its value;
  - the weights are rounded to the type for the product with v: eps / 2 of S;
  - a score is a sum of head_dim products in fp32, off by at most head_dim 2^-23 sum |q k| scale
    (twice 2^-24 where the products' sum is truncated), which moves the weights, and so the
    output, by twice that of S;
  - exponentials and the running sums over T keys: (T + 16) 2^-23 of S.
lse: the score's bound, plus (T + 16) 2^-23 for the sum, plus 2^-22 of its value.
"""
import math
import random

import pytest

import cache_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_12_gb300 as sv
    sv.lib()
    return sv


def make(seed, lens, drafts, k_max, Hq, Hk, D, page, dtype, window=0, sinks=0, ragged=True, layout="nhd", spare=2,
         sharpen=1.0):
    """Requests over pages in random order; slots past each length, and pages out of the window,
    hold NaN or nothing (-1)."""
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
    kc, vc = (torch.randn((len(ids), page, Hk, D), generator=g) for _ in range(2))
    kc, vc = kc.to(dt), vc.to(dt)
    for (b, x), p in zip(want, ids):
        table[b, x] = p
        if (x + 1) * page > lens[b]:
            kc[p, lens[b] - x * page:] = float("nan")
            vc[p, lens[b] - x * page:] = float("nan")
    for p in ids[len(want):]:
        kc[p] = vc[p] = float("nan")
    return dict(q=(torch.randn((R, Hq, D), generator=g) * sharpen).to(dt), kc=kc, vc=vc, table=table,
                lens=torch.tensor(lens, dtype=torch.int32), nd=torch.tensor(drafts, dtype=torch.int32),
                ro=torch.tensor(off, dtype=torch.int32) if ragged else None, k_max=k_max, layout=layout, dt=dt,
                window=window, sinks=sinks, scale=1 / math.sqrt(D))


def gpu(c, layout):
    if layout == "nhd":
        return c.cuda()
    if layout == "hnd":
        return c.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    both = torch.full((c.shape[0], 2) + tuple(c.shape[1:]), float("nan"), dtype=c.dtype, device="cuda")
    both[:, 0] = c.cuda()
    return both[:, 0]


class OnGpu:
    def __init__(self, sv, s):
        self.sv, self.s = sv, s
        c = lambda t: None if t is None else t.cuda()
        self.q, self.table, self.lens, self.nd, self.ro = (c(s[n]) for n in ("q", "table", "lens", "nd", "ro"))
        self.kc, self.vc = gpu(s["kc"], s["layout"]), gpu(s["vc"], s["layout"])
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        self.ws = torch.full((sv.sv_attention_workspace_bytes(self.q.shape[2]),), 255, dtype=torch.uint8, device="cuda")
        self.ws[:256] = 0

    def call(self, stream=None, lse=True):
        s = self.s
        self.sv.spec_attention(self.q, self.kc, self.vc, self.table, self.lens, self.nd, self.ro, s["k_max"], s["scale"],
                               s["window"], s["sinks"], self.out, self.lse if lse else None, self.ws, stream)

    def results(self):
        torch.cuda.synchronize()
        return self.out.cpu(), self.lse.cpu(), self.sv.sv_read_device_error(self.ws)


def check(s, out, lse, rows=None):
    ro, rl, size, score = plain.attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["nd"], s["ro"], s["k_max"],
                                          s["scale"], s["window"], s["sinks"])
    D, T, eps = s["q"].shape[2], int(s["lens"].max()), torch.finfo(s["dt"]).eps
    off = D * 2.0 ** -23 * score.double()
    tol = eps / 2 * ro.abs() + size * (eps / 2 + 2 * off + (T + 16) * 2.0 ** -23)[..., None] + torch.finfo(s["dt"]).tiny
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
    # Hq, Hk, D, page, dtype, layout
    (8, 2, 128, 16, "bf16", "nhd"), (8, 1, 64, 64, "fp16", "hnd"), (7, 1, 80, 8, "bf16", "both"),
    (6, 3, 96, 32, "fp16", "nhd"), (4, 4, 112, 256, "bf16", "hnd"), (32, 2, 40, 128, "fp16", "nhd"),
    (3, 1, 8, 8, "bf16", "nhd"), (5, 5, 16, 16, "fp16", "both"), (48, 1, 128, 16, "fp16", "nhd"),
    (2, 2, 72, 16, "bf16", "hnd"), (130, 1, 64, 16, "bf16", "nhd"), (1, 1, 128, 8, "bf16", "nhd"),
]
MASKS = [(0, 0), (1, 0), (7, 3), (100, 4), (128, 128), (200, 0), (1 << 30, 5), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("Hq,Hk,D,page,dtype,layout", HEADS)
def test_heads_types_and_layouts(sv, Hq, Hk, D, page, dtype, layout):
    """Lengths of one token, of just the new tokens, and around pages and multiples of 64 and 128."""
    lens = [1, 5, 63, 64, 65, 127, 128, 129, 130, 256, 385, 700]
    drafts = [0, 4, 2, 0, 1, 3, 4, 0, 4, 1, 4, 2]
    run_and_check(sv, make(D + Hq, lens, drafts, 4, Hq, Hk, D, page, dtype, layout=layout))


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("page", [8, 64, 256])
def test_windows_and_sinks(sv, window, sinks, page):
    lens = [1, 6, 130, 257, 300, 511, 640, 1000]
    drafts = [0, 5, 5, 0, 3, 2, 5, 4]
    run_and_check(sv, make(window % 1000 + sinks, lens, drafts, 5, 8, 2, 64, page, "fp16", window, sinks))


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("Hq,Hk", [(8, 1), (4, 4), (6, 2)])
def test_many_rows_per_request(sv, ragged, Hq, Hk):
    """Up to 65 rows: 65 x 8 rows share a key head; rows that no request uses are zero."""
    s = make(21, [65, 400, 66, 190, 5, 70], [64, 64, 31, 17, -1, 40], 64, Hq, Hk, 128, 16, "bf16", ragged=ragged)
    run_and_check(sv, s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(8, 1), (8, 2), (10, 2)])
@pytest.mark.parametrize("ragged", [True, False])
def test_last_row_tiles_of_any_height(sv, D, Hq, Hk, ragged):
    """520, 260 and 325 rows per key head, and all the smaller counts beside them, over one and many CTAs."""
    rng = random.Random(Hq * 10 + Hk)
    run_and_check(sv, make(31, [65], [64], 64, Hq, Hk, D, 16, "bf16", ragged=ragged))
    run_and_check(sv, make(32, [2900, 700], [64, 31], 64, Hq, Hk, D, 64, "fp16", ragged=ragged))
    drafts = [rng.choice([-1, 0, 1, 15, 25, 31, 32, 50, 63, 64]) for _ in range(21)]
    lens = [k + 1 + rng.choice([0, 1, 127, 600]) for k in drafts]
    run_and_check(sv, make(33, lens, drafts, 64, Hq, Hk, D, 32, "bf16", ragged=ragged))


def test_many_rows_with_a_window(sv):
    run_and_check(sv, make(22, [300, 70, 513, 65], [64, 64, 40, 64], 64, 8, 1, 64, 32, "fp16", window=50, sinks=20))


@pytest.mark.parametrize("L", [4096, 20011, 70001])
def test_long_contexts(sv, L):
    run_and_check(sv, make(L, [L, 3], [3, 0], 3, 8, 2, 128 if L < 50000 else 64, 16, "bf16" if L < 50000 else "fp16"))


@pytest.mark.parametrize("D", [64, 128])
def test_many_short_requests(sv, D):
    """More requests than one look at the batch takes, of one to five key tiles: segments of one
    group, of both, and cut between CTAs."""
    r = random.Random(D)
    drafts = [r.randint(0, 3) for _ in range(450)]
    lens = [r.randint(k + 1, 600) for k in drafts]
    run_and_check(sv, make(37, lens, drafts, 3, 4, 2, D, 32, "bf16"))


def test_uneven_batch(sv):
    """Many requests of very different lengths."""
    r = random.Random(5)
    drafts = [r.randint(0, 8) for _ in range(70)]
    lens = [max(k + 1, int(math.exp(r.uniform(0, math.log(3000))))) for k in drafts]
    run_and_check(sv, make(23, lens, drafts, 8, 12, 4, 64, 16, "fp16"))


@pytest.mark.parametrize("sharpen,scale", [(30.0, None), (1.0, 0.0), (1.0, -0.3), (0.001, None), (8.0, 3.0)])
def test_score_ranges(sv, sharpen, scale):
    """One-hot and flat softmaxes, scores of hundreds, a negative and a zero scale."""
    s = make(24, [300, 129, 33], [4, 1, 0], 4, 8, 2, 64, 16, "fp16", sharpen=sharpen)
    if scale is not None:
        s["scale"] = scale
    run_and_check(sv, s)


def test_scores_far_below_zero(sv):
    """Every score of a row near -1e4: the sum must not vanish."""
    s = make(25, [200, 131], [2, 0], 2, 4, 1, 64, 16, "fp16")
    s["q"] = s["q"].abs() * 16
    s["kc"] = torch.where(s["kc"].isnan(), s["kc"], -s["kc"].abs() * 16)
    run_and_check(sv, s)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 2)])
def test_masked_tokens_have_no_influence(sv, bad, window, sinks):
    """A non-finite key and value of a later draft, or of a token that left some rows' window, must
    not reach the rows that do not see it."""
    s = make(26, [200, 140], [4, 4], 4, 8, 2, 64, 16, "bf16", window, sinks, ragged=False)
    seen = []
    for b, L in enumerate([200, 140]):
        for j in ([L - 2] if not window else [L - 2, L - 5 - 60 + 2]):
            p, t = int(s["table"][b, j // 16]), j % 16
            s["kc"][p, t] = bad
            s["vc"][p, t] = bad
            seen += [5 * b + i for i in range(5) if j in plain.visible(L - 5 + i, window, sinks)]
    clean = [r for r in range(10) if r not in seen]
    assert clean and seen
    x = OnGpu(sv, s)
    x.call()
    out, lse, e = x.results()
    check(s, out, lse, clean)
    assert not bool(out[seen].isfinite().all(-1).any())
    assert e == (0, -1)


def test_non_finite_value_reaches_only_its_elements(sv):
    """One element of a visible value is infinite: that element of the rows that see it, no other."""
    s = make(27, [150], [4], 4, 4, 1, 64, 16, "bf16", ragged=False)
    p = int(s["table"][0, 148 // 16])
    s["vc"][p, 148 % 16, 0, 5] = float("inf")
    x = OnGpu(sv, s)
    x.call()
    out, lse, _ = x.results()
    ro, _, size, score = plain.attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["nd"], None, 4, s["scale"], 0, 0)
    hit = torch.zeros(5, 4, 64, dtype=torch.bool)
    hit[3:, :, 5] = True
    assert bool((out[hit] == float("inf")).all()) and bool(out[~hit].isfinite().all())
    assert float((out.double() - ro)[~hit].abs().max()) < 2.0 ** -6


def test_errors_stay_with_their_request(sv):
    base = make(28, [200, 260, 150, 40], [4, 3, 4, 2], 4, 4, 2, 64, 16, "bf16", ragged=False)
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
    """row_offsets that run backwards: the requests in error are reported, nothing else is touched."""
    s = make(29, [50, 60, 70], [2, 2, 2], 2, 2, 1, 64, 16, "bf16")
    s["ro"] = torch.tensor([0, 6, 3, 9], dtype=torch.int32)
    x = OnGpu(sv, s)
    x.call()
    _, _, e = x.results()
    assert e == (1, 1)


def test_idle_requests_that_own_no_row(sv):
    drafts = [-1] * 40 + [2, -1, 0] + [-1] * 500 + [3] + [-1] * 33 + [1] + [-1] * 50
    lens = [9 + b % 300 for b in range(len(drafts))]
    s = make(36, lens, drafts, 3, 4, 2, 64, 16, "bf16")
    rows = [k + 1 for k in drafts]
    off = [sum(rows[:b]) for b in range(len(rows) + 1)]
    s["ro"] = torch.tensor(off, dtype=torch.int32)
    s["q"] = s["q"][:off[-1] + 2]      # and two rows after the last request
    run_and_check(sv, s)


def test_page_table_of_pages_never_seen(sv):
    """Entries past the length, and out of the window, are not looked at."""
    s = make(30, [300, 40], [4, 4], 4, 4, 2, 64, 16, "bf16", window=40, sinks=2)
    s["table"][s["table"] == -1] = 1 << 30
    run_and_check(sv, s)


def test_same_bits_every_time_and_on_another_stream(sv):
    s = make(31, [5000, 1, 777, 64], [4, 0, 4, 3], 4, 16, 2, 128, 16, "bf16")
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
    """Captured once; the lengths, which the call reads on the device, then grow."""
    s = make(32, [300, 17, 1030], [2, 2, 2], 2, 8, 2, 64, 16, "fp16")
    s["kc"], s["vc"] = s["kc"].nan_to_num(0.5), s["vc"].nan_to_num(0.5)
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
    s = make(33, [90, 200], [3, 3], 3, 4, 2, 80, 16, "bf16")
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
    """Element offsets beyond 2^31: the same tokens at both ends of a large pool."""
    pages, page, Hk, D = 70000, 256, 1, 128
    s = make(34, [500], [3], 3, 4, Hk, D, page, "bf16", spare=0)
    x = OnGpu(sv, s)
    x.call()
    ref = x.results()
    big = [torch.zeros((pages, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far = [pages - 1, 35001]
    for c, o in zip(big, (x.kc, x.vc)):
        for i, p in enumerate(far):
            c[p] = o[int(s["table"][0, i])]
    x.kc, x.vc, x.table = big[0], big[1], torch.tensor([far], dtype=torch.int32, device="cuda")
    x.call()
    got = x.results()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_first_call_of_a_host_thread(sv):
    """A thread whose first CUDA call of all is this one: the library itself brings it to the device."""
    import threading

    s = make(48, [300], [2], 2, 4, 2, 64, 16, "bf16", ragged=False)
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


def test_threads_with_different_row_counts(sv):
    """Two threads, a stream and a workspace each, whose calls need different amounts of shared memory: every
    one is launched.  (The library is called without the interpreter's lock.)"""
    import threading

    from speculative_decoding_verification_12_gb300 import cache
    lib, want, fails = cache._lib(), [], []

    def prepare(G, k_max, D):
        s = make(50 + G, [k_max + 90], [k_max], k_max, G, 1, D, 16, "bf16", ragged=False)
        x = OnGpu(sv, s)
        x.call()
        want.append(x.results()[0])
        x.out.fill_(7.0)
        kc = x.kc
        view = sv.SvKvCache(kc.data_ptr(), x.vc.data_ptr(), *kc.stride()[:3], kc.shape[0], 16, 1, D, 1, x.table.shape[1],
                            x.table.data_ptr())
        stream = torch.cuda.Stream()
        args = (x.q.data_ptr(), x.q.stride(0), G, x.nd.data_ptr(), None, x.lens.data_ptr(), 1, k_max, k_max + 1, view,
                s["scale"], 0, 0, x.out.data_ptr(), None, x.ws.data_ptr(), x.ws.numel(), stream.cuda_stream)
        return x, args, stream

    calls = [prepare(1, 0, 128), prepare(8, 64, 128)]
    torch.cuda.synchronize()

    def run(args):
        fails.append([s for s in (lib.spec_attention(*args) for _ in range(4000)) if s])

    threads = [threading.Thread(target=run, args=(c[1],)) for c in calls]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert fails == [[], []]
    for (x, _, _), w in zip(calls, want):
        assert torch.equal(x.results()[0], w)


@pytest.mark.parametrize("G,k_max", [(4, 4), (8, 3), (1, 0)])
@pytest.mark.parametrize("tiles", [5, 6, 9])
def test_short_segments_of_both_groups_in_a_row(sv, tiles, G, k_max):
    """Narrow heads, up to 32 rows: segments that both groups share follow each other directly, each handing its
    maxima and sums over at the same place.  A segment whose scores are far above the next one's would show in it."""
    B = 120
    r = random.Random(tiles)
    lens = [tiles * 128 - r.randint(0, 100) for _ in range(B)]
    s = make(70 + tiles, lens, [k_max] * B, k_max, 4 * G, 4, 64, 32, "bf16", ragged=False)
    s["q"] *= torch.tensor([30.0, 0.02])[torch.arange(s["q"].shape[0]) // (k_max + 1) % 2][:, None, None].to(s["q"].dtype)
    x = OnGpu(sv, s)
    x.call()
    out, lse, e = x.results()
    assert e == (0, -1)
    check(s, out, lse)
    for _ in range(20):
        x.call()
        assert torch.equal(x.results()[0], out)
