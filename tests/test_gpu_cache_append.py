"""spec_append on the GPU against the 64-bit definition (cache_plain.append).

Tolerance: one rounding to the type (half a step, eps / 2 of the value) plus the fp32 arithmetic
before it.  A pair's error scales with |a| + |z|: the norm and two products round about six times
(2^-24 each), and the angle, reduced exactly and held in 24 bits of a half turn, is off by at most
pi 2^-25, its sine and cosine by a few 2^-24: 2^-20 (|a| + |z|) in all.
"""
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


def make(seed, lens, drafts, k_max, Hq, Hk, D, page, dtype, rotary, ragged=True, layout="nhd", norm=True, packed=True):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    B = len(lens)
    off = [0]
    for k in drafts:
        off.append(off[-1] + (max(k, 0) + 1 if ragged else k_max + 1))
    R = off[-1]
    M = max(1, -(-max(max(lens), 1) // page))
    # only the pages that hold new tokens; the rest of the table is -1
    table = torch.full((B, M), -1, dtype=torch.int32)
    want = [(b, x) for b, (L, k) in enumerate(zip(lens, drafts)) if k >= 0
            for x in range(max(L - k - 1, 0) // page, -(-L // page))]
    ids = torch.randperm(len(want) + 3, generator=g)
    for (b, x), p in zip(want, ids.tolist()):
        table[b, x] = p
    shape = (len(ids), page, Hk, D)
    kc, vc = (torch.randn(shape, generator=g).to(dt) for _ in range(2))
    width = (Hq + 2 * Hk) * D
    qkv = torch.randn((R, width if packed else width + 8), generator=g).to(dt)
    q, k, v = (x.reshape(R, -1, D) for x in qkv[:, :width].split([Hq * D, Hk * D, Hk * D], 1))
    w = (torch.rand(2, D, generator=g) + 0.5).to(dt) if norm else (None, None)
    inv = (10000.0 ** (-torch.arange(rotary // 2).double() * 2 / max(rotary, 1))).float() if rotary else None
    return dict(q=q, k=k, v=v, qkv=qkv, w=w, inv=inv, kc=kc, vc=vc, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                nd=torch.tensor(drafts, dtype=torch.int32), ro=torch.tensor(off, dtype=torch.int32) if ragged else None,
                k_max=k_max, layout=layout, D=D, Hq=Hq, Hk=Hk, R=R, dt=dt)


def gpu(c, layout):
    """A cache on the GPU in the given order of its dimensions, seen as [pages, slots, heads, D]."""
    if layout == "nhd":
        return c.cuda()
    if layout == "hnd":
        return c.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    both = torch.zeros((c.shape[0], 2) + tuple(c.shape[1:]), dtype=c.dtype, device="cuda")   # k and v interleaved
    both[:, 0] = c.cuda()
    return both[:, 0]


def call(sv, s, interleaved=False, rope_scale=1.0, inplace=False, stream=None, eps=1e-6):
    dev = s["qkv"].cuda()
    D, Hq, Hk, R = s["D"], s["Hq"], s["Hk"], s["R"]
    q = dev[:, :Hq * D].view(R, Hq, D)
    k = dev[:, Hq * D:(Hq + Hk) * D].view(R, Hk, D)
    v = dev[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(R, Hk, D)
    kc, vc = gpu(s["kc"], s["layout"]), gpu(s["vc"], s["layout"])
    out = q if inplace else torch.full((R, Hq, D), 7.0, dtype=s["dt"], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    c = lambda t: None if t is None else t.cuda()
    args = [q, k, v, c(s["w"][0]), c(s["w"][1]), eps, c(s["inv"]), kc, vc, c(s["table"]), c(s["lens"]), c(s["nd"]),
            c(s["ro"]), s["k_max"], out, ws]
    torch.cuda.synchronize()
    sv.spec_append(*args, interleaved=interleaved, rope_scale=rope_scale, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), kc.cpu(), vc.cpu(), sv.sv_read_device_error(ws)


def check(got, ref, size, dt):
    d = (got.double() - ref).abs()
    tol = torch.finfo(dt).eps / 2 * ref.abs() + 2.0 ** -20 * size + torch.finfo(dt).tiny
    assert bool((d <= tol).all()), (float((d - tol).max()), int((d > tol).sum()))


def run_and_check(sv, s, interleaved=False, rope_scale=1.0, inplace=False, eps=1e-6):
    out, kc, vc, err = call(sv, s, interleaved, rope_scale, inplace, eps=eps)
    ro, rk, rv, so, sk = plain.append(s["q"], s["k"], s["v"], *s["w"], eps, s["inv"], s["kc"], s["vc"], s["table"],
                                      s["lens"], s["nd"], s["ro"], s["k_max"], interleaved, rope_scale)
    check(out, ro, so, s["dt"])
    check(kc, rk, sk, s["dt"])
    assert torch.equal(vc.double(), rv)
    assert err == (0, -1)


CASES = [
    # D, rotary, Hq, Hk, page, dtype, interleaved, layout
    (128, 128, 32, 8, 16, "bf16", False, "nhd"), (128, 64, 8, 8, 8, "fp16", True, "hnd"),
    (64, 64, 7, 1, 256, "bf16", True, "both"), (64, 20, 12, 4, 64, "fp16", False, "nhd"),
    (80, 80, 10, 2, 32, "bf16", False, "hnd"), (96, 48, 9, 3, 128, "fp16", True, "nhd"),
    (72, 36, 5, 5, 16, "bf16", False, "nhd"), (8, 8, 3, 1, 8, "fp16", False, "nhd"), (8, 2, 1, 1, 8, "bf16", True, "hnd"),
    (256, 256, 6, 2, 16, "bf16", False, "nhd"), (136, 70, 4, 2, 16, "fp16", False, "both"), (16, 0, 2, 2, 8, "bf16", False, "nhd"),
    (112, 112, 64, 8, 16, "bf16", False, "nhd"),
]


@pytest.mark.parametrize("D,rotary,Hq,Hk,page,dtype,il,layout", CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_matches_definition(sv, D, rotary, Hq, Hk, page, dtype, il, layout, norm):
    s = make(D + rotary, [1, 5, page, page + 1, 3 * page + 2, 40], [0, 4, 2, 1, 3, 7], 7, Hq, Hk, D, page, dtype,
             rotary, layout=layout, norm=norm)
    run_and_check(sv, s, il, rope_scale=1.0 if norm else 0.83)


@pytest.mark.parametrize("ragged", [True, False])
def test_rows_of_both_layouts(sv, ragged):
    """Requests that use fewer rows than they own, idle ones, one token, k_max = 64."""
    s = make(3, [1, 70, 65, 300, 9], [0, 64, 64, 17, -1], 64, 4, 2, 64, 16, "bf16", 64, ragged=ragged)
    run_and_check(sv, s)


def test_idle_requests_that_own_no_row(sv):
    """Runs of more than 32 of them between, before and after the others."""
    drafts = [-1] * 40 + [2, -1, 0] + [-1] * 100 + [3] + [-1] * 33 + [1] + [-1] * 50
    lens = [9 + b % 40 for b in range(len(drafts))]
    s = make(12, lens, drafts, 3, 4, 2, 64, 16, "bf16", 64)
    rows = [k + 1 for k in drafts]
    off = [sum(rows[:b]) for b in range(len(rows) + 1)]
    s["R"] = off[-1] + 2              # and two rows after the last request
    s["ro"] = torch.tensor(off, dtype=torch.int32)
    for n in ("q", "k", "v", "qkv"):
        s[n] = s[n][:s["R"]]
    run_and_check(sv, s)


def test_rows_before_the_first_request(sv):
    s = make(13, [30, 40], [2, 1], 2, 4, 2, 64, 16, "bf16", 64)
    s["ro"] = torch.tensor([3, 4, 6], dtype=torch.int32)
    s["nd"] = torch.tensor([0, 1], dtype=torch.int32)
    s["R"] = 6
    for n in ("q", "k", "v", "qkv"):
        s[n] = torch.cat([s[n], s[n]])[:6]
    run_and_check(sv, s)


def test_one_row(sv):
    run_and_check(sv, make(4, [777], [0], 0, 32, 8, 128, 16, "bf16", 128, ragged=False))


@pytest.mark.parametrize("B,Hq,Hk,D,rotary,il,ragged", [(125, 2, 1, 16, 16, False, False), (130, 1, 1, 24, 20, False, True),
                                                       (30, 112, 8, 64, 64, False, True), (12, 60, 2, 128, 128, True, False),
                                                       (12, 60, 2, 128, 36, False, True)])
def test_many_rows(sv, B, Hq, Hk, D, rotary, il, ragged):
    """More rows than one wave of CTAs takes, and several rows per CTA of more heads than it holds at a time."""
    lens = [65 + 7 * b % 200 for b in range(B)]
    drafts = [64 if not ragged or b % 3 else 63 - b % 11 for b in range(B)]
    run_and_check(sv, make(6, lens, drafts, 64, Hq, Hk, D, 16, "bf16", rotary, ragged=ragged), il, inplace=bool(B % 2))


def test_padded_rows_and_in_place(sv):
    s = make(5, [12, 90], [4, 2], 4, 6, 3, 80, 16, "fp16", 80, packed=False)
    run_and_check(sv, s, inplace=True)


@pytest.mark.parametrize("pos", [1 << 20, 4194303, 100000007])
def test_far_positions(sv, pos):
    """The angle of a far position is exact: an fp32 product would be off by radians."""
    run_and_check(sv, make(6, [pos], [2], 2, 4, 1, 128, 256, "fp16", 128))


@pytest.mark.parametrize("freq", [[0.0, 1.0, 3.0, 1e-30], [-1.0, 8.5, 6.25e8, 1e-45], [7e-12, 1e-20, 123.456, 0.1]])
def test_any_frequency(sv, freq):
    s = make(7, [54321, 3], [3, 1], 3, 2, 1, 16, 16, "fp16", 8, norm=False)
    s["inv"] = torch.tensor(freq, dtype=torch.float32)
    # the definition in 64 bits is itself good for angles up to about 1e13
    run_and_check(sv, s)


def test_eps_carries_a_zero_head(sv):
    s = make(8, [10], [3], 3, 4, 2, 64, 16, "bf16", 64)
    for x in (s["q"], s["k"]):
        x[1] = 0
    s["qkv"] = torch.cat([s["q"].flatten(1), s["k"].flatten(1), s["v"].flatten(1)], 1)
    run_and_check(sv, s, eps=1e-5)


def test_errors_stay_with_their_request(sv):
    """A length below the new tokens, one past the table, drafts out of range, a bad page, a
    negative (failed) length: NaN queries for the rows in error, the cache untouched there."""
    page = 16
    base = make(9, [20, 20, 20, 20, 20], [4] * 5, 4, 4, 2, 64, page, "bf16", 64, ragged=False)
    for what, code in [("short", 1), ("long", 1), ("drafts", 1), ("page", 9), ("high page", 9), ("failed", 1)]:
        s = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in base.items()}
        if what == "short":
            s["lens"][2] = 4
        if what == "long":
            s["lens"][2] = 33
        if what == "drafts":
            s["nd"][2] = 5
        if what == "page":
            s["table"][2, 0:2] = -1
        if what == "high page":
            s["table"][2, 0:2] = s["kc"].shape[0]
        if what == "failed":
            s["lens"][2] = -21
        out, kc, vc, err = call(sv, s)
        assert err == (code, 2), (what, err)
        assert bool(out[10:15].isnan().all()), what
        ok = dict(s, nd=s["nd"].clone())
        ok["nd"][2] = -1
        ro, rk, rv, so, sk = plain.append(ok["q"], ok["k"], ok["v"], *ok["w"], 1e-6, ok["inv"], ok["kc"], ok["vc"],
                                          ok["table"], ok["lens"], ok["nd"], None, 4)
        good = [r for r in range(25) if not 10 <= r < 15]
        check(out[good], ro[good], so[good], s["dt"])
        check(kc, rk, sk, s["dt"])
        assert torch.equal(vc.double(), rv)


def test_offsets_out_of_order(sv):
    s = make(10, [50, 60, 70], [2, 2, 2], 2, 2, 1, 64, 16, "bf16", 64)
    s["ro"] = torch.tensor([0, 6, 3, 9], dtype=torch.int32)
    assert call(sv, s)[3] == (1, 1)


def test_pool_past_32_bits(sv):
    """Element offsets beyond 2^31."""
    pages, page, Hk, D = 70000, 256, 1, 128           # 2.3e9 elements
    kc = torch.zeros((pages, page, Hk, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.randn(2, 1, D, device="cuda").bfloat16()
    tab = torch.tensor([[pages - 1], [1]], dtype=torch.int32, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(x), torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.spec_append(x, x, x, None, None, 0.0, None, kc, vc, tab, i(256, 7), i(0, 0), None, 0, out, ws)
    assert torch.equal(kc[pages - 1, 255], x[0]) and torch.equal(vc[1, 6], x[1]) and torch.equal(out, x)
    assert int((kc != 0).any(-1).sum()) == 2


def test_another_stream_and_graph(sv):
    s = make(11, [33, 70], [4, 4], 4, 8, 2, 128, 16, "bf16", 128, ragged=False)
    ref = call(sv, s)
    got = call(sv, s, stream=torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(ref[:3], got[:3]))
    dev = {k: v.cuda() for k, v in s.items() if torch.is_tensor(v)}
    out, ws = torch.zeros(s["R"], 8, 128, dtype=s["dt"], device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    w = [x.cuda() for x in s["w"]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_append(dev["q"], dev["k"], dev["v"], *w, 1e-6, dev["inv"], dev["kc"], dev["vc"], dev["table"],
                       dev["lens"], dev["nd"], None, 4, out, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), ref[0]) and torch.equal(dev["kc"].cpu(), ref[1])


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("D,rotary,il", [(64, 64, False), (64, 64, True), (64, 20, False), (16, 0, False), (128, 128, False),
                                         (128, 64, True), (128, 70, False), (256, 256, False), (136, 36, False)])
def test_one_weight_alone(sv, which, D, rotary, il):
    """A norm of the queries or of the keys alone, with query, key and value heads of all counts in one warp."""
    for Hq, Hk in [(7, 7), (7, 1), (3, 3), (1, 1), (5, 5), (33, 11)]:
        s = make(D + Hq, [1, 9, 40], [0, 3, 4], 4, Hq, Hk, D, 16, "bf16", rotary)
        s["w"] = (s["w"][0], None) if which == 0 else (None, s["w"][1])
        run_and_check(sv, s, il)
