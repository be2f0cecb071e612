"""Page bookkeeping on the GPU against the one-page-at-a-time model (cache_plain.Pages): whole
numbers, so equality."""
import random

import pytest

import cache_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_12_gb300 as sv
    sv.lib()
    return sv


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


class Pool:
    """The state on the GPU beside the model's."""

    def __init__(self, sv, lens, table, ref, page):
        self.sv, self.page = sv, page
        self.model = plain.Pages(ints(lens), ints(table), ints(ref), page)
        self.len, self.table, self.ref = (ints(x).cuda() for x in (lens, table, ref))
        self.ws = torch.zeros(sv.sv_page_workspace_bytes(len(lens), len(ref)), dtype=torch.uint8, device="cuda")
        self.ws[256:] = 171    # everything past the header may hold anything

    def same(self):
        assert self.len.tolist() == self.model.len
        assert self.table.tolist() == self.model.table
        assert self.ref.tolist() == self.model.ref
        code, bad = self.sv.sv_read_device_error(self.ws)
        if self.model.errors:
            assert code in [c for c, _ in self.model.errors] and bad == min(b for _, b in self.model.errors)
        else:
            assert (code, bad) == (0, -1)

    def reserve(self, drafts):
        self.model.reserve(ints(drafts))
        self.sv.spec_page_reserve(ints(drafts).cuda(), self.len, self.table, self.ref, self.page, self.ws)
        self.same()

    def fork(self, parents, children, fork_len):
        F = len(parents)
        want = self.model.fork(ints(parents), ints(children), None if fork_len is None else ints(fork_len))
        src, dst = (torch.full((F,), 55, dtype=torch.int32, device="cuda") for _ in range(2))
        self.sv.spec_page_fork(ints(parents).cuda(), ints(children).cuda(),
                               None if fork_len is None else ints(fork_len).cuda(), self.len, self.table, self.ref,
                               self.page, src, dst, self.ws)
        assert list(zip(src.tolist(), dst.tolist())) == want
        self.same()
        return want

    def release(self, window=0, sinks=0):
        self.model.release(window, sinks)
        self.sv.spec_page_release(self.len, self.table, self.ref, self.page, window, sinks, self.ws)
        self.same()

    def compact(self, capacity):
        want = self.model.compact(capacity)
        src, dst = (torch.full((capacity,), 55, dtype=torch.int32, device="cuda") for _ in range(2))
        self.sv.spec_page_compact(self.table, self.ref, src, dst, self.ws)
        assert list(zip(src.tolist(), dst.tolist())) == want
        self.same()

    def set_len(self, b, L):
        self.model.len[b] = L
        self.len[b] = L


def filled(sv, r, B, M, N, page, share=0.5):
    """Requests of random lengths over pages in random order."""
    ids = list(range(N))
    r.shuffle(ids)
    lens, table, ref = [], [[-1] * M for _ in range(B)], [0] * N
    for b in range(B):
        L = r.randint(0, int(M * page * share)) if r.random() < 0.8 else 0
        if -(-L // page) > len(ids) - 2:
            L = 0
        for x in range(-(-L // page)):
            table[b][x] = p = ids.pop()
            ref[p] = 1
        lens.append(L)
    return Pool(sv, lens, table, ref, page)


@pytest.mark.parametrize("seed,B,M,N,page", [(0, 6, 10, 60, 4), (1, 40, 30, 700, 16), (2, 3, 1, 5, 1), (3, 9, 33, 129, 8),
                                             (4, 70, 12, 9001, 16), (5, 30, 260, 70001, 32), (6, 1100, 3, 2500, 8)])
def test_random_histories(sv, seed, B, M, N, page):
    """Steps, forks, ends and compactions in random order; the pool runs short now and then."""
    r = random.Random(seed)
    p = filled(sv, r, B, M, N, page)
    for _ in range(8):
        act = r.randrange(4)
        m = p.model
        if act == 0:
            drafts = [r.choice([-1, 0, 0, 1, 4, 3 * page]) if m.len[b] >= 0 else -1 for b in range(B)]
            p.reserve(drafts)
            for b in range(B):
                if drafts[b] > 0 and m.len[b] > drafts[b]:
                    p.set_len(b, m.len[b] - r.randint(0, drafts[b]))
                if m.len[b] < 0:
                    p.set_len(b, -1 - m.len[b])
            p.release()
        if act == 1:
            full = [b for b in range(B) if m.len[b] > 0]
            empty = [b for b in range(B) if m.len[b] == 0]
            n = min(len(empty), r.randint(1, 6))
            if full and n:
                pa = [r.choice(full) for _ in range(n)]
                p.fork(pa, r.sample(empty, n), [r.randint(1, m.len[b]) for b in pa] if r.random() < 0.7 else None)
                for b in range(B):
                    if m.len[b] < 0:
                        p.set_len(b, 0)
        if act == 2:
            for b in range(B):
                if r.random() < 0.3:
                    p.set_len(b, 0)
            p.release(r.choice([0, 3 * page + 1]), r.choice([0, 1, page]))
        if act == 3:
            p.compact(r.choice([1, 7, N]))


def test_reserve_serves_in_order_and_fails_whole(sv):
    """Three free pages: the request that does not fit fails, and so do those after it that ask for
    more than is left counting it; one that needs none still grows."""
    p = Pool(sv, [4, 4, 3, 8, 0], [[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, 4, -1], [-1, -1, -1]],
             [1, 1, 1, 1, 1, 0, 0, 0], 4)
    p.reserve([0, 7, 0, 3, 0])
    assert p.model.len == [5, 12, 4, -9, -1]


def test_reserve_errors(sv):
    tab = [[0, 1], [2, 3], [4, -1], [9, 1], [1, -1], [5, -1], [6, -1]]
    p = Pool(sv, [6, 8, -3, 2, 1, 2, 0], tab, [2, 2, 1, 1, 0, 0, 1, 0, 0], 4)
    # shared last page; past the table; failed before; a page that is none; shared; a count of 0; bad drafts
    p.reserve([0, 0, 0, 0, 0, 1, -2])
    assert [c for c, _ in p.model.errors] == [11, 1, 1, 9, 11, 9, 1]


def test_long_prompt_reservation(sv):
    p = Pool(sv, [0, 5], [[-1] * 700, [3] + [-1] * 699], [0, 0, 0, 1] + [0] * 2000, 8)
    p.reserve([8 * 700 - 1, 8 * 650 - 6])


def test_fork_errors(sv):
    """Bad indexes, a child that runs, lengths out of range, a child named twice, a chain through a
    child, a missing last page, no pages left."""
    tab = [[0, 1, 2], [3, -1, 9], [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3,
           [-1] * 3, [-1] * 3]
    p = Pool(sv, [10, 7, 0, 0, 0, 0, 0, 0, 0, 0], tab, [1, 1, 1, 1, 0], 4)
    p.fork([0, -1, 10, 0, 0, 0, 2, 1, 0, 0], [2, 3, 3, 12, 1, 2, 4, 5, 6, 7], [10, 1, 1, 1, 4, 8, 3, 6, 9, 11])
    assert p.model.len == [10, 7, 10, -1, -1, -1, -1, -1, 0, 0]


def test_fork_shares_a_page_that_is_none(sv):
    p = Pool(sv, [12, 0], [[0, 7, 2], [-1] * 3], [1, 0, 1], 4)
    src = torch.empty(1, dtype=torch.int32, device="cuda")
    sv.spec_page_fork(ints([0]).cuda(), ints([1]).cuda(), None, p.len, p.table, p.ref, 4, src, src.clone(), p.ws)
    assert p.table.tolist()[1] == [0, -1, 2] and p.ref.tolist() == [2, 0, 2]
    assert sv.sv_read_device_error(p.ws) == (9, 0)


@pytest.mark.parametrize("B,M,N,long", [(3, 5000, 15000, 3), (40, 300, 9000, 30), (1500, 40, 30000, 700), (1500, 40, 9000, 900),
                                        (1024, 9, 5000, 1024)])
def test_prompts_among_steps(sv, B, M, N, long):
    """Many pages for some requests and few or none for the others, with enough and too few in the pool."""
    r = random.Random(B + N)
    p = Pool(sv, [0] * B, [[-1] * M for _ in range(B)], [int(r.random() < 0.1) for _ in range(N)], 4)
    want = [r.randint(16, M * 4 - 1) if b < long else r.choice([-1, 0, 3, 4, 15]) for b in range(B)]
    r.shuffle(want)
    p.reserve(want)


@pytest.mark.parametrize("B,M,forks", [(40, 400, 20), (40, 1024, 20), (40, 1025, 20), (300, 1100, 150), (1300, 7, 1200)])
def test_many_forks(sv, B, M, forks):
    """Forks of several chunks of a table row and of one short of it; more forks than threads."""
    r = random.Random(B + M)
    parents = B - forks
    page, lens, ids = 4, [], list(range(parents * M + forks))
    r.shuffle(ids)
    table, ref = [[-1] * M for _ in range(B)], [0] * len(ids)
    for b in range(B):
        lens.append(r.randint(1, M * page) if b < parents else 0)
        for x in range(-(-lens[b] // page)):
            table[b][x] = p = ids.pop()
            ref[p] = 1
    p = Pool(sv, lens, table, ref, page)
    pa = [r.randrange(parents) for _ in range(forks)]
    p.fork(pa, r.sample(range(parents, B), forks), [r.randint(1, lens[b]) for b in pa])


def test_release_errors_and_windows(sv):
    p = Pool(sv, [4, 13, -5, 0], [[0, 7, 1], [2, 3, 4], [5, -1, -1], [-3, 6, -1]], [1, 0, 1, 1, 1, 1, 0], 4)
    sv.spec_page_release(p.len, p.table, p.ref, 4, 0, 0, p.ws)
    assert p.table.tolist() == [[0, -1, -1], [2, 3, 4], [5, -1, -1], [-1, -1, -1]]
    assert p.ref.tolist() == [1, 0, 1, 1, 1, 1, 0]
    assert sv.sv_read_device_error(p.ws) in [(9, 0), (1, 0)]
    for window in (1, 3, 4, 5, 8, 9, 17, 64, 1 << 30):
        for sinks in (0, 1, 4, 5, 1 << 30):
            q = Pool(sv, [64, 61, 3, 0], [list(range(16)), list(range(16, 32)), [32] + [-1] * 15, [33] + [-1] * 15],
                     [1] * 34, 4)
            q.release(window, sinks)


def test_release_many_pages(sv):
    N = 9000
    q = Pool(sv, [36000, 4], [list(range(N)), list(range(N, 2 * N))], [1] * 2 * N, 4)
    q.release(100, 9)


def test_compact_edges(sv):
    Pool(sv, [0], [[-1]], [0], 4).compact(3)                       # nothing in use
    Pool(sv, [4], [[0]], [1], 4).compact(1)                        # nothing to move
    Pool(sv, [8], [[9, 4]], [0] * 4 + [1] + [0] * 4 + [1], 4).compact(5)
    n = 20000
    Pool(sv, [4, 4], [[n - 1], [n - 1]], [0] * (n - 1) + [2], 4).compact(2)
    q = Pool(sv, [4, 4], [[7], [3]], [1, 0, 0, 0, 0], 4)           # entries that are no pages in use
    src = torch.empty(2, dtype=torch.int32, device="cuda")
    sv.spec_page_compact(q.table, q.ref, src, src.clone(), q.ws)
    assert q.table.tolist() == [[7], [3]] and sv.sv_read_device_error(q.ws) == (9, 0)


@pytest.mark.parametrize("shape,dtype", [((9, 16, 2, 64), torch.bfloat16), ((3, 9, 8, 1, 8), torch.float16),
                                         ((2, 9, 128, 8, 128), torch.bfloat16), ((9, 40), torch.float32)])
@pytest.mark.parametrize("layout", ["plain", "transposed", "apart"])
def test_copy(sv, shape, dtype, layout):
    g = torch.Generator(device="cuda").manual_seed(1)
    layers = len(shape) == 5
    if layout == "transposed":
        if len(shape) < 4:
            return
        shape = shape[:-3] + (shape[-2], shape[-3], shape[-1])
    both = torch.randn((2,) + shape, device="cuda", generator=g).to(dtype)
    if layout == "apart":      # keys and values of a page next to each other
        both = torch.randn(shape[:2 if layers else 1] + (2,) + shape[2 if layers else 1:], device="cuda", generator=g).to(dtype)
        k, v = both.unbind(2 if layers else 1)
    else:
        k, v = both
        if layout == "transposed":
            k, v = k.transpose(-2, -3), v.transpose(-2, -3)
    wk, wv = k.clone(), v.clone()
    pairs = [(0, 5), (-1, -1), (0, 8), (3, 2), (4, -1), (-1, 1)]
    for a, d in pairs:
        if a >= 0 and d >= 0:
            (wk[:, d] if layers else wk[d]).copy_(wk[:, a] if layers else wk[a])
            (wv[:, d] if layers else wv[d]).copy_(wv[:, a] if layers else wv[a])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    src, dst = ints([a for a, _ in pairs]).cuda(), ints([d for _, d in pairs]).cuda()
    sv.spec_page_copy(k, v, src, dst, ws)
    assert torch.equal(k, wk) and torch.equal(v, wv) and sv.sv_read_device_error(ws) == (0, -1)
    sv.spec_page_copy(k, None, ints([9, 1]).cuda(), ints([1, 9]).cuda(), ws)     # not pages: skipped
    assert torch.equal(k, wk) and sv.sv_read_device_error(ws) == (9, 0)


def test_copy_far_apart(sv):
    """Byte offsets past 2^32 and many pairs."""
    k = torch.zeros((2, 40000, 16, 1, 2048), dtype=torch.bfloat16, device="cuda")    # 5.2 GB
    k[:, 39000:] = torch.arange(1000, device="cuda").view(1, -1, 1, 1, 1).bfloat16()
    src, dst = torch.arange(39000, 40000, dtype=torch.int32, device="cuda"), torch.arange(1000, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.spec_page_copy(k, None, src, dst, ws)
    assert torch.equal(k[:, :1000], k[:, 39000:]) and int(k[:, 1000:39000].count_nonzero()) == 0


def test_graph_of_a_step(sv):
    """reserve, roll back, release captured once and replayed."""
    p = filled(sv, random.Random(8), 30, 20, 400, 8, share=0.3)
    nd, acc = ints([3] * 30).cuda(), ints([1] * 30).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_page_reserve(nd, p.len, p.table, p.ref, 8, p.ws)
        sv.spec_rollback(p.len, acc, nd, p.ws)
        sv.spec_page_release(p.len, p.table, p.ref, 8, 0, 0, p.ws)
    for _ in range(6):
        graph.replay()
        p.model.reserve(ints([3] * 30))
        p.model.len = [n - 2 for n in p.model.len]
        p.model.release()
        p.same()


@pytest.mark.parametrize("L,sinks,window", [(20479, 0, 4096), (20479, 4, 4096), (50000, 0, 4096), (50000, 4, 4096),
                                            (65536, 5000, 64), (16500, 16384, 1)])
def test_a_windowed_request_that_ends_gives_every_page_back(sv, L, sinks, window):
    """A long request whose middle pages went back under its window ends: its table row empties and every
    count returns to 0, and so again for the slot's next owner."""
    page, M = 16, 4096
    r = random.Random(L + sinks)
    need = -(-L // page)
    ids = list(range(need + 40))
    r.shuffle(ids)
    other = ids[need:need + 5]
    ref = [0] * len(ids)
    for p in ids[:need + 5]:
        ref[p] = 1
    p = Pool(sv, [L, 5 * page], [ids[:need] + [-1] * (M - need), other + [-1] * (M - 5)], ref, page)
    for n in (L, 3):
        p.release(window, sinks)
        p.set_len(0, 0)
        p.release(0 if n == 3 else window, sinks)
        assert p.table[0].tolist() == [-1] * M and int(p.ref.sum()) == 5
        p.reserve([n - 1, -1])
    p.release()


@pytest.mark.parametrize("L,window,keep", [(50000, 4096, 4), (50000, 4096, 16), (40000, 100, 33)])
def test_a_windowed_request_cut_to_its_first_tokens(sv, L, window, keep):
    """Whatever length a caller sets, the pages past it go back, also behind a gap."""
    page, M, need = 16, 3200, -(-L // 16)
    p = Pool(sv, [L], [list(range(need)) + [-1] * (M - need)], [1] * need + [0] * 8, page)
    p.release(window, 33)
    p.set_len(0, keep)
    p.release(window, 33)
    assert int(p.ref.sum()) == -(-keep // page)


def test_release_of_rows_of_every_length(sv):
    """Rows shorter and longer than one CTA's entries, at odd lengths and starts."""
    for M in (1, 2, 255, 257, 1023, 1024, 1025, 5001):
        r = random.Random(M)
        lens, table, ref, n = [], [], [], 0
        for b in range(5):
            held = r.randint(0, M)
            table.append(list(range(n, n + held)) + [-1] * (M - held))
            ref += [1] * held
            n += held
            lens.append(r.choice([0, -3, r.randint(0, held * 8), held * 8]))
        p = Pool(sv, lens, table, ref + [0], 8)
        p.release(r.choice([0, 1, 77, 5000]), r.choice([0, 9, 4000]))
        p.release()


def reserve_by_the_state_before(p, drafts):
    """p.reserve, where the model's counts are read as they were before the call: a partly filled page without
    a request is none, also once another request has been granted it."""
    m, hidden = p.model, {}
    for b, L in enumerate(m.len):
        if L > 0 and L % m.P:
            x = m.table[b][L // m.P]
            if 0 <= x < len(m.ref) and m.ref[x] < 1:
                hidden[b, L // m.P], m.table[b][L // m.P] = x, -1
    m.reserve(ints(drafts))
    for (b, i), x in hidden.items():
        m.table[b][i] = x
    p.sv.spec_page_reserve(ints(drafts).cuda(), p.len, p.table, p.ref, p.page, p.ws)
    p.same()


@pytest.mark.parametrize("B", [1023, 1024, 1025, 2100, 3000])
def test_reserve_judges_every_request_by_the_state_before_the_call(sv, B):
    """The last request's partly filled page is a free one, which the same call grants to the first request:
    still no page in use, however many requests lie between; and the requests behind it are served."""
    page, N = 4, B + 8
    lens = [0] * (B - 2) + [2, 0]
    table = [[-1, -1] for _ in range(B)]
    table[B - 2][0] = 0
    p = Pool(sv, lens, table, [0] * N, page)
    reserve_by_the_state_before(p, [0] * (B - 2) + [4, 7])
    assert p.model.errors == [(9, B - 2)]


def test_reserve_of_many_requests_with_errors_among_them(sv):
    r = random.Random(77)
    for N in (6000, 2200):
        B, M, page = 2600, 4, 8
        lens, table, ref, n = [], [], [0] * N, 0
        for b in range(B):
            L = r.choice([0, 0, r.randint(1, 2 * page)]) if n < 1500 else 0
            row = [-1] * M
            for x in range(-(-L // page)):
                row[x] = n
                ref[n] = 1
                n += 1
            what = r.random()
            if L % page and what < 0.1:
                row[L // page] = r.choice([-1, N, r.randrange(1600, 1700)])
            elif L % page and what < 0.2:
                ref[row[L // page]] = r.choice([0, 2])
            elif what < 0.22:
                L = -5
            lens.append(L)
            table.append(row)
        p = Pool(sv, lens, table, ref, page)
        reserve_by_the_state_before(p, [r.choice([-2, -1, 0, 1, 8, 15, 31]) for _ in range(B)])


@pytest.mark.parametrize("extra", [0, 2100])
def test_fork_shares_no_page_that_was_free_before_the_call(sv, extra):
    """Full pages of a parent that no request holds are no pages in use, for each of several children,
    also where the same call takes them as fresh pages, and with more forks than a CTA's list holds."""
    B, N, page = 8 + extra, 60 + 2 * extra, 4
    # parent 0: 6 tokens, pages 40 and 41; parent 1: 12 tokens, pages 0 and 5 free, 42 in use; parent 2: as parent 0
    table = [[-1] * 3 for _ in range(B)]
    table[0][:2], table[1][:], table[2][:2] = [40, 41], [0, 5, 42], [43, 44]
    ref = [0] * N
    for p in range(40, 45):
        ref[p] = 1
    lens = [6, 12, 6] + [0] * (B - 3)
    pa = [0, 1, 1, 2, 1] + [0] * extra
    ch = [3, 4, 5, 6, 7] + list(range(8, B))
    t, n, c = ints(table).cuda(), ints(lens).cuda(), ints(ref).cuda()
    F = len(pa)
    src, dst = torch.full((2, F), 55, dtype=torch.int32, device="cuda")
    ws = torch.zeros(sv.sv_page_workspace_bytes(B, N), dtype=torch.uint8, device="cuda")
    ws[256:] = 171
    sv.spec_page_fork(ints(pa).cuda(), ints(ch).cuda(), None, n, t, c, page, src, dst, ws)
    assert sv.sv_read_device_error(ws) == (9, 1)
    fresh = [p for p in range(N) if ref[p] == 0][:2 + extra]
    assert t[3].tolist() == [40, fresh[0], -1] and t[6].tolist() == [43, fresh[1], -1]
    for child in (4, 5, 7):
        assert t[child].tolist() == [-1, -1, 42]
    want = list(ref)
    for p in fresh:
        want[p] = 1
    want[40] += 1 + extra
    want[43] += 1
    want[42] += 3
    assert c.tolist() == want
    assert dst.tolist() == [fresh[0], -1, -1, fresh[1], -1] + fresh[2:]
    assert n.tolist()[:8] == [6, 12, 6, 6, 12, 12, 6, 12]
