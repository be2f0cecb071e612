"""Refusals of the cache-side calls that need no GPU: nothing is enqueued and no pointer is read."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_12_gb300 import build
    build.build()
    import speculative_decoding_verification_12_gb300 as sv
    from speculative_decoding_verification_12_gb300 import cache
    cache._lib()
    return sv


INV, WS, UNS = 1, 2, 4
PTR = 256   # a non-null, aligned placeholder


def kv(sv, **kw):
    d = dict(k=PTR, v=PTR, page_stride=16 * 8 * 128, token_stride=8 * 128, head_stride=128, num_pages=10,
             page_size=16, num_heads=8, head_dim=128, dtype=1, max_pages=4, block_table=PTR)
    d.update(kw)
    return sv.SvKvCache(*[d[n] for n, _ in sv.SvKvCache._fields_])


CACHE_BAD = [(dict(k=None), INV), (dict(v=None), INV), (dict(block_table=None), INV), (dict(num_pages=0), INV),
             (dict(num_heads=0), INV), (dict(head_dim=0), INV), (dict(max_pages=0), INV), (dict(dtype=0), INV),
             (dict(dtype=7), INV), (dict(page_stride=0), INV), (dict(token_stride=-8), INV),
             (dict(head_dim=12), UNS), (dict(head_dim=264), UNS), (dict(page_size=4), UNS), (dict(page_size=24), UNS),
             (dict(page_size=512), UNS), (dict(head_stride=4), UNS), (dict(token_stride=1028), UNS),
             (dict(k=264), UNS), (dict(v=264), UNS), (dict(max_pages=1 << 28), UNS)]


def append(sv, **kw):
    d = dict(q=PTR, k=PTR, v=PTR, qs=4096, ks=1024, vs=1024, Hq=32, qw=PTR, kw=PTR, eps=1e-6, inv=PTR, rot=128, il=0,
             rs=1.0, nd=PTR, ro=None, ln=PTR, B=2, k_max=4, R=10, cache=kv(sv), o=PTR, os=4096, ws=PTR)
    d.update(kw)
    return sv.lib().spec_append(*d.values(), None)


def attention(sv, **kw):
    d = dict(q=PTR, qs=4096, Hq=32, nd=PTR, ro=None, ln=PTR, B=2, k_max=4, R=10, cache=kv(sv), scale=1.0, window=0,
             sinks=0, out=PTR, lse=None, ws=PTR, wsb=1 << 30)
    d.update(kw)
    return sv.lib().spec_attention(*d.values(), None)


BATCH_BAD = [(dict(B=0), INV), (dict(k_max=-1), INV), (dict(k_max=65, R=132), UNS), (dict(R=11), INV),
             (dict(nd=None), INV), (dict(ln=None), INV), (dict(Hq=30), INV), (dict(Hq=0), INV),
             (dict(B=1 << 25, ro=PTR), UNS), (dict(q=None), INV), (dict(qs=4092), INV), (dict(qs=4100), UNS),
             (dict(q=264), UNS), (dict(ws=None), INV), (dict(ws=128), WS)]


@pytest.mark.parametrize("call", [append, attention])
def test_batch_and_cache_refusals(sv, call):
    for bad, want in BATCH_BAD:
        assert call(sv, **bad) == want, bad
    for bad, want in CACHE_BAD:
        assert call(sv, cache=kv(sv, **bad)) == want, bad


def test_append_refusals(sv):
    for bad, want in [(dict(rot=3), INV), (dict(rot=130), INV), (dict(inv=None), INV), (dict(eps=-1.0), INV),
                      (dict(eps=float("nan")), INV), (dict(rs=float("inf")), INV), (dict(o=None), INV),
                      (dict(ks=1016), INV), (dict(vs=1028), UNS), (dict(os=4090), INV), (dict(o=264), UNS),
                      (dict(qw=264), UNS)]:
        assert append(sv, **bad) == want, bad


def test_attention_refusals(sv):
    need = sv.sv_attention_workspace_bytes(128)
    for bad, want in [(dict(window=-1), INV), (dict(sinks=-1), INV), (dict(scale=float("nan")), INV),
                      (dict(out=None), INV), (dict(out=264), UNS), (dict(wsb=need - 1), WS),
                      (dict(cache=kv(sv, head_dim=136, head_stride=136), qs=8192), UNS)]:
        assert attention(sv, **bad) == want, bad
    assert sv.sv_attention_workspace_bytes(12) == sv.sv_attention_workspace_bytes(136) == 0
    assert need >= 256 and need % 256 == 0


def test_page_refusals(sv):
    l, big = sv.lib(), 1 << 30

    def reserve(nd=PTR, ln=PTR, B=2, tab=PTR, M=4, ref=PTR, N=10, P=16, ws=PTR, wsb=big):
        return l.spec_page_reserve(nd, ln, B, tab, M, ref, N, P, ws, wsb, None)

    def fork(pa=PTR, ch=PTR, fl=None, F=1, ln=PTR, B=2, tab=PTR, M=4, ref=PTR, N=10, P=16, s=PTR, d=PTR, ws=PTR,
             wsb=big):
        return l.spec_page_fork(pa, ch, fl, F, ln, B, tab, M, ref, N, P, s, d, ws, wsb, None)

    def release(ln=PTR, B=2, tab=PTR, M=4, ref=PTR, N=10, P=16, w=0, s=0, ws=PTR):
        return l.spec_page_release(ln, B, tab, M, ref, N, P, w, s, ws, None)

    def compact(B=2, tab=PTR, M=4, ref=PTR, N=10, s=PTR, d=PTR, cap=4, ws=PTR, wsb=big):
        return l.spec_page_compact(B, tab, M, ref, N, s, d, cap, ws, wsb, None)

    small = sv.sv_page_workspace_bytes(2, 10) - 1
    for call in (reserve, fork, release, compact):
        for bad, want in [(dict(B=0), INV), (dict(tab=None), INV), (dict(ref=None), INV), (dict(M=0), INV),
                          (dict(N=0), INV), (dict(ws=None), INV), (dict(ws=128), WS), (dict(B=1 << 25), UNS),
                          (dict(N=1 << 28), UNS), (dict(M=(1 << 20) + 1), UNS)]:
            assert call(**bad) == want, (call, bad)
    for call in (reserve, fork, compact):
        assert call(wsb=small) == WS
    for call in (reserve, fork, release):
        assert call(P=0) == INV and call(ln=None) == INV
        assert call(M=1 << 20, P=1 << 12) == UNS
    assert reserve(nd=None) == INV
    assert fork(pa=None) == fork(ch=None) == fork(s=None) == fork(d=None) == fork(F=0) == INV
    assert fork(F=3) == UNS
    assert release(w=-1) == release(s=-1) == INV
    assert compact(s=None) == compact(d=None) == compact(cap=0) == INV

    def copy(k=PTR, v=PTR, pb=1024, ps=1024, nl=1, ls=0, N=10, s=PTR, d=PTR, n=4, ws=PTR):
        return l.spec_page_copy(k, v, pb, ps, nl, ls, N, s, d, n, ws, None)

    for bad, want in [(dict(k=None), INV), (dict(s=None), INV), (dict(d=None), INV), (dict(ws=None), INV),
                      (dict(n=0), INV), (dict(N=0), INV), (dict(nl=0), INV), (dict(nl=2), INV), (dict(pb=0), INV),
                      (dict(ps=512), INV), (dict(ls=-16, nl=2), INV), (dict(k=264), UNS), (dict(v=264), UNS),
                      (dict(pb=1000), UNS), (dict(ps=1032), UNS), (dict(nl=2, ls=1000), UNS), (dict(ws=128), WS)]:
        assert copy(**bad) == want, bad
    assert sv.sv_page_workspace_bytes(0, 5) == sv.sv_page_workspace_bytes(5, 0) == 0
    assert sv.sv_page_workspace_bytes(1 << 25, 5) == sv.sv_page_workspace_bytes(5, 1 << 28) == 0


def test_binding_refuses_wrong_tensors(sv):
    """The binding's own checks come before the library is called: CPU tensors never reach it."""
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    tab = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_append(x, x, x, None, None, 1e-6, None, c, c, tab, i, i, None, 0, x, ws)
    with pytest.raises(ValueError):
        sv.spec_attention(x, c, c, tab, i, i, None, 0, 1.0, 0, 0, x, None, ws)
    with pytest.raises(ValueError):
        sv.spec_page_reserve(i, i, tab, i, 16, ws)
    with pytest.raises(ValueError):
        sv.spec_page_fork(i, i, None, i, tab, i, 16, i, i, ws)
    with pytest.raises(ValueError):
        sv.spec_page_release(i, tab, i, 16, 0, 0, ws)
    with pytest.raises(ValueError):
        sv.spec_page_compact(tab, i, i, i, ws)
    with pytest.raises(ValueError):
        sv.spec_page_copy(c, c, i, i, ws)


def test_cache_rollback_refusals(sv):
    def call(ln=PTR, acc=PTR, nd=PTR, B=2, ws=PTR):
        return sv.lib().spec_cache_rollback(ln, acc, nd, B, ws, None)

    for bad, want in [(dict(ln=None), INV), (dict(acc=None), INV), (dict(nd=None), INV), (dict(B=0), INV),
                      (dict(ws=None), INV), (dict(ws=128), WS), (dict(B=1 << 25), UNS)]:
        assert call(**bad) == want, bad
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_cache_rollback(i, i, i, torch.zeros(256, dtype=torch.uint8))


def test_the_library_is_built_without_pytorch(tmp_path, monkeypatch):
    """The binding is for PyTorch's users; the library needs neither it nor its headers."""
    from speculative_decoding_verification_12_gb300 import build
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    with monkeypatch.context() as m:
        m.setattr(build.importlib.util, "find_spec", lambda name: None)
        assert C.CDLL(build.build()).one() == 1
        assert sorted(p.name for p in tmp_path.iterdir()) == ["lib.so", "one.cu"]
    # and where the binding does not compile
    (tmp_path / "lib.so").unlink()
    (tmp_path / "binding.cpp").write_text("no C++\n")
    with pytest.raises(RuntimeError, match="_binding.so"):
        build.build()
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "binding.so").exists()


def test_rollback_without_the_compiled_binding(sv, monkeypatch):
    """spec_rollback needs libspecverify.so alone: its own checks, then the library."""
    import sys

    from speculative_decoding_verification_12_gb300 import cache

    class OnCuda:
        is_cuda, dtype = True, torch.int32

        def __init__(self, at, n=2):
            self.at, self.n = at, n

        def is_contiguous(self):
            return True

        def numel(self):
            return self.n

        def data_ptr(self):
            return self.at

    class Library:
        def spec_rollback(self, *args):
            self.args = args
            return sv.SV_OK

    monkeypatch.setattr(cache, "_native", None)
    monkeypatch.delattr(sv, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "speculative_decoding_verification_12_gb300._binding", None)
    library = Library()
    monkeypatch.setattr(sv, "lib", lambda: library)
    sv.spec_rollback(OnCuda(256), OnCuda(512), OnCuda(768), OnCuda(1024, 2), stream=7)
    assert library.args == (256, 512, 768, 2, 1024, 7)
    with pytest.raises(ValueError, match="accept_len"):
        sv.spec_rollback(OnCuda(256), OnCuda(512, 3), OnCuda(768), OnCuda(1024))
