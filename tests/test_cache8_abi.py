"""Refusals of the 8-bit cache's calls and of spec_logits that need no GPU: nothing is enqueued and no pointer is
read."""
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


def kv8(sv, **kw):
    d = dict(k=PTR, v=PTR, k_scale=PTR, v_scale=PTR, page_stride=16 * 8 * 128, token_stride=8 * 128, head_stride=128,
             scale_page_stride=8, scale_block_stride=8, scale_head_stride=1, num_pages=10, page_size=16, scale_tokens=16,
             num_heads=8, head_dim=128, max_pages=4, block_table=PTR)
    d.update(kw)
    return sv.SvKvCache8(*[d[n] for n, _ in sv.SvKvCache8._fields_])


CACHE_BAD = [(dict(k=None), INV), (dict(v=None), INV), (dict(k_scale=None), INV), (dict(v_scale=None), INV),
             (dict(block_table=None), INV), (dict(num_pages=0), INV), (dict(num_heads=0), INV), (dict(head_dim=0), INV),
             (dict(max_pages=0), INV), (dict(page_stride=0), INV), (dict(token_stride=-16), INV),
             (dict(scale_page_stride=0), INV), (dict(scale_block_stride=-1), INV), (dict(scale_head_stride=0), INV),
             (dict(head_dim=24), UNS), (dict(head_dim=144), UNS), (dict(page_size=4), UNS), (dict(page_size=24), UNS),
             (dict(page_size=512), UNS), (dict(head_stride=8), UNS), (dict(token_stride=1032), UNS), (dict(page_stride=1032), UNS),
             (dict(scale_tokens=4), UNS), (dict(scale_tokens=32), UNS), (dict(scale_tokens=12), UNS), (dict(scale_tokens=0), UNS),
             (dict(k=264), UNS), (dict(v=264), UNS), (dict(k_scale=258), UNS), (dict(v_scale=257), UNS),
             (dict(max_pages=1 << 28), UNS), (dict(scale_page_stride=1 << 38), UNS)]


def append(sv, **kw):
    d = dict(q=PTR, k=PTR, v=PTR, dtype=1, qs=4096, ks=1024, vs=1024, Hq=32, qw=PTR, kw=PTR, eps=1e-6, inv=PTR, rot=128,
             il=0, rs=1.0, nd=PTR, ro=None, ln=PTR, B=2, k_max=4, R=10, cache=kv8(sv), o=PTR, os=4096, ws=PTR)
    d.update(kw)
    return sv.lib().spec_append8(*d.values(), None)


def attention(sv, **kw):
    d = dict(q=PTR, dtype=1, qs=4096, Hq=32, nd=PTR, ro=None, ln=PTR, B=2, k_max=4, R=10, cache=kv8(sv), scale=1.0,
             window=0, sinks=0, out=PTR, lse=None, ws=PTR, wsb=1 << 30)
    d.update(kw)
    return sv.lib().spec_attention8(*d.values(), None)


BATCH_BAD = [(dict(B=0), INV), (dict(k_max=-1), INV), (dict(k_max=65, R=132), UNS), (dict(R=11), INV),
             (dict(nd=None), INV), (dict(ln=None), INV), (dict(Hq=30), INV), (dict(Hq=0), INV), (dict(dtype=0), INV),
             (dict(dtype=7), INV), (dict(B=1 << 25, ro=PTR), UNS), (dict(q=None), INV), (dict(qs=4092), INV),
             (dict(qs=4100), UNS), (dict(q=264), UNS), (dict(ws=None), INV), (dict(ws=128), WS)]


@pytest.mark.parametrize("call", [append, attention])
def test_batch_and_cache_refusals(sv, call):
    for bad, want in BATCH_BAD:
        assert call(sv, **bad) == want, bad
    for bad, want in CACHE_BAD:
        assert call(sv, cache=kv8(sv, **bad)) == want, bad


def test_append_refusals(sv):
    for bad, want in [(dict(rot=3), INV), (dict(rot=130), INV), (dict(inv=None), INV), (dict(eps=-1.0), INV),
                      (dict(eps=float("nan")), INV), (dict(rs=float("inf")), INV), (dict(o=None), INV),
                      (dict(ks=1016), INV), (dict(vs=1028), UNS), (dict(os=4090), INV), (dict(o=264), UNS),
                      (dict(qw=264), UNS)]:
        assert append(sv, **bad) == want, bad


def test_attention_refusals(sv):
    need = sv.sv_attention_workspace_bytes(128)
    for bad, want in [(dict(window=-1), INV), (dict(sinks=-1), INV), (dict(scale=float("nan")), INV),
                      (dict(out=None), INV), (dict(out=264), UNS), (dict(wsb=need - 1), WS)]:
        assert attention(sv, **bad) == want, bad


def rules(sv, **kw):
    d = dict(repetition=PTR, presence=PTR, frequency=PTR, prior_offsets=PTR, prior_tokens=PTR, prior_counts=PTR, prior_len=5,
             bias_len=5, bias_offsets=PTR, bias_tokens=PTR, bias_values=PTR, masks=PTR, mask_rows=PTR, num_masks=3, mask_words=32)
    d.update(kw)
    return sv.SvLogitRules(*[d[n] for n, _ in sv.SvLogitRules._fields_])


def test_logits_refusals(sv):
    def call(**kw):
        d = dict(z=PTR, dtype=1, toks=PTR, nd=PTR, ro=None, B=2, k_max=4, V=1000, R=10, rules=rules(sv), out=PTR, ws=PTR)
        d.update(kw)
        return sv.lib().spec_logits(*d.values(), None)

    for bad, want in [(dict(z=None), INV), (dict(out=None), INV), (dict(nd=None), INV), (dict(ws=None), INV), (dict(toks=None), INV),
                      (dict(B=0), INV), (dict(k_max=-1), INV), (dict(V=0), INV), (dict(R=0), INV), (dict(R=11), INV),
                      (dict(dtype=2), INV), (dict(dtype=9), INV), (dict(k_max=65, R=132), UNS), (dict(B=1 << 25, ro=PTR), UNS),
                      (dict(V=(1 << 21) + 1), UNS), (dict(z=264), UNS), (dict(out=264), UNS), (dict(ws=128), WS),
                      (dict(out=PTR + 1024), INV), (dict(z=PTR + 1024), INV)]:
        assert call(**bad) == want, bad
    for bad in [dict(prior_len=-1), dict(prior_tokens=None), dict(prior_counts=None), dict(bias_len=-1), dict(bias_tokens=None),
                dict(bias_values=None), dict(num_masks=-1), dict(masks=None), dict(mask_words=31)]:
        assert call(rules=rules(sv, **bad)) == INV, bad


def test_binding_refuses_wrong_tensors(sv):
    """The binding's own checks come before the library is called: CPU tensors never reach it."""
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    tab, sc, z = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(4, 1, 2), torch.zeros(2, 50)
    with pytest.raises(ValueError):
        sv.spec_append8(x, x, x, None, None, 1e-6, None, c, c, sc, sc, tab, i, i, None, 0, x, ws)
    with pytest.raises(ValueError):
        sv.spec_attention8(x, c, c, sc, sc, tab, i, i, None, 0, 1.0, 0, 0, x, None, ws)
    with pytest.raises(ValueError):
        sv.spec_logits(z, i[:0], i, None, 0, None, None, None, None, None, None, None, z, ws)


def test_a_cache_keeps_each_pages_scales_behind_its_numbers(sv):
    c = sv.PagedCache(2, 4, 10, 32, 5, 3, 64, dtype=torch.float8_e4m3fn, device="cpu", scale_tokens=8)
    assert c.k.shape == (2, 10, 32, 3, 64) and c.k.dtype == torch.float8_e4m3fn and c.k_scale.shape == (2, 10, 4, 3)
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert x.stride(1) % 16 == 0 and 4 * s.stride(1) == x.stride(1) and 4 * s.stride(0) == x.stride(0)
        end = x[1, 9].data_ptr() + 32 * 3 * 64
        assert s[1, 9].data_ptr() == end
        s[1, 9, 3, 2] = 5.0
        assert float(s[1, 9, 3, 2]) == 5.0 and int(s.count_nonzero()) == 1
    assert c._pages[0].view(torch.uint8).count_nonzero() > 0
    d = sv.PagedCache(1, 2, 4, 8, 3, 2, 64, dtype=torch.float8_e4m3fn, device="cpu")
    assert d.k_scale.shape == (1, 4, 1, 2)    # (a block is at most a page)
    with pytest.raises(ValueError):
        sv.PagedCache(1, 2, 4, 32, 3, 2, 64, dtype=torch.float8_e4m3fn, device="cpu", scale_tokens=12)
