"""The 8-bit cache's calls, spec_logits and spec_verify together, as a server runs them, and the attention kernel's
bounded waits."""
import os
import sys

import pytest

import cache8_plain as plain8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_12_gb300 as sv
    sv.lib()
    return sv


@pytest.mark.parametrize("dtype,ruled,limit", [(torch.bfloat16, True, 0.1), (E4M3, False, 0.5), (E4M3, True, 0.5)])
def test_verify_steps_under_rules_and_over_8_bits(sv, dtype, ruled, limit):
    """The example server.  With a bf16 cache the chosen tokens' logits lie as near the plain forward's largest as without
    rules (0.1: bf16 activations); a repetition penalty of 1.2 stretches that by no more than 1.2, of a gap that was far
    smaller.  An e4m3 number is off by up to 2^-4 of its value, 0.03 in the mean square, keys and values alike:
    scores of order 1 by 0.03, so weights and values by 3 to 5 %, averaged over the keys, and with them a part of the
    residual stream whose logits are of order 1.  0.5 is ten times that.  No refused token is ever chosen."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step
    seqs, gap, rate = verify_step.run(dtype=dtype, ruled=ruled)
    assert gap < limit
    assert all(len(s) > 20 + 8 for s in seqs)
    if ruled:
        assert all((a + b) % 3 for s in seqs for a, b in zip(s[19:], s[20:]))


def test_one_step_of_calls_against_the_definitions(sv):
    """reserve, append, attend, commit and release of a ragged batch on one 8-bit cache, each against its definition."""
    g = torch.Generator().manual_seed(5)
    B, Hq, Hk, D, drafts = 5, 8, 2, 128, [4, -1, 2, 4, 0]
    c = sv.PagedCache(1, B, 200, 16, 40, Hk, D, dtype=E4M3, scale_tokens=8)
    ints = lambda v: torch.tensor(v, dtype=torch.int32)
    c.reserve(ints([500, 127, 63, 0, 300]).cuda())
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x.view(torch.uint8).copy_((torch.randn(x.shape, generator=g) * 100).clamp(-448, 448).to(E4M3).view(torch.uint8))
        s.copy_(2.0 ** torch.randint(-9, -5, s.shape, generator=g).float())
    off = [0]
    for k in drafts:
        off.append(off[-1] + max(k, 0) + 1)
    nd, ro = ints(drafts), ints(off)
    c.reserve(nd.cuda())
    q, k, v = (torch.randn(off[-1], h, D, generator=g).bfloat16() for h in (Hq, Hk, Hk))
    inv = 1e4 ** (-torch.arange(D // 2) * 2 / D)
    before = [x[0].cpu() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    out_q, out = torch.empty_like(q, device="cuda"), torch.empty_like(q, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    c.append(0, q.cuda(), k.cuda(), v.cuda(), None, None, 1e-6, inv.cuda(), nd.cuda(), ro.cuda(), 4, out_q)
    c.attend(0, out_q, nd.cuda(), ro.cuda(), 4, D ** -0.5, out, 200, 4, lse)
    assert sv.sv_read_device_error(c.workspace) == (0, -1)
    import test_gpu_cache8_append as append
    import test_gpu_cache8_attention as attention
    state = dict(table=c.block_table.cpu(), lens=c.kv_seq_len.cpu(), nd=nd, ro=ro, k_max=4, dt=torch.bfloat16)
    kc, vc, ks, vs = before
    now = [x[0].cpu() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    append.check(dict(state, q=q, k=k, v=v, w=(None, None), inv=inv, kc=kc.view(E4M3), vc=vc.view(E4M3), ks=ks, vs=vs),
                 dict(q=out_q.cpu(), kc=now[0], vc=now[1], ks=now[2], vs=now[3]))
    attention.check(dict(state, q=out_q.cpu(), kc=now[0].view(E4M3), vc=now[1].view(E4M3), ks=now[2], vs=now[3],
                         scale=D ** -0.5, window=200, sinks=4), out.cpu(), lse.cpu())
    lens = c.kv_seq_len.tolist()
    c.commit(torch.zeros(B, dtype=torch.int32, device="cuda"), nd.cuda(), window=200, sinks=4)
    assert c.kv_seq_len.tolist() == [n - max(k, 0) for n, k in zip(lens, drafts)]
    assert int(c.ref_count.sum()) == int((c.block_table >= 0).sum())


def test_pages_move_with_their_scales(sv):
    """A fork's copied page and compacted pages stand for the numbers that they stood for before."""
    g = torch.Generator(device="cuda").manual_seed(7)
    c = sv.PagedCache(3, 4, 40, 16, 8, 3, 80, dtype=E4M3, scale_tokens=8)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    c.reserve(ints(70, 40, 9, -1))
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x.view(torch.uint8).copy_(torch.randint(0, 127, x.shape, device="cuda", generator=g, dtype=torch.uint8))
        s.copy_(torch.rand(s.shape, device="cuda", generator=g) + 0.1)

    def tokens(b, n):
        out = []
        for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            held = torch.stack([plain8.held(x[l].cpu(), s[l].cpu()) for l in range(3)])
            t = torch.arange(n)
            out.append(held[:, c.block_table[b].cpu()[t // 16].long(), t % 16])
        return torch.stack(out)

    was = tokens(0, 71), tokens(1, 41)
    c.fork(ints(0), ints(3), ints(71))
    assert torch.equal(tokens(3, 71), was[0])
    c.kv_seq_len[0] = 0          # the first request ends; what is left moves down
    c.release()
    c.compact(40)
    assert int((c.ref_count > 0).sum()) == int((c.ref_count > 0).nonzero().max()) + 1
    assert torch.equal(tokens(3, 71), was[0]) and torch.equal(tokens(1, 41), was[1])
    assert sv.sv_read_device_error(c.workspace) == (0, -1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,k_max", [(8, 2), (8, 7), (32, 4)])
def test_bounded_waits_run_out(sv, D, Hq, k_max):
    """With one tile of keys withheld from each range the call must still end, with its error word set and a device that
    the next call uses normally."""
    B, L, Hk, page, n = 3, 300, 2, 16, k_max + 1
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randint(0, 120, (60, page, Hk, D), device="cuda", generator=g, dtype=torch.uint8).view(E4M3) for _ in range(2))
    ks, vs = (torch.full((60, 1, Hk), 0.01, device="cuda") for _ in range(2))
    q = torch.randn(B * n, Hq, D, device="cuda", generator=g).bfloat16()
    table = torch.arange(B * 19, device="cuda", dtype=torch.int32).view(B, 19)
    lens, nd = (torch.full((B,), x, device="cuda", dtype=torch.int32) for x in (L, k_max))
    ws = torch.zeros(sv.sv_attention_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    out, again = torch.empty_like(q), torch.empty_like(q)
    call = lambda o: sv.spec_attention8(q, k, v, ks, vs, table, lens, nd, None, k_max, D ** -0.5, 0, 0, o, None, ws)
    call(out)
    assert sv.sv_read_device_error(ws) == (0, -1)
    assert sv.lib().sv_set_test_withhold(1) == sv.SV_OK
    try:
        call(again)
        torch.cuda.synchronize()
    finally:
        sv.lib().sv_set_test_withhold(0)
    assert sv.sv_read_device_error(ws)[0] == 7
    ws[:256] = 0
    call(again)
    assert sv.sv_read_device_error(ws) == (0, -1) and torch.equal(out, again)
