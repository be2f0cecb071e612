"""The cache-side calls and spec_verify together, as a server runs them (examples/verify_step.py),
and the attention kernel's bounded waits."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_12_gb300 as sv
    sv.lib()
    return sv


def test_verify_steps_give_the_models_own_tokens(sv):
    """Greedy requests: every token that comes out is, up to bf16 activations, the plain forward's
    largest logit.  The logits are of order 1 with a spread over 512 tokens; bf16 activations of a
    4-layer residual stream (each rounding 2^-9 of its value, a few tens of them) move one by less
    than 0.1."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step
    seqs, gap, rate = verify_step.run()
    assert gap < 0.1
    # a request's first wrong draft is its first, second or third in turn: 0, 1 or 2 are kept, 1 on
    # average, and a near tie of two logits may move a few of the 48
    assert abs(rate - 1.0) < 0.2
    assert all(len(s) > 20 + 8 for s in seqs)


def test_bounded_waits_run_out(sv):
    """With one tile of keys withheld the call must still end, with its error word set and a device
    that the next call uses normally."""
    B, L, Hq, Hk, D, page = 3, 300, 8, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    for D in (64, 128):
        k, v = (torch.randn(60, page, Hk, D, device="cuda", generator=g).bfloat16() for _ in range(2))
        q = torch.randn(B * 3, Hq, D, device="cuda", generator=g).bfloat16()
        table = torch.arange(B * 19, device="cuda", dtype=torch.int32).view(B, 19)
        lens, nd = (torch.full((B,), x, device="cuda", dtype=torch.int32) for x in (L, 2))
        ws = torch.zeros(sv.sv_attention_workspace_bytes(D), dtype=torch.uint8, device="cuda")
        out, again = torch.empty_like(q), torch.empty_like(q)
        call = lambda o: sv.spec_attention(q, k, v, table, lens, nd, None, 2, D ** -0.5, 0, 0, o, None, ws)
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
