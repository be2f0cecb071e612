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


def test_idle_slots_in_a_whole_step(sv):
    """Slots without a request (num_drafts -1), empty and resting ones, from the reservation to the commit: no
    length, page or error word of theirs changes, whatever accept_len holds for them."""
    c = sv.PagedCache(1, 6, 40, 8, 8, 1, 64)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    c.reserve(ints(9, -1, 20, 3, -1, 0))
    before = c.block_table[2].tolist()
    x = torch.randn(6 * 5, 1, 64, device="cuda").bfloat16()
    for nd, acc in [(ints(4, -1, -1, 0, -1, 2), ints(2, -1, 99, 0, -1, 2)), (ints(-1, -1, -1, 4, -1, -1), ints(0, 5, 1, 0, 0, 7))]:
        out, again = torch.empty_like(x), torch.empty_like(x)
        lens = c.kv_seq_len.tolist()
        c.reserve(nd)
        c.append(0, x, x, x, None, None, 0.0, None, nd, None, 4, out)
        c.attend(0, out, nd, None, 4, 0.125, again)
        c.commit(acc, nd)
        want = [n + 1 + a if k >= 0 else n for n, k, a in zip(lens, nd.tolist(), acc.tolist())]
        assert c.kv_seq_len.tolist() == want
        assert sv.sv_read_device_error(c.workspace) == (0, -1)
    assert c.block_table[2].tolist() == before and c.kv_seq_len[2] == 21
    assert int(c.ref_count.sum()) == sum(-(-n // 8) for n in c.kv_seq_len.tolist())


def test_commit_still_reports_what_is_wrong(sv):
    """Drafts below -1, accepted drafts below 0 or above the drafts, and failed reservations keep their length."""
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for nd, acc, length in [(-2, 0, 9), (2, -1, 9), (2, 3, 9), (2, 1, -10), (8, 0, 7)]:
        c = sv.PagedCache(1, 2, 10, 8, 4, 1, 64)
        c.reserve(ints(8, 4))
        c.kv_seq_len[0] = length
        c.commit(ints(acc, 1), ints(nd, 4))
        assert c.kv_seq_len.tolist() == [length, 2] and sv.sv_read_device_error(c.workspace) == (1, 0)


def test_rollback_itself_takes_no_idle_requests(sv):
    """spec_rollback's own rule is unchanged: drafts below 0 are an error."""
    kv, acc, nd = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([9, 9], [0, 1], [-1, 3]))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.spec_rollback(kv, acc, nd, ws)
    assert kv.tolist() == [9, 7] and sv.sv_read_device_error(ws) == (1, 0)


def test_rollback_takes_what_it_always_took(sv):
    """A workspace of a few words, and none at all refused by the library, with and without compiled checks."""
    from speculative_decoding_verification_12_gb300 import cache
    for native in (True, False):
        kv, acc, nd = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([9, 9], [0, 1], [2, 3]))
        ws = torch.zeros(8, dtype=torch.uint8, device="cuda")
        if native:
            sv.spec_rollback(kv, acc, nd, ws)
        else:
            with pytest.MonkeyPatch.context() as m:
                m.setattr(cache, "_native", None)
                m.delattr(sv, "_binding", raising=False)
                m.setitem(sys.modules, "speculative_decoding_verification_12_gb300._binding", None)
                sv.spec_rollback(kv, acc, nd, ws)
        assert kv.tolist() == [7, 7]
        with pytest.raises(sv.SvError):
            sv.spec_rollback(kv, acc, nd, None)
        with pytest.raises(ValueError):
            sv.spec_rollback(kv, acc.long(), nd, ws)


def test_calls_let_other_threads_run(sv, tmp_path):
    """The compiled calls release the interpreter's lock while the library works: with a library that takes
    0.3 s, another thread goes on.  In a process of its own, whose binding keeps the slow library."""
    import subprocess
    (tmp_path / "slow.c").write_text("#include <unistd.h>\nint slow(void) { usleep(300000); return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "slow.so"), str(tmp_path / "slow.c")], check=True)
    code = f"""
import ctypes, sys, threading, time
sys.path.insert(0, {ROOT!r})
import torch
from speculative_decoding_verification_12_gb300 import cache
binding = cache._load()
slow = ctypes.CDLL({str(tmp_path / "slow.so")!r}).slow
binding.init(*[ctypes.cast(slow, ctypes.c_void_p).value] * ENTRIES, torch._C._cuda_getCurrentRawStream)
t = torch.zeros(256, dtype=torch.int32, device="cuda")
ticks, stop = [0], []
def tick():
    while not stop:
        time.sleep(0.001)
        ticks[0] += 1
thread = threading.Thread(target=tick)
thread.start()
time.sleep(0.05)
before = ticks[0]
assert binding.rollback(t, t, t, t, 0) == 0
print(ticks[0] - before)
stop.append(1)
thread.join()
"""
    from speculative_decoding_verification_12_gb300 import cache
    code = code.replace("ENTRIES", str(len(cache.ENTRIES)))
    out = subprocess.run([sys.executable, "-c", code], check=True, capture_output=True, text=True).stdout
    assert int(out) > 30


def test_a_new_cache_is_ready_for_any_stream(sv):
    """What the constructor fills is there when it returns, however busy the stream it was filled on."""
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    nd, other = ints(20, -1, 3), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)      # (about 0.1 s)
    c = sv.PagedCache(1, 3, 30, 8, 8, 1, 64)
    c.reserve(nd, other)
    other.synchronize()
    assert c.kv_seq_len.tolist() == [21, 0, 4]
    assert c.block_table.tolist() == [[0, 1, 2] + [-1] * 5, [-1] * 8, [3] + [-1] * 7]
    assert c.ref_count.tolist() == [1] * 4 + [0] * 26 and sv.sv_read_device_error(c.workspace) == (0, -1)
