"""A server's verify steps with the library's own calls, from the tokens to the released pages.

A small random decoder (grouped-query attention with per-head norms and rotation, every other layer
with a sliding window and sinks) runs over a paged cache.  Each step drafts k tokens per request,
here by asking what the request would continue with and getting some of them wrong, and then:

    reserve -> per layer: append, attend -> spec_verify -> rollback -> release

Requests are greedy, so whatever the drafts are, the tokens that come out are the model's own greedy
continuation; `python examples/verify_step.py` checks them against a plain forward over the whole
sequence.  Half way, one request is forked, and the pool is compacted.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_12_gb300 import PagedCache, spec_verify, sv_read_device_error, sv_workspace_bytes  # noqa: E402


class Decoder:
    """Weights of a random decoder; `plain` is its forward over one whole sequence in fp32."""

    def __init__(self, vocab=512, layers=4, heads=8, kv_heads=2, head_dim=64, window=48, sinks=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, device=device, generator=g)
        self.vocab, self.layers, self.Hq, self.Hk, self.D = vocab, layers, heads, kv_heads, head_dim
        width = heads * head_dim
        self.embed = rand(vocab, width).bfloat16()
        self.qkv = [(rand(width, width + 2 * kv_heads * head_dim) / width ** 0.5).bfloat16() for _ in range(layers)]
        self.out = [(rand(width, width) / width ** 0.5).bfloat16() for _ in range(layers)]
        self.q_norm, self.k_norm = ([(torch.rand(head_dim, device=device, generator=g) + 0.5).bfloat16()
                                     for _ in range(layers)] for _ in range(2))
        self.inv_freq = 10000.0 ** (-torch.arange(head_dim // 2, device=device) * 2 / head_dim)
        self.windows = [window if i % 2 else 0 for i in range(layers)]
        self.sinks, self.eps, self.scale = sinks, 1e-6, head_dim ** -0.5

    def plain(self, tokens):
        """Logits [len(tokens), vocab] of one sequence, fp32 arithmetic on the bf16 weights."""
        n, D = len(tokens), self.D
        x = self.embed[tokens].float()
        pos = torch.arange(n, device=x.device)
        angle = pos[:, None].double() * self.inv_freq.double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turned(h, w):
            h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + self.eps) * w.float()
            a, z = h[..., :D // 2], h[..., D // 2:]
            return torch.cat((a * cos - z * sin, a * sin + z * cos), -1)

        for i in range(self.layers):
            q, k, v = (x @ self.qkv[i].float()).split([self.Hq * D, self.Hk * D, self.Hk * D], 1)
            q, k = turned(q.view(n, -1, D), self.q_norm[i]), turned(k.view(n, -1, D), self.k_norm[i])
            z = torch.einsum("ihgd,jhd->hgij", q.view(n, self.Hk, -1, D), k) * self.scale
            seen = pos[None] <= pos[:, None]
            if self.windows[i]:
                seen &= (pos[None] > pos[:, None] - self.windows[i]) | (pos[None] < self.sinks)
            p = z.masked_fill(~seen, -torch.inf).softmax(-1)
            o = torch.einsum("hgij,jhd->ihgd", p, v.view(n, -1, D)).reshape(n, -1)
            x = x + o @ self.out[i].float()
        return x @ self.embed.float().T / 8


class Server:
    """Greedy requests over a paged cache, k drafts a step."""

    def __init__(self, model, slots, k, pages=256, page_size=16, max_pages=32):
        self.m, self.k, self.B = model, k, slots
        self.cache = PagedCache(model.layers, slots, pages, page_size, max_pages, model.Hk, model.D)
        R, dev = slots * (k + 1), "cuda"
        self.q = torch.empty(slots * 65, model.Hq, model.D, dtype=torch.bfloat16, device=dev)   # (a prompt's rows too)
        self.attended = torch.empty_like(self.q)
        self.workspace = torch.empty(sv_workspace_bytes(slots, R, model.vocab), dtype=torch.uint8, device=dev)
        full = lambda v, t: torch.full((slots,), v, dtype=t, device=dev)
        self.params = (full(1, torch.float32), full(0, torch.int32), full(1, torch.float32), None, None, full(1, torch.uint8))
        self.uniforms = torch.zeros(R, 2, device=dev)
        self.draft_probs = torch.zeros(slots * k, model.vocab, device=dev)
        self.out_tokens = torch.empty(slots, k + 1, dtype=torch.int32, device=dev)
        self.accept_len = torch.empty(slots, dtype=torch.int32, device=dev)

    def forward(self, tokens, num_drafts, k_max):
        """Logits of the new tokens [B, k_max + 1], which are in the cache afterwards."""
        m, c = self.m, self.cache
        rows = tokens.numel()
        q, o = self.q[:rows], self.attended[:rows]
        c.reserve(num_drafts)
        x = m.embed[tokens.flatten()]
        for i in range(m.layers):
            qkv = x @ m.qkv[i]
            heads = qkv.view(rows, -1, m.D).split([m.Hq, m.Hk, m.Hk], 1)
            c.append(i, *heads, m.q_norm[i], m.k_norm[i], m.eps, m.inv_freq, num_drafts, None, k_max, q)
            c.attend(i, q, num_drafts, None, k_max, m.scale, o, m.windows[i], m.sinks)
            x = x + o.flatten(1) @ m.out[i]
        return x.float() @ m.embed.float().T / 8

    def prompt(self, tokens):
        """Prompts [B, n], n at most 65: their last token is the first row of the next step."""
        B, n = tokens.shape
        self.forward(tokens[:, :-1].contiguous(), torch.full((B,), n - 2, dtype=torch.int32, device="cuda"), n - 2)
        self.last = tokens[:, -1:]

    def step(self, drafts):
        """One verify step over drafts [B, k]; returns the new tokens of each request (-1: none)."""
        nd = torch.full((self.B,), self.k, dtype=torch.int32, device="cuda")
        logits = self.forward(torch.cat((self.last, drafts), 1), nd, self.k)
        spec_verify(logits, self.draft_probs, drafts.int().contiguous(), nd, None, self.k, *self.params, self.uniforms,
                    self.out_tokens, self.accept_len, None, self.workspace)
        self.cache.commit(self.accept_len, nd)
        self.last = self.out_tokens.long().gather(1, self.accept_len.long()[:, None])
        return self.out_tokens


def run(slots=6, prompt=20, steps=8, k=4, seed=1):
    """Runs the server; returns (sequences, the largest gap by which a chosen token's plain logit lies
    below the plain maximum, accepted drafts per step)."""
    model = Decoder()
    server = Server(model, slots, k)
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, model.vocab, (slots, prompt), device="cuda", generator=g)
    tokens[slots - 1] = tokens[0]          # the last slot will be a fork of the first: same prompt for now
    server.prompt(tokens)
    seqs = [t.tolist() for t in tokens]
    accepted = 0
    for s in range(steps):
        if s == steps // 2:
            # the last request ends; its slot continues from the first one's tokens
            server.cache.kv_seq_len[slots - 1] = 0
            server.cache.release()
            server.cache.fork(torch.tensor([0], dtype=torch.int32, device="cuda"),
                              torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
            seqs[slots - 1], server.last[slots - 1] = list(seqs[0]), server.last[0]
            server.cache.compact(64)
        # drafts: the plain continuation, with every third one wrong
        drafts = []
        for b, seq in enumerate(seqs):
            now = list(seq)
            for i in range(k):
                t = int(model.plain(torch.tensor(now, device="cuda"))[-1].argmax())
                now.append((t + 1) % model.vocab if (b + s + i) % 3 == 2 else t)
            drafts.append(now[-k:])
        out = server.step(torch.tensor(drafts, device="cuda")).tolist()
        accepted += int(server.accept_len.sum())
        for seq, new in zip(seqs, out):
            seq.extend(t for t in new if t >= 0)
    assert sv_read_device_error(server.cache.workspace) == (0, -1)
    assert sv_read_device_error(server.workspace) == (0, -1)
    lens = server.cache.kv_seq_len.tolist()
    assert lens == [len(s) - 1 for s in seqs], (lens, [len(s) for s in seqs])
    used = sum(-(-n // server.cache.page_size) for n in lens)
    held = int((server.cache.ref_count > 0).sum())
    assert held <= used and int(server.cache.ref_count.sum()) == used
    gap = 0.0
    for seq in seqs:
        z = model.plain(torch.tensor(seq, device="cuda"))[prompt - 1:-1]
        chosen = z.gather(1, torch.tensor(seq[prompt:], device="cuda")[:, None])[:, 0]
        gap = max(gap, float((z.amax(-1) - chosen).max()))
    return seqs, gap, accepted / (steps * slots)


if __name__ == "__main__":
    seqs, gap, rate = run()
    print(f"{len(seqs)} requests of {[len(s) for s in seqs]} tokens, {rate:.2f} drafts accepted a step")
    print(f"chosen tokens lie at most {gap:.4f} below the plain forward's largest logit")
