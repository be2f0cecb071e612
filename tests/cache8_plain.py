"""Plain 64-bit implementations of the 8-bit cache's operators, on CPU tensors, for the tests."""
import math

import torch

import cache_plain as plain

E4M3 = torch.float8_e4m3fn
LEAST, MOST, TOP = 2.0 ** -40, 2.0 ** 40, 448.0

# every e4m3 number that is finite, ascending
NUMBERS = sorted({s * (1 + m / 8) * 2.0 ** (e - 7) if e else s * m * 2.0 ** -9
                  for s in (-1, 1) for e in range(16) for m in range(8) if (e, m) != (15, 7)})


def clean(s):
    """A stored scale as it counts."""
    s = float(s)
    return LEAST if math.isnan(s) else min(max(s, LEAST), MOST)


def scale_for(amax):
    """The least power of two s in [LEAST, MOST] with amax <= 448 s."""
    k = -40
    while amax > TOP * 2.0 ** k and k < 40:
        k += 1
    return 2.0 ** k


def held(data, scales):
    """The numbers that a cache [pages, slots, heads, D] with scales [pages, blocks, heads] stands for."""
    n = data.view(torch.uint8).view(E4M3).double()
    s = scales.double().nan_to_num(LEAST).clamp(LEAST, MOST)
    return n * s.repeat_interleave(data.shape[1] // scales.shape[1], 1)[..., None]


def attention(q, k_cache, v_cache, k_scale, v_scale, *rest):
    return plain.attention(q, held(k_cache, k_scale), held(v_cache, v_scale), *rest)


def smallest(q, k_cache, v_cache, k_scale, v_scale, table, lens, num_drafts, row_offsets, k_max, scale, window, sinks):
    """For each output, the largest weight times its value's scale, times the sum of the magnitudes of the numbers that
    the row sees: an error of e times the largest weight in each of them moves the output by up to e of this."""
    R, Hq, D = q.shape
    P, Hk = k_cache.shape[1], k_cache.shape[2]
    k, one = held(k_cache, k_scale), held(v_cache, torch.ones_like(v_scale))
    s = v_scale.double().nan_to_num(LEAST).clamp(LEAST, MOST).repeat_interleave(P // v_scale.shape[1], 1)
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    for b, row, n, L in plain.spans(num_drafts, row_offsets, lens, k_max):
        for i in range(n):
            j = torch.tensor(plain.visible(L - n + i, window, sinks))
            page, slot = table[b][j // P].long(), j % P
            z = scale * torch.einsum("hgd,jhd->hgj", q[row + i].double().view(Hk, Hq // Hk, D), k[page, slot])
            w = (torch.softmax(z, -1) * s[page, slot].T[:, None]).amax(-1)
            out[row + i] = (w[..., None] * one[page, slot].abs().sum(0)[:, None]).reshape(Hq, D)
    return out


def append(q, k, v, q_weight, k_weight, eps, inv_freq, k_cache, v_cache, k_scale, v_scale, table, lens, num_drafts,
           row_offsets, k_max, interleaved=False, rope_scale=1.0):
    """(q, its errors' magnitudes) in float64, and for keys and values a list of blocks:
    (page, block, head, [scales that fp32 arithmetic may choose], older tokens' stored numbers, new elements in
    float64 and their errors' magnitudes)."""
    P, T = k_cache.shape[1], k_cache.shape[1] // k_scale.shape[1]
    wide = (torch.zeros(k_cache.shape, dtype=torch.float64) for _ in range(2))
    out, kc, vc, out_size, kc_size = plain.append(q, k, v, q_weight, k_weight, eps, inv_freq, *wide, table, lens,
                                                  num_drafts, row_offsets, k_max, interleaved, rope_scale)
    sides = []
    for data, scales, new, size in ((k_cache, k_scale, kc, kc_size), (v_cache, v_scale, vc, torch.zeros_like(kc_size))):
        numbers = data.view(torch.uint8).view(E4M3).double()
        blocks = []
        for b, row, n, L in plain.spans(num_drafts, row_offsets, lens, k_max):
            for block in range((L - n) // T, (L - 1) // T + 1):
                page, sub = int(table[b, block * T // P]), block % (P // T)
                lo, hi = max(L - n, block * T), min(L, (block + 1) * T)
                slots, before = slice(lo % P, (hi - 1) % P + 1), slice(sub * T, lo % P)
                older = lo - block * T
                for h in range(data.shape[2]):
                    x, e = new[page, slots, h], 2.0 ** -20 * size[page, slots, h]
                    finite = x.abs() < math.inf
                    tops = [max([0.0] + (x.abs() + f * e)[finite].tolist()) for f in (-1, 1)]
                    had = clean(scales[page, sub, h]) if older else 0.0
                    may = sorted({max(had, scale_for(t)) for t in tops})
                    blocks.append((page, sub, h, may, had, numbers[page, before, h] if older else numbers[page, :0, h], slots, x, e))
        sides.append(blocks)
    return out, out_size, sides


def nearest(x):
    """The e4m3 number nearest to a float64 within its range, ties to even."""
    if math.isnan(x):
        return x
    m, e = math.frexp(abs(x))
    step = 2.0 ** (max(e, -5) - 4)
    return math.copysign(round(abs(x) / step) * step, x)
