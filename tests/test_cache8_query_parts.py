"""How many bits of a query spec_attention8 keeps, by arithmetic alone (no GPU): every 16-bit number goes through the
splitting into 8-bit parts beside row maxima of every fraction, and the bounds that come out are those the interface states."""
import math
import os
import re

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"SV_BF16": (torch.bfloat16, 1), "SV_F16": (torch.float16, 2)}      # and the parts after the first


def rest(x, top, dt, parts):
    """What the parts of elements x (float64) leave of them in a row whose largest magnitude is top."""
    m, e = math.frexp(top)                        # 448 = 0.875 * 2^9
    k = max(e - 9 + (m > 0.875), -126)
    assert 448 * 2.0 ** k >= top and (top > 224 * 2.0 ** k or k == -126)
    x = x * 2.0 ** -k
    left = x - x.float().to(torch.float8_e4m3fn).double()
    for _ in range(parts):
        half = left.half()
        assert bool(((half.double() - left).abs() <= 2.0 ** -25).all())   # (the rest has few bits, but for what is tiny)
        left = left - half.float().to(torch.float8_e5m2).double()
    return left.abs() * 2.0 ** k


def tops(dt):
    if dt == torch.float16:
        return [n * 2.0 ** e for e in (-5, 5) for n in range(1024, 2048, 17)] + [2047 * 2.0 ** 5, 2.0 ** -24, 449 * 2.0 ** -10]
    return [n * 2.0 ** e for e in (-8, 120, -127) for n in range(128, 256)] + [n * 2.0 ** -133 for n in (1, 3, 100, 255)]


@pytest.mark.parametrize("name", TYPES)
def test_the_bounds_that_the_interface_states(name):
    dt, parts = TYPES[name]
    with open(os.path.join(ROOT, "include", "spec_cache.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    whole = 2.0 ** float(re.search(r"exact for elements from 2\^(-[\d.]+) of the row's largest on", text).group(1))
    off = 2.0 ** float(re.search(r"2\^(-[\d.]+) \(%s" % name, text[text.index("smaller ones are off"):]).group(1))
    x = torch.arange(0, 1 << 15).to(torch.int16).view(dt).double()
    x = x[x.isfinite()]
    worst = 0.0
    for top in tops(dt):
        assert float(torch.tensor(top).to(dt)) == top
        y = x[x <= top]
        left = rest(y, top, dt, parts) / top
        assert not bool(left[y >= whole * top].any()), top
        assert float(left.max()) <= off, (top, math.log2(float(left.max())))
        worst = max(worst, float(left.max()))
    assert worst > off / 1.05        # (and is reached)
