"""The routing's own 64-bit exponential (csrc/experts.cu, exp_64), its steps carried out on the host with the source's numbers,
against 40 digits."""
import os
import re
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "sparse_embeddings_feature_gb300", "csrc", "experts.cu")


def _source():
    text = open(SOURCE).read()
    at = text.index("kPowers[64]")
    table = [float(v) for v in re.findall(r"\d+\.\d+(?:e-?\d+)?", text[at:text.index("};", at)])]
    body = text[text.index("double exp_64(double x)"):]
    down = body[body.index("double exp_64_down(double x)"):]
    body, down = body[:body.index("\n}\n")], down[:down.index("\n}\n")]
    per = float(re.search(r"shifted = x \* ([\d.]+)", body).group(1))
    less = [float(v) for v in re.findall(r"fma\(k, (-[\d.e-]+), [xr]\)", body)]
    assert "x < -700.0 ? exp_64(x + 700.0) *" in down
    tiny = float(re.search(r"\* ([\d.e-]+) : exp_64\(x\)", down).group(1))
    low, high = (float(v) for v in re.search(r"fmax\(x, (-[\d.]+)\), ([\d.]+)\)", body).groups())
    return table, per, less, tiny, low, high


def _fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def _exp(x, table, per, less, tiny, low, high):
    small = x < -700.0
    x = min(max(x + 700.0 if small else x, low), high)
    k = float(np.float64(x * per + 1.5 * 2.0 ** 52) - 1.5 * 2.0 ** 52)
    n = int(k)
    r = _fma(k, less[1], _fma(k, less[0], x))
    p = _fma(r, 1 / 120, 1 / 24)
    for c in (1 / 6, 0.5, 1.0):
        p = _fma(p, r, c)
    p *= r
    y = _fma(table[n & 63], p, table[n & 63])
    z = float(np.ldexp(y, n >> 6))
    return z * tiny if small else z


def test_the_tables_are_powers_of_two():
    getcontext().prec = 40
    table, per, less, tiny, _, _ = _source()
    ln2 = Decimal(2).ln()
    assert len(table) == 64 and len(less) == 2
    for j, v in enumerate(table):
        assert v == float((ln2 * j / 64).exp())
    assert abs(Decimal(per) - 64 / ln2) <= Decimal(2) ** -46          # half a last place of 92
    assert abs(Decimal(less[0]) + Decimal(less[1]) + ln2 / 64) <= Decimal(2) ** -89
    assert Fraction(less[0]).numerator.bit_length() <= 31             # its product with k is exact
    assert tiny == float(Decimal(-700).exp())


def test_the_exponential_is_within_two_last_places():
    # the table half a place, the last step half a place, p within a place of 2^-7; below e^-700 a product's half place more, and
    # half of 2^-1074 where the result is that small
    getcontext().prec = 40
    numbers = _source()
    rng = np.random.default_rng(0)
    points = np.concatenate([rng.uniform(-744.0, 709.0, 1500), rng.uniform(-1, 1, 300), rng.uniform(-745, -699, 300),
                             [0.0, -700.0, -0.0, 1e-300, 709.0]])
    for x in points.tolist():
        got, ref = Decimal(_exp(x, *numbers)), Decimal(x).exp()
        assert abs(got - ref) <= ref * Decimal(2) ** -51 + Decimal(2) ** -1074, x
    assert _exp(-np.inf, *numbers) == 0.0 and _exp(-746.0, *numbers) == 0.0 and np.isfinite(_exp(np.inf, *numbers))
