"""32-bit products by three bf16 parts: the parts, a bound on what the six
products of them may be off by as a whole, and inputs whose results show every one
of the products exactly.

The parts x1 + x2 + x3 are x, each of 8 bits.  A dropped product x2 y2, x1 y3 or
x3 y1 is some 2^-19 of the result's norm (a rounding to 8 bits is off by 0.38 * 2^-8
in the mean square, and so squared), 36 u of u = 2^-24.  The kernels' own error is
that of adding up: k / 32 additions of instructions at the size of the whole sum
and as many at 2^-8 and 2^-16 of it, errors of either sign, which grows as sqrt(k):
0.15 sqrt(k) u was measured for k of 64 to 4104, 1 to 2 u for short sums.  Twice
that, and 4 u, is the bound.
"""
import torch

from encoder_util import F64, U

# in the order of their size: the planes of the operands
PRODUCTS = [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)]


def whole_bound(*k):
    """Bound on ||error|| / ||result|| of sums over k one after another."""
    return (4 + 0.3 * sum(k) ** 0.5) * U


def parts(x):
    """The three bf16 parts of a 32-bit tensor, as 64-bit values."""
    out, rest = [], x.to(F64)
    for _ in range(3):
        p = rest.to(torch.bfloat16).to(F64)
        out.append(p)
        rest = rest - p
    return out


def product(x, y, but=None, held=False):
    """x @ y.T by the products of parts without ``but``; held: x is one part."""
    px, py = parts(x), parts(y)
    if held:
        px = px[:1]
    out = 0
    for p in PRODUCTS:
        if p != but and p[0] < len(px):
            out = out + px[p[0]] @ py[p[1]].t()
    return out


# Numbers whose parts are 1 and 2^-10, or 1, 2^-10 and 2^-20: times powers of two
# they show a part each, and the first of them squared, 1 + 2^-9 + 2^-20, the
# product of both second parts.  All these products are 32-bit numbers.
TWO, THREE = 1 + 2.0 ** -10, 1 + 2.0 ** -10 + 2.0 ** -20
EXACT_PAIRS = [(THREE, 1.0), (1.0, THREE), (TWO, TWO)]


def pattern(shape, value, seed, device):
    """``value`` times 1, 2 or 4."""
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.exp2(torch.randint(0, 3, shape, generator=g, device=device).float()) * value


def one_of_each_row(rows, cols, first, value, seed, device):
    """[rows, cols] with one value in each row, at a column from ``first`` on; the columns."""
    g = torch.Generator(device=device).manual_seed(seed)
    at = torch.randint(first, cols, (rows,), generator=g, device=device)
    out = torch.zeros((rows, cols), device=device)
    out[torch.arange(rows, device=device), at] = pattern((rows,), value, seed + 1, device)
    return out, at
