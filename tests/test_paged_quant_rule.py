"""The FP8 append divides by Markstein's method (paged_cache.cu: r = RN(1 / s), q = RN(x r),
RN(q + r RN(x - q s))) where the rule divides in fp32.  The two quotients can differ only where x / s
is next to the middle of two floats, and their E4M3 codes only where that middle is next to a border
between codes (a number of five bits): x = M s (1 +- about 2^-24), which for 24-bit x asks for s
within 2 ulp of a multiple of 2^-3 of its binade.  All of those, in exact arithmetic: there the two quotients
are one.  CPU only."""
import random
from fractions import Fraction as F


def rn(v, bits=24):
    """v to the nearest number of `bits` significant bits, ties to even."""
    if v == 0:
        return F(0)
    a, e = abs(v), 0
    while a >= 2:
        a, e = a / 2, e + 1
    while a < 1:
        a, e = a * 2, e - 1
    n = a * 2 ** (bits - 1)
    lo = n.numerator // n.denominator
    r = n - lo
    if r > F(1, 2) or (r == F(1, 2) and lo & 1):
        lo += 1
    return (1 if v > 0 else -1) * F(lo, 2 ** (bits - 1)) * F(2) ** e


def quotient(x, s):
    r = rn(1 / s)
    q = rn(x * r)
    return rn(q + r * rn(x - q * s))


def same(x, s):
    return rn(x / s) == quotient(x, s)


def test_every_quotient_next_to_a_border_of_codes():
    n = 0
    for k in range(8, 17):
        for ds in range(-3, 4):
            S = k * 2 ** 20 + ds
            if not 2 ** 23 <= S < 2 ** 24:
                continue
            for M in range(16, 32):
                T = F(S * M, 16)  # x = X 2^e with x / s = M / 16 (2^e chosen for 24 bits)
                e = 0
                while T >= 2 ** 24:
                    T, e = T / 2, e + 1
                for X in range(int(T) - 4, int(T) + 6):
                    if 2 ** 23 <= X < 2 ** 24:
                        n += 1
                        assert same(F(X) * 2 ** e, F(S)), (S, M, X)
    assert n > 5000


def test_random_quotients():
    g = random.Random(1)
    for _ in range(3000):
        S = g.randrange(2 ** 23, 2 ** 24)
        # a bf16 value, any fp32 value, and one next to a border
        for X in (F(g.randrange(128, 256)), F(g.randrange(2 ** 23, 2 ** 24)), F(int(F(S * g.randrange(16, 32), 16)) + g.randrange(-2, 3))):
            if X < 2 ** 24:
                assert same(X, F(S))
