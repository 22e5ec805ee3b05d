"""How far results of random inputs may be off, relative to the norm.

The bounds of an element's error in the tests of the operators are for the
worst case; errors of random inputs lie far below, so that they would hide a
product that is left out or a rounding too many.  These limits are twice (float32)
or 1.1 times (bf16) what the roundings give at random.

A rounding to nearest is off by 0.42 u of the value in the root mean square (u the largest: 2^-8 in
bf16, 2^-24 in float32; 1 / sqrt(3) of it, times the mean of 1 / mantissa).  A sum of random
terms that is taken in n steps has partial sums that grow as a random walk, half its
square on average: 0.42 / sqrt(2) sqrt(n) = 0.3 sqrt(n) u.  Sums inside a matrix instruction, of few
terms: 2 u."""
import math

U32, U16 = 2.0 ** -24, 2.0 ** -8


def attend_f32(keys: int) -> float:
    """A probability: its score (D / 16 steps, at most 16, after the smaller terms: 3.2 u), the scale (2 u), the scaled
    difference of up to 8 (2.3 u), the exponential (1.2 u): 4.6 u.  Their sum, positive, over the keys / 2 of a lane: 0.24
    sqrt(keys / 2) u.  The second product in 6 keys / 16 steps: 0.3 sqrt(6 keys / 16) u."""
    return 2 * U32 * math.sqrt(4.6 ** 2 + 0.24 ** 2 * keys / 2 + 0.3 ** 2 * 6 * keys / 16)


def attend_bf16() -> float:
    """The probabilities and the result, each rounded once."""
    return 1.1 * math.sqrt(2) * 0.42 * U16


def experts_f32(H: int, I: int, fp8: bool = False) -> float:
    """Gate and up: 3 H / 32 steps, and for fp8 a ratio, itself rounded, every 128 k.  The hidden activation has both and 2 u
    for exponential and reciprocal; the output keeps that and its own sum's, the result a rounding."""
    def total(k):
        return math.sqrt((0.3 * math.sqrt(3 * k / 32)) ** 2 + 2 ** 2 + (2 * (0.3 * math.sqrt(k / 128)) ** 2 if fp8 else 0))
    hidden = math.sqrt(2 * (1.1 * total(H)) ** 2 + 2 ** 2)
    return 2 * U32 * math.sqrt(hidden ** 2 + total(I) ** 2 + 1)


def experts_bf16() -> float:
    """The hidden activations and the result, each rounded once."""
    return 1.1 * math.sqrt(2) * 0.42 * U16


def off(got, ref) -> float:
    """The error's norm over the result's."""
    return float((got.double() - ref.double()).norm() / ref.double().norm())
