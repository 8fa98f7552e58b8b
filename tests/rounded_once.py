"""That a result is its exact value rounded once to bf16: its error, all
elements together, against that of the rounding alone.

A value of 16 or more significant bits that is stored in 8 adds nothing that
shows: 2^-17 of it against the store's 2^-9 on average.  A value that has been
rounded to bf16 on the way adds an error of its own of the store's size times
its part of the result, and independent errors add in squares: sqrt(2) of the
store's where all of the result went through it, sqrt(1.5) = 1.22 where half
of its variance did.  1.1 lies between; weights rounded to fp16 (1/8 of the
store's error) stay below it at 1.01.  The norms' own spread over a thousand
or more elements is 1.5 % at most.
"""
import torch

LIMIT = 1.1


def error_ratio(got, want):
    """|got - want| / |bf16(want) - want| over all elements (want in 64 bits)."""
    got = got.double().cpu()
    own = (want.float().bfloat16().double() - want).norm()
    return float((got - want).norm() / own)


def rounded_once(got, want, what):
    assert want.numel() >= 1000 and torch.isfinite(want).all()
    ratio = error_ratio(got, want)
    assert ratio <= LIMIT, "%s: %.3f times the error of one rounding" % (what, ratio)
