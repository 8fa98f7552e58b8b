"""linear_logprobs takes many tokens in runs, and every run's shares must fit the workspace that the call asks for: a
shorter last run may take more of it than the others, since fewer tokens are cut into more shares each.  Sizes alone:
no GPU."""
import random

import pytest

import weight_only_bit_q4_amd as q

RUN, LOGITS = 128, 1 << 25  # a run holds at most 2^25 logits, or 128 tokens


def al256(b):
    return (b + 255) // 256 * 256


def run_lengths(n, t):
    most = max(RUN, LOGITS // n)
    runs = -(-t // most)
    run = -(-t // runs)
    return run, t - (runs - 1) * run


def check(n, k, t, top):
    run, last = run_lengths(n, t)
    assert 1 <= last <= run
    have = q.q4lin_linear_logprobs_workspace_bytes(n, k, t, top)
    before = al256(2 * t * k) + al256(4 * t * (k // 64)) + al256(4 * run * n)
    for c in (run, last):
        need = before + q.q4lin_logprobs_workspace_bytes(n, c, top)
        assert have >= need, "n=%d t=%d top=%d: a run of %d tokens (of %d) needs %d bytes, %d are asked for" % (
            n, t, top, c, run, need, have)


@pytest.mark.parametrize("n,t", [(131072, 293), (131072, 409), (128256, 409), (50257, 1023), (65000, 1023),
                                 (65000, 683), (256000, 137), (1 << 24, 257), (1000, 40000)])
@pytest.mark.parametrize("top", [0, 1, 20, 32])
def test_a_shorter_last_run_fits(n, t, top):
    check(n, 64, t, top)


def test_any_run_fits():
    rng = random.Random(5)
    for _ in range(4000):
        n = int(2 ** rng.uniform(5, 24))
        check(n, 64 * rng.randint(1, 40), int(2 ** rng.uniform(0, 13)), rng.randint(0, min(32, n)))
