"""Inputs and bounds shared by the tests of the gradients and the 4-bit operators.

Bounds. Products of two bf16 values are exact in binary32, so what a sum of n
of them in the matrix cores is off by are its additions: at most n of them,
each by at most one unit of the last place (2^-23) of a partial sum, which the
sum S of the magnitudes bounds. One more covers the start. A sum of 4-bit
values rounds less: the 32 products of a block are multiples of 1/4 scale and
add up to at most 1152 scales, exact in binary32 in any order, so only the
additions of the K / 32 block sums round.

A result rounded to bf16 once lies between the bf16 roundings of the ends of
its interval, as rounding is monotone.
"""

import numpy as np
import pytest

import oracle
import workloads as wl

ULP = 2.0 ** -23


def bits(rng, *shape, scale=1.0):
    return wl.f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def int_bits(rng, *shape, most=3):
    return wl.f32_to_bf16_bits(rng.integers(-most, most + 1, size=shape).astype(np.float32))


def offsets_of(sizes):
    return wl.offsets_from_sizes(sizes)


def sum_bound(n, S):
    return (np.asarray(n) + 1) * ULP * S


def check_f32(got, ref, err, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), "%s: non-finite output" % what
    d = np.abs(got - ref)
    bad = d > err
    assert not bad.any(), "%s: %d elements beyond their bound, the first at %s: %g for %g, bound %g" % (
        what, int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][0], ref[bad][0],
        np.broadcast_to(err, ref.shape)[bad][0])


def check_bf16(got, ref, err, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), "%s: non-finite output" % what
    bad = (got < oracle.round_to_bf16(ref - err)) | (got > oracle.round_to_bf16(ref + err))
    assert not bad.any(), "%s: %d bf16 elements outside their interval, the first at %s: %g for %g" % (
        what, int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][0], ref[bad][0])


def to_dev(x, device="cuda:0"):
    import torch
    x = np.ascontiguousarray(x)
    if x.dtype == np.uint16:
        return torch.from_numpy(x.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(x).to(device)


def host(t):
    """A device tensor as a numpy array (bf16 widened)."""
    import torch
    t = t.detach()
    return (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def bits_of(t):
    """The bf16 bit patterns of a device tensor."""
    import torch
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


SLEEP = 100_000_000  # cycles: tens of milliseconds


def beside(attempt, tries=12):
    """Runs attempt(stream) until it says that the stream and the present one ran beside
    each other. (Streams share a few hardware queues, which the runtime deals out anew as
    they fall idle: on one queue they run in turn, and the attempt shows nothing.)"""
    import torch
    for _ in range(tries):
        torch.cuda.synchronize()
        if attempt(torch.cuda.Stream()):
            return
    pytest.skip("no two streams ran beside each other")
