"""Inputs and error bounds shared by the GPU tests of the gated recurrence.

The bound on an fp32 result is c times the oracle's magnitude (the recursion run on absolute
values, adding at each step the terms that the step rounds), with

  c = ((1.25 S + 3) 2 + 8) 2^-24,   S = the largest |g + bias|:

the gate's exponential takes the sum s (one rounding, |s| 2^-24 relative on exp), the
product with log2 e (its rounding and the constant's, together under 1.5 |s| 2^-24), the
hardware's exp2 and reciprocal (one unit in the last place each, 2^-23) and one addition
(2^-24), so q and a are each within (2.5 S + 5) 2^-24 of themselves, rounded up to
(1.25 S + 3) 2^-23; and no step of either recursion rounds more than eight times (products
of decays over a span count once per step of the span).  A stored output adds half a step of
its type: 2^-8 relative in bf16, 2^-24 in fp32.  d_bias adds one rounding per summed term in
the worst order.
"""
import numpy as np
import torch

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def make(B, T, D, dtype, seed=0, bias=True, init=True, nseq=0, slow=3.0):
    """CPU tensors; x and g are the halves of one projection's rows (odd offsets included)."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dt = DTYPES[dtype]
    xg = rand(B, T, 2 * D + 3).to(dt)
    v = dict(xg=xg, bias=(torch.rand((D,), generator=gen) * 2 * slow - 1) if bias else None,
             init=rand(B, D) if init and not nseq else None, cu=None,
             dh=rand(B, T, D).to(dt), d_final=rand(nseq or B, D))
    if nseq:
        cuts = torch.sort(torch.randint(0, T + 1, (nseq - 1,), generator=gen)).values
        v["cu"] = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(torch.int32)
    return v


def halves(xg):
    D = (xg.shape[-1] - 3) // 2
    return xg[..., :D], xg[..., D + 3:]


def c_of(g, bias):
    s = np.abs(np.asarray(g, np.float64) + (0.0 if bias is None else bias)).max() if g.size else 0
    return ((1.25 * s + 3) * 2 + 8) * 2.0 ** -24


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(name, got, want, mag, c, half=2.0 ** -24):
    """Every element of got within c * mag + half * |want|; returns the largest share used."""
    got = n64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    lim = c * mag + half * np.abs(want) + 1e-36
    bad = ~(np.abs(got - want) <= lim)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside, first at {tuple(i)}: "
                             f"{got[tuple(i)]!r} for {want[tuple(i)]!r} +- {lim[tuple(i)]:.3g}")
    return float((np.abs(got - want) / lim).max()) if got.size else 0.0
