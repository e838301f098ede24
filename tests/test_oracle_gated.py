"""The fp64 oracle of the gated recurrence and of the 8-bit checkpoints, pinned on the CPU.

The forward against its closed form (the lower-triangular matrix of decay products) and a
hand-worked example; the backward against torch's reverse mode in fp64 and against central
differences; packed rows against each sequence alone; the checkpoints against their
definition.  Tolerances: fp64 rounding of a few hundred operations (1e-11 relative), and for
differences with step 1e-5 a truncation of order 1e-10 and a rounding of order 1e-11.
"""
import numpy as np
import pytest
import torch

from oracle import gated


def inputs(B, T, D, seed=0):
    r = np.random.RandomState(seed)
    return dict(x=r.randn(B, T, D), g=2 * r.randn(B, T, D), bias=r.rand(D) * 3,
                init=r.randn(B, D), dh=r.randn(B, T, D), d_final=r.randn(B, D))


def test_four_steps_by_hand():
    """g = log 3 makes q = 1/4 and a = 3/4."""
    x = np.array([4.0, 8.0, 0.0, -4.0]).reshape(1, 4, 1)
    g = np.full((1, 4, 1), np.log(3.0))
    r = gated.gated_ref(x, g, None, np.array([[16.0]]))
    np.testing.assert_allclose(r["h"][0, :, 0], [13.0, 11.75, 8.8125, 5.609375], rtol=1e-14)
    np.testing.assert_allclose(r["final"], [[5.609375]], rtol=1e-14)


def test_forward_is_the_triangular_matrix():
    v = inputs(2, 70, 3)
    q, a = gated.gate(v["g"] + v["bias"])
    r = gated.gated_ref(v["x"], v["g"], v["bias"], v["init"])
    for b in range(2):
        for d in range(3):
            M = np.zeros((70, 70))
            for t in range(70):
                for s in range(t + 1):
                    M[t, s] = np.prod(a[b, s + 1:t + 1, d]) * q[b, s, d]
            h = M @ v["x"][b, :, d] + np.cumprod(a[b, :, d]) * v["init"][b, d]
            np.testing.assert_allclose(r["h"][b, :, d], h, rtol=1e-11, atol=1e-13)
    np.testing.assert_array_equal(r["entry"][:, 0], v["init"])
    np.testing.assert_array_equal(r["entry"][:, 1], r["h"][:, 63])


def torch_grads(v, cu=None):
    t = {k: torch.tensor(a, dtype=torch.float64, requires_grad=k in ("x", "g", "bias", "init"))
         for k, a in v.items()}
    T = v["x"].shape[1]
    first, last = (set(), {}) if cu is None else gated._sequences(cu, T)
    h = t["init"] if cu is None else torch.zeros_like(t["init"])
    loss = 0.0
    for i in range(T):
        if i in first:
            h = torch.zeros_like(h)
        q = torch.sigmoid(-(t["g"][:, i] + t["bias"]))
        h = (1 - q) * h + q * t["x"][:, i]
        loss = loss + (h * t["dh"][:, i]).sum()
        if i in last:
            loss = loss + (h[0] * t["d_final"][last[i]]).sum()
    if cu is None:
        loss = loss + (h * t["d_final"]).sum()
    loss.backward()
    return {k: t[k].grad.numpy() for k in ("x", "g", "bias", "init") if t[k].grad is not None}


@pytest.mark.parametrize("T", [1, 64, 65, 150])
def test_backward_matches_reverse_mode(T):
    v = inputs(2, T, 5, seed=T)
    r = gated.gated_ref(v["x"], v["g"], v["bias"], v["init"])
    got = gated.gated_bwd_ref(v["x"], v["g"], v["bias"], r["entry"], v["dh"], v["d_final"])
    want = torch_grads(v)
    for k, n in (("x", "dx"), ("g", "dg"), ("bias", "d_bias"), ("init", "d_init")):
        np.testing.assert_allclose(got[n], want[k], rtol=1e-11, atol=1e-12)


def test_backward_matches_differences():
    v = inputs(1, 67, 2, seed=3)

    def loss(w):
        r = gated.gated_ref(w["x"], w["g"], w["bias"], w["init"])
        return (r["h"] * w["dh"]).sum() + (r["final"] * w["d_final"]).sum()

    r = gated.gated_ref(v["x"], v["g"], v["bias"], v["init"])
    got = gated.gated_bwd_ref(v["x"], v["g"], v["bias"], r["entry"], v["dh"], v["d_final"])
    for k, n in (("x", "dx"), ("g", "dg"), ("bias", "d_bias"), ("init", "d_init")):
        flat = got[n].reshape(-1)
        for i in range(0, v[k].size, 7):
            lo, hi = dict(v), dict(v)
            lo[k], hi[k] = v[k].copy(), v[k].copy()
            lo[k].reshape(-1)[i] -= 1e-5
            hi[k].reshape(-1)[i] += 1e-5
            assert abs((loss(hi) - loss(lo)) / 2e-5 - flat[i]) < 1e-8


def test_packed_row_is_its_sequences_alone():
    cu = [0, 0, 5, 69, 69, 70, 133, 133]
    v = inputs(1, 133, 4, seed=9)
    v["d_final"] = np.random.RandomState(1).randn(7, 4)
    r = gated.gated_ref(v["x"], v["g"], v["bias"], cu=cu)
    got = gated.gated_bwd_ref(v["x"], v["g"], v["bias"], r["entry"], v["dh"], v["d_final"], cu=cu)
    want = torch_grads(v, cu)
    for k, n in (("x", "dx"), ("g", "dg"), ("bias", "d_bias")):
        np.testing.assert_allclose(got[n], want[k], rtol=1e-11, atol=1e-12)
    for s in range(7):
        i, j = cu[s], cu[s + 1]
        if i == j:
            np.testing.assert_array_equal(r["final"][s], 0.0)
            continue
        one = gated.gated_ref(v["x"][:, i:j], v["g"][:, i:j], v["bias"])
        np.testing.assert_allclose(r["h"][:, i:j], one["h"], rtol=1e-13)
        np.testing.assert_allclose(r["final"][s], one["final"][0], rtol=1e-13)


def test_checkpoint_codes_follow_their_definition():
    r = np.random.RandomState(0)
    v = (r.randn(9, 200) * np.exp(3 * r.randn(9, 1))).astype(np.float32)
    v[0, :64] = 0.0
    v[1, 3] = np.inf
    v[2, 70] = np.nan
    v[3, :64] = 2.0 ** -101
    v[4, 128:192] = np.arange(64) - 32.0    # m = 32: values at multiples of 127/32
    codes, scales = gated.ckpt_pack(v)
    assert codes.shape == v.shape and scales.shape == (9, 4) and scales.dtype == np.float32
    back = gated.ckpt_unpack(codes, scales)
    assert scales[0, 0] == 0 and not codes[0, :64].any() and not back[0, :64].any()
    assert np.isnan(scales[1, 0]) and np.isnan(back[1, :64]).all() and not codes[1, :64].any()
    assert np.isnan(back[2, 64:128]).all() and np.isfinite(back[2, :64]).all()
    assert scales[3, 0] == 0 and not back[3, :64].any()
    assert codes[4, 128] == -127 and codes[4, 128 + 32] == 0
    fine = np.isfinite(back)
    step = np.repeat(scales, 64, -1)[:, :200]
    # half a step, plus the roundings of scale, inverse and value (2^-24 each of up to 127 steps)
    lim = step * (0.5 + 3 * 127 * 2.0 ** -24)
    ok = np.abs(back.astype(np.float64) - v)[fine] <= np.where(step > 0, lim, 2.0 ** -100)[fine]
    assert ok.all()
    assert (np.abs(codes.astype(int)) <= 127).all()


def test_checkpoint_ties_go_to_even():
    v = np.zeros((1, 64), np.float32)
    v[0, :5] = [127.0, 0.5, 1.5, -2.5, 3.5]    # scale 1
    codes, scales = gated.ckpt_pack(v)
    assert scales[0, 0] == 1.0
    np.testing.assert_array_equal(codes[0, :5], [127, 0, 2, -2, 4])


def test_checkpoint_extremes_stay_finite():
    """The largest fp32 and bf16 values and the smallest group that keeps its codes."""
    for m in (np.finfo(np.float32).max, 3.3895313892515355e38, 2.0 ** -100):
        v = np.full((1, 64), m, np.float32)
        codes, scales = gated.ckpt_pack(v)
        back = gated.ckpt_unpack(codes, scales)
        assert (codes == 127).all() and np.isfinite(back).all()
        np.testing.assert_allclose(back, v, rtol=2.0 ** -22)
