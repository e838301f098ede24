"""The gated recurrence on the GPU against the fp64 oracle: forward, backward, single step,
8-bit checkpoints in between, packed rows, strides, graphs, streams.  Bounds: gated_cases."""
import numpy as np
import pytest
import torch

from gated_cases import DTYPES, HALF_STEP, c_of, check, halves, make, n64
from mamba_ssd_chunked_03_amd import binding
from oracle import gated
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    binding.library()


def cuda(v):
    return {k: None if t is None else t.cuda() for k, t in v.items()}


def forward(d, saved=None, **kw):
    x, g = halves(d["xg"])
    return binding.ssd_gated_fwd(x, g, d["bias"], init_state=d["init"], cu_seqlens=d["cu"],
                                 saved=saved, **kw)


def reference(v):
    x, g = (n64(t) for t in halves(v["xg"]))
    cu = None if v["cu"] is None else v["cu"].tolist()
    return x, g, n64(v["bias"]), cu, gated.gated_ref(x, g, n64(v["bias"]), n64(v["init"]), cu)


SHAPES = [  # B, T, D: one step, around a chunk's and a tile's borders, odd widths, long
    (1, 1, 1), (3, 1, 64), (2, 2, 7), (1, 63, 65), (2, 64, 64), (1, 65, 130), (5, 127, 33),
    (1, 128, 66), (2, 255, 100), (1, 256, 64), (1, 257, 192), (2, 513, 1001), (1, 1025, 20),
    (1, 2049, 256), (1, 5003, 48), (300, 3, 5),
    # chains that the tile counters share out evenly, nearly, or not at all
    (9, 50, 64), (7, 300, 64), (63, 20, 40), (3, 700, 576), (67, 260, 8), (1, 400, 3000),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward_and_backward(B, T, D, dtype):
    v = make(B, T, D, dtype, seed=B + T + D, bias=D % 2 == 1 or T > 100, init=T % 2 == 1)
    say(f"[gated] B={B} T={T} D={D} {dtype}")
    x, g, bias, _, r = reference(v)
    d = cuda(v)
    saved = binding.ssd_gated_saved(halves(d["xg"])[0])
    h, final = forward(d, saved)
    c, half = c_of(g, bias), HALF_STEP[dtype]
    used = [check("h", h, r["h"], r["h_mag"], c, half),
            check("final", final, r["final"], r["final_mag"], c),
            check("entry", saved["entry_states"], r["entry"], r["entry_mag"], c)]
    # the backward from the states that were saved
    want = gated.gated_bwd_ref(x, g, bias, n64(saved["entry_states"]), n64(v["dh"]),
                               n64(v["d_final"]))
    xd, gd = halves(d["xg"])
    out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, d_final=d["d_final"])
    used += check_grads(out, want, c, half, B * T)
    say("    share of the bound used: " + " ".join(f"{u:.3f}" for u in used))


def check_grads(out, want, c, half, terms):
    used = [check(k, out[k], want[k], want[k + "_mag"], c, half) for k in ("dx", "dg")]
    used.append(check("d_bias", out["d_bias"], want["d_bias"], want["d_bias_mag"],
                      c + terms * 2.0 ** -24))
    if out["d_init"] is not None:
        used.append(check("d_init", out["d_init"], want["d_init"], want["d_init_mag"], c))
    return used


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,D,nseq", [(1, 3, 1), (64, 64, 2), (130, 33, 40), (700, 65, 5),
                                      (1500, 128, 9), (2050, 24, 300), (4100, 64, 2)])
def test_packed_row(T, D, nseq, dtype):
    """Sequences of every length (many empty) against the oracle, forward and backward, with
    slow gates so that a state leaking over a start would show."""
    v = make(1, T, D, dtype, seed=T + nseq, nseq=nseq, slow=5.0)
    say(f"[gated packed] T={T} D={D} nseq={nseq} {dtype}")
    x, g, bias, cu, r = reference(v)
    d = cuda(v)
    saved = binding.ssd_gated_saved(halves(d["xg"])[0])
    h, final = forward(d, saved)
    c, half = c_of(g, bias), HALF_STEP[dtype]
    check("h", h, r["h"], r["h_mag"], c, half)
    check("final", final, r["final"], r["final_mag"], c)
    check("entry", saved["entry_states"], r["entry"], r["entry_mag"], c)
    want = gated.gated_bwd_ref(x, g, bias, n64(saved["entry_states"]), n64(v["dh"]),
                               n64(v["d_final"]), cu)
    xd, gd = halves(d["xg"])
    out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, d_final=d["d_final"],
                                cu_seqlens=d["cu"])
    assert out["d_init"] is None
    check_grads(out, want, c, half, T)


@pytest.mark.parametrize("nseq", [0, 3])
def test_long_row(nseq):
    """So many tiles to a chain that the carry goes over all of its levels (tiles, 16 and 256
    of them), with gates that remember hundreds of steps."""
    T, D = 67000, 5
    v = make(1, T, D, "fp32", seed=6, nseq=nseq, slow=3.5)
    x, g, bias, cu, r = reference(v)
    d = cuda(v)
    saved = binding.ssd_gated_saved(halves(d["xg"])[0])
    h, final = forward(d, saved)
    c = c_of(g, bias)
    check("h", h, r["h"], r["h_mag"], c)
    check("final", final, r["final"], r["final_mag"], c)
    check("entry", saved["entry_states"], r["entry"], r["entry_mag"], c)
    want = gated.gated_bwd_ref(x, g, bias, n64(saved["entry_states"]), n64(v["dh"]),
                               n64(v["d_final"]), cu)
    xd, gd = halves(d["xg"])
    out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, d_final=d["d_final"],
                                cu_seqlens=d["cu"])
    check_grads(out, want, c, 2.0 ** -24, T)


def test_every_call_on_a_stream_of_its_own():
    """The stream argument: outputs and workspaces made inside belong to that stream."""
    v = make(2, 700, 130, "bf16", seed=13)
    d = cuda(v)
    xd, gd = halves(d["xg"])

    def run(**kw):
        saved = binding.ssd_gated_saved(xd, ckpt=True)
        torch.cuda.synchronize()
        h, final = forward(d, saved, **kw)
        a = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, d_final=d["d_final"], **kw)
        b = binding.ssd_gated_bwd_ckpt(d["bias"], d["dh"], saved, d_final=d["d_final"], **kw)
        y = binding.ssd_gated_step(xd[:, 0], gd[:, 0], d["bias"], final, **kw)
        torch.cuda.synchronize()
        return [h, final, y, *(o[k] for o in (a, b) for k in ("dx", "dg", "d_bias", "d_init"))]

    want = run()
    got = run(stream=torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("cu", [[0, 64, 128, 192, 256, 320], [0, 0, 0, 256, 256, 512, 512],
                                [0, 255, 256, 257, 511, 513, 600]])
def test_packed_starts_on_borders(cu):
    T = cu[-1]
    v = make(1, T, 70, "fp32", seed=T, nseq=len(cu) - 1, slow=5.0)
    v["cu"] = torch.tensor(cu, dtype=torch.int32)
    x, g, bias, _, r = reference(v)
    d = cuda(v)
    saved = binding.ssd_gated_saved(halves(d["xg"])[0])
    h, final = forward(d, saved)
    c = c_of(g, bias)
    check("h", h, r["h"], r["h_mag"], c)
    check("final", final, r["final"], r["final_mag"], c)
    want = gated.gated_bwd_ref(x, g, bias, n64(saved["entry_states"]), n64(v["dh"]), None, cu)
    xd, gd = halves(d["xg"])
    out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, cu_seqlens=d["cu"])
    check_grads(out, want, c, 2.0 ** -24, T)


@pytest.mark.parametrize("nseq", [0, 6])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(2, 1, 5), (1, 64, 64), (2, 300, 130), (1, 1111, 97),
                                   (3, 515, 256)])
def test_training_pass_with_8_bit_inputs(B, T, D, dtype, nseq):
    """The forward's codes are ssd_ckpt_pack's, and the backward is the formula at the values
    they stand for, restarted from the forward's states at every chunk."""
    B = 1 if nseq else B
    v = make(B, T, D, dtype, seed=T, nseq=nseq)
    x, g, bias, cu, r = reference(v)
    d = cuda(v)
    xd, gd = halves(d["xg"])
    saved = binding.ssd_gated_saved(xd, ckpt=True)
    h, final = forward(d, saved)
    c, half = c_of(g, bias), HALF_STEP[dtype]
    check("h", h, r["h"], r["h_mag"], c, half)
    check("final", final, r["final"], r["final_mag"], c)
    values = []
    for n, t, src in (("x", xd, x), ("g", gd, g)):
        codes, scales = binding.ssd_ckpt_pack(t)
        assert torch.equal(saved[n + "_codes"], codes) and torch.equal(saved[n + "_scales"], scales)
        want_codes, want_scales = gated.ckpt_pack(src)
        assert np.array_equal(codes.cpu().numpy(), want_codes)
        assert np.array_equal(scales.cpu().numpy(), want_scales)
        values.append(gated.ckpt_unpack(want_codes, want_scales).astype(np.float64))
    want = gated.gated_bwd_ref(*values, bias, n64(saved["entry_states"]), n64(v["dh"]),
                               n64(v["d_final"]), cu)
    out = binding.ssd_gated_bwd_ckpt(d["bias"], d["dh"], saved, d_final=d["d_final"],
                                     cu_seqlens=d["cu"])
    check_grads(out, want, c_of(values[1], bias), half, B * T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("batch,D", [(1, 1), (1, 1536), (7, 65), (64, 1001), (513, 256)])
def test_single_steps_continue_a_forward(batch, D, dtype):
    """Three steps from a forward's final state are three steps of the oracle's recurrence."""
    v = make(batch, 5, D, dtype, seed=D)
    x, g, bias, _, r = reference(v)
    d = cuda(v)
    xd, gd = halves(d["xg"])
    h, state = binding.ssd_gated_fwd(xd[:, :2].contiguous(), gd[:, :2].contiguous(), d["bias"],
                                     init_state=d["init"])
    c, half = c_of(g, bias), HALF_STEP[dtype]
    check("h", h, r["h"][:, :2], r["h_mag"][:, :2], c, half)
    for t in range(2, 5):
        y = binding.ssd_gated_step(xd[:, t], gd[:, t], d["bias"], state)
        check("step", y, r["h"][:, t], r["h_mag"][:, t], c, half)
    check("state", state, r["final"], r["final_mag"], c)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_outputs_as_column_ranges_leave_the_rest(dtype):
    B, T, D = 2, 333, 77
    v = make(B, T, D, dtype, seed=5)
    d = cuda(v)
    xd, gd = halves(d["xg"])
    saved = binding.ssd_gated_saved(xd)
    forward(d, saved)
    plain = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved)
    wide = torch.full((B, T, 2 * D + 9), 7.0, dtype=DTYPES[dtype], device="cuda")
    dhw = torch.zeros((B, T, D + 5), dtype=DTYPES[dtype], device="cuda")
    dhw[..., 1:D + 1] = d["dh"]
    binding.ssd_gated_bwd(xd, gd, d["bias"], dhw[..., 1:D + 1], saved,
                          out=dict(dx=wide[..., 1:D + 1], dg=wide[..., D + 4:2 * D + 4]))
    assert torch.equal(wide[..., 1:D + 1], plain["dx"])
    assert torch.equal(wide[..., D + 4:2 * D + 4], plain["dg"])
    rest = torch.cat([wide[..., :1], wide[..., D + 1:D + 4], wide[..., 2 * D + 4:]], -1)
    assert bool((rest == 7.0).all())


def test_aligned_and_unaligned_rows_agree():
    """Contiguous tensors and column ranges at odd offsets give the same bits."""
    v = make(2, 300, 128, "bf16", seed=11)
    d = cuda(v)
    xd, gd = halves(d["xg"])
    a, fa = binding.ssd_gated_fwd(xd, gd, d["bias"])
    b, fb = binding.ssd_gated_fwd(xd.contiguous(), gd.contiguous(), d["bias"])
    assert torch.equal(a, b) and torch.equal(fa, fb)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_extreme_gates(dtype):
    """Gates that close or open entirely, beyond where exp over- and underflows."""
    B, T, D = 1, 300, 64
    v = make(B, T, D, dtype, seed=2, bias=False)
    x, g = halves(v["xg"])
    g[:, :, :16] = 200.0      # the state never changes
    g[:, :, 16:32] = -200.0   # the state is the input
    g[:, 100:200, 32:48] = 60.0
    _, gn, bias, _, r = reference(v)
    d = cuda(v)
    xd, gd = halves(d["xg"])
    saved = binding.ssd_gated_saved(xd)
    h, final = forward(d, saved)
    half = HALF_STEP[dtype]
    # |s| = 200 is outside the range where c holds; there q is exactly 0 or 1
    c = c_of(np.clip(gn, -60, 60), None)
    check("h", h, r["h"], r["h_mag"], c, half)
    assert torch.equal(final[:, :16], d["init"][:, :16])
    want = gated.gated_bwd_ref(n64(x), gn, None, n64(saved["entry_states"]), n64(v["dh"]))
    out = binding.ssd_gated_bwd(xd, gd, None, d["dh"], saved)
    for k in ("dx", "dg"):
        check(k, out[k], want[k], want[k + "_mag"], c, half)
    assert bool(torch.isfinite(out["d_bias"]).all())


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_stay_in_their_channel_and_sequence(bad, ckpt):
    T, D, cu = 900, 130, [0, 300, 301, 650, 900]
    v = make(1, T, D, "bf16", seed=4, nseq=4)
    v["cu"] = torch.tensor(cu, dtype=torch.int32)

    def run(w):
        d = cuda(w)
        xd, gd = halves(d["xg"])
        saved = binding.ssd_gated_saved(xd, ckpt=ckpt)
        h, final = forward(d, saved)
        if ckpt:
            out = binding.ssd_gated_bwd_ckpt(d["bias"], d["dh"], saved, cu_seqlens=d["cu"])
        else:
            out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, cu_seqlens=d["cu"])
        return [t.float().cpu() for t in (h, final, out["dx"], out["dg"], out["d_bias"])]

    clean = run(v)
    w = dict(v, xg=v["xg"].clone())
    halves(w["xg"])[0][0, 400, 70] = bad  # sequence 2, channel 70
    dirty = run(w)
    group = slice(64, 128) if ckpt else slice(70, 71)  # 8 bits: the group shares a scale
    assert not torch.isfinite(dirty[0][0, 400:650, 70]).any()
    assert not torch.isfinite(dirty[1][2, 70])
    for t in (dirty[0], clean[0]):
        t[0, 400:650, 70] = 0
    for t in (dirty[1], clean[1]):
        t[2, 70] = 0
    assert torch.equal(dirty[0], clean[0]) and torch.equal(dirty[1], clean[1])
    for k in (2, 3):
        for t in (dirty[k], clean[k]):
            t[0, 301:650, group] = 0
        assert torch.equal(dirty[k], clean[k])
    for t in (dirty[4], clean[4]):
        t[group] = 0
    assert torch.equal(dirty[4], clean[4])


def test_no_steps_and_no_channels():
    init, dfin = torch.randn(3, 5).cuda(), torch.randn(3, 5).cuda()
    x = torch.zeros(3, 0, 5, device="cuda")
    h, final = binding.ssd_gated_fwd(x, x, init_state=init)
    assert h.shape == x.shape and torch.equal(final, init)
    assert not binding.ssd_gated_fwd(x, x)[1].any()
    saved = binding.ssd_gated_saved(x)
    out = binding.ssd_gated_bwd(x, x, None, x, saved, d_final=dfin)
    assert torch.equal(out["d_init"], dfin) and not out["d_bias"].any()
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    h, final = binding.ssd_gated_fwd(x[:1], x[:1], cu_seqlens=cu)
    assert final.shape == (3, 5) and not final.any()
    for shape in ((0, 9, 5), (2, 9, 0)):
        x = torch.zeros(shape, device="cuda")
        h, _ = binding.ssd_gated_fwd(x, x)
        out = binding.ssd_gated_bwd(x, x, None, x, binding.ssd_gated_saved(x))
        assert h.shape == shape and not out["d_bias"].any()
    e = torch.zeros(0, 5, device="cuda")
    assert binding.ssd_gated_step(e, e, None, e.clone()).shape == (0, 5)


def test_gradient_along_a_direction_matches_differences():
    """<gradient, u> against central differences of the GPU's own loss: truncation of order
    e^2 and the fp32 rounding of h (2^-24 of each term) over 2 e, both under the bound."""
    B, T, D, e = 1, 400, 64, 2.0 ** -7
    v = make(B, T, D, "fp32", seed=8)
    d = cuda(v)
    xd, gd = (t.contiguous() for t in halves(d["xg"]))
    saved = binding.ssd_gated_saved(xd)

    def loss(x, g, bias, init):
        h, final = binding.ssd_gated_fwd(x, g, bias, init_state=init)
        return float((h.double() * d["dh"].double()).sum()
                     + (final.double() * d["d_final"].double()).sum())

    binding.ssd_gated_fwd(xd, gd, d["bias"], init_state=d["init"], saved=saved)
    out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, d_final=d["d_final"])
    at = [xd, gd, d["bias"], d["init"]]
    torch.manual_seed(0)
    for i, k in enumerate(("dx", "dg", "d_bias", "d_init")):
        u = torch.randn_like(at[i]).sign()
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - e * u, at[i] + e * u
        slope = (loss(*hi) - loss(*lo)) / (2 * e)
        want = float((out[k].double() * u.double()).sum())
        # each of the B*T*D terms of the loss: |third derivative| e^2 / 6 and 2^-22 / e of
        # values of order 1, added at random signs (times 8)
        lim = 8 * (B * T * D) ** 0.5 * (e * e + 2.0 ** -22 / e)
        say(f"    {k}: {slope:.6f} by differences, {want:.6f} (bound {lim:.3g})")
        assert abs(slope - want) <= lim


@pytest.mark.parametrize("nseq", [0, 5])
def test_bitwise_reproducible(nseq):
    v = make(1 if nseq else 4, 3000, 320, "bf16", seed=1, nseq=nseq)
    d = cuda(v)
    xd, gd = halves(d["xg"])
    first = None
    for _ in range(4):
        saved = binding.ssd_gated_saved(xd, ckpt=True)
        h, final = forward(d, saved)
        out = binding.ssd_gated_bwd(xd, gd, d["bias"], d["dh"], saved, cu_seqlens=d["cu"])
        out8 = binding.ssd_gated_bwd_ckpt(d["bias"], d["dh"], saved, cu_seqlens=d["cu"])
        now = [h, final, *saved.values(), *(o[k] for o in (out, out8)
                                            for k in ("dx", "dg", "d_bias"))]
        if first is None:
            first = [t.clone() for t in now]
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_two_streams_with_their_own_workspaces():
    """Calls in flight at once on two streams, each with its own buffers."""
    vs = [cuda(make(2, 4000, 256, "bf16", seed=s)) for s in (1, 2)]
    want = []
    for d in vs:
        xd, _ = halves(d["xg"])
        saved = binding.ssd_gated_saved(xd)
        want.append((forward(d, saved)[0], saved["entry_states"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in vs]
    held = []
    for _ in range(5):
        for d, st in zip(vs, streams):
            saved = binding.ssd_gated_saved(halves(d["xg"])[0])
            held.append((forward(d, saved, stream=st)[0], saved["entry_states"]))
    torch.cuda.synchronize()
    for i, got in enumerate(held):
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2]))


@pytest.mark.parametrize("nseq", [0, 7])
def test_graph_of_a_training_pass(nseq):
    """Forward with checkpoints and both backwards captured and replayed on new inputs, with
    eager calls of the same operators in between, on their own and on the graph's buffers."""
    B, T, D = 1 if nseq else 2, 1500, 192
    srcs = [cuda(make(B, T, D, "bf16", seed=s, nseq=nseq)) for s in (1, 2)]
    cap = {k: None if t is None else t.clone() for k, t in srcs[0].items()}
    xd, gd = halves(cap["xg"])
    saved = binding.ssd_gated_saved(xd, ckpt=True)
    ws = binding.ssd_gated_workspace(xd)
    h, final = torch.empty_like(cap["dh"]), torch.empty_like(cap["d_final"])
    outs = [dict(dx=torch.empty_like(h), dg=torch.empty_like(h),
                 d_bias=torch.empty(D, device="cuda"),
                 d_init=None if nseq else torch.empty(B, D, device="cuda")) for _ in range(2)]

    def call():
        kw = dict(cu_seqlens=cap["cu"], workspace=ws, check_cu_seqlens=False)
        binding.ssd_gated_fwd(xd, gd, cap["bias"], init_state=cap["init"], saved=saved, h=h,
                              final_state=final, **kw)
        binding.ssd_gated_bwd(xd, gd, cap["bias"], cap["dh"], saved, d_final=cap["d_final"],
                              out=outs[0], **kw)
        binding.ssd_gated_bwd_ckpt(cap["bias"], cap["dh"], saved, d_final=cap["d_final"],
                                   out=outs[1], **kw)

    results = [h, final, *saved.values(),
               *(t for o in outs for t in o.values() if t is not None)]

    def load(src):
        for k, t in cap.items():
            if t is not None:
                t.copy_(src[k])

    refs = []
    for src in srcs:
        load(src)
        call()
        torch.cuda.synchronize()
        refs.append([t.clone() for t in results])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep, k in enumerate((0, 1, 0, 1, 1)):
        load(srcs[k])
        for t in results:
            t.zero_()
        ws.fill_(0x5a + rep)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, refs[k])), rep
        load(srcs[1 - k])
        call()  # eager, in the same buffers
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, refs[1 - k])), rep


def test_more_than_2_to_32_elements():
    """One row past 2^32 values: the last steps against a run over those steps alone.  The
    gates forget at least half of the state per step, so after 200 steps nothing older than
    2^-200 of it is left."""
    D, T = 4096, (1 << 20) + 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((1, T, D), dtype=torch.bfloat16, device="cuda")
    g = torch.empty_like(x)
    for t in range(0, T, 1 << 17):
        x[:, t:t + (1 << 17)].normal_(generator=gen)
        g[:, t:t + (1 << 17)].uniform_(-2, 0, generator=gen)
    saved = binding.ssd_gated_saved(x)
    h, final = binding.ssd_gated_fwd(x, g, None, saved=saved)
    tail = slice(T - 44 - 256, T)  # starts on a chunk of the row
    xt, gt = x[:, tail], g[:, tail]
    ts = binding.ssd_gated_saved(xt)
    ht, ft = binding.ssd_gated_fwd(xt, gt, None, saved=ts)
    assert (T - 300) % 64 == 0
    s = c_of(np.array([2.0]), None) * 400  # magnitudes: |values| < 8 over a memory of 2 steps
    assert float((h[:, tail].float() - ht.float())[:, 200:].abs().max()) <= 8 * 2 ** -8 + s
    assert float((final - ft).abs().max()) <= s
    dh = x  # any upstream gradient
    out = binding.ssd_gated_bwd(x, g, None, dh, saved, out=dict(dx=torch.empty_like(x)))
    ot = binding.ssd_gated_bwd(xt, gt, None, dh[:, tail], saved=ts)
    for k in ("dx", "dg"):
        a, b = out[k][:, tail].float(), ot[k].float()
        assert float((a - b)[:, 200:].abs().max()) <= 64 * 2 ** -8 + s
    # the first steps do not depend on the last ones
    xh, gh = x[:, :640], g[:, :640]
    hs = binding.ssd_gated_saved(xh)
    hh, _ = binding.ssd_gated_fwd(xh, gh, None, saved=hs)
    oh = binding.ssd_gated_bwd(xh, gh, None, dh[:, :640], saved=hs)
    assert float((hh.float() - h[:, :640].float()).abs().max()) <= 8 * 2 ** -8 + s
    for k in ("dx", "dg"):
        a, b = out[k][:, :640].float(), oh[k].float()
        assert float((a - b)[:, :440].abs().max()) <= 64 * 2 ** -8 + s


@pytest.mark.parametrize("nseq", [0, 9])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_small_and_large_calls_agree(dtype, nseq):
    """Rows are loaded in another way where a call has many: the same bits as for a part of its
    channels alone."""
    T, D, n = 4096, 12288 if dtype == "bf16" else 6144, 192  # 300 MB of rows or more
    v = cuda(make(1, T, D, dtype, seed=2, nseq=nseq))
    x, g = halves(v["xg"])
    part = slice(128, 128 + n)

    def run(x, g, bias, init, dh, d_final):
        saved = binding.ssd_gated_saved(x, ckpt=True)
        kw = dict(cu_seqlens=v["cu"])
        res = [*binding.ssd_gated_fwd(x, g, bias, init_state=init, saved=saved, **kw)]
        bare = binding.ssd_gated_saved(x)
        res += [*binding.ssd_gated_fwd(x, g, bias, init_state=init, saved=bare, **kw)]
        for o in (binding.ssd_gated_bwd(x, g, bias, dh, saved, d_final=d_final, **kw),
                  binding.ssd_gated_bwd_ckpt(bias, dh, saved, d_final=d_final, **kw)):
            res += [o[k] for k in ("dx", "dg", "d_bias", "d_init") if o[k] is not None]
        return res + [saved["entry_states"], bare["entry_states"], saved["x_codes"],
                      saved["g_codes"]]

    full = (x, g, v["bias"], v["init"], v["dh"], v["d_final"])
    cols = [None if t is None else t[..., part] for t in full]
    cols[2:4] = [None if t is None else t.contiguous() for t in cols[2:4]]
    cols[5] = cols[5].contiguous()
    for a, b in zip(run(*full), run(*cols)):
        assert torch.equal(a[..., part], b)


@pytest.mark.parametrize("B,T,stride", [(3, 1, 2 ** 29 + 8), (2, 4, 2 ** 27 - 1)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_far_apart(B, T, stride, dtype):
    """Rows as far apart as their offsets inside a tile allow, inputs and gradients: the bits of
    contiguous rows, and 8-bit checkpoints of them the same."""
    D = 9
    v = make(B, T, D, dtype, seed=T)
    d = cuda(v)
    xc, gc = (t.contiguous() for t in halves(d["xg"]))
    rows = torch.empty((B * T - 1) * stride + 5 * D, dtype=DTYPES[dtype], device="cuda")
    x, g, dh, dx, dg = (rows.as_strided((B, T, D), (T * stride, stride, 1), i * D)
                        for i in range(5))
    for to, of in ((x, xc), (g, gc), (dh, d["dh"])):
        to.copy_(of)
    got, want = [], []
    for xs, gs, dhs, out, res in ((x, g, dh, dict(dx=dx, dg=dg), got),
                                  (xc, gc, d["dh"], None, want)):
        saved = binding.ssd_gated_saved(xc, ckpt=True)
        res += binding.ssd_gated_fwd(xs, gs, d["bias"], init_state=d["init"], saved=saved)
        res += saved.values()
        o = binding.ssd_gated_bwd(xs, gs, d["bias"], dhs, saved, d_final=d["d_final"], out=out)
        res += [o[k] for k in ("dx", "dg", "d_bias", "d_init")]
        o = binding.ssd_gated_bwd_ckpt(d["bias"], dhs, saved, d_final=d["d_final"])
        res += [o[k] for k in ("dx", "dg", "d_bias", "d_init")]
        state = d["init"].clone()
        res += [binding.ssd_gated_step(xs[:, 0], gs[:, 0], d["bias"], state), state]
    assert len(got) == len(want) and all(torch.equal(p, q) for p, q in zip(got, want))


def test_calls_on_the_layer_s_own_tensors():
    """The recurrence next to the layer: the block's prologue makes x and the gate's rows come
    from the same projection; the epilogue takes its output."""
    H, P, N, G, B, T = 4, 16, 16, 1, 2, 200
    gen = torch.Generator().manual_seed(0)
    width = 2 * H * P + 2 * G * N + H
    zx = torch.randn((B, T, width), generator=gen).to(torch.bfloat16).cuda()
    z, xbc, dtr = zx[..., :H * P], zx[..., H * P:-H], zx[..., -H:]
    cw = torch.randn((H * P + 2 * G * N, 4), generator=gen).cuda() * 0.5
    pro = binding.ssd_block_prologue(xbc, cw, None, dtr, None, H, P, N, G)
    x = pro["x"].view(B, T, H * P)
    h, _ = binding.ssd_gated_fwd(x, z, None)
    w = torch.ones(H * P, device="cuda")
    out = binding.ssd_block_epilogue(h.view(B, T, H, P), z, w, None, 1)
    r = gated.gated_ref(n64(x), n64(z))
    check("h", h, r["h"], r["h_mag"], c_of(n64(z), None), 2.0 ** -8)
    assert bool(torch.isfinite(out).all())
