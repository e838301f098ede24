"""What the gated recurrence and the 8-bit checkpoints refuse (CPU only): the C ABI returns
its status before any launch, the binding raises before any call into the library."""
import ctypes

import pytest
import torch

from mamba_ssd_chunked_03_amd import binding

f32, bf16, i8 = torch.float32, torch.bfloat16, torch.int8
NULL, DIMS, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
P = 256  # a pointer that no call below gets to use


@pytest.fixture(scope="module")
def lib():
    return binding.library()


def gdims(b=2, t=100, d=64):
    return ctypes.byref(binding.SsdGatedDims(b, t, d))


def saved(entry=P, xc=None, xs=None, gc=None, gs=None):
    return ctypes.byref(binding.SsdGatedSaved(entry, xc, xs, gc, gs))


def fwd(lib, dims=None, dtype=1, x=P, xs=64, g=P, gs=64, bias=P, cu=None, nseq=0, init=None, h=P,
        final=P, sv=None, ws=P, nb=1 << 40):
    return lib.ssd_gated_fwd(dims or gdims(), dtype, x, xs, g, gs, bias, cu, nseq, init, h, final,
                             sv, ws, nb, None)


def bwd(lib, dims=None, dtype=1, x=P, xs=64, g=P, gs=64, bias=P, cu=None, nseq=0, sv=None, dh=P,
        hs=64, dfin=None, dx=P, dxs=64, dg=P, dgs=64, db=P, di=None, ws=P, nb=1 << 40):
    return lib.ssd_gated_bwd(dims or gdims(), dtype, x, xs, g, gs, bias, cu, nseq, sv or saved(),
                             dh, hs, dfin, dx, dxs, dg, dgs, db, di, ws, nb, None)


def bwd8(lib, sv, dims=None, dtype=1, cu=None, nseq=0, dh=P, hs=64, di=None, ws=P, nb=1 << 40):
    return lib.ssd_gated_bwd_ckpt(dims or gdims(), dtype, P, cu, nseq, sv, dh, hs, None, P, 64, P,
                                  64, P, di, ws, nb, None)


def test_forward_refusals(lib):
    assert fwd(lib, gdims(b=-1)) == DIMS and fwd(lib, gdims(t=-1)) == DIMS
    assert fwd(lib, gdims(d=-1)) == DIMS and fwd(lib, gdims(d=(1 << 20) + 1)) == DIMS
    assert fwd(lib, gdims(b=1 << 31)) == DIMS and fwd(lib, gdims(t=1 << 31)) == DIMS
    assert fwd(lib, gdims(b=1 << 20, t=1 << 20)) == DIMS
    assert fwd(lib, gdims(b=1 << 30, t=1, d=1 << 20), xs=1 << 20, gs=1 << 20) == DIMS
    assert fwd(lib, gdims(b=1 << 62, t=4)) == DIMS
    assert fwd(lib, xs=63) == DIMS and fwd(lib, gs=63) == DIMS
    assert fwd(lib, xs=1 << 62) == DIMS and fwd(lib, gs=-1) == DIMS
    assert fwd(lib, gdims(t=300), xs=1 << 21) == DIMS and fwd(lib, gs=1 << 23) == DIMS
    assert fwd(lib, gdims(t=300), xs=(1 << 21) - 1, h=None) == NULL  # the stride is taken
    assert fwd(lib, gdims(t=1), xs=1 << 40, h=None) == NULL
    assert fwd(lib, dtype=2) == UNSUPPORTED and fwd(lib, dtype=-1) == UNSUPPORTED
    assert lib.ssd_gated_fwd(None, 1, P, 64, P, 64, P, None, 0, None, P, P, None, P, 1 << 40,
                             None) == NULL
    for k in ("x", "g", "h"):
        assert fwd(lib, **{k: None}) == NULL
        assert fwd(lib, **{k: 257}) == ALIGN
        assert fwd(lib, dtype=0, **{k: 258}) == ALIGN
    for k in ("bias", "init", "final"):
        assert fwd(lib, **{k: 258}) == ALIGN
    assert fwd(lib, ws=None) == WORKSPACE and fwd(lib, nb=3) == WORKSPACE
    assert fwd(lib, ws=264) == ALIGN
    # packed rows
    assert fwd(lib, cu=P, nseq=1) == DIMS  # batch 2
    one = gdims(b=1)
    assert fwd(lib, one, cu=P, nseq=0) == DIMS and fwd(lib, one, cu=P, nseq=1 << 30) == DIMS
    assert fwd(lib, one, cu=P, nseq=2, init=P) == UNSUPPORTED
    assert fwd(lib, one, cu=257, nseq=2) == ALIGN
    # what is kept for the backward
    assert fwd(lib, sv=saved(entry=None)) == NULL
    assert fwd(lib, sv=saved(xc=P)) == NULL and fwd(lib, sv=saved(P, P, P, P, None)) == NULL
    assert fwd(lib, sv=saved(entry=258)) == ALIGN
    assert fwd(lib, sv=saved(P, 1, 258, 1, P)) == ALIGN


def test_backward_refusals(lib):
    assert bwd(lib, gdims(t=-1)) == DIMS and bwd(lib, dtype=9) == UNSUPPORTED
    for k in ("xs", "gs", "hs", "dxs", "dgs"):
        assert bwd(lib, **{k: 63}) == DIMS
    for k in ("x", "g", "dh", "dx", "dg"):
        assert bwd(lib, **{k: None}) == NULL
        assert bwd(lib, **{k: 257}) == ALIGN
    for k in ("bias", "dfin", "db", "di"):
        assert bwd(lib, **{k: 258}) == ALIGN
    assert bwd(lib, sv=saved(entry=None)) == NULL and bwd(lib, sv=saved(entry=257)) == ALIGN
    assert bwd(lib, ws=None) == WORKSPACE and bwd(lib, nb=0) == WORKSPACE
    one = gdims(b=1)
    assert bwd(lib, cu=P, nseq=1) == DIMS
    assert bwd(lib, one, cu=P, nseq=1, di=P) == UNSUPPORTED
    full = saved(P, 1, P, 1, P)
    assert bwd8(lib, saved()) == NULL and bwd8(lib, saved(P, 1, P, 1, None)) == NULL
    assert bwd8(lib, saved(None, 1, P, 1, P)) == NULL and bwd8(lib, None) == NULL
    assert bwd8(lib, full, dh=None) == NULL and bwd8(lib, full, hs=1) == DIMS
    assert bwd8(lib, saved(P, 1, 257, 1, P)) == ALIGN
    assert bwd8(lib, full, ws=None) == WORKSPACE and bwd8(lib, full, dtype=5) == UNSUPPORTED
    assert bwd8(lib, full, one, cu=P, nseq=3, di=P) == UNSUPPORTED


def test_step_refusals(lib):
    def step(dims=None, dtype=1, x=P, xs=64, g=P, gs=64, bias=None, state=P, h=P):
        return lib.ssd_gated_step(dims or gdims(), dtype, x, xs, g, gs, bias, state, h, None)
    assert step(gdims(b=-1)) == DIMS and step(xs=63) == DIMS and step(gs=0) == DIMS
    assert step(dtype=3) == UNSUPPORTED
    assert step(gdims(b=1 << 15, d=1 << 18), xs=1 << 18, gs=1 << 18) == DIMS
    for k in ("x", "g", "state", "h"):
        assert step(**{k: None}) == NULL
        assert step(**{k: 257}) == ALIGN
    assert step(bias=258) == ALIGN
    assert step(gdims(b=0)) == 0 and step(gdims(d=0), xs=0, gs=0) == 0
    assert lib.ssd_gated_step(None, 1, P, 64, P, 64, None, P, P, None) == NULL


def test_checkpoint_refusals(lib):
    def pack(rows=3, width=64, dtype=1, src=P, stride=64, codes=1, scales=P):
        return lib.ssd_ckpt_pack(rows, width, dtype, src, stride, codes, scales, None)

    def unpack(rows=3, width=64, dtype=1, codes=1, scales=P, dst=P, stride=64):
        return lib.ssd_ckpt_unpack(rows, width, dtype, codes, scales, dst, stride, None)
    for call, end in ((pack, "src"), (unpack, "dst")):
        assert call(rows=-1) == DIMS and call(width=-1) == DIMS and call(stride=63) == DIMS
        assert call(rows=1 << 31) == DIMS and call(rows=1 << 62, stride=1 << 62) == DIMS
        assert call(width=1 << 31, stride=1 << 31) == DIMS
        assert call(rows=1 << 21, stride=1 << 40) == DIMS
        assert call(dtype=2) == UNSUPPORTED
        for k in ("codes", "scales", end):
            assert call(**{k: None}) == NULL
        assert call(scales=258) == ALIGN and call(**{end: 257}) == ALIGN
        assert call(dtype=0, **{end: 258}) == ALIGN
        assert call(rows=0) == 0 and call(width=0) == 0
    assert binding.ssd_ckpt_scale_count(3, 65) == 6 and binding.ssd_ckpt_scale_count(3, 0) == 0
    assert binding.ssd_ckpt_scale_count(-1, 5) == 0


def test_layer_backward_refusals(lib):
    d = ctypes.byref(binding.SsdDims(1, 100, 2, 16, 16, 1))

    def call(dims=d, dtype=1, nb=1 << 40, **k):
        p = dict(xc=1, xs=P, dt=P, A=P, Bc=1, Bs=P, Cc=1, Cs=P, D=P, init=None, dy=P, df=None,
                 dx=P, ddt=P, dA=P, dB=P, dC=P, dD=P, di=None, ws=P)
        p.update(k)
        return lib.ssd_bwd_ckpt(dims, dtype, p["xc"], p["xs"], p["dt"], p["A"], p["Bc"], p["Bs"],
                                p["Cc"], p["Cs"], p["D"], 64, p["init"], p["dy"], p["df"], p["dx"],
                                p["ddt"], p["dA"], p["dB"], p["dC"], p["dD"], p["di"], p["ws"], nb,
                                None)
    assert call(ctypes.byref(binding.SsdDims(1, 100, 2, 24, 16, 1))) == UNSUPPORTED
    assert call(dtype=4) == UNSUPPORTED
    for k in ("xc", "xs", "dt", "A", "Bc", "Bs", "Cc", "Cs", "D", "dy", "dx", "ddt", "dA", "dB",
              "dC", "dD"):
        assert call(**{k: None}) == NULL, k
    for k in ("xs", "Bs", "Cs", "dt", "A", "init", "di"):
        assert call(**{k: 258}) == ALIGN
    assert call(dy=264) == ALIGN and call(ws=264) == ALIGN
    assert call(ws=None) == WORKSPACE and call(nb=100) == WORKSPACE
    dims = binding.SsdDims(1, 100, 2, 16, 16, 1)
    need = binding.ssd_bwd_ckpt_workspace_size(dims, bf16, 64)
    assert need > binding.ssd_bwd_workspace_size(dims, 64)
    assert call(nb=need - 1) == WORKSPACE


def test_binding_refuses_mismatched_tensors():
    x = torch.zeros(2, 10, 6)
    with pytest.raises(ValueError, match="GPU"):
        binding.ssd_gated_fwd(x, x)
    with pytest.raises(TypeError):
        binding.ssd_gated_fwd(x.half(), x.half())
    with pytest.raises(TypeError):
        binding.ssd_gated_fwd(x, x.to(bf16))
    for bad in (dict(g=torch.zeros(2, 10, 7)), dict(bias=torch.zeros(5)),
                dict(init_state=torch.zeros(2, 5)), dict(h=torch.zeros(2, 9, 6)),
                dict(final_state=torch.zeros(1, 6)), dict(x=torch.zeros(2, 6, 10).transpose(1, 2)),
                dict(x=torch.zeros(1, 10, 6).expand(2, 10, 6)),
                dict(g=torch.zeros(2, 20, 6)[:, ::2][:, :, :][:2].flip(0)[:, 1:]),
                dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)),
                dict(saved=dict(entry_states=torch.zeros(2, 2, 6)))):
        a = dict(x=x, g=x)
        a.update(bad)
        with pytest.raises(ValueError):
            binding.ssd_gated_fwd(a.pop("x"), a.pop("g"), **a)
    one = torch.zeros(1, 10, 6)
    for cu in ([0, 9], [1, 10], [0, 6, 5, 10], [0]):
        with pytest.raises(ValueError):
            binding.ssd_gated_fwd(one, one, cu_seqlens=torch.tensor(cu, dtype=torch.int32))
    with pytest.raises(TypeError):
        binding.ssd_gated_fwd(one, one, cu_seqlens=torch.tensor([0, 10]))
    sv = dict(entry_states=torch.zeros(2, 1, 6))
    with pytest.raises(ValueError, match="x_codes"):
        binding.ssd_gated_bwd_ckpt(None, x, sv)
    with pytest.raises(ValueError):
        binding.ssd_gated_bwd(x, x, None, x[:, :9], sv)
    with pytest.raises(ValueError):
        binding.ssd_gated_bwd(x, x, None, x, sv, out=dict(dx=torch.zeros(2, 10, 5)))
    with pytest.raises(ValueError):
        binding.ssd_gated_bwd(x, x, None, x, sv, d_final=torch.zeros(1, 6))
    s = torch.zeros(3, 6)
    with pytest.raises(ValueError):
        binding.ssd_gated_step(s, s, None, torch.zeros(3, 5))
    with pytest.raises(TypeError):
        binding.ssd_gated_step(s.to(bf16), s.to(bf16), None, s.to(bf16))
    with pytest.raises(ValueError):
        binding.ssd_ckpt_pack(torch.zeros(4, 70), scales=torch.zeros(4, 1))
    with pytest.raises(TypeError):
        binding.ssd_ckpt_pack(torch.zeros(4, 70, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.ssd_ckpt_unpack(torch.zeros(4, 70, dtype=i8), torch.zeros(4, 1))
    with pytest.raises(ValueError):
        binding.ssd_bwd_ckpt((torch.zeros(1, 5, 32, dtype=i8), torch.zeros(1, 5, 1)),
                             torch.zeros(1, 5, 2), torch.zeros(2),
                             (torch.zeros(1, 5, 16, dtype=i8), torch.zeros(1, 5, 1)),
                             (torch.zeros(1, 5, 17, dtype=i8), torch.zeros(1, 5, 1)),
                             torch.zeros(2), 64, torch.zeros(1, 5, 2, 16), 1)


def test_row_strides():
    """Evenly spaced rows are taken as they lie; others are refused."""
    rows = binding._rows
    w = torch.zeros(4, 6, 20)
    assert rows(w[..., 3:10], "w") == 20 and rows(w[:, :1, 3:10], "w") == 120
    assert rows(w[:1, :, 3:10], "w") == 20 and rows(w[:1, :1, 3:10], "w") == 7
    assert rows(w[..., 3:4], "w") == 20
    assert rows(torch.zeros(0, 3, 5), "w") == 5
    assert rows(w[:, ::2, :], "w") == 40  # 3 rows 40 apart are 120: evenly spaced
    for bad in (w[:, :4:2, :], w[:, 1:, :], w[::2], w[..., ::2], w.transpose(0, 1)):
        with pytest.raises(ValueError):
            rows(bad, "w")
