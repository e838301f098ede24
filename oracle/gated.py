"""The gated recurrence and the 8-bit checkpoints in fp64 (numpy), step by step.

  q = 1 / (1 + exp(g + bias)),  a = 1 - q,  h_t = a h_{t-1} + q x_t  (per channel)

and the reverse-mode derivative of exactly these steps.  The backward restarts h in every
chunk of CHUNK steps from the entry state it is given (which matters where x and g are not
the forward's own, but 8-bit checkpoints of them).

Next to each result goes a magnitude that its rounding errors are measured against: the
same recursions run on absolute values, adding at every step the size of the terms that
the step rounds.  A computation in fp32 that rounds each term a few times, in any order of
combining steps, stays within a small multiple of 2^-24 of it.
"""
import numpy as np

CHUNK = 64
GROUP = 64
# the largest fp32 value that stays finite 127 times
SCALE_MOST = np.nextafter(np.float32(np.finfo(np.float32).max / 127.0), np.float32(0))


def gate(s):
    """q and a = 1 - q, each accurate by itself."""
    s = np.asarray(s, dtype=np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(s)), 1.0 / (1.0 + np.exp(-s))


def _sequences(cu, T):
    """(first steps, {last step: sequence}) of a packed row; empty sequences have neither."""
    first, last = set(), {}
    for k in range(len(cu) - 1):
        if cu[k + 1] > cu[k]:
            first.add(int(cu[k]))
            last[int(cu[k + 1]) - 1] = k
    return first, last


def gated_ref(x, g, bias=None, init=None, cu=None):
    """x, g [B,T,D], bias [D], init [B,D].  Returns a dict: h [B,T,D], final [B or nseq,D],
    entry [B,nC,D], and the magnitudes h_mag, final_mag."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    B, T, D = x.shape
    q, a = gate(g + (0.0 if bias is None else np.asarray(bias, np.float64)))
    first, last = (set(), {}) if cu is None else _sequences(cu, T)
    v = np.zeros((B, D)) if init is None else np.asarray(init, np.float64).copy()
    size, err = np.abs(v), np.zeros((B, D))
    nC = -(-T // CHUNK)
    h, mag = np.empty((B, T, D)), np.empty((B, T, D))
    entry, entry_mag = np.empty((B, nC, D)), np.empty((B, nC, D))
    ends = B if cu is None else len(cu) - 1
    final, final_mag = np.zeros((ends, D)), np.zeros((ends, D))
    for t in range(T):
        if t % CHUNK == 0:
            entry[:, t // CHUNK], entry_mag[:, t // CHUNK] = v, err
        if t in first:
            v, size, err = np.zeros((B, D)), np.zeros((B, D)), np.zeros((B, D))
        u = q[:, t] * (np.abs(x[:, t]) + size)
        v = a[:, t] * v + q[:, t] * x[:, t]
        size = a[:, t] * size + q[:, t] * np.abs(x[:, t])
        err = a[:, t] * err + u + size
        h[:, t], mag[:, t] = v, err
        if t in last:
            final[last[t]], final_mag[last[t]] = v[0], err[0]
    if cu is None:
        final, final_mag = v, err
    return dict(h=h, final=final, entry=entry, h_mag=mag, final_mag=final_mag,
                entry_mag=entry_mag)


def gated_bwd_ref(x, g, bias, entry, dh, d_final=None, cu=None):
    """Returns a dict: dx, dg [B,T,D], d_bias [D], d_init [B,D] and their magnitudes *_mag."""
    x, g, dh = (np.asarray(v, np.float64) for v in (x, g, dh))
    B, T, D = x.shape
    q, a = gate(g + (0.0 if bias is None else np.asarray(bias, np.float64)))
    first, last = (set(), {}) if cu is None else _sequences(cu, T)
    zero = np.zeros((B, D))
    before, bsize, berr = (np.empty((B, T, D)) for _ in range(3))
    v = size = err = zero
    for t in range(T):
        if t % CHUNK == 0:
            v = np.asarray(entry, np.float64)[:, t // CHUNK]
            size, err = np.abs(v), np.abs(v)
        if t in first:
            v, size, err = zero, zero, zero
        before[:, t], bsize[:, t], berr[:, t] = v, size, err
        u = q[:, t] * (np.abs(x[:, t]) + size)
        v = a[:, t] * v + q[:, t] * x[:, t]
        size = a[:, t] * size + q[:, t] * np.abs(x[:, t])
        err = a[:, t] * err + u + size
    out = {k: np.empty((B, T, D)) for k in ("dx", "dg", "dx_mag", "dg_mag")}
    dfin = None if d_final is None else np.asarray(d_final, np.float64)
    c = zero if dfin is None or cu is not None else dfin
    csize, cerr = np.abs(c), zero
    for t in range(T - 1, -1, -1):
        if t in last:
            c = zero if dfin is None else dfin[last[t]][None]
            csize, cerr = np.abs(c), zero
        G = dh[:, t] + c
        size = np.abs(dh[:, t]) + csize
        err = cerr + size
        d = before[:, t] - x[:, t]
        out["dx"][:, t], out["dx_mag"][:, t] = q[:, t] * G, q[:, t] * (err + size)
        out["dg"][:, t] = G * d * q[:, t] * a[:, t]
        out["dg_mag"][:, t] = q[:, t] * a[:, t] * (
            (err + size) * (bsize[:, t] + np.abs(x[:, t])) + size * berr[:, t])
        keep = 0.0 if t in first else 1.0
        c = keep * a[:, t] * G
        cerr = keep * (a[:, t] * err + q[:, t] * size + size)
        csize = keep * a[:, t] * size
    out.update(d_bias=out["dg"].sum((0, 1)), d_init=c, d_init_mag=cerr + csize,
               d_bias_mag=out["dg_mag"].sum((0, 1)) + np.abs(out["dg"]).sum((0, 1)))
    return out


def ckpt_pack(v):
    """codes (int8), scales (fp32) of rows v [..., width] (fp32 or bf16 values)."""
    v = np.asarray(v, np.float64)
    width = v.shape[-1]
    groups = -(-width // GROUP)
    pad = np.zeros(v.shape[:-1] + (groups * GROUP - width,))
    w = np.concatenate([v, pad], -1).reshape(v.shape[:-1] + (groups, GROUP))
    with np.errstate(all="ignore"):
        most = np.abs(w).max(-1)  # NaN where any value is
        tiny, bad = most < 2.0 ** -100, ~np.isfinite(most)
        scale = np.where(tiny, 0.0, np.where(bad, np.nan, most / 127)).astype(np.float32)
        scale = np.minimum(scale, SCALE_MOST)
        inverse = np.where(tiny | bad, 0.0, 127 / most).astype(np.float32).astype(np.float64)
        codes = np.where(bad[..., None], 0.0, np.rint(w * inverse[..., None]))
    codes = codes.reshape(v.shape[:-1] + (groups * GROUP,))[..., :width]
    return codes.astype(np.int8), scale


def ckpt_unpack(codes, scales):
    """The fp32 values that codes and scales stand for."""
    s = np.repeat(np.asarray(scales, np.float32), GROUP, axis=-1)[..., :codes.shape[-1]]
    with np.errstate(over="ignore"):
        return codes.astype(np.float32) * s
