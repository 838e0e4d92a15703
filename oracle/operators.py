"""fp64 reference of the operators beside the block: q/k norm with rotation, gated scan, 8-bit projection.

Every function also returns, or takes part in, a bound on what fp32 arithmetic may add to its result: `c` roundings of
2^-24 relative to the sum of the magnitudes that enter a value.  The tests add half a step of the output's type.
"""
import numpy as np

EPS32 = 2.0 ** -24


def half_step(dtype: str) -> float:
    """Largest relative error of one rounding to the type."""
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def rope_table(count, dims, start=0, theta=10000.0):
    i = np.arange(dims // 2, dtype=np.float64)
    ang = (start + np.arange(count, dtype=np.float64))[:, None] * theta ** (-2.0 * i / dims)
    return np.stack((np.cos(ang), np.sin(ang)), axis=-1)


def _rotation(cfg, tables):
    """Per token and channel: partner channel, cos, signed sin (z_c = y_c cos + y_partner sin)."""
    n = cfg.T * cfg.H * cfg.W
    r = np.arange(n)
    at = (r // (cfg.H * cfg.W), r // cfg.W % cfg.H, r % cfg.W)
    partner = np.arange(cfg.tp)
    co, si = np.ones((n, cfg.tp)), np.zeros((n, cfg.tp))
    c0 = 0
    for axis, (dims, tab) in enumerate(zip((cfg.rt, cfg.rh, cfg.rw), tables)):
        for i in range(dims // 2):
            u, v = (c0 + 2 * i, c0 + 2 * i + 1) if cfg.pairing == "adjacent" else (c0 + i, c0 + i + dims // 2)
            partner[u], partner[v] = v, u
            cs = np.asarray(tab, np.float64)[at[axis], i]
            co[:, u] = co[:, v] = cs[:, 0]
            si[:, u], si[:, v] = -cs[:, 1], cs[:, 1]
        c0 += dims
    return partner, co, si


def qk_norm_rope(qkv, wq, wk, tables, cfg):
    """(out [rows, width], bound on the fp32 error of its q and k columns [rows, hq + hk, tp])."""
    nh, tp = cfg.hq + cfg.hk, cfg.tp
    x = np.asarray(qkv, np.float64).reshape(cfg.B, -1, cfg.width)
    q = x[..., :nh * tp].reshape(cfg.B, -1, nh, tp)
    w = np.stack([np.ones(tp) if wq is None else wq] * cfg.hq + [np.ones(tp) if wk is None else wk] * cfg.hk)
    y = q / np.sqrt((q * q).mean(-1, keepdims=True) + np.float64(np.float32(cfg.eps))) * w
    partner, co, si = _rotation(cfg, tables)
    z = y * co[None, :, None] + y[..., partner] * si[None, :, None]
    mag = np.abs(y) + np.abs(y[..., partner])
    out = np.concatenate([z.reshape(cfg.B, -1, nh * tp), x[..., nh * tp:]], axis=-1)
    return out.reshape(-1, cfg.width), 32 * EPS32 * mag.reshape(-1, nh, tp)


def qk_norm_rope_backward(qkv, wq, wk, tables, dout, cfg):
    """(dqkv, bound of its q and k columns, (dwq, dwk), their bounds)."""
    nh, tp = cfg.hq + cfg.hk, cfg.tp
    x = np.asarray(qkv, np.float64).reshape(cfg.B, -1, cfg.width)[..., :nh * tp].reshape(cfg.B, -1, nh, tp)
    d = np.asarray(dout, np.float64).reshape(cfg.B, -1, cfg.width)
    dz = d[..., :nh * tp].reshape(cfg.B, -1, nh, tp)
    w = np.stack([np.ones(tp) if wq is None else wq] * cfg.hq + [np.ones(tp) if wk is None else wk] * cfg.hk)
    partner, co, si = _rotation(cfg, tables)
    co, si = co[None, :, None], si[None, :, None]
    dy = dz * co - dz[..., partner] * si
    mdy = np.abs(dz) + np.abs(dz[..., partner])
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(cfg.eps)))
    n = x * r
    g, mg = dy * w, mdy * np.abs(w)
    dx = r * (g - n * (g * n).mean(-1, keepdims=True))
    bound = 64 * EPS32 * r * (mg + np.abs(n) * (mg * np.abs(n)).mean(-1, keepdims=True))
    dw, mdw = (dy * n).sum((0, 1)), (mdy * np.abs(n)).sum((0, 1))
    out = np.concatenate([dx.reshape(cfg.B, -1, nh * tp), d[..., nh * tp:]], axis=-1).reshape(-1, cfg.width)
    # a sum of k terms in any order is off by at most k - 1 roundings of the sum of magnitudes; the longest chain of
    # additions is that of one thread and the joins behind it, below 256 for the tests' sizes
    grads = (dw[:cfg.hq].sum(0), dw[cfg.hq:].sum(0))
    return out, bound.reshape(-1, nh, tp), grads, (256 * EPS32 * mdw[:cfg.hq].sum(0), 256 * EPS32 * mdw[cfg.hq:].sum(0))


def scan_rows(cfg):
    """Grid row of every step of the recurrence."""
    r = np.arange(cfg.T * cfg.H * cfg.W)
    t, h, w = r // (cfg.H * cfg.W), r // cfg.W % cfg.H, r % cfg.W
    pos = (r, (t * cfg.W + w) * cfg.H + h, (h * cfg.W + w) * cfg.T + t, (w * cfg.H + h) * cfg.T + t)[cfg.order]
    rows = np.argsort(pos)
    return rows[::-1] if cfg.reverse else rows


def _sigmoid(z):
    return 1 / (1 + np.exp(-np.clip(z, -700, 700)))


def gated_scan(x, g, cfg, bias=None, h0=None, dy=None, dh_last=None):
    """dict of (value, bound on the fp32 error): y, h_last, and with dy also dx, dg, dbias, dh0.

    Bounds: with H = the recurrence of magnitudes, every step adds at most c roundings of H_t, where c counts the
    gate's (its argument's sum, product and constant move it by up to 2.2 |z| half steps, of which the 24 hold 0.2 |z|;
    then exp, reciprocal), the products and the additions, in whichever order the steps are joined; E_t = a_t E_{t-1} + c 2^-24 H_t.  The adjoint state likewise."""
    rows = scan_rows(cfg)
    x = np.asarray(x, np.float64).reshape(cfg.B, -1, cfg.D)[:, rows]
    z = np.asarray(g, np.float64).reshape(cfg.B, -1, cfg.D)[:, rows] + (0 if bias is None else np.asarray(bias, np.float64))
    n = x.shape[1]
    a, na = _sigmoid(z), _sigmoid(-z)
    c = (24 + 2 * np.minimum(np.abs(z), 100)) * EPS32
    h = np.zeros((cfg.B, cfg.D)) if h0 is None else np.asarray(h0, np.float64)
    before, hs = np.empty_like(x), np.empty_like(x)
    mag, mag_before, err, err_before = np.abs(h), np.empty_like(x), np.zeros_like(h), np.empty_like(x)
    errs = np.empty_like(x)
    for t in range(n):
        before[:, t], mag_before[:, t], err_before[:, t] = h, mag, err
        h = a[:, t] * h + na[:, t] * x[:, t]
        mag = a[:, t] * mag + na[:, t] * np.abs(x[:, t])
        err = a[:, t] * err + c[:, t] * mag
        hs[:, t], errs[:, t] = h, err

    def grid(v):
        o = np.empty_like(v)
        o[:, rows] = v
        return o

    out = dict(y=(grid(hs), grid(errs)), h_last=(h, err))
    if dy is None:
        return out
    dy = np.asarray(dy, np.float64).reshape(cfg.B, -1, cfg.D)[:, rows]
    lam = np.zeros((cfg.B, cfg.D)) if dh_last is None else np.asarray(dh_last, np.float64)
    mag, err = np.abs(lam), np.zeros_like(lam)
    dx, dg, ex, eg, mg = (np.empty_like(x) for _ in range(5))
    for t in range(n - 1, -1, -1):
        l, ml, el = dy[:, t] + lam, np.abs(dy[:, t]) + mag, err + c[:, t] * (np.abs(dy[:, t]) + mag)
        dx[:, t], ex[:, t] = na[:, t] * l, na[:, t] * (el + c[:, t] * ml)
        aa, hx = a[:, t] * na[:, t], mag_before[:, t] + np.abs(x[:, t])
        dg[:, t] = l * (before[:, t] - x[:, t]) * aa
        eg[:, t] = aa * (el * hx + ml * err_before[:, t] + 2 * c[:, t] * ml * hx)
        mg[:, t] = aa * ml * hx
        lam, mag, err = a[:, t] * l, a[:, t] * ml, a[:, t] * (el + c[:, t] * ml)
    out.update(dx=(grid(dx), grid(ex)), dg=(grid(dg), grid(eg)), dh0=(lam, err),
               dbias=(dg.sum((0, 1)), eg.sum((0, 1)) + 256 * EPS32 * mg.sum((0, 1))))
    return out


def quantize_rows(x):
    """(q, scale): the fp32 scale max|x| / 127, q to the nearest integer of the quotient in 64 bits, ties to even."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.abs(x).max(1)
        scale = (m / np.float32(127)).astype(np.float32)
        bad = ~np.isfinite(x).all(1)
        quot = x.astype(np.float64) / scale.astype(np.float64)[:, None]
        q = np.where((scale[:, None] > 0) & ~bad[:, None], np.clip(np.rint(quot), -127, 127), 0)
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def project_int8(A, a_scale, Wt, w_scale, bias=None):
    """(C, bound): the sum is exact; its conversion, two products and the bias round."""
    acc = A.astype(np.int64) @ Wt.astype(np.int64).T
    v = acc.astype(np.float64) * np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)
    b = 0 if bias is None else np.asarray(bias, np.float64)
    return v + b, 4 * EPS32 * (np.abs(v) + np.abs(b))
