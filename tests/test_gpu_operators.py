"""The operators beside the block on the GPU against their fp64 reference (oracle/operators.py): q/k norm with
rotation, gated scan and 8-bit projection, alone and in a run as a mixing block uses them.

Tolerances: half a step of the output's type (bf16 2^-8, fp32 2^-24 of the value) and the reference's bound on the
fp32 arithmetic before that rounding."""
import dataclasses

import numpy as np
import pytest

from helpers import requires_gpu
import mate_inputs as mi
from oracle import operators as OP

pytestmark = [pytest.mark.gpu, requires_gpu]

torch = pytest.importorskip("torch")
from linear_complexity_video_mate_b200 import _lib, mate as M  # noqa: E402


def _host(rng, shape, dtype, scale=1.0):
    a = (scale * rng.standard_normal(shape)).astype(np.float32)
    return mi.round_to_bf16(a) if dtype == "bf16" else a


def _dev(a, dtype="f32"):
    return torch.as_tensor(np.ascontiguousarray(a)).to(device="cuda",
                                                       dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _strided(a, dtype, pad):
    """Rows of `a` [rows, cols] inside a wider buffer whose other columns hold NaN."""
    big = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), device="cuda",
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    big[:, 8:8 + a.shape[1]] = _dev(a, dtype)
    return big, big[:, 8:8 + a.shape[1]]


def _close(got, ref, bound, dtype, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = OP.half_step(dtype) * (np.abs(ref) + bound) + bound + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol):.3g} tolerances"


# ------------------------------------------------------------------------------------ q/k norm with rotation
QK = [
    M.QkConfig(B=1, T=1, H=1, W=1, hq=1, hk=1, hv=0, tp=8, rt=2, rh=2, rw=2),
    M.QkConfig(B=1, T=1, H=1, W=1, hq=16, hk=4, hv=4, tp=128, rt=44, rh=42, rw=42),
    M.QkConfig(B=2, T=3, H=5, W=7, hq=4, hk=4, hv=4, tp=128, rt=32, rh=48, rw=48),
    M.QkConfig(B=2, T=3, H=5, W=7, hq=5, hk=2, hv=2, tp=80, rt=16, rh=24, rw=24, pairing="halves"),
    M.QkConfig(B=1, T=129, H=1, W=1, hq=3, hk=3, hv=3, tp=64, rt=64, pairing="halves"),
    M.QkConfig(B=1, T=2, H=9, W=4, hq=2, hk=1, hv=0, tp=256, rt=0, rh=130, rw=126),
    M.QkConfig(B=3, T=4, H=3, W=2, hq=1, hk=2, hv=1, tp=24, rt=6, rh=0, rw=10, pairing="halves"),
    M.QkConfig(B=1, T=4, H=3, W=2, hq=2, hk=2, hv=2, tp=72),
    M.QkConfig(B=1, T=2, H=2, W=2, hq=2, hk=1, hv=1, tp=4, rt=2, dtype="f32"),
    M.QkConfig(B=2, T=3, H=5, W=7, hq=6, hk=2, hv=0, tp=80, rt=16, rh=24, rw=24, pairing="halves", dtype="f32"),
    M.QkConfig(B=2, T=5, H=3, W=3, hq=4, hk=4, hv=4, tp=256, rt=86, rh=86, rw=84, dtype="f32"),
    M.QkConfig(B=1, T=40, H=20, W=9, hq=3, hk=1, hv=1, tp=128, rt=32, rh=48, rw=48, pairing="halves", eps=1e-3),
]


def _qk_id(c):
    return f"{c.B}x{c.T}x{c.H}x{c.W}_{c.hq}-{c.hk}-{c.hv}x{c.tp}_{c.rt}-{c.rh}-{c.rw}_{c.pairing}_{c.dtype}"


def _qk_inputs(cfg, seed, weights=True, start=(0, 0, 0)):
    rng = np.random.default_rng(seed)
    qkv = _host(rng, (cfg.rows, cfg.width), cfg.dtype)
    qkv *= mi.round_to_bf16(np.exp2(rng.integers(-3, 4, (cfg.rows, 1))).astype(np.float32))   # rows of other sizes
    if cfg.rows > 2:
        qkv[1, :cfg.tp] = 0     # a head of zeros
    w = [(1 + 0.3 * rng.standard_normal(cfg.tp)).astype(np.float32) if weights else None for _ in range(2)]
    tabs = [M.rope_table(n, r, start=s) for n, r, s in zip((cfg.T, cfg.H, cfg.W), (cfg.rt, cfg.rh, cfg.rw), start)]
    return rng, qkv, w, tabs, [t.cpu().numpy() for t in tabs]


def _qk_check(got, ref, bound, cfg, what):
    got = _np(got).reshape(cfg.rows, cfg.width)
    nqk = (cfg.hq + cfg.hk) * cfg.tp
    _close(got[:, :nqk].reshape(bound.shape), ref[:, :nqk].reshape(bound.shape), bound, cfg.dtype, what)
    np.testing.assert_array_equal(got[:, nqk:], ref[:, nqk:], err_msg=what)   # value columns pass unchanged


@pytest.mark.parametrize("cfg", QK, ids=_qk_id)
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rope(cfg, weights):
    _, qkv, (wq, wk), tabs, tabs_h = _qk_inputs(cfg, 1, weights, start=(1000, 0, 3))
    ref, bound = OP.qk_norm_rope(qkv, wq, wk, tabs_h, cfg)
    dw = [None if w is None else _dev(w) for w in (wq, wk)]
    x = _dev(qkv, cfg.dtype)
    out = M.qk_norm_rope(x, *dw, tabs, cfg)
    _qk_check(out, ref, bound, cfg, "out of place")
    # strided rows of a wider buffer, in place: the value columns and the other columns stay
    big, view = _strided(qkv, cfg.dtype, 24)
    M.qk_norm_rope(view, *dw, tabs, cfg, out=view)
    assert torch.equal(view.contiguous(), out)
    assert torch.isnan(big[:, :8]).all() and torch.isnan(big[:, 8 + cfg.width:]).all()
    # into strided rows
    big, view = _strided(np.zeros_like(qkv), cfg.dtype, 40)
    M.qk_norm_rope(x, *dw, tabs, cfg, out=view)
    assert torch.equal(view.contiguous(), out)
    assert torch.isnan(big[:, :8]).all() and torch.isnan(big[:, 8 + cfg.width:]).all()


@pytest.mark.parametrize("cfg", QK, ids=_qk_id)
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rope_backward(cfg, weights):
    rng, qkv, (wq, wk), tabs, tabs_h = _qk_inputs(cfg, 2, weights)
    dout = _host(rng, (cfg.rows, cfg.width), cfg.dtype)
    ref, bound, dws, dwb = OP.qk_norm_rope_backward(qkv, wq, wk, tabs_h, dout, cfg)
    dw = [None if w is None else _dev(w) for w in (wq, wk)]
    x, d = _dev(qkv, cfg.dtype), _dev(dout, cfg.dtype)
    got = M.qk_norm_rope_backward(x, *dw, tabs, d, cfg)
    _qk_check(got["dqkv"], ref, bound, cfg, "dqkv")
    _close(got["dwq"], dws[0], dwb[0], "f32", "dwq")
    _close(got["dwk"], dws[1], dwb[1], "f32", "dwk")
    # over the output gradient, over the input, and again: the same bits
    for target in ("dout", "qkv"):
        x2, d2 = x.clone(), d.clone()
        again = M.qk_norm_rope_backward(x2, *dw, tabs, d2, cfg, dqkv=d2 if target == "dout" else x2)
        for k in got:
            assert torch.equal(again[k], got[k]), (target, k)
    big, view = _strided(np.zeros_like(qkv), cfg.dtype, 16)
    _, dview = _strided(dout, cfg.dtype, 32)
    M.qk_norm_rope_backward(x, *dw, tabs, dview, cfg, dqkv=view)
    assert torch.equal(view.contiguous(), got["dqkv"])
    assert torch.isnan(big[:, :8]).all() and torch.isnan(big[:, 8 + cfg.width:]).all()


# every way a head's channels lie over the lanes: lanes per head, two units per lane, pairs inside a lane or through
# shared memory; more heads than one warp's share of a row
QK_LANES = [M.QkConfig(B=1, T=2, H=3, W=2, hq=3, hk=2, hv=1, tp=tp, rt=r[0], rh=r[1], rw=r[2], pairing=pair, dtype=dt)
            for dt, shapes in (("bf16", ((256, (88, 88, 80)), (256, (86, 84, 86)), (136, (48, 40, 48)), (32, (8, 8, 16)),
                                         (32, (10, 10, 12)), (16, (8, 0, 8)))),
                               ("f32", ((256, (88, 84, 84)), (256, (86, 84, 82)), (200, (68, 64, 60)), (132, (44, 40, 48)),
                                        (64, (20, 20, 24)), (12, (4, 0, 4)), (12, (6, 2, 4)))))
            for tp, r in shapes for pair in ("adjacent", "halves")]
QK_LANES += [M.QkConfig(B=1, T=1, H=1, W=1, hq=40, hk=33, hv=5, tp=32, rt=32),
             M.QkConfig(B=2, T=3, H=1, W=1, hq=1, hk=17, hv=2, tp=64, rt=6, pairing="halves")]


@pytest.mark.parametrize("cfg", QK_LANES, ids=_qk_id)
def test_qk_lane_layouts(cfg):
    rng, qkv, (wq, wk), tabs, tabs_h = _qk_inputs(cfg, 18)
    x, dw = _dev(qkv, cfg.dtype), [_dev(w) for w in (wq, wk)]
    ref, bound = OP.qk_norm_rope(qkv, wq, wk, tabs_h, cfg)
    _qk_check(M.qk_norm_rope(x, *dw, tabs, cfg), ref, bound, cfg, "out")
    dout = _host(rng, (cfg.rows, cfg.width), cfg.dtype)
    ref, bound, dws, dwb = OP.qk_norm_rope_backward(qkv, wq, wk, tabs_h, dout, cfg)
    got = M.qk_norm_rope_backward(x, *dw, tabs, _dev(dout, cfg.dtype), cfg)
    _qk_check(got["dqkv"], ref, bound, cfg, "dqkv")
    _close(got["dwq"], dws[0], dwb[0], "f32", "dwq")
    _close(got["dwk"], dws[1], dwb[1], "f32", "dwk")


def test_qk_gradient_against_differences():
    """The gradient against central differences of the fp64 forward pass along random directions: the fp32 kernel's
    gradient rounds at 2^-24 per term, the difference quotient is off by its third-order term, h^2 = 1e-10 relative."""
    cfg = dataclasses.replace(QK[9], B=1)
    rng, qkv, (wq, wk), tabs, tabs_h = _qk_inputs(cfg, 3)
    qkv[1, :cfg.tp] = 1
    dout = _host(rng, qkv.shape, "f32")
    g = M.qk_norm_rope_backward(_dev(qkv), _dev(wq), _dev(wk), tabs, _dev(dout), cfg)
    f = lambda x, a, b: (OP.qk_norm_rope(x, a, b, tabs_h, cfg)[0] * dout).sum()
    h = 1e-5
    for _ in range(3):
        vx, vq, vk = (rng.standard_normal(s) for s in (qkv.shape, wq.shape, wk.shape))
        vx *= np.abs(qkv).mean(1, keepdims=True)
        num = (f(qkv + h * vx, wq + h * vq, wk + h * vk) - f(qkv - h * vx, wq - h * vq, wk - h * vk)) / (2 * h)
        terms = [_np(g["dqkv"]) * vx, _np(g["dwq"]) * vq, _np(g["dwk"]) * vk]
        ana, mag = sum(t.sum() for t in terms), sum(np.abs(t).sum() for t in terms)
        assert abs(num - ana) <= 1e-6 * mag, (num, ana, mag)


@pytest.mark.parametrize("start", [0, 12345, 1 << 24, (1 << 40) + 1])
@pytest.mark.parametrize("dims,theta", [(2, 10000.0), (44, 10000.0), (128, 5e5)])
def test_rope_table(start, dims, theta):
    """Angles in 64 bits: the position times a frequency that is right to a few 2^-53 (pow is good to 2 of its steps)."""
    got = _np(M.rope_table(37, dims, start=start, theta=theta))
    ref = OP.rope_table(37, dims, start, theta)
    assert np.abs(got - ref).max() <= 2.0 ** -24 + 8 * 2.0 ** -53 * (start + 37)


# ------------------------------------------------------------------------------------------------ gated scan
SCAN = [
    M.GatedScanConfig(B=1, T=1, H=1, W=1, D=8),
    M.GatedScanConfig(B=64, T=1, H=1, W=1, D=264),
    M.GatedScanConfig(B=3, T=2, H=1, W=1, D=16, reverse=True),
    M.GatedScanConfig(B=2, T=3, H=5, W=7, D=40, order=1),
    M.GatedScanConfig(B=2, T=3, H=5, W=7, D=40, order=2, reverse=True),
    M.GatedScanConfig(B=1, T=4, H=4, W=4, D=128, order=3),
    M.GatedScanConfig(B=1, T=5, H=13, W=1, D=72, order=3, reverse=True),
    M.GatedScanConfig(B=2, T=1025, H=1, W=1, D=136),
    M.GatedScanConfig(B=1, T=127, H=3, W=11, D=24, order=2),
    M.GatedScanConfig(B=1, T=16, H=16, W=16, D=256, order=1, reverse=True),
    M.GatedScanConfig(B=1, T=1, H=1, W=1, D=4, dtype="f32"),
    M.GatedScanConfig(B=2, T=9, H=13, W=5, D=44, order=3, reverse=True, dtype="f32"),
    M.GatedScanConfig(B=1, T=33, H=8, W=8, D=132, order=2, dtype="f32"),
    M.GatedScanConfig(B=3, T=64, H=2, W=1, D=128, order=1, dtype="f32"),
    M.GatedScanConfig(B=1, T=9001, H=1, W=1, D=12, dtype="f32"),
]


def _scan_id(c):
    return f"{c.B}x{c.T}x{c.H}x{c.W}_D{c.D}_o{c.order}{'r' if c.reverse else ''}_{c.dtype}"


def _scan_inputs(cfg, seed, extras, gate=2.0, spread=1.0):
    rng = np.random.default_rng(seed)
    shape = (cfg.B, cfg.T * cfg.H * cfg.W, cfg.D)
    x, dy = _host(rng, shape, cfg.dtype), _host(rng, shape, cfg.dtype)
    g = (gate + spread * rng.standard_normal(shape)).astype(np.float32)
    g = mi.round_to_bf16(g) if cfg.dtype == "bf16" else g
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)
    kw = dict(bias=f32(cfg.D), h0=f32(cfg.B, cfg.D), dh_last=f32(cfg.B, cfg.D)) if extras else \
        dict(bias=None, h0=None, dh_last=None)
    return x, g, dy, kw


def _scan_check(cfg, x, g, dy, kw):
    ref = OP.gated_scan(x, g, cfg, kw["bias"], kw["h0"], dy, kw["dh_last"])
    dkw = {k: None if v is None else _dev(v) for k, v in kw.items()}
    xd, gd, dyd = (_dev(v, cfg.dtype) for v in (x, g, dy))
    states = M.gated_scan_states(cfg)
    y, hl = M.gated_scan(xd, gd, cfg, bias=dkw["bias"], h0=dkw["h0"])
    y2, hl2 = M.gated_scan(xd, gd, cfg, bias=dkw["bias"], h0=dkw["h0"], states=states)
    assert torch.equal(y, y2) and torch.equal(hl, hl2)
    _close(y, *ref["y"], cfg.dtype, "y")
    _close(hl, *ref["h_last"], "f32", "h_last")
    gr = M.gated_scan_backward(xd, gd, states, dyd, cfg, bias=dkw["bias"], dh_last=dkw["dh_last"])
    again = M.gated_scan_backward(xd, gd, states, dyd, cfg, bias=dkw["bias"], dh_last=dkw["dh_last"])
    assert ("dbias" in gr) == (kw["bias"] is not None)
    for k, v in gr.items():
        _close(v, *ref[k], cfg.dtype if k in ("dx", "dg") else "f32", k)
        assert torch.equal(v, again[k]), k
    assert M.device_status() == 0
    return y, hl, gr, xd, gd, dyd, dkw, states


@pytest.mark.parametrize("cfg", SCAN, ids=_scan_id)
@pytest.mark.parametrize("extras", [True, False])
def test_gated_scan(cfg, extras):
    x, g, dy, kw = _scan_inputs(cfg, 4, extras)
    y, hl, gr, xd, gd, dyd, dkw, states = _scan_check(cfg, x, g, dy, kw)
    # strided rows: columns of wider buffers, the others left alone
    rows = lambda a: a.reshape(-1, cfg.D)
    (_, xs), (_, gs), (_, ds) = (_strided(rows(a), cfg.dtype, p) for a, p in ((x, 16), (g, 24), (dy, 32)))
    outs = [_strided(rows(np.zeros_like(x)), cfg.dtype, p) for p in (40, 16, 24)]
    st2 = M.gated_scan_states(cfg)
    M.gated_scan(xs, gs, cfg, bias=dkw["bias"], h0=dkw["h0"], y=outs[0][1], states=st2)
    M.gated_scan_backward(xs, gs, st2, ds, cfg, bias=dkw["bias"], dh_last=dkw["dh_last"], dx=outs[1][1], dg=outs[2][1])
    for (big, view), want in zip(outs, (y, gr["dx"], gr["dg"])):
        assert torch.equal(view.contiguous(), want.reshape(-1, cfg.D))
        assert torch.isnan(big[:, :8]).all() and torch.isnan(big[:, 8 + cfg.D:]).all()


@pytest.mark.parametrize("gate,spread", [(-6.0, 1.0), (9.0, 2.0), (0.0, 30.0), (200.0, 0.0), (-200.0, 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_scan_extreme_gates(gate, spread, dtype):
    """Gates that forget at once, hardly forget, saturate either way: no overflow on the way."""
    cfg = M.GatedScanConfig(B=1, T=300, H=2, W=1, D=64, order=1, dtype=dtype)
    x, g, dy, kw = _scan_inputs(cfg, 5, True, gate, spread)
    _scan_check(cfg, x, g, dy, kw)


@pytest.mark.parametrize("size", [8.0, 30.0, 100.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_scan_cancelling_bias(size, dtype):
    """Large biases and gates that cancel: the gate is as good as that of the sum, whatever its parts were."""
    cfg = M.GatedScanConfig(B=2, T=100, H=2, W=1, D=64, order=1, dtype=dtype)
    x, g, dy, kw = _scan_inputs(cfg, 21, True)
    kw["bias"] = (size * np.random.default_rng(22).standard_normal(cfg.D)).astype(np.float32)
    g = (g - 2 - kw["bias"]).astype(np.float32)
    g = mi.round_to_bf16(g) if dtype == "bf16" else g
    _scan_check(cfg, x, g, dy, kw)


@pytest.mark.parametrize("B", [512, 128, 64])
def test_gated_scan_long_chunks(B):
    """Batches with so many channels that a thread walks 128, 64 or 32 rows: against the recurrence in 64 bits on the GPU,
    with the bounds of the reference (oracle/operators.py)."""
    cfg = M.GatedScanConfig(B=B, T=10, H=5, W=6, D=1024, order=1, reverse=True)
    gen = torch.Generator(device="cuda").manual_seed(B)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy = (rnd(B, 300, 1024).bfloat16() for _ in range(2))
    g, bias, h0, dhl = (rnd(B, 300, 1024) + 2).bfloat16(), rnd(1024), rnd(B, 1024), rnd(B, 1024)
    states = M.gated_scan_states(cfg)
    y, hl = M.gated_scan(x, g, cfg, bias=bias, h0=h0, states=states)
    got = M.gated_scan_backward(x, g, states, dy, cfg, bias=bias, dh_last=dhl)
    rows = torch.as_tensor(np.ascontiguousarray(OP.scan_rows(cfg))).cuda()
    eps, worst = OP.EPS32, {}

    def check(name, v, ref, bound, half):
        tol = half * (ref.abs() + bound) + bound + 1e-37
        worst[name] = max(worst.get(name, 0.0), ((v.double() - ref).abs() / tol).max().item())

    h, mag, err = h0.double(), h0.double().abs(), torch.zeros_like(h0, dtype=torch.float64)
    before = []
    for r in rows:
        z = g[:, r].double() + bias.double()
        a, na, c = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z)), (24 + 2 * z.abs()) * eps
        before.append((h, mag, err, a, na, c))
        h = a * h + na * x[:, r].double()
        mag = a * mag + na * x[:, r].double().abs()
        err = a * err + c * mag
        check("y", y[:, r], h, err, OP.half_step("bf16"))
    check("h_last", hl, h, err, OP.half_step("f32"))
    lam, mag, err = dhl.double(), dhl.double().abs(), torch.zeros_like(h)
    db, dbm = torch.zeros(1024, dtype=torch.float64, device="cuda"), torch.zeros(1024, dtype=torch.float64, device="cuda")
    for r, (hb, hm, he, a, na, c) in zip(reversed(rows), reversed(before)):
        d = dy[:, r].double()
        l, ml, el = d + lam, d.abs() + mag, err + c * (d.abs() + mag)
        check("dx", got["dx"][:, r], na * l, na * (el + c * ml), OP.half_step("bf16"))
        xv, aa = x[:, r].double(), a * na
        hx = hm + xv.abs()
        dg, eg = l * (hb - xv) * aa, aa * (el * hx + ml * he + 2 * c * ml * hx)
        check("dg", got["dg"][:, r], dg, eg, OP.half_step("bf16"))
        db += dg.sum(0)
        # 300 B terms in sums of at most 512 additions on any path
        dbm += (eg + 512 * eps * aa * ml * hx).sum(0)
        lam, mag, err = a * l, a * ml, a * (el + c * ml)
    check("dh0", got["dh0"], lam, err, OP.half_step("f32"))
    check("dbias", got["dbias"], db, dbm, OP.half_step("f32"))
    assert all(v <= 1 for v in worst.values()), worst


def test_gated_scan_infinite_gates():
    """A gate of -inf starts the state afresh from x, of +inf keeps it as it is, exactly."""
    cfg = M.GatedScanConfig(B=1, T=200, H=1, W=1, D=8, dtype="f32")
    x, g, dy, kw = _scan_inputs(cfg, 6, True)
    g[:, 50], g[:, 51:100] = -np.inf, np.inf
    y, _ = M.gated_scan(_dev(x), _dev(g), cfg, bias=_dev(kw["bias"]), h0=_dev(kw["h0"]))
    y = _np(y)
    assert np.isfinite(y).all()
    np.testing.assert_array_equal(y[:, 50:100], np.repeat(x[:, 50:51], 50, 1).astype(np.float64))


def _classes(t):
    """0: finite, 1: inf, -1: -inf, 2: NaN."""
    a = _np(t) if isinstance(t, torch.Tensor) else t
    return np.where(np.isnan(a), 2, np.where(np.isinf(a), np.sign(a), 0)).astype(int)


def _same_classes(got, ref, bound, dtype, what):
    """Infinities and NaN as the recurrence gives them, and the finite values within their bounds."""
    np.testing.assert_array_equal(_classes(got), _classes(ref), err_msg=what)
    ok = np.isfinite(ref)
    _close(_np(got)[ok], ref[ok], np.broadcast_to(bound, ref.shape)[ok], dtype, what)


def _infinite_inputs(cfg, seed):
    """Gates whose products leave fp32's range in a chunk (column 1 of 4), in eight rows (2), in two (3), or not at all."""
    x, g, dy, kw = _scan_inputs(cfg, seed, True, gate=0.0)
    g += np.array([2.0, -9.0, -20.0, -60.0], np.float32)[np.arange(cfg.D) % 4]
    g = mi.round_to_bf16(g) if cfg.dtype == "bf16" else g
    return x, g, dy, kw


@pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order,reverse", [(0, False), (2, True)])
def test_gated_scan_infinite_states(order, reverse, dtype):
    """An infinite state stays infinite and a NaN stays NaN behind the row that brings it, wherever chunks begin: from x,
    from h0, from the gradients dy and dh_last; opposite infinities meet in a NaN."""
    cfg = M.GatedScanConfig(B=2, T=50, H=7, W=2, D=32, order=order, reverse=reverse, dtype=dtype)
    x, g, dy, kw = _infinite_inputs(cfg, 23)
    row = OP.scan_rows(cfg)
    plain = [a.copy() for a in (x, dy)]
    x[0, row[50], 0:8], x[0, row[333], 4:12], x[1, row[699], :] = np.inf, -np.inf, -np.inf
    x[1, row[100], 8:12] = np.nan
    kw["h0"][1, 12:24] = -np.inf
    kw["h0"][0, 20:24] = np.nan
    ref = OP.gated_scan(x, g, cfg, kw["bias"], kw["h0"])
    d = {k: _dev(v) for k, v in kw.items()}
    y, hl = M.gated_scan(_dev(x, dtype), _dev(g, dtype), cfg, bias=d["bias"], h0=d["h0"])
    _same_classes(y, *ref["y"], dtype, "y")
    _same_classes(hl, *ref["h_last"], "f32", "h_last")
    assert {-1, 0, 1, 2} == set(_classes(y).ravel())
    # the adjoint state runs back from the gradients
    x, dy = plain
    _, _, _, kw = _infinite_inputs(cfg, 23)
    dy[0, row[600], 0:8], dy[0, row[30], 4:12], dy[1, row[350], 8:12] = np.inf, -np.inf, np.nan
    kw["dh_last"][1, 12:24] = -np.inf
    ref = OP.gated_scan(x, g, cfg, kw["bias"], kw["h0"], dy, kw["dh_last"])
    d = {k: _dev(v) for k, v in kw.items()}
    xd, gd, states = _dev(x, dtype), _dev(g, dtype), M.gated_scan_states(cfg)
    M.gated_scan(xd, gd, cfg, bias=d["bias"], h0=d["h0"], states=states)
    gr = M.gated_scan_backward(xd, gd, states, _dev(dy, dtype), cfg, bias=d["bias"], dh_last=d["dh_last"])
    # dg = l (h - x) a (1 - a): where h and x agree to the rounding of an fp32 h (a repeated bf16 x behind a gate of e^-60),
    # the difference may come out as 0 or with either sign, and an infinite l times it as NaN or either infinity
    h, err = (v[:, row] for v in ref["y"])
    before, eb = np.concatenate([kw["h0"][:, None], h[:, :-1]], axis=1), np.concatenate([0 * err[:, :1], err[:, :-1]], axis=1)
    free = np.zeros(h.shape, bool)
    free[:, row] = np.abs(before - x[:, row]) <= eb + OP.EPS32 * (np.abs(before) + np.abs(x[:, row]))
    free &= ~np.isfinite(ref["dg"][0])
    assert free.mean() < 0.01 and not np.isfinite(_np(gr["dg"])[free]).any()
    gr["dg"][torch.as_tensor(free).cuda()] = 0
    ref["dg"][0][free], ref["dg"][1][free] = 0, 0
    for k, v in gr.items():
        _same_classes(v, *ref[k], dtype if k in ("dx", "dg") else "f32", k)
    assert {-1, 0, 1, 2} <= set(_classes(gr["dx"]).ravel()) | set(_classes(gr["dh0"]).ravel())


@pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")
@pytest.mark.parametrize("at", [3, 150, 700 - 9])
def test_gated_scan_infinite_state_meets_a_zero_gate(at):
    """0 times infinity: a gate of -inf makes an infinite state NaN from its row on, and starts a finite one afresh."""
    cfg = M.GatedScanConfig(B=1, T=700, H=1, W=1, D=16, dtype="f32")
    x, g, _, kw = _infinite_inputs(cfg, 24)
    kw["h0"][0, :8] = np.inf
    g[:, at] = -np.inf
    ref = OP.gated_scan(x, np.maximum(g, -700), cfg, kw["bias"], kw["h0"])["y"]
    y, _ = M.gated_scan(_dev(x), _dev(g), cfg, bias=_dev(kw["bias"]), h0=_dev(kw["h0"]))
    want = np.zeros((1, 700, 16), int)
    want[:, :at, :8], want[:, at:, :8] = 1, 2
    np.testing.assert_array_equal(_classes(y), want)
    _close(y[..., 8:], ref[0][..., 8:], ref[1][..., 8:], "f32", "y")
    np.testing.assert_array_equal(_np(y)[:, at, 8:], x[:, at, 8:])


@pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")
def test_gated_scan_infinite_states_whatever_the_chunks():
    """The same rows alone, in a batch that walks 128 rows at a time, in parts and token by token."""
    cfg = M.GatedScanConfig(B=1, T=300, H=1, W=1, D=1024)
    x, g, _, kw = _infinite_inputs(cfg, 25)
    x[0, 17, :500], x[0, 200, 400:900] = np.inf, -np.inf
    ref = OP.gated_scan(x, g, cfg, kw["bias"], kw["h0"])
    xd, gd, b, h0 = _dev(x, "bf16"), _dev(g, "bf16"), _dev(kw["bias"]), _dev(kw["h0"])
    y, _ = M.gated_scan(xd, gd, cfg, bias=b, h0=h0)
    _same_classes(y, *ref["y"], "bf16", "alone")
    many = lambda t: t.expand(512, *t.shape[1:]).contiguous()
    yb, _ = M.gated_scan(many(xd), many(gd), dataclasses.replace(cfg, B=512), bias=b, h0=many(h0))
    assert torch.equal(yb.view(torch.int16), yb[:1].view(torch.int16).expand_as(yb))
    _same_classes(yb[:1], *ref["y"], "bf16", "batch")
    h, parts = h0, []
    cuts = [0, 100, *range(195, 206), 300]
    for lo, hi in zip(cuts, cuts[1:]):
        yp, h = M.gated_scan(xd[:, lo:hi].contiguous(), gd[:, lo:hi].contiguous(), dataclasses.replace(cfg, T=hi - lo), bias=b, h0=h)
        parts.append(yp)
    _same_classes(torch.cat(parts, dim=1), *ref["y"], "bf16", "parts")


@pytest.mark.parametrize("order,reverse", [(0, False), (0, True)])
def test_gated_scan_in_parts(order, reverse):
    """A video in parts, the last token by token: h_last handed on as h0 gives the whole run's rows and state."""
    cfg = M.GatedScanConfig(B=2, T=150, H=1, W=1, D=40, order=order, reverse=reverse, dtype="f32")
    x, g, _, kw = _scan_inputs(cfg, 7, True)
    ref = OP.gated_scan(x, g, cfg, kw["bias"], kw["h0"])
    h, parts = _dev(kw["h0"]), []
    cuts = [0, 70, 135, *range(136, 151)]
    spans = list(zip(cuts, cuts[1:]))
    for lo, hi in (reversed(spans) if reverse else spans):
        c = dataclasses.replace(cfg, T=hi - lo)
        y, h = M.gated_scan(_dev(x[:, lo:hi]), _dev(g[:, lo:hi]), c, bias=_dev(kw["bias"]), h0=h)
        parts.append(y)
    y = torch.cat(list(reversed(parts)) if reverse else parts, dim=1)
    _close(y, *ref["y"], "f32", "y")
    _close(h, *ref["h_last"], "f32", "h_last")


@pytest.mark.parametrize("cfg", [SCAN[1], SCAN[7], SCAN[13]], ids=_scan_id)
def test_gated_scan_state_in_place(cfg):
    """The last state written over the first, as a stream of calls on one state buffer does, one chunk and several."""
    x, g, _, kw = _scan_inputs(cfg, 17, True)
    xd, gd, b, h0 = _dev(x, cfg.dtype), _dev(g, cfg.dtype), _dev(kw["bias"]), _dev(kw["h0"])
    y, hl = M.gated_scan(xd, gd, cfg, bias=b, h0=h0)
    for _ in range(5):
        h = h0.clone()
        y2, hl2 = M.gated_scan(xd, gd, cfg, bias=b, h0=h, h_last=h)
        assert hl2 is h and torch.equal(y, y2) and torch.equal(hl, h)


def test_gated_scan_gradient_against_differences():
    cfg = M.GatedScanConfig(B=2, T=7, H=3, W=5, D=8, order=3, dtype="f32")
    x, g, dy, kw = _scan_inputs(cfg, 8, True)
    states = M.gated_scan_states(cfg)
    M.gated_scan(_dev(x), _dev(g), cfg, bias=_dev(kw["bias"]), h0=_dev(kw["h0"]), states=states)
    gr = M.gated_scan_backward(_dev(x), _dev(g), states, _dev(dy), cfg, bias=_dev(kw["bias"]), dh_last=_dev(kw["dh_last"]))

    def f(x, g, b, h):
        o = OP.gated_scan(x, g, cfg, b, h)
        return (o["y"][0] * dy).sum() + (o["h_last"][0] * kw["dh_last"]).sum()

    rng, h = np.random.default_rng(9), 1e-5
    base = (x.astype(np.float64), g.astype(np.float64), kw["bias"].astype(np.float64), kw["h0"].astype(np.float64))
    for _ in range(3):
        v = [rng.standard_normal(b.shape) for b in base]
        num = (f(*(b + h * d for b, d in zip(base, v))) - f(*(b - h * d for b, d in zip(base, v)))) / (2 * h)
        terms = [_np(gr[k]) * d for k, d in zip(("dx", "dg", "dbias", "dh0"), v)]
        ana, mag = sum(t.sum() for t in terms), sum(np.abs(t).sum() for t in terms)
        assert abs(num - ana) <= 1e-6 * mag, (num, ana, mag)


# ------------------------------------------------------------------------------------------ 8-bit projection
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M_,K", [(1, 1), (1, 16), (3, 100), (7, 129), (130, 1024), (33, 4096), (2, 20000)])
def test_quantize_rows(M_, K, dtype):
    rng = np.random.default_rng(10)
    x = _host(rng, (M_, K), dtype) * np.exp2(rng.integers(-40, 40, (M_, 1))).astype(np.float32)
    ref_q, ref_s = OP.quantize_rows(x)
    q, s = M.quantize_rows(_dev(np.pad(x, ((0, 0), (0, -K % 8))), dtype)[:, :K])
    np.testing.assert_array_equal(s.cpu().numpy(), ref_s)
    np.testing.assert_array_equal(q.cpu().numpy(), ref_q)


def test_quantize_rows_ties_and_edges():
    """Exact midpoints go to the even neighbour, their fp32 neighbours to their own side; rows of zeros, of the smallest
    and largest values; rows with an infinity or NaN."""
    mid = np.arange(-126, 127) + 0.5
    rows = [np.concatenate([mid, [127.0, -127.0, 0.0]])]
    rows += [np.concatenate([np.nextafter(mid.astype(np.float32), np.float32(to)), [127.0, -127.0, 0.0]])
             for to in (-200, 200)]
    rows += [r * np.float32(2.0 ** e) for r in rows for e in (-100, -20, 3, 100)]
    rows += [r * np.float32(1.37) for r in rows[:3]]
    rows += [np.zeros(256), np.full(256, 1e-45), np.linspace(-3e-44, 3e-44, 256), np.linspace(-1e-38, 1e-38, 256),
             np.linspace(-3.4e38, 3.4e38, 256), np.linspace(-2e-30, 2e-30, 256)]
    for v in (np.inf, -np.inf, np.nan):
        r = np.linspace(-1, 1, 256)
        r[200] = v
        rows.append(r)
    x = np.stack(rows).astype(np.float32)
    ref_q, ref_s = OP.quantize_rows(x)
    q, s = M.quantize_rows(_dev(x))
    np.testing.assert_array_equal(s.cpu().numpy(), ref_s)
    np.testing.assert_array_equal(q.cpu().numpy(), ref_q)


def _quantised(x):
    """(q, scale) of OP.quantize_rows on the GPU: a quotient in 64 bits rounds to 32, or to an integer, as the exact one
    does, since one that is no midpoint of them is 2^-34 of itself or more away from it."""
    scale = (x.abs().amax(1).double() / 127).float()
    q = torch.round(x.double() / scale.double()[:, None]).nan_to_num(0)
    return q.clamp(-127, 127).to(torch.int8), scale


# per type: lengths that a warp holds as 1, 2, 4 and 8 vectors a lane, odd ones among them
WARP_ROWS = {"bf16": (249, 256, 257, 512, 1021, 1024, 2041, 2048), "f32": (125, 128, 255, 256, 511, 512, 1023, 1024)}


@pytest.mark.parametrize("dtype,K", [(d, k) for d in WARP_ROWS for k in WARP_ROWS[d]])
@pytest.mark.parametrize("M_", [901, 20011])
def test_quantize_many_rows(M_, K, dtype):
    """A warp per row, one row or several each."""
    assert M_ >= 6 * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M_, (K + 7) // 8 * 8, generator=gen, device="cuda") * torch.exp2(
        torch.randint(-30, 30, (M_, 1), generator=gen, device="cuda").float())
    x = (x.bfloat16() if dtype == "bf16" else x)[:, :K]
    x[7] = 0
    ref_q, ref_s = _quantised(x.contiguous())
    big = torch.full((M_, (K + 15) // 16 * 16 + 16), 77, dtype=torch.int8, device="cuda")
    q, s = M.quantize_rows(x, q=big[:, :K])
    assert torch.equal(s, ref_s) and torch.equal(q, ref_q) and (big[:, K:] == 77).all()


@pytest.mark.parametrize("dtype,K", [("bf16", 2056), ("bf16", 4801), ("bf16", 12000), ("bf16", 16500),
                                     ("f32", 1028), ("f32", 2303), ("f32", 6000), ("f32", 8300)])
def test_quantize_blocks_of_several_rows(dtype, K):
    """Rows too long for a warp, more of them than blocks."""
    M_ = 8 * torch.cuda.get_device_properties(0).multi_processor_count + 333
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M_, (K + 7) // 8 * 8, generator=gen, device="cuda") * (1 + torch.arange(M_, device="cuda") % 5)[:, None]
    x = (x.bfloat16() if dtype == "bf16" else x)[:, :K]
    q, s = M.quantize_rows(x)
    ref_q, ref_s = _quantised(x)
    assert torch.equal(s, ref_s) and torch.equal(q, ref_q)


@pytest.mark.parametrize("few", [True, False])
def test_quantize_bf16_midpoints(few):
    """Every bf16 row maximum, with all midpoints of the integers' multiples and their bf16 neighbours: rows of a few and of
    many (a block and a warp per row).  Exact midpoints need a scale that is a power of two (maxima 127 * 2^e)."""
    top = torch.arange(1, 0x7f80, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    if few:
        top = torch.cat((top[::97], 127 * torch.exp2(torch.arange(-90, 90, 9, device="cuda")).bfloat16()))[:880]
    mid = torch.arange(-126, 126, device="cuda") + 0.5
    near = ((top.double() / 127)[:, None] * mid).bfloat16()
    step = near.view(torch.int16)
    x = torch.cat([top[:, None], near, (step - 1).view(torch.bfloat16), (step + 1).view(torch.bfloat16)], dim=1)
    # the tiniest rows' midpoints round to 0 and to the maximum: neighbours that leave the row's range are left out
    x = torch.where(x.abs() <= top[:, None], x, torch.zeros_like(x))
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 8))
    ref_q, ref_s = _quantised(x)
    q, s = M.quantize_rows(x)
    assert torch.equal(s, ref_s) and torch.equal(q, ref_q)
    exact = (x.double() / ref_s.double()[:, None] % 1 == 0.5).any(1)
    assert exact.any() and (few or len(x) >= 6 * torch.cuda.get_device_properties(0).multi_processor_count)


@pytest.mark.parametrize("K", [769, 1024])
def test_project_int8_f32_streams_long_rows(K):
    """fp32 output beyond 768 bytes of K: the weights are streamed where bf16 output keeps them, to the same sums."""
    assert _int8_rule(20000, K, 600, "f32") == (256, False) and _int8_rule(20000, K, 600, "bf16") == (256, True)
    gen = torch.Generator(device="cuda").manual_seed(K)
    A, W = (torch.randint(-128, 128, (r, (K + 15) // 16 * 16), generator=gen, device="cuda", dtype=torch.int8)[:, :K]
            for r in (20000, 600))
    one = torch.ones(20000, device="cuda")
    out = M.project_int8(A, one, W, one[:600], out_dtype=torch.float32)
    assert torch.equal(out.double(), A.double() @ W.double().t())   # sums below 2^24: exact in fp32, too
    assert torch.equal(M.project_int8(A, one, W, one[:600]), out.bfloat16())


INT8 = [(1, 16, 1), (1, 1024, 96), (2, 2048, 1001), (5, 100, 37), (8, 4096, 4096), (9, 1040, 513), (16, 512, 264),
        (17, 256, 256), (64, 333, 2048), (129, 128, 255), (257, 144, 288), (300, 1024, 1000), (513, 2048, 520), (1000, 80, 4368),
        (2000, 1024, 300), (600, 48, 19240), (10000, 250, 600), (4000, 1025, 777), (4, 4096, 100), (3, 31, 9),
        (16, 1024, 6000), (40, 4096, 70)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M_,K,N", INT8)
def test_project_int8(M_, K, N, dtype):
    rng = np.random.default_rng(11)
    pad = lambda k: k + (-k % 16)
    A = rng.integers(-128, 128, (M_, pad(K))).astype(np.int8)    # the padding holds values too: they do not count
    W = rng.integers(-128, 128, (N, pad(K))).astype(np.int8)
    A[0], W[-1] = -128, -128
    sa, sw, bias = (rng.uniform(0.5, 2, n).astype(np.float32) / 127 for n in (M_, N, N))
    ref, bound = OP.project_int8(A[:, :K], sa, W[:, :K], sw)
    dA, dW, dsa, dsw, db = (torch.as_tensor(a).cuda() for a in (A, W, sa, sw, bias * 127))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = M.project_int8(dA[:, :K], dsa, dW[:, :K], dsw, out_dtype=dt)
    _close(out, ref, bound, dtype, "no bias")
    ref, bound = OP.project_int8(A[:, :K], sa, W[:, :K], sw, bias * 127)
    for shift in (8, 1):   # rows of C that start on 16 bytes, and not
        big = torch.full((M_, N + (-N % 8) + 16 + (shift == 1)), float("nan"), dtype=dt, device="cuda")
        view = big[:, 8:8 + N]
        M.project_int8(dA[:, :K], dsa, dW[:, :K], dsw, bias=db, out=view)
        _close(view, ref, bound, dtype, f"bias, strided {shift}")
        assert torch.isnan(big[:, :8]).all() and torch.isnan(big[:, 8 + N:]).all()
    assert M.device_status() == 0


def _int8_rule(M_, K, N, dtype):
    """(tile columns, whether W's column tiles are kept in shared memory) that the library's rule gives on this GPU."""
    up = lambda a, b: -(-a // b)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    mb, bn = up(M_, 256), 256
    if mb * up(N, 256) < pairs:
        bn = min((256, 128, 64, 32), key=lambda b: up(mb * up(N, b), pairs) * (b + 32))
    nt = up(N, bn)
    slots = min(nt, pairs)
    groups = min(pairs // slots, mb)
    return bn, K <= (1024 if dtype == "bf16" else 768) and bn == 256 and up(nt, slots) * up(mb, groups) < 1.1 * up(mb * nt, min(mb * nt, pairs))


@pytest.mark.parametrize("M_,K,N,dtype", [
    (65536, 1024, 512, "bf16"), (65536, 768, 512, "f32"),    # 7 row tiles a pair, the ring of A wraps, accumulators reused
    (20000, 1000, 600, "bf16"), (20000, 700, 600, "f32"),    # the last block of K and the last tiles cut
    (512, 144, 37888, "bf16"), (512, 144, 37888, "f32"),     # a second column tile over the first
    (512, 1000, 56700, "bf16"), (512, 760, 56700, "f32")])   # a third one, cut, with more blocks of K than the ring holds
def test_project_int8_kept_weights(M_, K, N, dtype):
    """W kept in shared memory while a pair walks down the rows: reused accumulators and ring stages, column tiles loaded
    over earlier ones; launch after launch, since a CTA may not leave before its last arrivals are in."""
    assert _int8_rule(M_, K, N, dtype) == (256, True)
    gen = torch.Generator(device="cuda").manual_seed(M_ + K)
    ints = lambda r: torch.randint(-128, 128, (r, (K + 15) // 16 * 16), generator=gen, device="cuda", dtype=torch.int8)[:, :K]
    A, W = ints(M_), ints(N)
    sa, sw = ((0.5 + torch.rand(n, generator=gen, device="cuda")) / 127 for n in (M_, N))
    bias = torch.randn(N, generator=gen, device="cuda")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    outs = [M.project_int8(A, sa, W, sw, bias=bias, out_dtype=dt) for _ in range(4)]
    again = outs[1]
    for _ in range(20):
        M.project_int8(A, sa, W, sw, bias=bias, out=again)
    assert M.device_status() == 0
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    for r in range(0, M_, 8192):   # integers below 2^53 add up exactly in 64 bits
        v = (A[r:r + 8192].double() @ W.double().t()) * sa[r:r + 8192, None].double() * sw.double()
        ref, bound = v + bias.double(), 4 * OP.EPS32 * (v.abs() + bias.double().abs())
        tol = OP.half_step(dtype) * (ref.abs() + bound) + bound
        assert ((outs[0][r:r + 8192].double() - ref).abs() <= tol).all(), r


def test_project_int8_largest_sums():
    """The longest K with all products at their largest: the sum stays exact in 32 bits (2^31 - 16384)."""
    K = 131071
    A = torch.full((3, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    W = torch.full((40, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    one = torch.ones(40, device="cuda")
    out = M.project_int8(A, one[:3].contiguous(), W, one, out_dtype=torch.float32)
    want = np.float32(K * 16384)
    assert (out.cpu().numpy() == want).all()


def test_project_int8_empty_and_nan_rows():
    W, sw = torch.ones((24, 32), dtype=torch.int8, device="cuda"), torch.ones(24, device="cuda")
    q, s = M.quantize_rows(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    assert M.project_int8(q, s, W, sw).shape == (0, 24)
    x = torch.randn(4, 32, device="cuda")
    x[1, 3], x[2] = float("inf"), 0
    q, s = M.quantize_rows(x)
    out = M.project_int8(q, s, W, sw, out_dtype=torch.float32)
    assert torch.isnan(out[1]).all() and (out[2] == 0).all() and torch.isfinite(out[[0, 3]]).all()


# ------------------------------------------------------------------------------------------------ alignment
def _at8(t):
    """The same values in a tensor that starts 8 bytes behind a multiple of 16."""
    n = 8 // t.element_size()
    big = torch.zeros(t.numel() + n, dtype=t.dtype, device=t.device)
    big[n:] = t.flatten()
    return big[n:].view(t.shape)


def test_vectors_on_8_bytes():
    """Weights, biases, scales and states that are slices of larger tensors: the same bits as on 16 bytes."""
    qk = QK[2]
    rng, qkv, (wq, wk), tabs, _ = _qk_inputs(qk, 26)
    x, d, wq, wk = _dev(qkv, "bf16"), _dev(_host(rng, qkv.shape, "bf16"), "bf16"), _dev(wq), _dev(wk)
    tabs8 = [_at8(t) for t in tabs]
    assert torch.equal(M.qk_norm_rope(x, wq, wk, tabs, qk), M.qk_norm_rope(x, _at8(wq), _at8(wk), tabs8, qk))
    want, got = M.qk_norm_rope_backward(x, wq, wk, tabs, d, qk), M.qk_norm_rope_backward(x, _at8(wq), _at8(wk), tabs8, d, qk)
    assert all(torch.equal(want[k], got[k]) for k in want)
    for cfg in (SCAN[2], SCAN[7], SCAN[11]):
        x, g, dy, kw = _scan_inputs(cfg, 27, True)
        x, g, dy, kw = _dev(x, cfg.dtype), _dev(g, cfg.dtype), _dev(dy, cfg.dtype), {k: _dev(v) for k, v in kw.items()}
        kw8 = {k: _at8(v) for k, v in kw.items()}
        res = []
        for w, at in ((kw, lambda t: t), (kw8, _at8)):
            st, hl = at(M.gated_scan_states(cfg)), at(torch.zeros((cfg.B, cfg.D), device="cuda"))
            y, _ = M.gated_scan(x, g, cfg, bias=w["bias"], h0=w["h0"], h_last=hl, states=st)
            res.append((y, hl, *M.gated_scan_backward(x, g, st, dy, cfg, bias=w["bias"], dh_last=w["dh_last"]).values()))
        assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M_,K,N", [(2, 256, 96), (300, 1024, 1000), (20000, 1000, 600)])
def test_project_int8_on_8_bytes(M_, K, N, dtype):
    """Scales and biases of some of the channels, and an output whose rows start 8 bytes behind a multiple of 16."""
    gen = torch.Generator(device="cuda").manual_seed(28)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    A, W = (torch.randint(-127, 128, (r, (K + 15) // 16 * 16), generator=gen, device="cuda", dtype=torch.int8)[:, :K]
            for r in (M_, N))
    sa, sw, b = (torch.rand(n, generator=gen, device="cuda") for n in (M_, N, N))
    want = M.project_int8(A, sa, W, sw, bias=b, out_dtype=dt)
    c0 = 8 // want.element_size()
    big = torch.full((M_, N + (-N % 8) + 16), float("nan"), dtype=dt, device="cuda")
    M.project_int8(A, sa, W, _at8(sw), bias=_at8(b), out=big[:, c0:c0 + N])
    assert torch.equal(big[:, c0:c0 + N], want)
    assert torch.isnan(big[:, :c0]).all() and torch.isnan(big[:, c0 + N:]).all()


def test_refusals_name_the_tensor():
    """What starts at an odd place is refused by name."""
    A, s = torch.ones((4, 32), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(_lib.MateError, match="w_scale: starts 4 bytes"):
        M.project_int8(A, s[:4], A, s[1:5])
    with pytest.raises(_lib.MateError, match="out: starts 2 bytes"):
        M.project_int8(A, s[:4], A, s[:4], out=torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")[:, 1:5])
    with pytest.raises(_lib.MateError, match="x: .* rows 200 bytes apart"):
        M.quantize_rows(torch.zeros((4, 100), dtype=torch.bfloat16, device="cuda"))
    cfg = M.GatedScanConfig(B=1, T=4, H=1, W=1, D=32, dtype="f32")
    x = torch.zeros((4, 32), device="cuda")
    with pytest.raises(_lib.MateError, match="h0: starts 4 bytes"):
        M.gated_scan(x, x, cfg, h0=s[1:33])


# ---------------------------------------------------------------------------- graphs, streams, the run together
def _together_ref(cfg, qk, gs, w):
    """The mixing block in fp64, with the rounding of every stored tensor."""
    r16 = lambda a: mi.round_to_bf16(np.asarray(a, np.float32)).astype(np.float64)
    q, s = OP.quantize_rows(w["x"])
    z = r16(OP.project_int8(q, s, w["wq8"], w["ws"])[0])
    a = qk.width
    qkv = r16(OP.qk_norm_rope(z[:, :a], w["nq"], w["nk"], w["tabs"], qk)[0])
    from oracle import mate_oracle as O
    att = r16(O.tesa_attention(qkv.reshape(cfg.T, cfg.H, cfg.W, -1), cfg.th, cfg.tp, (cfg.wt, cfg.wh, cfg.ww),
                               (cfg.st, cfg.sh, cfg.sw), True))
    ys = [r16(OP.gated_scan(z[:, a:a + gs.D], z[:, a + gs.D:], dataclasses.replace(gs, reverse=rev))["y"][0])
          for rev in (False, True)]
    cat = np.concatenate([att.reshape(cfg.n, -1), ys[0][0], ys[1][0]], axis=1)
    return cat, cat @ w["wo"].astype(np.float64).T


def test_run_together():
    """One mixing block: 8-bit projection to q | k | v | x | g rows, q/k norm with rotation in place, window attention
    on the rows, the gated scan both ways over the x and g columns, and the out-projection of all three."""
    cfg = dataclasses.replace(mi.TEST_CONFIGS["bf16_b2_20x16x16_d512"], B=1, T=8, R=0)
    a, D, n = 3 * cfg.th * cfg.tp, 256, cfg.n
    qk = M.QkConfig(B=1, T=cfg.T, H=cfg.H, W=cfg.W, hq=cfg.th, hk=cfg.th, hv=cfg.th, tp=cfg.tp, rt=32, rh=48, rw=48)
    gs = M.GatedScanConfig(B=1, T=cfg.T, H=cfg.H, W=cfg.W, D=D, order=2)
    rng = np.random.default_rng(12)
    w = dict(x=_host(rng, (n, cfg.d), "bf16"))
    W = rng.standard_normal((a + 2 * D, cfg.d)) / np.sqrt(cfg.d)
    w["wq8"], w["ws"] = OP.quantize_rows(W)
    w["nq"], w["nk"] = ((1 + 0.2 * rng.standard_normal(cfg.tp)).astype(np.float32) for _ in range(2))
    w["wo"] = _host(rng, (cfg.d, cfg.th * cfg.tp + 2 * D), "bf16", 1 / 32)
    tabs = [M.rope_table(k, r) for k, r in zip((cfg.T, cfg.H, cfg.W), (32, 48, 48))]
    w["tabs"] = [t.cpu().numpy() for t in tabs]
    cat_ref, ref = _together_ref(cfg, qk, gs, w)
    x, wq8, ws, wo = _dev(w["x"], "bf16"), torch.as_tensor(w["wq8"]).cuda(), _dev(w["ws"]), _dev(w["wo"], "bf16")
    nq, nk = _dev(w["nq"]), _dev(w["nk"])
    ao = cfg.th * cfg.tp

    def block():
        z = M.project_int8(*M.quantize_rows(x), wq8, ws)
        qkv = M.qk_norm_rope(z[:, :a], nq, nk, tabs, qk, out=torch.empty((n, a), dtype=torch.bfloat16, device="cuda"))
        cat = torch.empty((n, ao + 2 * D), dtype=torch.bfloat16, device="cuda")
        cat[:, :ao] = M.tesa_forward(qkv, True, cfg).view(n, ao)
        M.gated_scan(z[:, a:a + D], z[:, a + D:], gs, y=cat[:, ao:ao + D])
        M.gated_scan(z[:, a:a + D], z[:, a + D:], dataclasses.replace(gs, reverse=True), y=cat[:, ao + D:])
        return cat, M.project_bf16(cat, wo)

    cat, out = block()
    # the reference rounds every stored tensor as the kernels do, so what differs are values next to a rounding
    # border: half a step of the stored type, carried through at most four stored tensors
    for got, want in ((cat, cat_ref), (out, ref)):
        rms = np.sqrt((want ** 2).mean())
        assert np.sqrt(((_np(got) - want) ** 2).mean()) <= 4 * 2.0 ** -8 * rms
    # captured and replayed: the same bits, new inputs included
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cat_g, out_g = block()
    for k in range(2):
        x.copy_(_dev(_host(np.random.default_rng(20 + k), (n, cfg.d), "bf16"), "bf16"))
        graph.replay()
        cat_e, out_e = block()
        torch.cuda.synchronize()
        assert torch.equal(cat_g, cat_e) and torch.equal(out_g, out_e)
    assert M.device_status() == 0


def test_training_run_together():
    """q/k norm -> window attention and back: the chained gradients of the library against the chained fp64 ones."""
    from oracle import backward as BW, mate_oracle as O
    cfg = dataclasses.replace(mi.TEST_CONFIGS["bf16_b2_20x16x16_d512"], B=1, T=8, R=0, th=1)
    qk = M.QkConfig(B=1, T=cfg.T, H=cfg.H, W=cfg.W, hq=1, hk=1, hv=1, tp=cfg.tp, rt=32, rh=48, rw=48, pairing="halves")
    rng, qkv, (wq, wk), tabs, tabs_h = _qk_inputs(qk, 13)
    qkv = _host(rng, qkv.shape, "bf16")
    dO = _host(rng, (cfg.n, cfg.tp), "bf16")
    win, sh = (cfg.wt, cfg.wh, cfg.ww), (cfg.st, cfg.sh, cfg.sw)
    mid = mi.round_to_bf16(OP.qk_norm_rope(qkv, wq, wk, tabs_h, qk)[0].astype(np.float32))
    grid = (cfg.T, cfg.H, cfg.W, -1)
    dmid = BW.tesa_attention_backward(mid.reshape(grid), 1, cfg.tp, win, sh, True, dO.reshape(grid))
    ref, _, dws, _ = OP.qk_norm_rope_backward(qkv, wq, wk, tabs_h, dmid, qk)
    x = _dev(qkv, "bf16")
    m = M.qk_norm_rope(x, _dev(wq), _dev(wk), tabs, qk)
    o = M.tesa_forward(m, True, cfg)
    dm = M.tesa_backward(m, o, _dev(dO, "bf16"), True, cfg)
    g = M.qk_norm_rope_backward(x, _dev(wq), _dev(wk), tabs, dm, qk, dqkv=dm)
    # the attention's own gradient is good to 2e-2 of its largest value; the norm's backward adds three roundings
    for got, want in ((g["dqkv"], ref), (g["dwq"], dws[0]), (g["dwk"], dws[1])):
        got = _np(got).reshape(want.shape)
        assert np.abs(got - want).max() <= 2.5e-2 * np.abs(want).max()


def test_streams():
    """Calls on two streams at once, each with memory of its own, and a stream that is not the current one."""
    cfg = M.GatedScanConfig(B=1, T=3000, H=1, W=1, D=128, order=0)
    qk = QK[2]
    x, g, _, kw = _scan_inputs(cfg, 14, True)
    xd, gd, b, h0 = _dev(x, "bf16"), _dev(g, "bf16"), _dev(kw["bias"]), _dev(kw["h0"])
    _, qkv, (wq, wk), tabs, _ = _qk_inputs(qk, 15)
    qd, wq, wk = _dev(qkv, "bf16"), _dev(wq), _dev(wk)
    want_y, want_h = M.gated_scan(xd, gd, cfg, bias=b, h0=h0)
    want_q = M.qk_norm_rope(qd, wq, wk, tabs, qk)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        for s in (s1, s2):
            got.append((M.gated_scan(xd, gd, cfg, bias=b, h0=h0, stream=s), M.qk_norm_rope(qd, wq, wk, tabs, qk, stream=s)))
    torch.cuda.synchronize()
    for (y, h), q in got:
        assert torch.equal(y, want_y) and torch.equal(h, want_h) and torch.equal(q, want_q)
    assert M.device_status() == 0


def _everything(seed):
    """One call of every operator, forward and backward, that returns all outputs; and its inputs, to be changed between runs."""
    qk, gs = QK[3], dataclasses.replace(SCAN[7], T=700, D=264)
    rng, qkv, (wq, wk), tabs, _ = _qk_inputs(qk, seed)
    x, g, dy, kw = _scan_inputs(gs, seed, True)
    W, sw = M.quantize_rows(_dev(rng.standard_normal((5000, 304))))
    io = dict(qkv=_dev(qkv, "bf16"), dz=_dev(_host(rng, qkv.shape, "bf16"), "bf16"), x=_dev(x, "bf16"), g=_dev(g, "bf16"),
              dy=_dev(dy, "bf16"), a=_dev(rng.standard_normal((12000, 304)), "bf16"))
    wq, wk, bias, sb = _dev(wq), _dev(wk), _dev(kw["bias"]), _dev(rng.standard_normal(5000))
    h0, dhl = _dev(kw["h0"]), _dev(kw["dh_last"])

    def run():
        out = [M.qk_norm_rope(io["qkv"], wq, wk, tabs, qk)]
        out += M.qk_norm_rope_backward(io["qkv"], wq, wk, tabs, io["dz"], qk).values()
        st = M.gated_scan_states(gs)
        out += M.gated_scan(io["x"], io["g"], gs, bias=bias, h0=h0, states=st)
        out += M.gated_scan_backward(io["x"], io["g"], st, io["dy"], gs, bias=bias, dh_last=dhl).values()
        q, s = M.quantize_rows(io["a"])
        for rows, dt in ((12000, torch.bfloat16), (12000, torch.float32), (40, torch.bfloat16), (3, torch.float32)):
            out.append(M.project_int8(q[:rows], s[:rows], W, sw, bias=sb, out_dtype=dt))
        return out

    return io, run


def test_training_graphs_replayed_beside_each_other():
    """Every forward and backward pass captured into two graphs that are replayed at the same time on two streams, with new
    inputs, beside eager calls on a third: the bits of eager calls alone."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    graphs, ios, runs, outs = [], [], [], []
    for k, s in enumerate(sides):
        io, run = _everything(30 + k)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(run())
        graphs.append(graph), ios.append(io), runs.append(run)
    for rep in range(3):
        for io in ios:
            for t in io.values():
                t.copy_(t.flip(0) * (0.5 + rep))
        want = [run() for run in runs]
        torch.cuda.synchronize()
        for s, graph in zip(sides, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        beside = runs[0]()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert len(w) == len(o) and all(torch.equal(a, b) for a, b in zip(w, o))
        assert all(torch.equal(a, b) for a, b in zip(want[0], beside))
    assert M.device_status() == 0


def test_offsets_past_32_bits():
    """Rows a million elements apart, so that the last ones lie more than 2^32 elements in: the bits of packed rows."""
    ld, rows = (1 << 20) + 32, 4200
    assert ld * rows > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(33)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    big = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")

    def far(t, at):
        view = big[:, at:at + t.shape[1]]
        view.copy_(t)
        return view

    none = torch.zeros((rows, 1), dtype=torch.bfloat16, device="cuda")
    qk = M.QkConfig(B=2, T=21, H=10, W=10, hq=2, hk=1, hv=1, tp=64, rt=16, rh=24, rw=24)
    tabs, w = [M.rope_table(n, r) for n, r in ((21, 16), (10, 24), (10, 24))], torch.rand(64, generator=gen, device="cuda")
    x, d = rnd(rows, 256), rnd(rows, 256)
    want, got = M.qk_norm_rope(x, w, w, tabs, qk), far(none.expand(rows, 256), 1024)
    M.qk_norm_rope(far(x, 0), w, w, tabs, qk, out=got)
    assert torch.equal(got, want)
    want = M.qk_norm_rope_backward(x, w, w, tabs, d, qk)
    grads = M.qk_norm_rope_backward(far(x, 0), w, w, tabs, far(d, 512), qk, dqkv=got)
    assert all(torch.equal(grads[k], want[k]) for k in want)
    gs = M.GatedScanConfig(B=2, T=21, H=10, W=10, D=256, order=3, reverse=True)
    g, st, st2 = rnd(rows, 256), M.gated_scan_states(gs), M.gated_scan_states(gs)
    y, hl = M.gated_scan(x, g, gs, states=st)
    yf, hf = M.gated_scan(far(x, 0), far(g, 512), gs, y=got, states=st2)
    assert torch.equal(yf, y) and torch.equal(hf, hl) and torch.equal(st, st2)
    want = M.gated_scan_backward(x, g, st, d, gs)
    dx, dg = far(none.expand(rows, 256), 2048), far(none.expand(rows, 256), 4096)
    grads = M.gated_scan_backward(big[:, :256], big[:, 512:768], st, far(d, 1024), gs, dx=dx, dg=dg)
    assert all(torch.equal(grads[k], want[k]) for k in want)
    wide = torch.empty((rows, ld), dtype=torch.int8, device="cuda")
    q, s = M.quantize_rows(x)
    qf, sf = M.quantize_rows(big[:, :256], q=wide[:, 64:320])
    assert torch.equal(qf, q) and torch.equal(sf, s)
    W, sw = M.quantize_rows(rnd(300, 256))
    want = M.project_int8(q, s, W, sw)
    assert torch.equal(M.project_int8(qf, s, W, sw, out=big[:, 8192:8192 + 300]), want)
    assert torch.equal(M.project_int8(qf[-3:], s[-3:], W, sw, out=big[-3:, 8192:8192 + 300]), want[-3:])
    # the weights' rows as far apart
    Wf = wide[:, 512:768]
    Wf.copy_(q)
    assert torch.equal(M.project_int8(q[:64], s[:64], Wf, s), M.project_int8(q[:64], s[:64], q, s))
    assert torch.equal(M.project_int8(q[:2], s[:2], Wf, s), M.project_int8(q[:2], s[:2], q, s))
