"""Host-side checks of the operators beside the block (no GPU): every refusal comes before any device work."""
import copy
import ctypes
import pickle

import numpy as np
import pytest

from linear_complexity_video_mate_b200 import _lib, build
from oracle import operators as OP

torch = pytest.importorskip("torch")
from linear_complexity_video_mate_b200 import mate as M  # noqa: E402

OK, ARG, SHAPE, WS, UNS = (_lib.MATE_OK, _lib.MATE_ERR_ARG, _lib.MATE_ERR_SHAPE, _lib.MATE_ERR_WORKSPACE,
                           _lib.MATE_ERR_UNSUPPORTED)
F, MIS = 1 << 20, (1 << 20) + 4      # never dereferenced: aligned to 16 bytes, and to 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _refused(fn, args, changes):
    for kw, want in changes:
        a = dict(args, **kw)
        assert fn(*a.values()) == want, kw


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hk=0), SHAPE), (dict(hv=-1), SHAPE),
    (dict(tp=0), SHAPE), (dict(tp=12), SHAPE), (dict(tp=264), UNS), (dict(rt=3), SHAPE), (dict(rt=-2), SHAPE),
    (dict(rt=64, rh=64, rw=2), SHAPE), (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(T=1 << 16, H=1 << 15), SHAPE), (dict(T=1 << 30, H=1 << 30, W=1 << 30), SHAPE), (dict(hq=1 << 30), SHAPE),
])
def test_qk_config_refusals(lib, kw, want):
    base = dict(B=2, T=3, H=4, W=5, hq=4, hk=4, hv=4, tp=128, rt=32, rh=48, rw=48)
    c = M.QkConfig(**{**base, **kw}).ccfg
    assert lib.mate_qk_norm_rope(F, 1 << 20, F, F, F, F, F, F, 1 << 20, ctypes.byref(c), None) == want
    assert lib.mate_qk_norm_rope_backward_workspace_bytes(ctypes.byref(c)) == 0
    assert lib.mate_qk_norm_rope_backward(F, 1 << 20, F, F, F, F, F, F, 1 << 20, F, 1 << 20, F, F, ctypes.byref(c), F,
                                          1 << 40, None) == want


def test_qk_argument_refusals(lib):
    cfg = M.QkConfig(B=2, T=3, H=4, W=5, hq=4, hk=4, hv=4, tp=128, rt=32, rh=48, rw=48)
    c, wd = ctypes.byref(cfg.ccfg), cfg.width
    args = dict(qkv=F, ldi=wd, wq=F, wk=F, tt=F, th=F, tw=F, out=2 * F, ldo=wd, cfg=c, stream=None)
    both = [(dict(qkv=None), ARG), (dict(qkv=MIS), ARG), (dict(ldi=wd - 8), ARG), (dict(ldi=wd + 4), ARG),
            (dict(wq=MIS), ARG), (dict(wk=MIS), ARG), (dict(tt=None), ARG), (dict(th=MIS), ARG), (dict(tw=None), ARG)]
    _refused(lib.mate_qk_norm_rope, args, both + [
        (dict(out=None), ARG), (dict(out=MIS), ARG), (dict(ldo=wd - 8), ARG), (dict(out=F, ldo=wd + 8), ARG),
        (dict(cfg=None), ARG)])
    nb = lib.mate_qk_norm_rope_backward_workspace_bytes(c)
    assert nb > 0
    args = dict(qkv=F, ldi=wd, wq=F, wk=F, tt=F, th=F, tw=F, dout=2 * F, ldg=wd, dqkv=3 * F, ldd=wd, dwq=F, dwk=F, cfg=c,
                ws=F, nb=nb, stream=None)
    _refused(lib.mate_qk_norm_rope_backward, args, both + [
        (dict(dout=None), ARG), (dict(dout=MIS), ARG), (dict(dqkv=None), ARG), (dict(ws=None), ARG), (dict(ws=MIS), ARG),
        (dict(ldg=wd - 8), ARG), (dict(ldd=wd + 4), ARG), (dict(dqkv=2 * F, ldd=wd + 8), ARG),
        (dict(dqkv=F, ldd=wd + 8), ARG), (dict(nb=nb - 1), WS)])
    for args, want in (((None, 0, 4, 8, 1e4), ARG), ((MIS, 0, 4, 8, 1e4), ARG), ((F, 0, 0, 8, 1e4), SHAPE),
                       ((F, 0, 4, 7, 1e4), SHAPE), ((F, 0, 4, 0, 1e4), SHAPE), ((F, 0, 4, 8, 0.0), ARG),
                       ((F, 0, 4, 8, float("inf")), ARG)):
        assert lib.mate_rope_table(*args, None) == want, args


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), SHAPE), (dict(W=0), SHAPE), (dict(D=0), SHAPE), (dict(D=12), SHAPE), (dict(order=4), ARG),
    (dict(order=-1), ARG), (dict(T=1 << 16, H=1 << 15), SHAPE),
])
def test_gated_scan_config_refusals(lib, kw, want):
    c = ctypes.byref(M.GatedScanConfig(**{**dict(B=2, T=3, H=4, W=5, D=64), **kw}).ccfg)
    assert lib.mate_gated_scan(F, 64, 2 * F, 64, None, None, 3 * F, 64, None, None, c, F, 1 << 40, None) == want
    assert lib.mate_gated_scan_backward(F, 64, 2 * F, 64, None, F, 3 * F, 64, None, 4 * F, 64, 5 * F, 64, None, None, c, F,
                                        1 << 40, None) == want
    for q in (lib.mate_gated_scan_workspace_bytes, lib.mate_gated_scan_states_bytes,
              lib.mate_gated_scan_backward_workspace_bytes):
        assert q(c) == 0


def test_gated_scan_argument_refusals(lib):
    cfg = M.GatedScanConfig(B=2, T=30, H=4, W=5, D=64)
    c = ctypes.byref(cfg.ccfg)
    nb, ns = lib.mate_gated_scan_workspace_bytes(c), lib.mate_gated_scan_states_bytes(c)
    assert nb > 0 and ns >= 2 * 64 * 4
    args = dict(x=F, ldx=64, g=2 * F, ldg=64, bias=F, h0=F, y=3 * F, ldy=64, hl=F, st=F, cfg=c, ws=F, nb=nb, stream=None)
    _refused(lib.mate_gated_scan, args, [
        (dict(x=None), ARG), (dict(g=None), ARG), (dict(y=None), ARG), (dict(ws=None), ARG), (dict(x=MIS), ARG),
        (dict(bias=MIS), ARG), (dict(h0=MIS), ARG), (dict(hl=MIS), ARG), (dict(st=MIS), ARG), (dict(ldx=56), ARG),
        (dict(ldg=68), ARG), (dict(ldy=60), ARG), (dict(y=F), ARG), (dict(y=2 * F), ARG), (dict(nb=nb - 1), WS),
        (dict(cfg=None), ARG)])
    nb = lib.mate_gated_scan_backward_workspace_bytes(c)
    args = dict(x=F, ldx=64, g=2 * F, ldg=64, bias=F, st=F, dy=3 * F, lddy=64, dhl=F, dx=4 * F, lddx=64, dg=5 * F, lddg=64,
                db=F, dh0=F, cfg=c, ws=F, nb=nb, stream=None)
    _refused(lib.mate_gated_scan_backward, args, [
        (dict(x=None), ARG), (dict(st=None), ARG), (dict(dy=None), ARG), (dict(dx=None), ARG), (dict(dg=None), ARG),
        (dict(ws=None), ARG), (dict(dy=MIS), ARG), (dict(dhl=MIS), ARG), (dict(db=MIS), ARG), (dict(dh0=MIS), ARG),
        (dict(lddy=56), ARG), (dict(lddx=60), ARG), (dict(lddg=56), ARG), (dict(dx=F), ARG), (dict(dg=3 * F), ARG),
        (dict(dx=5 * F), ARG), (dict(nb=nb - 1), WS)])


def test_int8_argument_refusals(lib):
    args = dict(x=F, ldx=64, M=4, K=64, dt=0, q=2 * F, ldq=64, s=F, stream=None)
    _refused(lib.mate_quantize_rows, args, [
        (dict(x=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG), (dict(x=MIS), ARG), (dict(q=MIS), ARG),
        (dict(s=F + 2), ARG), (dict(ldx=56), ARG), (dict(ldx=68), ARG), (dict(ldq=72), ARG), (dict(ldq=48), ARG),
        (dict(M=-1), ARG), (dict(K=0), ARG), (dict(dt=2), ARG), (dict(M=1 << 31), ARG), (dict(M=0), OK)])
    args = dict(A=F, lda=64, sa=F, M=4, K=64, W=2 * F, ldw=64, sw=F, N=32, bias=F, C=3 * F, ldc=32, dt=0, stream=None)
    _refused(lib.mate_project_int8, args, [
        (dict(A=None), ARG), (dict(sa=None), ARG), (dict(W=None), ARG), (dict(sw=None), ARG), (dict(C=None), ARG),
        (dict(A=MIS), ARG), (dict(W=MIS), ARG), (dict(C=MIS), ARG), (dict(sw=MIS), ARG), (dict(bias=MIS), ARG),
        (dict(sa=F + 1), ARG), (dict(lda=72), ARG), (dict(ldw=48), ARG), (dict(ldc=31), ARG), (dict(M=-1), ARG),
        (dict(K=0), ARG), (dict(N=0), ARG), (dict(dt=2), ARG), (dict(K=131072, lda=131072, ldw=131072), UNS),
        (dict(M=0), OK)])


def test_int8_sizes_next_to_the_index_range(lib):
    """Row and column counters are 32-bit and run past the last row or column before they are compared: sizes that leave
    them no room below 2^31 are refused (one more than the documented most; the largest a caller can pass)."""
    most, top = (1 << 31) - (1 << 14), (1 << 31) - 16
    for n in (most + 1, (1 << 31) - 9472, (1 << 31) - 256, (1 << 31) - 1):
        for dt in (0, 1):
            assert lib.mate_quantize_rows(F, 16, n, 8, dt, 2 * F, 16, F, None) == ARG, n
            assert lib.mate_project_int8(F, 16, F, n, 16, 2 * F, 16, F, 32, None, 3 * F, 32, dt, None) == ARG, n
            assert lib.mate_project_int8(F, 16, F, 4, 16, 2 * F, 16, F, n, None, 3 * F, (1 << 31) - 1, dt, None) == ARG, n
    for k in (most + 1, (1 << 31) - 256, top):
        assert lib.mate_quantize_rows(F, top, 1, k, 0, 2 * F, top, F, None) == ARG, k


def test_binding_refusals():
    """The Python layer names the argument: wrong type, shape, place or stride (CPU tensors stand in)."""
    cfg = M.QkConfig(B=1, T=2, H=1, W=1, hq=1, hk=1, hv=1, tp=16)
    gs = M.GatedScanConfig(B=1, T=2, H=1, W=1, D=16)
    x = torch.zeros(2, 48, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="qkv"):
        M.qk_norm_rope(x, None, None, (None, None, None), cfg)
    with pytest.raises(ValueError, match="qkv"):
        M.qk_norm_rope_backward(x, None, None, (None, None, None), x, cfg)
    with pytest.raises(ValueError, match="x:"):
        M.gated_scan(x[:, :16], x[:, :16], gs)
    with pytest.raises(ValueError, match="x:"):
        M.quantize_rows(x)
    with pytest.raises(ValueError, match="x:"):
        M.quantize_rows(x[0])
    with pytest.raises(ValueError, match="x:"):
        M.quantize_rows(x.half())
    with pytest.raises(ValueError, match="A"):
        M.project_int8(x.to(torch.int8), x, x.to(torch.int8), x)
    with pytest.raises(ValueError, match="pairing"):
        M.QkConfig(B=1, T=2, H=1, W=1, hq=1, hk=1, hv=1, tp=16, pairing="odd")
    with pytest.raises(ValueError, match="dtype"):
        M.GatedScanConfig(B=1, T=2, H=1, W=1, D=16, dtype="f16")
    with pytest.raises(ValueError, match="T ="):
        M.GatedScanConfig(B=1, T=1 << 32, H=1, W=1, D=16)


def test_binding_sizes_are_not_cut():
    """Sizes of 2^32 and a little fit a 64-bit tensor, not the library's ints: refused, where cut to 32 bits they would be
    a small job that leaves most of the output unwritten (expanded CPU tensors stand in)."""
    wide = lambda rows, cols, dtype: torch.zeros((1, 1), dtype=dtype).expand(rows, cols)
    big = (1 << 32) + 16
    with pytest.raises(ValueError, match="K = "):
        M.quantize_rows(wide(2, big, torch.bfloat16))
    s = torch.zeros(1)
    with pytest.raises(ValueError, match="K = "):
        M.project_int8(wide(2, big, torch.int8), s, wide(2, big, torch.int8), s)
    with pytest.raises(ValueError, match="N = "):
        M.project_int8(wide(2, 16, torch.int8), s, wide(big, 16, torch.int8), s)
    for kw, name in ((dict(count=big, dims=2), "count"), (dict(count=2, dims=big), "dims"),
                     (dict(count=2, dims=2, start=(1 << 64) + 5), "start"), (dict(count=2, dims=2, start=-(1 << 63) - 1), "start")):
        with pytest.raises(ValueError, match=f"{name} = "):
            M.rope_table(**kw, device="cuda:0")


@pytest.mark.parametrize("cfg", [
    M.QkConfig(B=1, T=2, H=3, W=4, hq=5, hk=2, hv=2, tp=128, rt=32, rh=48, rw=48, pairing="halves", eps=1e-5, dtype="f32"),
    M.GatedScanConfig(B=2, T=300, H=4, W=5, D=64, order=3, reverse=True, dtype="f32")], ids=["qk", "scan"])
def test_configs_copy_and_pickle(lib, cfg):
    """A module that holds a configuration can be copied, saved and sent to another process: before and after its cached
    sizes were asked for."""
    for _ in range(2):
        for c in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), copy.deepcopy([cfg, cfg])[1]):
            assert c == cfg and hash(c) == hash(cfg) and bytes(c.ccfg) == bytes(cfg.ccfg)
            assert c.ref._obj is c.ccfg and c.ccfg is not cfg.ccfg and (c.rows, c.tdtype) == (cfg.rows, cfg.tdtype)
            assert c.backward_workspace_bytes == cfg.backward_workspace_bytes > 0


# -------------------------------------------------------------------------------- pins of the fp64 reference
def test_reference_rotation_by_hand():
    """One head, two pairs: the norm leaves (3, 4, 0, 0) at twice its direction, the quarter turn swaps a pair."""
    cfg = M.QkConfig(B=1, T=1, H=1, W=1, hq=1, hk=1, hv=0, tp=4, rt=4, eps=1e-30, dtype="f32")
    tab = np.array([[[0.0, 1.0], [1.0, 0.0]]])        # pair 0 by 90 degrees, pair 1 not at all
    x = np.array([[3.0, 4.0, 0.0, 0.0, 0.0, 0.0, 5.0, 0.0]])
    out, _ = OP.qk_norm_rope(x, None, None, (tab, None, None), cfg)
    np.testing.assert_allclose(out, [[-1.6, 1.2, 0, 0, 0, 0, 2, 0]], atol=1e-12)
    halves = M.QkConfig(B=1, T=1, H=1, W=1, hq=1, hk=1, hv=0, tp=4, rt=4, eps=1e-30, dtype="f32", pairing="halves")
    out, _ = OP.qk_norm_rope(x, None, None, (tab, None, None), halves)     # pairs (0, 2) and (1, 3)
    np.testing.assert_allclose(out, [[0, 1.6, 1.2, 0, -2, 0, 0, 0]], atol=1e-12)


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    cfg = M.QkConfig(B=2, T=2, H=1, W=3, hq=2, hk=1, hv=1, tp=12, rt=4, rh=0, rw=6, pairing="halves", dtype="f32")
    tabs = [OP.rope_table(n, max(r, 2)) for n, r in zip((2, 1, 3), (4, 0, 6))]
    x, w, d = rng.standard_normal((cfg.rows, cfg.width)), rng.standard_normal((2, 12)), rng.standard_normal((cfg.rows, cfg.width))
    dx, _, dw, _ = OP.qk_norm_rope_backward(x, w[0], w[1], tabs, d, cfg)
    f = lambda x, w: (OP.qk_norm_rope(x, w[0], w[1], tabs, cfg)[0] * d).sum()
    vx, vw, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-6
    num = (f(x + h * vx, w + h * vw) - f(x - h * vx, w - h * vw)) / (2 * h)
    assert abs(num - (dx * vx).sum() - (dw * vw).sum()) < 1e-7 * (np.abs(dx * vx).sum() + 1)
    gs = M.GatedScanConfig(B=2, T=3, H=2, W=4, D=4, order=2, reverse=True, dtype="f32")
    base = [rng.standard_normal(s) for s in ((2, 24, 4), (2, 24, 4), (4,), (2, 4))]
    dy, dh = rng.standard_normal((2, 24, 4)), rng.standard_normal((2, 4))
    g = OP.gated_scan(base[0], base[1], gs, base[2], base[3], dy, dh)

    def fs(x, g, b, h0):
        o = OP.gated_scan(x, g, gs, b, h0)
        return (o["y"][0] * dy).sum() + (o["h_last"][0] * dh).sum()

    v = [rng.standard_normal(b.shape) for b in base]
    num = (fs(*(b + h * d for b, d in zip(base, v))) - fs(*(b - h * d for b, d in zip(base, v)))) / (2 * h)
    terms = [g[k][0] * d for k, d in zip(("dx", "dg", "dbias", "dh0"), v)]
    assert abs(num - sum(t.sum() for t in terms)) < 1e-7 * sum(np.abs(t).sum() for t in terms)


def test_reference_scan_order():
    """The rows of the recurrence are the Rotary Major Scan's (oracle/mate_oracle.py)."""
    from oracle import mate_oracle as O
    X = np.arange(3 * 4 * 5, dtype=np.float64).reshape(3, 4, 5, 1)
    for order in range(4):
        cfg = M.GatedScanConfig(B=1, T=3, H=4, W=5, D=8, order=order)
        np.testing.assert_array_equal(OP.scan_rows(cfg), O.rms_permute(X, order).reshape(-1))
