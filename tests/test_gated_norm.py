"""The gated recurrence and the RMS norm without a GPU: refusals of the C entry points and of the
binding, workspace sizes, and the 64-bit reference's gradients against differences."""
import ctypes

import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from gated_reference import grad_one, norm, norm_grad, scan_one

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
BUF = [(i + 1) << 40 for i in range(24)]  # fake buffers, never dereferenced
(X, R, G, SL, H0, O, HF, IDX, CU, WS, ERR, DOUT, DX, DR, DG, DSL, DH0, DHF, ACC, RES, W, SC, RO, Y) = BUF


def scan(**over):
    a = dict(x=X, r=R, g=G, sl=SL, h0=None, idx=None, cu=None, o=O, hf=None, ldx=64, ldr=64, ldg=64, ldo=64, B=2, T=300,
             N=2, C=64, P=0, dt=0, ws=WS, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lap.load_library().la_gated_scan_fwd(*a.values())


def back(**over):
    a = dict(x=X, r=R, g=G, sl=SL, h0=None, o=O, dout=DOUT, dhf=None, idx=None, cu=None, dx=DX, dr=DR, dg=DG, dsl=DSL,
             dh0=None, ldx=64, ldr=64, ldg=64, ldo=64, lddout=64, lddx=64, lddr=64, lddg=64, B=2, T=300, N=2, C=64, P=0,
             dt=0, ws=WS, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lap.load_library().la_gated_scan_bwd(*a.values())


def decode(fn="la_gated_decode", **over):
    a = dict(x=X, r=R, g=G, sl=SL, st=H0, idx=None, o=O, ldx=64, ldr=64, ldg=64, ldo=64, B=2, T=4, C=64, P=2, dt=0,
             err=None, stream=None)
    a.update(over)
    if fn == "la_gated_commit":
        del a["ldo"]
    return getattr(lap.load_library(), fn)(*a.values())


def fwd(fp8=False, **over):
    a = dict(x=X, res=None, w=W, eps=1e-5, y=Y, sc=SC, ro=None, ldx=64, ldres=64, ldy=64, ldro=64, rows=4, C=64, group=0,
             dt=0, err=None, stream=None)
    a.update(over)
    if not fp8:
        del a["sc"], a["group"]
    return getattr(lap.load_library(), "la_rms_norm_fwd_fp8" if fp8 else "la_rms_norm_fwd")(*a.values())


def nback(**over):
    a = dict(s=X, w=W, eps=1e-5, dy=DOUT, dres=None, dx=DX, dw=DSL, lds=64, lddy=64, lddres=64, lddx=64, rows=4, C=64,
             dt=0, ws=WS, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lap.load_library().la_rms_norm_bwd(*a.values())


BAD_SCAN = [
    (dict(C=0), INVALID), (dict(dt=2), UNSUPPORTED), (dict(N=3), INVALID), (dict(B=-1, N=-1), INVALID),
    (dict(cu=CU, B=2), INVALID), (dict(T=1 << 30, B=4, N=4), UNSUPPORTED), (dict(ldx=63), INVALID), (dict(ldr=0), INVALID),
    (dict(x=X + 1), INVALID), (dict(dt=1, g=G + 2), INVALID), (dict(sl=SL + 2), INVALID), (dict(sl=None), INVALID),
    (dict(x=None), INVALID), (dict(h0=H0, P=1), INVALID), (dict(h0=H0, idx=IDX, P=0), INVALID),
    (dict(h0=H0 + 1, P=2), INVALID), (dict(err=ERR + 1), INVALID),
]


@pytest.mark.parametrize("over,status", BAD_SCAN + [(dict(o=None), INVALID), (dict(ldo=1 << 50), INVALID),
                                                    (dict(cu=CU, B=1, T=600, ws=None), INVALID),
                                                    (dict(cu=CU, B=1, T=600, wsb=1), INVALID),
                                                    (dict(cu=CU, B=1, T=600, ws=WS + 16), INVALID)])
def test_scan_refusals(over, status):
    assert scan(**over) == status
    assert lap.load_library().la_last_error() != b""


@pytest.mark.parametrize("over,status", BAD_SCAN + [(dict(dx=None), INVALID), (dict(dsl=None), INVALID),
                                                    (dict(dout=None), INVALID), (dict(lddg=3), INVALID),
                                                    (dict(ws=None), INVALID), (dict(wsb=16), INVALID)])
def test_scan_gradient_refusals(over, status):
    assert back(**over) == status
    assert lap.load_library().la_last_error() != b""


# B = 2, T = 300, C = 64 bf16: a compact matrix holds 76800 bytes, a row 128
@pytest.mark.parametrize("over", [
    dict(o=X), dict(o=G + 76800 - 2), dict(o=SL - 64), dict(hf=X, P=2), dict(h0=H0, hf=H0 + 64, P=2),
    dict(o=X + 64, ldx=256, ldo=256),           # rows interleave, columns 32..95 against 0..63
    dict(o=X + 2 * 200, ldx=256, ldo=256),      # columns 200..263 run into the next row's
    dict(o=X + 128, ldx=256, ldo=200),          # different strides: whole ranges count
    dict(ws=O, cu=CU, B=1, T=600), dict(err=O + 4), dict(idx=HF + 4, hf=HF, P=4),
])
def test_scan_overlaps_are_refused(over):
    assert scan(**over) == INVALID
    assert b"overlaps" in lap.load_library().la_last_error()


@pytest.mark.parametrize("over", [dict(dx=DR), dict(dx=X), dict(dg=DOUT), dict(dsl=SL), dict(dh0=H0, h0=H0, P=2),
                                  dict(dh0=DHF, dhf=DHF, P=2), dict(dr=O), dict(ws=DX)])
def test_scan_gradient_overlaps_are_refused(over):
    assert back(**over) == INVALID
    assert b"overlaps" in lap.load_library().la_last_error()


def test_column_ranges_of_one_matrix_are_no_overlap():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    # past every host check: the device query fails
    ld = dict(ldx=192, ldr=192, ldg=192)
    assert scan(r=X + 128, g=X + 256, **ld) == CUDA
    assert scan(r=X + 128, g=X + 256, o=X + 384, ldx=256, ldr=256, ldg=256, ldo=256) == CUDA
    assert back(dr=DX + 128, dg=DX + 256, lddx=192, lddr=192, lddg=192) == CUDA
    assert scan(h0=H0, hf=H0, P=2) == CUDA
    assert scan(B=1, N=1, T=1, ws=None, wsb=0) == CUDA
    assert decode() == decode("la_gated_verify") == decode("la_gated_commit", o=ACC) == CUDA
    assert fwd(res=RES, ro=RES) == fwd(fp8=True, group=128) == nback() == CUDA


@pytest.mark.parametrize("fn", ["la_gated_decode", "la_gated_verify", "la_gated_commit"])
@pytest.mark.parametrize("over,status", [
    (dict(T=0), INVALID), (dict(C=0), INVALID), (dict(dt=7), UNSUPPORTED), (dict(P=1), INVALID),
    (dict(idx=IDX, P=0), INVALID), (dict(st=None), INVALID), (dict(o=None), INVALID), (dict(ldg=60), INVALID),
    (dict(x=X + 1), INVALID), (dict(B=-1), INVALID), (dict(err=H0), INVALID)])
def test_decode_refusals(fn, over, status):
    if fn == "la_gated_verify" and "err" in over:
        over = dict(err=O)
    assert decode(fn, **over) == status
    assert lap.load_library().la_last_error() != b""


def test_nothing_to_do():
    assert scan(B=0, N=0) == OK and decode(B=0) == OK and fwd(rows=0) == OK and fwd(fp8=True, rows=0) == OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over,status", [
    (dict(C=0), INVALID), (dict(C=16385, ldx=20000, ldy=20000), UNSUPPORTED), (dict(rows=-1), INVALID),
    (dict(dt=3), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(ro=RO), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(w=None), INVALID), (dict(ldy=63), INVALID), (dict(y=X), INVALID),
    (dict(res=RES, ro=RES, ldro=128), INVALID), (dict(err=Y + 4), INVALID), (dict(res=RES, ro=X), INVALID), (dict(res=RES, ldres=1), INVALID)])
def test_norm_refusals(fp8, over, status):
    assert fwd(fp8, **over) == status
    assert lap.load_library().la_last_error() != b""


def test_norm_fp8_refusals():
    assert fwd(True, group=64) == UNSUPPORTED and fwd(True, sc=None) == INVALID and fwd(True, sc=Y) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=8), INVALID),
    (dict(dx=DOUT), INVALID), (dict(dx=X), INVALID), (dict(dw=W), INVALID), (dict(dres=RES, lddres=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(C=20000, lds=20000, lddy=20000, lddx=20000), UNSUPPORTED)])
def test_norm_gradient_refusals(over, status):
    assert nback(**over) == status
    assert lap.load_library().la_last_error() != b""


def test_workspace_queries():
    torch = pytest.importorskip("torch")
    assert lap.la_gated_scan_workspace(1, 1, 1, 64, False, torch.bfloat16, False) == 0
    assert lap.la_gated_scan_workspace(1, 600, 3, 64, True, torch.bfloat16, True) % 256 == 0
    assert lap.la_rms_norm_bwd_workspace(0, 64) == 0 and lap.la_rms_norm_bwd_workspace(100, 64) >= 256
    with pytest.raises(lap.LaError):
        lap.la_gated_scan_workspace(2, 600, 3, 64, False, torch.bfloat16, False)
    lib = lap.load_library()
    assert lib.la_gated_scan_workspace(1, 1, 1, 64, 0, 0, 0, None) == INVALID
    assert lib.la_rms_norm_bwd_workspace(1, 0, ctypes.byref(ctypes.c_size_t())) == INVALID


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    s = torch.zeros(64)
    for call in (lambda t: lap.la_gated_scan_fwd(t, t, t, s, seq_len=8), lambda t: lap.la_gated_decode(t, t, t, s, s, 1),
                 lambda t: lap.la_gated_scan_bwd(t, t, t, s, t, t, seq_len=8), lambda t: lap.la_rms_norm_fwd(t, s, 1e-5),
                 lambda t: lap.la_gated_verify(t, t, t, s, s, 1), lambda t: lap.la_gated_commit(t, t, t, s, s, 1, None),
                 lambda t: lap.la_rms_norm_fwd_fp8(t, s, 1e-5), lambda t: lap.la_rms_norm_bwd(t, s, 1e-5, t)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(x)
        with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
            call(x.half())
        with pytest.raises(ValueError, match="2 dims"):
            call(x[0])
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call([0])


def random_sequence(seed, L, C):
    rng = np.random.default_rng(seed)
    x, r, g, dout = rng.standard_normal((4, L, C)) * 1.5
    slopes, h0, dhf = np.exp(rng.standard_normal(C) - 1), rng.standard_normal(C), rng.standard_normal(C)
    return x, r, g, dout, slopes, h0, dhf


def test_reference_gradients_against_differences():
    x, r, g, dout, slopes, h0, dhf = random_sequence(0, 9, 5)
    o, hf, _, _ = scan_one(x, r, g, slopes, h0)
    ref = grad_one(x, r, g, slopes, h0, o, dout, dhf)
    args = dict(x=x, r=r, g=g, slopes=slopes, h0=h0)

    def loss(**over):
        o, hf, _, _ = scan_one(**{**args, **over})
        return (o * dout).sum() + (hf * dhf).sum()
    for name, key in (("x", "dx"), ("r", "dr"), ("g", "dg"), ("slopes", "ds"), ("h0", "dh0")):
        v, grad = args[name], ref[key][0]
        for i in np.ndindex(*v.shape):
            d = np.zeros_like(v)
            d[i] = 1e-5
            diff = (loss(**{name: v + d}) - loss(**{name: v - d})) / 2e-5
            assert abs(diff - grad[i]) <= 1e-7 * (1 + abs(diff)), (name, i, diff, grad[i])


def test_reference_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    s, dy, dres = rng.standard_normal((3, 4, 6))
    w = rng.standard_normal(6)
    ref = norm_grad(s, w, 1e-2, dy, dres)

    def loss(s, w):
        return (norm(s, None, w, 1e-2)[0] * dy).sum() + (s * dres).sum()
    for i in np.ndindex(*s.shape):
        d = np.zeros_like(s)
        d[i] = 1e-5
        assert abs((loss(s + d, w) - loss(s - d, w)) / 2e-5 - ref["dx"][0][i]) <= 1e-8
    for i in range(6):
        d = np.zeros(6)
        d[i] = 1e-5
        assert abs((loss(s, w + d) - loss(s, w - d)) / 2e-5 - ref["dweight"][0][i]) <= 1e-8


def test_recurrence_special_cases():
    """Closed form on the reference: a constant decay is a geometric sum; beta keeps the variance."""
    L, C = 12, 3
    x, slopes = np.ones((L, C)), np.array([0.1, 1.0, 5.0])
    r, g = np.full((L, C), 40.0), np.full((L, C), 40.0)  # open gates: sigmoid = 1 to 64 bits
    o, hf, _, _ = scan_one(x, r, g, slopes, np.zeros(C))
    lam = np.exp(-slopes)
    for t in range(L):
        np.testing.assert_allclose(o[t], np.sqrt(1 - lam ** 2) * (1 - lam ** (t + 1)) / (1 - lam), rtol=1e-12)
    o, hf, _, _ = scan_one(x, np.full((L, C), -800.0), g, slopes, np.arange(3.0))
    np.testing.assert_array_equal(o, np.tile(np.arange(3.0), (L, 1)))
