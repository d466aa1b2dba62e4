"""The RMS norm on the GPU (include/la_norm.h) against its plain 64-bit form: residual addition,
both 8-bit scalings, gradients, strides, odd sizes, and a layer of the operators together."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from gated_reference import HALF_STEP, norm, norm_grad

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def f64(t):
    return t.detach().double().cpu().numpy()


def mat(rng, rows, C, dtype, scale=1.0, off=0, extra=0):
    a = torch.from_numpy(rng.standard_normal((rows, off + C + extra)).astype(np.float32) * np.float32(scale))
    return a.to(DT[dtype]).cuda()[:, off:off + C]


def near(got, ref, bound, dtype, label):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    tol = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + 1e-30
    worst = np.max(np.abs(got - ref) / tol) if ref.size else 0.0
    assert worst <= 1, f"{label}: {worst:.3g} of its bound"


SIZES = [(1, 1), (1, 64), (3, 7), (5, 100), (2, 127), (2, 128), (9, 129), (700, 64), (4, 1001), (3, 2048), (2, 4100),
         (2, 8192), (1, 16384), (2, 16383), (1300, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C", SIZES)
def test_forward(rows, C, dtype):
    rng = np.random.default_rng(rows * 7 + C)
    for off, extra in ((0, 0), (1, 2), (8, 8)):
        x, w = mat(rng, rows, C, dtype, 1.0, off, extra), torch.from_numpy(rng.standard_normal(C).astype(np.float32)).cuda()
        y, none = lap.la_rms_norm_fwd(x, w, EPS)
        ref, _, bound = norm(f64(x), None, f64(w), EPS)
        near(y, ref, bound, dtype, "y")
        assert none is None
        res = mat(rng, rows, C, dtype, 3.0, off, extra)
        y, s = lap.la_rms_norm_fwd(x, w, EPS, residual=res)
        ref, rs, bound = norm(f64(x), f64(res), f64(w), EPS)
        near(y, ref, bound + 2.0 ** -23 * np.abs(ref), dtype, "y of the sum")
        near(s, rs, 2.0 ** -24 * np.abs(rs), dtype, "residual_out")
        keep = res.clone()
        y2, s2 = lap.la_rms_norm_fwd(x, w, EPS, residual=keep, residual_out=keep)
        assert s2 is keep and torch.equal(keep, s) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,C", SIZES)
def test_forward_fp8(rows, C, group, dtype):
    rng = np.random.default_rng(rows * 5 + C + group)
    for off, extra, residual in ((0, 0, True), (1, 2, False), (16, 16, True)):
        x, w = mat(rng, rows, C, dtype, 1.0, off, extra), torch.from_numpy(rng.standard_normal(C).astype(np.float32)).cuda()
        res = mat(rng, rows, C, dtype, 2.0, off, extra) if residual else None
        y, scales, s = lap.la_rms_norm_fwd_fp8(x, w, EPS, residual=res, group=group)
        ref, rs, bound = norm(f64(x), f64(res) if residual else None, f64(w), EPS)
        width = group or C
        sc = np.stack([np.abs(ref[:, k:k + width]).max(1) for k in range(0, C, width)], 1)
        rel = (0.5 * C + 4) * 2.0 ** -24 + 2.0 ** -20  # of y, of its maximum and of the quotient
        near(scales, np.maximum(sc, 2.0 ** -40) / 448, rel * sc / 448, "fp32", "scales")
        full = np.repeat(f64(scales), width, axis=1)[:, :C]
        q = f64(y)
        want = ref / full
        # half a step of e4m3 (2^-4 relative, 2^-10 below its normal range) beyond the quotient's error
        assert np.all(np.abs(q - want) <= 2 * rel * np.abs(want) + np.maximum(HALF_STEP["e4m3"] * np.abs(want), 2.0 ** -10)
                      * (1 + 2.0 ** -10) + 1e-30)
        assert np.abs(q).max() <= 448
        if residual:
            near(s, rs, 2.0 ** -24 * np.abs(rs), dtype, "residual_out")


def test_zero_rows_and_non_finite_rows():
    rng = np.random.default_rng(1)
    x = mat(rng, 6, 300, "bf16")
    w = torch.ones(300, device="cuda")
    ref = lap.la_rms_norm_fwd_fp8(x, w, EPS, group=128)
    x[1] = 0
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    y, scales, _ = lap.la_rms_norm_fwd_fp8(x, w, EPS, group=128)
    assert torch.equal(f(y[1]), torch.zeros(300)) and torch.all(scales[1] > 0)
    assert torch.isnan(f(y[2])).all()                       # the row's norm is NaN
    assert torch.isnan(f(y[4])[7]) and (f(y[4])[8:] == 0).all()  # inf / inf, and x / inf
    for row in (0, 3, 5):
        assert torch.equal(f(y[row]), f(ref[0][row])) and torch.equal(scales[row], ref[1][row])
    y = lap.la_rms_norm_fwd(torch.zeros((3, 70), device="cuda"), torch.ones(70, device="cuda"), EPS)[0]
    assert torch.equal(y, torch.zeros_like(y))


def f(t):
    return t.float().cpu()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C", SIZES + [(0, 64), (2500, 200), (5000, 64), (1500, 1024)])
def test_backward(rows, C, dtype):
    rng = np.random.default_rng(rows * 3 + C)
    for off, extra, with_dres in ((0, 0, True), (1, 2, False), (8, 8, True)):
        s, dy = mat(rng, rows, C, dtype, 2.0, off, extra), mat(rng, rows, C, dtype, 1.0, off, extra)
        dres = mat(rng, rows, C, dtype, 1.0, off, extra) if with_dres else None
        w = torch.from_numpy(rng.standard_normal(C).astype(np.float32)).cuda()
        dx, dw = lap.la_rms_norm_bwd(s, w, EPS, dy, dres=dres)
        ref = norm_grad(f64(s), f64(w), EPS, f64(dy), f64(dres) if with_dres else None)
        near(dx, *ref["dx"], dtype, "dx")
        near(dw, *ref["dweight"], "fp32", "dweight")
        dx2, dw2 = lap.la_rms_norm_bwd(s, w, EPS, dy, dres=dres)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_captured_and_replayed():
    rng = np.random.default_rng(4)
    x, res, dy = (mat(rng, 900, 520, "bf16") for _ in range(3))
    w = torch.from_numpy(rng.standard_normal(520).astype(np.float32)).cuda()

    def step():
        y, s = lap.la_rms_norm_fwd(x, w, EPS, residual=res)
        q, sc, _ = lap.la_rms_norm_fwd_fp8(x, w, EPS, residual=res, group=128)
        return y, s, q.view(torch.uint8), sc, *lap.la_rms_norm_bwd(s, w, EPS, dy, dres=dy)
    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_past_32_bit_offsets():
    rows, ld, C = (1 << 18) + 3, 8256, 40
    wide = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide[:, :2 * C] = torch.randn((rows, 2 * C), generator=gen, device="cuda").to(torch.bfloat16)
    x, dy = wide[:, :C], wide[:, C:2 * C]
    w = torch.ones(C, device="cuda")
    y, _ = lap.la_rms_norm_fwd(x, w, EPS, y=wide[:, 3 * C:4 * C])
    assert torch.equal(y, lap.la_rms_norm_fwd(x.contiguous(), w, EPS)[0])
    dx, dw = lap.la_rms_norm_bwd(x, w, EPS, dy, dx=wide[:, 5 * C:6 * C])
    dx2, dw2 = lap.la_rms_norm_bwd(x.contiguous(), w, EPS, dy.contiguous())
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_a_training_step_of_a_layer():
    """Residual + norm, projection, packed gated scan, and back: the chained gradients against
    autograd in 64 bits over the same rounded intermediates."""
    torch.manual_seed(0)
    tokens, C = 300, 64
    cu = torch.tensor([0, 120, 120, 300], dtype=torch.int32, device="cuda")
    x, res = (torch.randn(tokens, C, device="cuda") for _ in range(2))
    w = 1 + 0.1 * torch.randn(C, device="cuda")
    proj = torch.randn(C, 3 * C, device="cuda") / 8
    slopes = torch.exp2(-8.0 * torch.arange(1, C + 1, device="cuda") / C)
    dout, ds = torch.randn(tokens, C, device="cuda"), torch.randn(tokens, C, device="cuda")
    y, s = lap.la_rms_norm_fwd(x, w, EPS, residual=res)
    xrg = y @ proj
    parts = xrg.split(C, 1)
    o = lap.la_gated_scan_fwd(*parts, slopes, cu_seqlens=cu)
    dxrg = torch.empty_like(xrg)
    _, _, _, dslopes, _ = lap.la_gated_scan_bwd(*parts, slopes, o, dout, cu_seqlens=cu,
                                                **dict(zip(("dx", "dr", "dg"), dxrg.split(C, 1))))
    dx, dw = lap.la_rms_norm_bwd(s, w, EPS, dxrg @ proj.t(), dres=ds)

    xd, wd, pd, sd = (t.double().requires_grad_() for t in (x, w, proj, slopes))
    sd_ = xd + res.double()
    yd = sd_ / (sd_.pow(2).mean(1, keepdim=True) + EPS).sqrt() * wd
    a, r, g = (yd @ pd).split(C, 1)
    u = sd * torch.sigmoid(r)
    lam, b = torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u)) * torch.sigmoid(g) * a
    hs, h = [], None
    for t in range(tokens):
        h = b[t] if t in (0, 120) else lam[t] * h + b[t]
        hs.append(h)
    od = torch.stack(hs)
    ((od * dout.double()).sum() + (sd_ * ds.double()).sum()).backward()
    # FP32 throughout; TF32 is off, so the products are FP32 sums of 64 and 192 terms: 2^-14 relative
    # to the largest value covers their roundings and the scan's memory of 1 / (1 - lambda) <= 512 steps
    for got, want, name in ((o, od, "o"), (dx, xd.grad, "dx"), (dw, wd.grad, "dweight"), (dslopes, sd.grad, "dslopes")):
        err = float((got.double() - want.detach()).abs().max() / want.detach().abs().max())
        assert err <= 2.0 ** -14, (name, err)


def test_a_serving_step_after_lightning_attention():
    """A packed prompt through la_prefill_fwd, its output into the residual stream and the 8-bit
    norm, then the gated layer's scan and decode from the pool: each against its plain form."""
    from gated_reference import scan_one
    torch.manual_seed(1)
    H, T, B = 2, 70, 3
    C = H * 128
    q, k, v = (torch.randn(B * T, H, 128, device="cuda").to(torch.bfloat16) for _ in range(3))
    q, k = (t / 11.3 for t in (q, k))
    att = lap.la_prefill_fwd(q, k, v, torch.tensor([0.5, 0.1], device="cuda"), 1.0, seq_len=T).view(B * T, C)
    res = torch.randn(B * T, C, device="cuda").to(torch.bfloat16)
    w = torch.ones(C, device="cuda")
    y8, sc, s = lap.la_rms_norm_fwd_fp8(att, w, EPS, residual=res)
    ref, rs, bound = norm(f64(att), f64(res), f64(w), EPS)
    near(s, rs, 2.0 ** -24 * np.abs(rs), "bf16", "residual")
    assert np.abs(f64(y8) * f64(sc) - ref).max() <= 448 / 16 * float(sc.max()) * 1.01
    xrg = ((y8.float() * sc) @ (torch.randn(C, 3 * C, device="cuda") / 16)).to(torch.bfloat16)
    x, r, g = xrg.split(C, 1)
    slopes = torch.exp2(-8.0 * torch.arange(1, C + 1, device="cuda") / C)
    pool = torch.zeros(5, C, device="cuda")
    idx = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    o = lap.la_gated_scan_fwd(x, r, g, slopes, h0=pool, h_final=pool, state_indices=idx, seq_len=T)
    at = torch.arange(B, device="cuda") * T
    o1 = lap.la_gated_decode(x[at], r[at], g[at], slopes, pool, 1, state_indices=idx)
    for n in range(B):
        rows = list(range(n * T, n * T + T)) + [n * T]
        ro, rh, eo, eh = scan_one(f64(x[rows]), f64(r[rows]), f64(g[rows]), f64(slopes), np.zeros(C))
        near(torch.cat([o[n * T:n * T + T], o1[n:n + 1]]), ro, eo, "bf16", f"sequence {n}")
        near(pool[int(idx[n])], rh, eh, "fp32", f"state {n}")
