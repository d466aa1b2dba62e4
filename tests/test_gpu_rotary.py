"""The norm and rotation of queries and keys on the GPU (include/la_rotary.h) against its plain 64-bit
form: head sizes, rotated parts, pair orders, strides, far positions, gradients."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_reference import HALF_STEP, norm_rope, norm_rope_grad

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, bound, dtype, label):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    tol = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + 1e-30
    worst = np.max(np.abs(got - ref) / tol) if ref.size else 0.0
    assert worst <= 1, f"{label}: {worst:.3g} of its bound"


def heads(rng, tokens, H, D, dtype, layout="dense"):
    """[tokens, H, D]: dense, a column range of a wider matrix (16-byte or odd offsets), or heads first."""
    n = {"dense": 0, "range": 64, "odd": 3}.get(layout, 0)
    a = torch.from_numpy(rng.standard_normal((tokens, n + H * D + n)).astype(np.float32) * 2).to(DT[dtype]).cuda()
    a = a[:, n:n + H * D].unflatten(1, (H, D))
    return a.permute(1, 0, 2).contiguous().permute(1, 0, 2) if layout == "heads" else a


def inputs(rng, tokens, H, HK, D, R, dtype, layout="dense", start=0):
    q, k = heads(rng, tokens, H, D, dtype, layout), heads(rng, tokens, HK, D, dtype, layout)
    wq, wk = (torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda() for _ in range(2))
    pos = torch.arange(start, start + tokens, dtype=torch.int32).cuda()
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)).cuda()
    return q, k, wq, wk, pos, freq


CASES = [(1, 1, 1, 64, 64), (3, 4, 2, 64, 64), (7, 5, 1, 128, 128), (130, 8, 8, 128, 64), (2, 3, 3, 256, 256), (33, 2, 1, 256, 32),
         (5, 6, 2, 128, 2), (5, 6, 2, 128, 90), (9, 1, 1, 64, 0), (1000, 3, 2, 128, 48), (3, 70, 7, 64, 62), (5000, 2, 1, 64, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,H,HK,D,R", CASES)
def test_forward(tokens, H, HK, D, R, interleaved, dtype):
    rng = np.random.default_rng(tokens + D + R)
    for layout in ("dense", "range", "odd", "heads"):
        q, k, wq, wk, pos, freq = inputs(rng, tokens, H, HK, D, R, dtype, layout, start=17)
        if layout == "range":
            wq = None
        qo, ko = lap.la_qk_norm_rope_fwd(q, k, wq, wk, EPS, pos, freq, interleaved=interleaved)
        for got, x, w, label in ((qo, q, wq, "q"), (ko, k, wk, "k")):
            ref, bound = norm_rope(f64(x), None if w is None else f64(w), EPS, f64(pos), f64(freq), interleaved)
            near(got, ref, bound, dtype, f"{label} {layout}")
        q2, k2 = q, k  # in place, in the inputs' own layout
        keep = (qo.clone(), ko.clone())
        lap.la_qk_norm_rope_fwd(q2, k2, wq, wk, EPS, pos, freq, interleaved=interleaved, q_out=q2, k_out=k2)
        assert torch.equal(q2, keep[0]) and torch.equal(k2, keep[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,H,HK,D,R", CASES)
def test_backward(tokens, H, HK, D, R, interleaved, dtype):
    rng = np.random.default_rng(tokens + D + R + 1)
    for layout in ("dense", "range", "odd", "heads"):
        q, k, wq, wk, pos, freq = inputs(rng, tokens, H, HK, D, R, dtype, layout, start=5)
        if layout == "odd":
            wk = None
        gq, gk = heads(rng, tokens, H, D, dtype, layout), heads(rng, tokens, HK, D, dtype, layout)
        got = lap.la_qk_norm_rope_bwd(q, k, wq, wk, EPS, gq, gk, pos, freq, interleaved=interleaved)
        for i, (x, w, g) in enumerate(((q, wq, gq), (k, wk, gk))):
            ref = norm_rope_grad(f64(x), None if w is None else f64(w), EPS, f64(g), f64(pos), f64(freq), interleaved)
            near(got[i], *ref["dx"], dtype, f"dx {i} {layout}")
            near(got[2 + i], *ref["dw"], "fp32", f"dw {i} {layout}")
        again = lap.la_qk_norm_rope_bwd(q, k, wq, wk, EPS, gq, gk, pos, freq, interleaved=interleaved, dq=gq, dk=gk)
        assert again[0] is gq and all(torch.equal(a, b) for a, b in zip(got, again))


def test_no_rotation_is_the_norm_of_each_head():
    rng = np.random.default_rng(1)
    q, k, wq, wk, _, _ = inputs(rng, 40, 4, 2, 128, 0, "fp32")
    qo, ko = lap.la_qk_norm_rope_fwd(q, k, wq, wk, EPS)
    y, _ = lap.la_rms_norm_fwd(q.reshape(-1, 128), wq, EPS)
    ref, bound = norm_rope(f64(q), f64(wq), EPS, np.zeros(40), [], False)
    near(qo, ref, bound, "fp32", "q")
    near(y.view_as(qo), ref, bound, "fp32", "la_rms_norm_fwd")


@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_of_any_size(interleaved):
    """Angles of frequencies from denormal to 2^25, of either sign.  The products are exact in 64 bits; the kernels' turn
    is off by position (1 + frequency) 2^-64 of a turn and by 2^-24 when it becomes FP32; the norm by 32 2^-24 + 2^-21 of
    its value, which is less than 2^-18; sine and cosine by 2^-21."""
    freq = np.array([1e-42, -3e-39, 1e-30, 2.0 ** -66, 1e-12, -1e-7, 1e-3, 0.7, 1.0, -1.0, 3.3, 1e3, -65537.0, 2.0 ** 23 + 1,
                     2.0 ** 24 + 2, -33554430.0], dtype=np.float32)
    pos = np.array([0, 1, -1, 2, 17, 4095, -65536, 2 ** 20 - 1], dtype=np.int32)
    rng = np.random.default_rng(51)
    q = torch.from_numpy(rng.standard_normal((len(pos), 3, 64)).astype(np.float32)).cuda()
    out, _ = lap.la_qk_norm_rope_fwd(q, q, None, None, EPS, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(),
                                     interleaved=interleaved)
    x = q.double().cpu().numpy()
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    a = pos.astype(np.float64)[:, None, None] * freq.astype(np.float64)
    lo, hi = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    ref = y.copy()
    ref[..., lo], ref[..., hi] = y[..., lo] * np.cos(a) - y[..., hi] * np.sin(a), y[..., lo] * np.sin(a) + y[..., hi] * np.cos(a)
    off = 2 * np.pi * (np.abs(pos)[:, None, None] * (1 + np.abs(freq.astype(np.float64))) * 2.0 ** -64 + 2.0 ** -24) + 2.0 ** -21
    tol = np.abs(ref) * 2.0 ** -18 + 1e-30
    both = (np.abs(y[..., lo]) + np.abs(y[..., hi])) * (off + 2.0 ** -18)
    tol[..., lo], tol[..., hi] = both, both
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("start", [-5, 2 ** 24 - 3, 2 ** 31 - 9])
def test_far_positions(start):
    rng = np.random.default_rng(2)
    q, k, wq, wk, pos, freq = inputs(rng, 8, 2, 1, 64, 64, "fp32", start=start)
    freq[1] = -3.7  # more than half a turn per token, backwards
    freq[2] = 1234.5
    qo, ko = lap.la_qk_norm_rope_fwd(q, k, wq, wk, EPS, pos, freq)
    # the angle modulo a turn in more than 64 bits: position and frequency are exact in integers of
    # 2^-149, and a turn is 2 pi to 40 digits
    from fractions import Fraction
    turn = 2 * Fraction("3.1415926535897932384626433832795028841972")
    ang = np.array([[float(Fraction(int(p)) * Fraction(float(f)) % turn) for f in f64(freq)] for p in f64(pos)])
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        x, w = f64(x), f64(w)
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
        a, b = y[..., :32], y[..., 32:]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        ref = np.concatenate([a * c - b * s, a * s + b * c], -1)
        size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
        # 2^-21 of sine and cosine, |position frequency| 2^-51 of the angle
        far = np.abs(f64(pos))[:, None] * np.abs(f64(freq)) * 2.0 ** -51
        e = 2.0 ** -20 + np.concatenate([far, far], 1)[:, None]
        assert np.all(np.abs(f64(got) - ref) <= size * e)


def test_captured_and_replayed_on_another_stream():
    rng = np.random.default_rng(4)
    q, k, wq, wk, pos, freq = inputs(rng, 300, 8, 2, 128, 128, "bf16", "range")
    gq, gk = heads(rng, 300, 8, 128, "bf16"), heads(rng, 300, 2, 128, "bf16")

    def step(stream=None):
        return (*lap.la_qk_norm_rope_fwd(q, k, wq, wk, EPS, pos, freq, stream=stream),
                *lap.la_qk_norm_rope_bwd(q, k, wq, wk, EPS, gq, gk, pos, freq, stream=stream))
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_past_32_bit_offsets():
    tokens, ld = (1 << 18) + 3, 8256
    wide = torch.empty((tokens, ld), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide[:, :192] = torch.randn((tokens, 192), generator=gen, device="cuda").to(torch.bfloat16)
    q, k = wide[:, :128].unflatten(1, (2, 64)), wide[:, 128:192].unflatten(1, (1, 64))
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    freq = torch.rand(32, device="cuda")
    qo, ko = lap.la_qk_norm_rope_fwd(q.contiguous(), k.contiguous(), None, None, EPS, pos, freq)
    lap.la_qk_norm_rope_fwd(q, k, None, None, EPS, pos, freq, q_out=wide[:, 512:640].unflatten(1, (2, 64)),
                            k_out=wide[:, 8192:].unflatten(1, (1, 64)))
    assert torch.equal(wide[:, 512:640].unflatten(1, (2, 64)), qo) and torch.equal(wide[:, 8192:].unflatten(1, (1, 64)), ko)
    got = lap.la_qk_norm_rope_bwd(q, k, None, None, EPS, qo, ko, pos, freq, dq=wide[:, 512:640].unflatten(1, (2, 64)))
    ref = lap.la_qk_norm_rope_bwd(q.contiguous(), k.contiguous(), None, None, EPS, qo, ko, pos, freq)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_empty_batch_writes_zero_weight_gradients():
    e = torch.empty((0, 2, 64), device="cuda")
    out = lap.la_qk_norm_rope_bwd(e, e, None, None, EPS, e, e)
    assert out[0].shape == e.shape and not out[2].any() and not out[3].any()
    assert lap.la_qk_norm_rope_fwd(e, e, None, None, EPS)[0].shape == e.shape


def test_wrong_arguments_are_refused():
    q = torch.zeros((4, 2, 64), device="cuda")
    pos, freq = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(32, device="cuda")
    for over, kind in ((dict(positions=None), ValueError), (dict(inv_freq=None), ValueError),
                       (dict(positions=pos[:3]), ValueError), (dict(positions=pos.long()), TypeError),
                       (dict(inv_freq=freq.double()), TypeError), (dict(k=q[:3]), ValueError), (dict(k=q.bfloat16()), TypeError),
                       (dict(q_weight=freq), ValueError), (dict(q_out=q[:, :1]), ValueError), (dict(q=q.transpose(1, 2)), ValueError),
                       (dict(inv_freq=torch.zeros(33, device="cuda")), lap.LaError), (dict(q_out=q, q=q[:, :1].expand(4, 2, 64)), lap.LaError)):
        a = dict(q=q, k=q, q_weight=None, k_weight=None, eps=EPS, positions=pos, inv_freq=freq)
        with pytest.raises(kind):
            lap.la_qk_norm_rope_fwd(**{**a, **over})
