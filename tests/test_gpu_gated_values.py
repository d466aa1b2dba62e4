"""The gated recurrence on the GPU where its values are hard: NaN in one input, steep slopes, gates
far open and far closed.  Each kernel form is entered (whole sequences in a tile, chains, tiles,
mixed rows, rows that are not 16-byte aligned).

Tolerances are those computed beside the 64-bit reference (gated_reference.py) or, where a factor is
small, derived here from the same roundings, relative to the value itself."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from gated_reference import HALF_STEP, gate_errors, gates, grad_one, scan_one
from test_gpu_gated import Batch, f64, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FORMS = {
    "whole sequences": dict(lens=[40] * 7, C=72, packed=False),
    "chains": dict(lens=[300] * 3, C=72, packed=False),
    "tiles": dict(lens=[3000], C=72, packed=False),
    "mixed rows": dict(lens=[50, 3, 0, 90, 41, 7, 120, 60], C=72),
    "packed tiles": dict(lens=[700, 0, 900, 412], C=72),
    "packed chains": dict(lens=[0, 600, 700, 1, 517, 300, 129, 128, 700, 64, 725, 812, 0, 333, 901, 499], C=4096),
    "unaligned": dict(lens=[300, 41, 900], C=67),
    "fp32": dict(lens=[300, 41, 900], C=72, dtype="fp32"),
}


def grads(b, o, dout, **kw):
    dx, dr, dg = b.three(float("nan"))
    dh0 = torch.full((b.P, b.C), float("nan"), device="cuda") if b.h0 is not None else None
    res = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dx=dx, dr=dr, dg=dg, dh0=dh0, **b.kw, **kw)
    torch.cuda.synchronize()
    return res


@pytest.mark.parametrize("what", ["x", "r", "g", "h0"])
@pytest.mark.parametrize("form", FORMS)
def test_a_nan_reaches_what_depends_on_it(form, what):
    """One NaN at one token of one channel: o from that token on and h_final are NaN, as the definition
    has it; every other value keeps its bits."""
    b = Batch(40, **FORMS[form])
    o, hf = b.fwd()
    n = int(np.argmax(b.lens))
    s, slot, c = b.rows(n), int(b.slots[n]), 5
    t = s.start if what == "h0" else (s.start + s.stop) // 2
    if what == "h0":
        b.h0[slot, c] = float("nan")
    else:
        getattr(b, what)[t, c] = float("nan")
    o2, hf2 = b.fwd()
    assert torch.isnan(o2[t:s.stop, c]).all() and torch.isnan(hf2[slot, c])
    o2[t:s.stop, c], hf2[slot, c] = o[t:s.stop, c], hf[slot, c]
    assert torch.equal(o2, o) and torch.equal(hf2, hf)


@pytest.mark.parametrize("form", FORMS)
def test_a_nan_gate_reaches_its_gradients(form):
    """NaN in g at one token: dx, dr, dg of that token and dslopes of its channel, nothing else."""
    b = Batch(41, **FORMS[form])
    o, _ = b.fwd()
    dout = b.mat()
    want = grads(b, o, dout)
    n = int(np.argmax(b.lens))
    t, c = (b.rows(n).start + b.rows(n).stop) // 2, 5
    b.g[t, c] = float("nan")
    got = grads(b, o, dout)
    for k in range(3):
        assert torch.isnan(got[k][t, c]), ("dx", "dr", "dg")[k]
        got[k][t, c] = want[k][t, c]
        assert torch.equal(got[k], want[k]), ("dx", "dr", "dg")[k]
    assert torch.isnan(got[3][c])
    got[3][c] = want[3][c]
    assert torch.equal(got[3], want[3]) and torch.equal(got[4], want[4])


@pytest.mark.parametrize("what", ["x", "r", "g", "state"])
@pytest.mark.parametrize("C", [64, 67])
def test_a_nan_in_decode(C, what):
    B, T, c, t = 5, 6, 9, 3
    b = Batch(42, lens=[T] * B, C=C, packed=False, pool=8)
    slot, row = int(b.slots[2]), 2 * T + t

    def calls():
        st, cm = b.h0.clone(), b.h0.clone()
        o = lap.la_gated_decode(b.x, b.r, b.g, b.slopes, st, T, state_indices=b.idx)
        v = lap.la_gated_verify(b.x, b.r, b.g, b.slopes, b.h0, T, state_indices=b.idx)
        lap.la_gated_commit(b.x, b.r, b.g, b.slopes, cm, T, torch.tensor([T, t, t + 1, T, 0], dtype=torch.int32,
                                                                         device="cuda"), state_indices=b.idx)
        return o, v, st, cm
    want = calls()
    if what == "state":
        b.h0[slot, c] = float("nan")
        row = 2 * T
    else:
        getattr(b, what)[row, c] = float("nan")
    for k, (got, ref) in enumerate(zip(calls(), want)):
        part = (slice(row, 3 * T), c) if k < 2 else (slot, c)
        assert torch.isnan(got[part]).all(), ("decode", "verify", "state", "commit")[k]
        got[part] = ref[part]
        assert torch.equal(got, ref)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("form", FORMS)
def test_other_sequences_keep_their_bits(form, value):
    """Non-finite inputs and states of one sequence leave the others, in both directions."""
    b = Batch(43, **FORMS[form])
    o, hf = b.fwd()
    dout, bad = b.mat(), int(np.argmax(b.lens))
    want = grads(b, o, dout)
    s, slot = b.rows(bad), int(b.slots[bad])
    for t in (b.x, b.r, b.g, dout):
        t[s] = value
    b.h0[slot] = value
    o2, hf2 = b.fwd()
    got = grads(b, o2, dout)
    for now, was, at in [(o2, o, s), (hf2, hf, slot), *((got[k], want[k], s) for k in range(3)), (got[4], want[4], slot)]:
        now, was = now.clone(), was.clone()
        now[at] = was[at] = 0
        assert torch.equal(now, was)


def test_other_requests_keep_their_bits_in_decode():
    B, T, C = 4, 3, 72
    b = Batch(44, lens=[T] * B, C=C, packed=False, pool=6)
    st = b.h0.clone()
    o = lap.la_gated_decode(b.x, b.r, b.g, b.slopes, st, T, state_indices=b.idx)
    s, slot = b.rows(1), int(b.slots[1])
    for t in (b.x, b.r, b.g):
        t[s] = float("inf")
    st2 = b.h0.clone()
    st2[slot] = float("nan")
    o2 = lap.la_gated_decode(b.x, b.r, b.g, b.slopes, st2, T, state_indices=b.idx)
    o2[s], st2[slot] = o[s], st[slot]
    assert torch.equal(o2, o) and torch.equal(st2, st)


# ---------------------------------------------------------------- steep slopes

def steep(b, hi):
    """Slopes from 2^-8 to `hi`, neighbours far apart."""
    k = (np.arange(b.C) * 37) % b.C
    b.slopes = torch.from_numpy((hi * np.exp2(-(8 + np.log2(hi)) * k / max(b.C - 1, 1))).astype(np.float32)).cuda()
    return b


@pytest.mark.parametrize("form", FORMS)
def test_steep_slopes(form):
    b = steep(Batch(45, **FORMS[form]), 64.0)
    cols = slice(0, min(b.C, 72))
    o, hf = b.fwd()
    dout, dhf = b.mat(), b.state()
    got = grads(b, o, dout, dh_final=dhf)
    sums = esum = terms = 0.0
    for n, L in enumerate(b.lens):
        s, slot = b.rows(n), int(b.slots[n])
        args = [f64(t[s, cols]) for t in (b.x, b.r, b.g)] + [f64(b.slopes[cols]), f64(b.h0[slot, cols])]
        ro, rh, eo, eh = scan_one(*args)
        near(o[s, cols], ro, eo, b.dtype, f"o of sequence {n} ({L} tokens)")
        near(hf[slot, cols], rh, eh, "fp32", f"h_final of sequence {n} ({L} tokens)")
        ref = grad_one(*args, f64(o[s, cols]), f64(dout[s, cols]), f64(dhf[slot, cols]))
        for t, name in zip(got, ("dx", "dr", "dg")):
            near(t[s, cols], *ref[name], b.dtype, f"{name} of sequence {n} ({L} tokens)")
        near(got[4][slot, cols], *ref["dh0"], "fp32", f"dh0 of sequence {n} ({L} tokens)")
        sums, esum, terms = sums + ref["ds"][0], esum + ref["ds"][1], terms + np.abs(ref["ds"][0])
    near(got[3][cols], sums, esum + len(b.lens) * 2.0 ** -24 * terms, "fp32", "dslopes")


def relative(got, ref, bound, label, dtype="fp32"):
    """As near, for values of any size: `bound` counts every rounding but the output's; results under the
    smallest normal number (2^-126) may be lost."""
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    tol = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + 2.0 ** -125
    worst = np.max(np.abs(got - ref) / tol)
    assert worst <= 1, f"{label}: {worst:.3g} of its bound at {np.argmax(np.abs(got - ref) / tol)}"


@pytest.mark.parametrize("T,C", [(1, 64), (3, 67), (5, 96)])
def test_a_decayed_state_keeps_its_digits(T, C):
    """Closed input gates: o is the state times the decays alone, exp(-u) of up to u = 16 a token."""
    b = steep(Batch(46, lens=[T] * 9, C=C, dtype="fp32", packed=False), 16.0)
    b.g[:] = float("-inf")
    o, hf = b.fwd()
    st = b.h0.clone()
    od = lap.la_gated_decode(b.x, b.r, b.g, b.slopes, st, T)
    dout = torch.zeros_like(o)
    dh0 = torch.empty_like(b.h0)
    lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dh_final=b.h0, dh0=dh0, seq_len=T)
    for n in range(9):
        s = b.rows(n)
        ro, rh, eo, eh = scan_one(np.zeros((T, C)), f64(b.r[s]), np.zeros((T, C)), f64(b.slopes), f64(b.h0[n]))
        for name, got, ref, e in (("o", o[s], ro, eo), ("h_final", hf[n], rh, eh), ("decode", od[s], ro, eo),
                                  ("state", st[n], rh, eh), ("dh0", dh0[n], rh, eh)):
            relative(got, ref, e, f"{name} of sequence {n}")


# ---------------------------------------------------------------- gates far open and far closed

@pytest.mark.parametrize("dtype,C", [("fp32", 64), ("bf16", 64), ("fp32", 67), ("bf16", 67)])
@pytest.mark.parametrize("lo,hi", [(-86, -44), (30, 100)])
def test_an_input_gate_far_closed_or_open(lo, hi, dtype, C):
    """sigmoid(g) down to exp(-86), and 1: o = beta sigmoid(g) x of one token, relative to itself."""
    b = Batch(47, lens=[1] * 40, C=C, dtype=dtype, packed=False, states=False)
    b.g = (lo + (hi - lo) * torch.from_numpy(b.rng.random((40, C))).cuda()).to(b.g.dtype)
    if lo > 0:
        b.g[::3] = float("inf")
    o = lap.la_gated_scan_fwd(b.x, b.r, b.g, b.slopes, seq_len=1)
    od = lap.la_gated_decode(b.x, b.r, b.g, b.slopes, torch.zeros(40, C, device="cuda"), 1)
    dx = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, b.x, seq_len=1)[0]
    x, r, g = f64(b.x), f64(b.r), f64(b.g)
    _, sg, u, _, beta = gates(x, r, g, f64(b.slopes))
    _, eg, _, eb = gate_errors(r, g, u)
    ref = beta * sg * x
    for name, got in (("scan", o), ("decode", od), ("dx", dx)):  # dout = x: dx = beta sigmoid(g) x too
        relative(got, ref, np.abs(ref) * (eb + eg + 2.0 ** -21), name, dtype)


def complement(z):
    """1 - sigmoid(z) and its error: exp(-z) / (1 + exp(-z)) from the argument's rounding |z| 2^-23, exp2
    and the reciprocal (2^-22 each), a sum and a product."""
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, e / (1 + e), 1 / (1 + e)), 2.0 ** -20 + np.abs(z) * 2.0 ** -23


@pytest.mark.parametrize("C", [64, 67])
@pytest.mark.parametrize("lo,hi,slope", [(-4, 4, 1.0), (8, 20, 1.0), (20, 80, 1.0), (-80, -8, 1.0), (-4, 4, 20.0),
                                         (8, 20, 20.0)])
def test_gradients_are_relative_to_their_factors(lo, hi, slope, C):
    """One token: dg = dx x (1 - sigmoid(g)) and dr = du u (1 - sigmoid(r)) keep their digits however far
    the gates are open, and du those of lambda however steep the slopes."""
    b = steep(Batch(48, lens=[1] * 30, C=C, dtype="fp32", packed=False), slope)
    gen = torch.Generator(device="cuda").manual_seed(48)
    for t in (b.r, b.g):
        t.copy_(lo + (hi - lo) * torch.rand(t.shape, generator=gen, device="cuda"))
    o, _ = b.fwd()
    dout = b.mat()
    dx, dr, dg, ds, dh0 = grads(b, o, dout)
    x, r, g, h, G = (f64(t) for t in (b.x, b.r, b.g, b.h0, dout))
    sr, sg, u, lam, beta = gates(x, r, g, f64(b.slopes))
    er, eg, d, eb = gate_errors(r, g, u)
    (cg, ecg), (cr, ecr) = complement(g), complement(r)
    rdx = G * beta * sg
    edx = np.abs(rdx) * (eb + eg + 2.0 ** -21)
    relative(dx, rdx, edx, "dx")
    rdg = rdx * x * cg
    relative(dg, rdg, np.abs(rdg) * (eb + eg + ecg + 2.0 ** -20), "dg")
    a1, a2 = sg * x * lam * lam / beta, lam * h
    du, size = G * (a1 - a2), np.abs(G) * (np.abs(a1) + np.abs(a2))
    edu = size * (eb + eg + 2 * d + 2.0 ** -20)
    rdr = du * u * cr
    relative(dr, rdr, edu * u * cr + np.abs(rdr) * (er + ecr + 2.0 ** -21), "dr")
    relative(dh0, lam * G, np.abs(lam * G) * (d + 2.0 ** -23), "dh0")
    terms, eterms = du * sr, edu * sr + np.abs(du * sr) * (er + 2.0 ** -22)
    relative(ds, terms.sum(0), eterms.sum(0) + 30 * 2.0 ** -24 * np.abs(terms).sum(0), "dslopes")


# ---------------------------------------------------------------- a single column

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_single_column_of_any_stride(dtype):
    """[rows, 1] tensors whose column stride is not 1, from a transposed or a wider matrix."""
    gen = torch.Generator(device="cuda").manual_seed(49)
    wide = torch.randn((7, 300), generator=gen, device="cuda").to(dtype)
    cols = [wide[k:k + 1].t() for k in range(5)]  # strides (1, 300)
    slopes = torch.tensor([0.3], device="cuda")
    x, r, g, d, y = cols
    o = lap.la_gated_scan_fwd(x, r, g, slopes, seq_len=300)
    got = lap.la_gated_scan_bwd(x, r, g, slopes, o, d, seq_len=300)
    want = [t.contiguous(memory_format=torch.contiguous_format).clone().reshape(300, 1) for t in cols]
    x, r, g, d, y = want
    ref = lap.la_gated_scan_fwd(x, r, g, slopes, seq_len=300)
    assert torch.equal(o, ref)
    for a, b in zip(got[:4], lap.la_gated_scan_bwd(x, r, g, slopes, ref, d, seq_len=300)[:4]):
        assert torch.equal(a, b)
    w = torch.tensor([1.5], device="cuda")
    for a, b in zip(lap.la_rms_norm_fwd(cols[4], w, 1e-5, residual=cols[0]), lap.la_rms_norm_fwd(y, w, 1e-5, residual=x)):
        assert torch.equal(a, b)
