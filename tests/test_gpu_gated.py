"""The gated recurrence on the GPU (include/la_gated.h) against its plain 64-bit form: forward,
gradients, decode / verify / commit, over lengths around the kernels' tiles, odd channel counts,
row strides, pools, padded and empty sequences, closed gates, and non-finite neighbours.

Tolerances are the bounds computed beside the reference values (tests/gated_reference.py)."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from gated_reference import HALF_STEP, grad_one, scan_one

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TINY = 1e-30


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """Seeded inputs of one call: x, r, g (apart, or column ranges of one matrix), slopes, states."""

    def __init__(self, seed, lens, C, dtype="bf16", packed=True, fused=False, pool=0, pad=(), states=True, tail=0,
                 offset=0):
        self.rng = np.random.default_rng(seed)
        self.lens, self.C, self.dtype, self.packed = list(lens), C, dtype, packed
        self.cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        self.tokens = int(self.cu[-1]) + tail
        N = len(self.lens)
        self.fused, self.offset = fused, offset
        self.x, self.r, self.g = self.three()
        self.slopes = torch.from_numpy(np.exp2(-8.0 * np.arange(1, C + 1) / C).astype(np.float32)).cuda()
        self.slots = np.arange(N) if not pool else self.rng.permutation(pool)[:N]
        self.slots = self.slots.astype(np.int32)
        self.slots[list(pad)] = -1
        self.idx = torch.from_numpy(self.slots).cuda() if pool else None
        self.P = pool or N
        self.h0 = self.state() if states else None
        self.cu_dev = torch.from_numpy(self.cu).cuda() if packed else None
        self.kw = dict(state_indices=self.idx, cu_seqlens=self.cu_dev, seq_len=None if packed else self.lens[0])

    def mat(self, scale=1.0, cols=None):
        a = self.rng.standard_normal((self.tokens, cols or self.C)).astype(np.float32) * np.float32(scale)
        return torch.from_numpy(a).to(DT[self.dtype]).cuda()

    def state(self):
        return torch.from_numpy(self.rng.standard_normal((self.P, self.C)).astype(np.float32)).cuda()

    def three(self, fill=None):
        C, off = self.C, self.offset
        if not self.fused:
            return tuple(self.mat(1.5) if fill is None else self.blank(fill) for _ in range(3))
        m = self.mat(1.5, 3 * C + off)
        if fill is not None:
            m.fill_(fill)
        return m[:, off:off + C], m[:, off + C:off + 2 * C], m[:, off + 2 * C:]

    def blank(self, fill=float("nan")):
        return torch.full((self.tokens, self.C), fill, dtype=DT[self.dtype], device="cuda")

    def start(self, n, h=None):
        h = self.h0 if h is None else h
        return np.zeros(self.C) if h is None else f64(h[int(self.slots[n])])

    def fwd(self, o=None, hf=None, **kw):
        o = self.blank() if o is None else o
        hf = torch.full((self.P, self.C), float("nan"), device="cuda") if hf is None else hf
        lap.la_gated_scan_fwd(self.x, self.r, self.g, self.slopes, h0=self.h0, o=o, h_final=hf, **self.kw, **kw)
        torch.cuda.synchronize()
        return o, hf

    def rows(self, n):
        return slice(int(self.cu[n]), int(self.cu[n + 1]))


def near(got, ref, bound, dtype, label):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    tol = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + TINY
    worst = np.max(np.abs(got - ref) / tol) if ref.size else 0.0
    assert worst <= 1, f"{label}: {worst:.3g} of its bound at {np.argmax(np.abs(got - ref) / tol)}"


def check_fwd(b, o, hf):
    live = np.zeros(b.tokens, bool)
    for n, L in enumerate(b.lens):
        if b.slots[n] < 0:
            continue
        s = b.rows(n)
        live[s] = True
        ro, rh, eo, eh = scan_one(f64(b.x[s]), f64(b.r[s]), f64(b.g[s]), f64(b.slopes), b.start(n))
        near(o[s], ro, eo, b.dtype, f"o of sequence {n} ({L} tokens)")
        near(hf[int(b.slots[n])], rh, eh, "fp32", f"h_final of sequence {n} ({L} tokens)")
    assert torch.isnan(o[torch.from_numpy(~live).cuda()]).all(), "rows of no sequence were written"
    other = np.setdiff1d(np.arange(b.P), b.slots)
    assert torch.isnan(hf[torch.from_numpy(other).cuda()]).all(), "unselected slots were written"


EDGE = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257]
FORMS = {
    "one token": dict(lens=[1], C=64, packed=False),
    "one odd sequence": dict(lens=[77], C=67, packed=False),
    "one channel": dict(lens=[300], C=1, packed=False, dtype="fp32"),
    "fixed": dict(lens=[129] * 5, C=130, packed=False),
    "fixed, no states": dict(lens=[64] * 3, C=96, packed=False, states=False),
    "fixed short": dict(lens=[3] * 100, C=200, packed=False, pool=120, pad=(0, 7, 99)),
    "edges": dict(lens=EDGE, C=72, pool=30, pad=(4,)),
    "edges fp32": dict(lens=EDGE[::-1], C=33, dtype="fp32", pool=30, pad=(0, 17)),
    "fused": dict(lens=[200, 0, 0, 311], C=128, fused=True),
    "fused odd": dict(lens=[200, 5, 311], C=37, fused=True, offset=1, pool=5, pad=(1,)),
    "fused fp32": dict(lens=[40, 90], C=66, fused=True, dtype="fp32", offset=2),
    "rows behind": dict(lens=[10, 300, 4], C=64, tail=130),
    "long": dict(lens=[5000], C=20, packed=False),
    "long packed": dict(lens=[1500, 2500, 1, 700], C=130, pool=9, pad=(2,)),
    "long fp32": dict(lens=[3333], C=9, packed=False, dtype="fp32"),
    "many short": dict(lens=list(np.random.default_rng(5).integers(0, 6, 700)), C=65, pool=800),
    "long sequences": dict(lens=[2000, 0, 1, 1300, 129, 128, 127, 900], C=72, pool=12, pad=(4,)),
    "long sequences odd": dict(lens=[112, 2000, 113, 0, 48, 1, 1300, 336], C=67, fused=True, offset=1, pool=9, pad=(7,)),
    "long sequences fp32": dict(lens=[64, 900, 0, 65, 1, 1300], C=68, dtype="fp32", tail=9),
    "many sequences": dict(lens=list(np.random.default_rng(6).integers(0, 260, 700)), C=64, pool=701, pad=(699,)),
    "thousands": dict(lens=list(np.random.default_rng(7).integers(0, 3, 5000)), C=3, dtype="fp32"),
    "groups": dict(lens=[1100] * 20, C=200, packed=False, pool=23, pad=(11,)),
    "groups packed": dict(lens=list(np.random.default_rng(9).integers(700, 1500, 20)), C=200, pool=23, pad=(3,)),
    "groups fp32": dict(lens=[9000], C=9, packed=False, dtype="fp32"),
    "groups of mixed rows": dict(lens=list(np.random.default_rng(8).integers(0, 5, 5000)), C=3, dtype="fp32"),
    "all padded": dict(lens=[5, 9], C=64, pool=4, pad=(0, 1)),
    "empty sequences": dict(lens=[0, 0, 0], C=64, pool=4),
}


@pytest.mark.parametrize("form", FORMS)
def test_forward(form):
    b = Batch(1, **FORMS[form])
    check_fwd(b, *b.fwd())


@pytest.mark.parametrize("form", FORMS)
def test_backward(form):
    b = Batch(2, **FORMS[form])
    o, _ = b.fwd()
    dout, dhf = b.mat(), b.state() if b.h0 is not None else None
    dx, dr, dg = b.three(float("nan"))
    dh0 = torch.full((b.P, b.C), float("nan"), device="cuda") if b.h0 is not None else None
    res = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dh_final=dhf, dx=dx, dr=dr, dg=dg, dh0=dh0,
                                **b.kw)
    torch.cuda.synchronize()
    assert res[0] is dx and res[4] is dh0
    sums, esum, terms = np.zeros(b.C), np.zeros(b.C), 0.0
    live = np.zeros(b.tokens, bool)
    for n, L in enumerate(b.lens):
        if b.slots[n] < 0:
            continue
        s = b.rows(n)
        live[s] = True
        ref = grad_one(f64(b.x[s]), f64(b.r[s]), f64(b.g[s]), f64(b.slopes), b.start(n), f64(o[s]), f64(dout[s]),
                       np.zeros(b.C) if dhf is None else b.start(n, dhf))
        for name, t in (("dx", dx), ("dr", dr), ("dg", dg)):
            near(t[s], *ref[name], b.dtype, f"{name} of sequence {n} ({L} tokens)")
        if dh0 is not None:
            near(dh0[int(b.slots[n])], *ref["dh0"], "fp32", f"dh0 of sequence {n} ({L} tokens)")
        sums, esum, terms = sums + ref["ds"][0], esum + ref["ds"][1], terms + np.abs(ref["ds"][0])
    near(res[3], sums, esum + len(b.lens) * 2.0 ** -24 * terms, "fp32", "dslopes")
    dead = torch.from_numpy(~live).cuda()
    assert all(torch.isnan(t[dead]).all() for t in (dx, dr, dg)), "rows of no sequence were written"
    if dh0 is not None:
        other = torch.from_numpy(np.setdiff1d(np.arange(b.P), b.slots)).cuda()
        assert torch.isnan(dh0[other]).all()


def test_gradients_against_differences_of_the_kernel():
    """FP32: a directional difference of the forward kernel against its gradients' product."""
    b = Batch(3, lens=[150], C=40, packed=False, dtype="fp32")
    o, hf = b.fwd()
    dout, dhf = b.mat(), b.state()
    dh0 = torch.zeros_like(b.h0)
    grads = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dh_final=dhf, dh0=dh0, **b.kw)
    for k, name in enumerate(("x", "r", "g", "slopes", "h0")):
        v = getattr(b, name)
        step = torch.from_numpy(b.rng.standard_normal(tuple(v.shape)).astype(np.float32)).cuda()
        if name == "slopes":
            step *= v
        eps, vals = 2.0 ** -8, []
        for sgn in (1, -1):
            setattr(b, name, v + sgn * eps * step)
            p, q = b.fwd()
            vals.append(float((p.double() * dout.double()).sum() + (q.double() * dhf.double()).sum()))
        setattr(b, name, v)
        diff, dot = (vals[0] - vals[1]) / (2 * eps), float((grads[k].double() * step.double()).sum())
        # FP32 outputs: 2 * 2^-20 relative noise over 2^-7; the third-order term 2^-16 / 6
        size = float((grads[k].double() * step.double()).norm()) * np.sqrt(v.numel())
        noise = float((o.double() * dout.double()).abs().sum()) * 2.0 ** -20 / eps
        assert abs(diff - dot) <= 2.0 ** -14 * size + noise, (name, diff, dot)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place_pool_and_continuation(dtype):
    """h_final == h0, and two halves of every sequence through the pool."""
    b = Batch(4, lens=[300, 7, 0, 129], C=70, dtype=dtype, pool=6)
    o, hf = b.fwd()
    pool = b.h0.clone()
    first = [min(L, 130) for L in b.lens]
    pieces = [(0, first), (1, [L - f for L, f in zip(b.lens, first)])]
    for part, lens in pieces:
        rows = np.concatenate([np.arange(b.cu[n] + part * first[n], b.cu[n] + part * first[n] + L)
                               for n, L in enumerate(lens)]).astype(np.int64)
        at = torch.from_numpy(rows).cuda()
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        o2 = lap.la_gated_scan_fwd(b.x[at], b.r[at], b.g[at], b.slopes, h0=pool, h_final=pool, state_indices=b.idx,
                                   cu_seqlens=cu)
        torch.testing.assert_close(o2, o[at], rtol=2 * HALF_STEP[dtype] + 1e-4, atol=1e-4)
    sel = b.idx.long()
    torch.testing.assert_close(pool[sel], hf[sel], rtol=1e-4, atol=1e-4)
    other = torch.from_numpy(np.setdiff1d(np.arange(b.P), b.slots)).cuda()
    assert torch.equal(pool[other], b.h0[other])


def test_closed_gates_keep_the_state():
    """r = -inf keeps the state and adds nothing; g = -inf adds nothing.  The state is kept up to the
    rounding of a blocked evaluation, which composes the rows before a tile in another order than
    it walks them: each value is within its bound E of the exact one, two of them within 2 E."""
    b = Batch(5, lens=[400], C=96, packed=False, dtype="fp32")
    b.r[100:] = float("-inf")
    o, hf = b.fwd()
    ro, _, eo, _ = scan_one(f64(b.x), f64(b.r), f64(b.g), f64(b.slopes), b.start(0))
    near(o, ro, eo, "fp32", "o under closed decay gates")
    assert np.array_equal(ro[100:], np.tile(ro[99], (300, 1)))
    assert np.all(np.abs(f64(o[100:]) - f64(o[99])) <= eo[100:] + eo[99] + 2.0 ** -23 * np.abs(ro[99]))
    assert torch.equal(hf[0], o[399])
    b = Batch(6, lens=[400], C=96, packed=False)
    b.g[:] = float("-inf")
    b.r[:] = float("inf")
    o, hf = b.fwd()
    ro, rh, eo, eh = scan_one(np.zeros((400, 96)), np.full((400, 96), 800.0), np.zeros((400, 96)), f64(b.slopes),
                              f64(b.h0[0]))
    near(o, ro, eo + 1e-30, "bf16", "o under closed input gates")
    dr = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, b.mat(), h0=b.h0, seq_len=400)[1]
    assert torch.isfinite(dr.float()).all()


def test_gradients_of_closed_decay_gates_and_zero_slopes_are_finite():
    b = Batch(7, lens=[130], C=64, packed=False)
    b.r[::3] = float("-inf")
    b.slopes[::2] = 0.0
    o, _ = b.fwd()
    grads = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, b.mat(), h0=b.h0, seq_len=130)
    assert all(torch.isfinite(t.float()).all() for t in grads[:4])
    ref = grad_one(f64(b.x), f64(b.r), f64(b.g), f64(b.slopes), b.start(0), f64(o), np.zeros((130, 64)), np.zeros(64))
    assert np.all(np.isfinite(ref["dr"][0]))


@pytest.mark.parametrize("lens", [[100, 37, 250, 64, 300], [700, 537, 850, 264, 900]])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_sequences_are_isolated(value, lens):
    """Non-finite inputs and states of one sequence, and of padded ones, leave the others bitwise."""
    b = Batch(8, lens=lens, C=72, pool=7, pad=(3,))
    o, hf = b.fwd()
    dout = b.mat()
    good = [n for n in range(5) if n not in (1, 3)]
    ref = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dx=b.blank(), dr=b.blank(), dg=b.blank(),
                                **b.kw)
    for n in (1, 3):
        for t in (b.x, b.r, b.g, dout):
            t[b.rows(n)] = value
    b.h0[int(b.slots[1])] = value
    o2, hf2 = b.fwd()
    got = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o2, dout, h0=b.h0, dx=b.blank(), dr=b.blank(), dg=b.blank(),
                                **b.kw)
    torch.cuda.synchronize()
    for n in good:
        s = b.rows(n)
        assert torch.equal(o2[s], o[s]), f"sequence {n} changed"
        assert torch.equal(hf2[int(b.slots[n])], hf[int(b.slots[n])])
        for t, u in zip(got[:3], ref[:3]):
            assert torch.equal(t[s], u[s]), f"a gradient of sequence {n} changed"


def test_sequences_may_share_a_slot_that_is_read():
    """A common prompt's state: both sequences begin with it, and no state is written."""
    b = Batch(13, lens=[300, 41], C=64, pool=3)
    b.slots[:] = 2
    b.idx.fill_(2)
    o = b.blank()
    lap.la_gated_scan_fwd(b.x, b.r, b.g, b.slopes, h0=b.h0, o=o, **b.kw)
    torch.cuda.synchronize()
    for n, L in enumerate(b.lens):
        s = b.rows(n)
        ro, _, eo, _ = scan_one(f64(b.x[s]), f64(b.r[s]), f64(b.g[s]), f64(b.slopes), b.start(n))
        near(o[s], ro, eo, b.dtype, f"o of sequence {n} ({L} tokens)")


def test_bad_bounds_and_indices_are_reported():
    b = Batch(9, lens=[200, 100, 300], C=64, pool=5)
    for cu in ([0, 250, 200, 600], [0, 200, 300, 601], [-1, 200, 300, 600]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        b.kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, hf = b.fwd(dev_error=err)
        assert int(err) == lap.DEV_ERR_BAD_SEQLENS and torch.isnan(o).all() and torch.isnan(hf).all()
    b.kw["cu_seqlens"] = b.cu_dev
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.slots[1] = 5
    b.kw["state_indices"] = torch.from_numpy(b.slots).cuda()
    o, hf = b.fwd(dev_error=err)
    assert int(err) == lap.DEV_ERR_BAD_INDEX
    b.slots[1] = -1
    check_fwd(b, o, hf)


def test_repeated_captured_and_replayed_calls_agree_bitwise():
    b = Batch(10, lens=[700, 3, 1400], C=200, pool=4)
    o, hf = b.fwd()
    dout, dhf = b.mat(), b.state()

    def bwd():
        return lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dh_final=dhf, **b.kw)[:4]
    grads = bwd()
    for _ in range(3):
        o2, hf2 = b.fwd()
        assert torch.equal(o2.view(torch.int16), o.view(torch.int16))
        assert torch.equal(hf2.view(torch.int32), hf.view(torch.int32))
        assert all(torch.equal(x, y) for x, y in zip(bwd(), grads))
    side = torch.cuda.Stream()
    o3, hf3 = b.blank(), torch.full_like(hf, float("nan"))
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        lap.la_gated_scan_fwd(b.x, b.r, b.g, b.slopes, h0=b.h0, o=o3, h_final=hf3, **b.kw)
        grads3 = bwd()
    for _ in range(3):
        o3.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o3.view(torch.int16), o.view(torch.int16))
        assert all(torch.equal(x, y) for x, y in zip(grads3, grads))


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces, against the same calls one after another."""
    bs = [Batch(20 + k, lens=[900, 1100 + k], C=160, pool=4) for k in range(2)]
    refs = [b.fwd() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    outs = [(b.blank(), torch.full((b.P, b.C), float("nan"), device="cuda")) for b in bs]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, st, (o, hf) in zip(bs, streams, outs):
            lap.la_gated_scan_fwd(b.x, b.r, b.g, b.slopes, h0=b.h0, o=o, h_final=hf, stream=st, **b.kw)
    torch.cuda.synchronize()
    for (o, hf), (ro, rh) in zip(outs, refs):
        assert torch.equal(o, ro) and torch.equal(hf[~torch.isnan(rh)], rh[~torch.isnan(rh)])


def test_garbage_workspace():
    b = Batch(11, lens=[700, 3, 1400], C=200, pool=4)
    o, hf = b.fwd()
    ref = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, o, h0=b.h0, **b.kw)
    for fill in (0x00, 0x7F, 0xFF):
        for back in (False, True):
            n = lap.la_gated_scan_workspace(1, b.tokens, 3, 200, True, torch.bfloat16, back)
            ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
            if back:
                got = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, o, h0=b.h0, workspace=ws, **b.kw)
                assert all(torch.equal(x, y) for x, y in zip(got[:4], ref[:4]))
            else:
                assert torch.equal(b.fwd(workspace=ws)[0], o)


def test_calls_in_a_row_share_a_workspace():
    """Calls of different batches on one stream, one workspace, nothing in between."""
    bs = [Batch(60 + k, lens=lens, C=C, pool=6) for k, (lens, C) in enumerate((
        ([900, 3, 1200], 72), ([5, 0, 700, 2], 200), ([2100], 40), ([300, 301, 302, 303, 1], 136)))]
    refs = [b.fwd() for b in bs]
    douts = [b.mat() for b in bs]
    grads = [lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, d, h0=b.h0, **b.kw)[:4]
             for b, (o, _), d in zip(bs, refs, douts)]
    n = max(lap.la_gated_scan_workspace(1, b.tokens, len(b.lens), b.C, True, torch.bfloat16, True) for b in bs)
    ws = torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda")
    outs = [(b.blank(), torch.full((b.P, b.C), float("nan"), device="cuda")) for b in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for b, (o, hf), d in zip(bs, outs, douts):
            lap.la_gated_scan_fwd(b.x, b.r, b.g, b.slopes, h0=b.h0, o=o, h_final=hf, workspace=ws, **b.kw)
            got.append(lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, d, h0=b.h0, workspace=ws, **b.kw)[:4])
    torch.cuda.synchronize()
    for (o, hf), (ro, rh), g, rg in zip(outs, refs, got, grads):
        assert torch.equal(o, ro) and torch.equal(hf[~torch.isnan(rh)], rh[~torch.isnan(rh)])
        assert all(torch.equal(a, b) for a, b in zip(g, rg))


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31 give what a compact copy gives, bit for bit."""
    T, ld, C = (1 << 18) + 77, 8256, 24
    wide = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide[:, :3 * C] = torch.randn((T, 3 * C), generator=gen, device="cuda").to(torch.bfloat16)
    x, r, g = (wide[:, k * C:(k + 1) * C] for k in range(3))
    o = wide[:, 4 * C:5 * C]
    slopes = torch.exp2(-8.0 * torch.arange(1, C + 1, device="cuda") / C)
    assert T * ld > 1 << 31
    lap.la_gated_scan_fwd(x, r, g, slopes, o=o, seq_len=T)
    ref = lap.la_gated_scan_fwd(x.contiguous(), r.contiguous(), g.contiguous(), slopes, seq_len=T)
    assert torch.equal(o, ref)
    d = [wide[:, k * C:(k + 1) * C] for k in (6, 7, 8)]
    got = lap.la_gated_scan_bwd(x, r, g, slopes, o, x, dx=d[0], dr=d[1], dg=d[2], seq_len=T)
    want = lap.la_gated_scan_bwd(x.contiguous(), r.contiguous(), g.contiguous(), slopes, ref, x.contiguous(), seq_len=T)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_row_strides_and_alignment(dtype):
    """The same values at any alignment and stride: each within its bound (16-byte rows are cut into
    other tiles than the rest, and a sum's order follows the tiles, so the bits may differ)."""
    b = Batch(12, lens=[333, 70], C=64, pool=2, dtype=dtype)
    dout = b.mat()
    want = b.fwd()[0]
    grads = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, want, dout, h0=b.h0, **b.kw)
    for off, ld in ((0, 64 + 8), (1, 67), (2, 66), (4, 72), (8, 80), (3, 65)):
        views = []
        for t in (b.x, b.r, b.g, dout, *[b.blank() for _ in range(4)]):
            w = torch.full((b.tokens, ld + off), 7.0, dtype=DT[dtype], device="cuda")
            v = w[:, off:off + 64]
            v.copy_(t)
            views.append((w, v))
        x, r, g, do, o, dx, dr, dg = (v for _, v in views)
        lap.la_gated_scan_fwd(x, r, g, b.slopes, h0=b.h0, o=o, **b.kw)
        lap.la_gated_scan_bwd(x, r, g, b.slopes, o, do, h0=b.h0, dx=dx, dr=dr, dg=dg, **b.kw)
        for n in range(2):
            s = b.rows(n)
            ro, _, eo, _ = scan_one(f64(b.x[s]), f64(b.r[s]), f64(b.g[s]), f64(b.slopes), b.start(n))
            near(o[s], ro, eo, dtype, f"o at offset {off}, stride {ld}")
            ref = grad_one(f64(b.x[s]), f64(b.r[s]), f64(b.g[s]), f64(b.slopes), b.start(n), f64(o[s]), f64(dout[s]),
                           np.zeros(64))
            for t, name in ((dx, "dx"), (dr, "dr"), (dg, "dg")):
                near(t[s], *ref[name], dtype, f"{name} at offset {off}, stride {ld}")
        for w, _ in views[4:]:  # nothing beside the columns was written
            assert (w[:, :off] == 7).all() and (w[:, off + 64:] == 7).all()


CHAINS = [0, 600, 2000, 1, 517, 300, 1290, 128, 700, 64, 1025, 812, 0, 333, 901, 499]


@pytest.mark.parametrize("dtype,back", [("bf16", False), ("bf16", True), ("fp32", False), ("fp32", True)])
def test_packed_batches_by_chains(dtype, back):
    """Wide packed batches of long sequences, which blocks take a sequence's channels at a time:
    padded, empty and out-of-range sequences among them; checked on a range of channels."""
    b = Batch(14, lens=CHAINS, C=4096, dtype=dtype, pool=20, pad=(4,))
    b.slots[9] = 20
    b.idx = b.kw["state_indices"] = torch.from_numpy(b.slots).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, hf = b.fwd(dev_error=err)
    assert int(err) == lap.DEV_ERR_BAD_INDEX
    b.slots[9] = -1
    C, cols = 4096, slice(4000, 4064)
    dout, dhf = (b.mat(), b.state()) if back else (None, None)
    dh0 = torch.full_like(hf, float("nan"))
    got = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dh_final=dhf, dx=b.blank(), dr=b.blank(),
                                dg=b.blank(), dh0=dh0, **b.kw) if back else None
    dead = torch.ones(b.tokens, dtype=torch.bool, device="cuda")
    sums = esum = terms = 0.0
    for n, L in enumerate(CHAINS):
        if b.slots[n] < 0:
            continue
        s, slot = b.rows(n), int(b.slots[n])
        dead[s] = False
        args = [f64(t[s, cols]) for t in (b.x, b.r, b.g)] + [f64(b.slopes[cols]), f64(b.h0[slot, cols])]
        if not back:
            ro, rh, eo, eh = scan_one(*args)
            near(o[s, cols], ro, eo, dtype, f"o of sequence {n} ({L} tokens)")
            near(hf[slot, cols], rh, eh, "fp32", f"h_final of sequence {n} ({L} tokens)")
            continue
        ref = grad_one(*args, f64(o[s, cols]), f64(dout[s, cols]), f64(dhf[slot, cols]))
        for t, name in zip(got, ("dx", "dr", "dg")):
            near(t[s, cols], *ref[name], dtype, f"{name} of sequence {n} ({L} tokens)")
        near(dh0[slot, cols], *ref["dh0"], "fp32", f"dh0 of sequence {n} ({L} tokens)")
        sums, esum, terms = sums + ref["ds"][0], esum + ref["ds"][1], terms + np.abs(ref["ds"][0])
    if back:
        near(got[3][cols], sums, esum + len(CHAINS) * 2.0 ** -24 * terms, "fp32", "dslopes")
        assert all(torch.isnan(t[dead]).all() for t in got[:3])
    else:
        assert torch.isnan(o[dead]).all()
        b.kw["cu_seqlens"] = b.cu_dev.flip(0).contiguous()
        err.zero_()
        o, hf = b.fwd(dev_error=err)
        assert int(err) & lap.DEV_ERR_BAD_SEQLENS and torch.isnan(o).all() and torch.isnan(hf).all()


UNEVEN = [90, 6000, 0, 33, 128, 1, 5000] + [70] * 60


@pytest.mark.parametrize("dtype,C", [("bf16", 1024), ("bf16", 1001), ("fp32", 1024)])
def test_long_sequences_among_many_short_ones(dtype, C):
    """Sequences far longer than the others, which blocks share by tiles while the others go by chains;
    padded ones of either kind, both directions, checked on a range of channels, bitwise repeatable."""
    b = Batch(15, lens=UNEVEN, C=C, dtype=dtype, pool=70, pad=(0, 6))
    cols = slice(C - 41, C)
    o, hf = b.fwd()
    dout, dhf = b.mat(), b.state()

    def bwd():
        dh0 = torch.full_like(hf, float("nan"))
        return lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, dout, h0=b.h0, dh_final=dhf, dx=b.blank(),
                                     dr=b.blank(), dg=b.blank(), dh0=dh0, **b.kw)
    got = bwd()
    torch.cuda.synchronize()
    live = torch.zeros(b.tokens, dtype=torch.bool, device="cuda")
    sums = esum = terms = 0.0
    for n, L in enumerate(UNEVEN):
        if b.slots[n] < 0:
            continue
        s, slot = b.rows(n), int(b.slots[n])
        live[s] = True
        args = [f64(t[s, cols]) for t in (b.x, b.r, b.g)] + [f64(b.slopes[cols]), f64(b.h0[slot, cols])]
        ro, rh, eo, eh = scan_one(*args)
        near(o[s, cols], ro, eo, dtype, f"o of sequence {n} ({L} tokens)")
        near(hf[slot, cols], rh, eh, "fp32", f"h_final of sequence {n} ({L} tokens)")
        ref = grad_one(*args, f64(o[s, cols]), f64(dout[s, cols]), f64(dhf[slot, cols]))
        for t, name in zip(got, ("dx", "dr", "dg")):
            near(t[s, cols], *ref[name], dtype, f"{name} of sequence {n} ({L} tokens)")
        near(got[4][slot, cols], *ref["dh0"], "fp32", f"dh0 of sequence {n} ({L} tokens)")
        sums, esum, terms = sums + ref["ds"][0], esum + ref["ds"][1], terms + np.abs(ref["ds"][0])
    near(got[3][cols], sums, esum + len(UNEVEN) * 2.0 ** -24 * terms, "fp32", "dslopes")
    assert all(torch.isnan(t[~live]).all() for t in (o, *got[:3]))
    again = bwd()
    assert torch.equal(b.fwd()[0][live], o[live])
    assert all(torch.equal(t[live], u[live]) for t, u in zip(again[:3], got[:3])) and torch.equal(again[3], got[3])


@pytest.mark.parametrize("lens,C", [(UNEVEN, 1024), ([300] * 240, 256), ([1] * 900, 70)])
def test_garbage_workspace_of_lists_and_tables(lens, C):
    b = Batch(16, lens=lens, C=C, pool=len(lens))
    o, _ = b.fwd()
    ref = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, o, h0=b.h0, **b.kw)
    for fill in (0x00, 0x7F, 0xFF):
        for back in (False, True):
            n = lap.la_gated_scan_workspace(1, b.tokens, len(lens), C, True, torch.bfloat16, back)
            ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
            if back:
                got = lap.la_gated_scan_bwd(b.x, b.r, b.g, b.slopes, o, o, h0=b.h0, workspace=ws, **b.kw)
                assert all(torch.equal(x, y) for x, y in zip(got[:4], ref[:4]))
            else:
                assert torch.equal(b.fwd(workspace=ws)[0], o)


# ---------------------------------------------------------------- decode, verify, commit

DECODE = {
    "one request": dict(B=1, T=1, C=64, P=1, dtype="bf16", idx=None),
    "serving": dict(B=40, T=1, C=520, P=64, dtype="bf16", idx="pad"),
    "drafts": dict(B=17, T=8, C=130, P=20, dtype="bf16", idx="pad"),
    "odd": dict(B=5, T=3, C=67, P=9, dtype="fp32", idx="pad"),
    "long": dict(B=3, T=70, C=33, P=3, dtype="bf16", idx=None),
    "fused": dict(B=6, T=4, C=96, P=8, dtype="bf16", idx="pad", fused=True),
    "fused odd": dict(B=6, T=5, C=41, P=8, dtype="fp32", idx="pad", fused=True, offset=3),
}


@pytest.mark.parametrize("form", DECODE)
def test_decode_verify_commit(form):
    f = DECODE[form]
    B, T, C, P = f["B"], f["T"], f["C"], f["P"]
    b = Batch(30, lens=[T] * B, C=C, dtype=f["dtype"], packed=False, pool=P if f["idx"] else 0,
              pad=range(1, B, 5) if f["idx"] else (), fused=f.get("fused", False), offset=f.get("offset", 0))
    pool0 = b.h0.clone()
    state, o = pool0.clone(), b.blank()
    lap.la_gated_decode(b.x, b.r, b.g, b.slopes, state, T, state_indices=b.idx, o=o)
    ov = b.blank()
    vstate = pool0.clone()
    lap.la_gated_verify(b.x, b.r, b.g, b.slopes, vstate, T, state_indices=b.idx, o=ov)
    torch.cuda.synchronize()
    assert torch.equal(vstate, pool0)
    live = torch.from_numpy(np.repeat(b.slots >= 0, T)).cuda()
    assert torch.equal(ov[live], o[live]) and torch.isnan(o[~live]).all() and torch.isnan(ov[~live]).all()
    acc = np.random.default_rng(31).integers(-1, T + 2, B).astype(np.int32)
    acc[0] = T
    cstate = pool0.clone()
    lap.la_gated_commit(b.x, b.r, b.g, b.slopes, cstate, T, torch.from_numpy(acc).cuda(), state_indices=b.idx)
    full = pool0.clone()
    lap.la_gated_commit(b.x, b.r, b.g, b.slopes, full, T, torch.full((B,), T, dtype=torch.int32, device="cuda"),
                        state_indices=b.idx)
    assert torch.equal(full, state)
    touched = []
    for n in range(B):
        slot = int(b.slots[n])
        if slot < 0:
            continue
        s = b.rows(n)
        args = f64(b.x[s]), f64(b.r[s]), f64(b.g[s])
        ro, rh, eo, eh = scan_one(*args, f64(b.slopes), f64(pool0[slot]))
        near(o[s], ro, eo, f["dtype"], f"o of request {n}")
        near(state[slot], rh, eh, "fp32", f"state of request {n}")
        L = int(np.clip(acc[n], 0, T))
        if L == 0:
            assert torch.equal(cstate[slot], pool0[slot])
        _, rh, _, eh = scan_one(*(v[:L] for v in args), f64(b.slopes), f64(pool0[slot]))
        near(cstate[slot], rh, eh, "fp32", f"committed state of request {n} ({L} of {T})")
        touched.append(slot)
    other = torch.from_numpy(np.setdiff1d(np.arange(b.P), touched)).cuda()
    for t in (state, cstate):
        assert torch.equal(t[other], pool0[other])


def test_decode_bad_index_is_reported():
    b = Batch(32, lens=[2] * 4, C=64, packed=False, pool=4)
    b.slots[2] = 4
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    state, o = b.h0.clone(), b.blank()
    lap.la_gated_decode(b.x, b.r, b.g, b.slopes, state, 2, state_indices=torch.from_numpy(b.slots).cuda(), o=o,
                        dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == lap.DEV_ERR_BAD_INDEX and torch.isnan(o[4:6]).all() and torch.isfinite(o[:4].float()).all()


def test_decode_continues_a_scan():
    """A prompt by the scan, then its next tokens by decode from the pool: one longer scan."""
    b = Batch(33, lens=[260, 260], C=72, packed=False, pool=5)
    o, hf = b.fwd()
    pool = b.h0.clone()
    at = torch.cat([torch.arange(256), 260 + torch.arange(256)]).cuda()
    lap.la_gated_scan_fwd(b.x[at], b.r[at], b.g[at], b.slopes, h0=pool, h_final=pool, state_indices=b.idx, seq_len=256)
    tail = torch.cat([torch.arange(256, 260), 260 + torch.arange(256, 260)]).cuda()
    o2 = lap.la_gated_decode(b.x[tail], b.r[tail], b.g[tail], b.slopes, pool, 4, state_indices=b.idx)
    torch.testing.assert_close(o2, o[tail], rtol=2.0 ** -7, atol=1e-4)
    torch.testing.assert_close(pool[b.idx.long()], hf[b.idx.long()], rtol=1e-4, atol=1e-4)


def test_fixed_length_zero_keeps_the_states():
    """T == 0 through the C entry points: final states are the initial ones, gradients likewise."""
    lib = lap.load_library()
    h0, hf, dh0 = torch.randn(2, 70, device="cuda"), torch.empty(2, 70, device="cuda"), torch.empty(2, 70, device="cuda")
    slopes, dsl = torch.ones(70, device="cuda"), torch.full((70,), float("nan"), device="cuda")
    n = lap.la_gated_scan_workspace(2, 0, 2, 70, False, torch.bfloat16, True)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert lib.la_gated_scan_fwd(None, None, None, slopes.data_ptr(), h0.data_ptr(), None, None, None, hf.data_ptr(),
                                 70, 70, 70, 70, 2, 0, 2, 70, 2, 0, ws.data_ptr(), n, None, s) == 0
    assert lib.la_gated_scan_bwd(None, None, None, slopes.data_ptr(), None, None, None, h0.data_ptr(), None, None, None,
                                 None, None, dsl.data_ptr(), dh0.data_ptr(), *[70] * 8, 2, 0, 2, 70, 2, 0, ws.data_ptr(),
                                 n, None, s) == 0
    assert torch.equal(hf, h0) and torch.equal(dh0, h0) and torch.equal(dsl, torch.zeros(70, device="cuda"))
