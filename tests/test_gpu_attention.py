"""Softmax attention over whole prompts on the GPU (include/la_attention.h) against its plain 64-bit
form: lengths around the kernels' tiles, packed batches, grouped heads, strides, foreign rows,
gradients, and a layer of the operators together."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_reference import BF16, attend, attend_grad, causal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, bound, label, half=BF16):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    tol = bound + half * (np.abs(ref) + bound) + 1e-30
    worst = np.max(np.abs(got - ref) / tol) if ref.size else 0.0
    assert worst <= 1, f"{label}: {worst:.3g} of its bound"


def make(rng, tokens, counts, D, layout="dense", scale=1.0):
    """bf16 [tokens, n, D] for each n: dense, column ranges of one matrix, or heads first."""
    if layout == "fused":
        a = torch.from_numpy(rng.standard_normal((tokens, sum(counts) * D)).astype(np.float32) * np.float32(scale))
        return [t.unflatten(1, (-1, D)) for t in a.to(torch.bfloat16).cuda().split([n * D for n in counts], 1)]
    out = [torch.from_numpy(rng.standard_normal((tokens, n, D)).astype(np.float32) * np.float32(scale)).to(torch.bfloat16).cuda()
           for n in counts]
    return [t.permute(1, 0, 2).contiguous().permute(1, 0, 2) for t in out] if layout == "heads" else out


def check_forward(q, k, v, scale, bounds, o, lse, label=""):
    H, HK = q.shape[1], k.shape[1]
    Q, K, V = f64(q), f64(k), f64(v)
    for lo, hi in bounds:
        for h in range(H):
            hk = h // (H // HK)
            ro, rl, eo, el = attend(Q[lo:hi, h], K[lo:hi, hk], V[lo:hi, hk], causal(hi - lo, hi - lo), scale)
            near(o[lo:hi, h], ro, eo, f"{label} o rows {lo}..{hi} head {h}")
            near(lse[h, lo:hi], rl, el, f"{label} lse rows {lo}..{hi} head {h}", 2.0 ** -24)


def check_backward(q, k, v, scale, bounds, o, lse, do, grads, label=""):
    H, HK = q.shape[1], k.shape[1]
    G = H // HK
    Q, K, V, O, L, DO = (f64(t) for t in (q, k, v, o, lse, do))
    dq, dk, dv = grads
    for lo, hi in bounds:
        for hk in range(HK):
            sums = {"dk": [0, 0], "dv": [0, 0]}
            for h in range(hk * G, (hk + 1) * G):
                ref = attend_grad(Q[lo:hi, h], K[lo:hi, hk], V[lo:hi, hk], scale, O[lo:hi, h], L[h, lo:hi], DO[lo:hi, h])
                near(dq[lo:hi, h], *ref["dq"], f"{label} dq rows {lo}..{hi} head {h}")
                for n in sums:
                    sums[n] = [a + b for a, b in zip(sums[n], ref[n])]
            near(dk[lo:hi, hk], *sums["dk"], f"{label} dk rows {lo}..{hi} head {hk}")
            near(dv[lo:hi, hk], *sums["dv"], f"{label} dv rows {lo}..{hi} head {hk}")


LENGTHS = [1, 2, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 520]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", LENGTHS)
def test_fixed_lengths(T, D):
    rng = np.random.default_rng(T + D)
    for B, H, HK, layout in ((1, 1, 1, "dense"), (3, 4, 2, "fused"), (2, 5, 1, "heads")):
        q, k, v = make(rng, B * T, (H, HK, HK), D, layout)
        o, lse = lap.la_attn_prefill_fwd(q, k, v, D ** -0.5, seq_len=T)
        bounds = [(b * T, (b + 1) * T) for b in range(B)]
        check_forward(q, k, v, D ** -0.5, bounds, o, lse, layout)
        do, = make(rng, B * T, (H,), D, layout if layout != "fused" else "dense")
        grads = lap.la_attn_prefill_bwd(q, k, v, D ** -0.5, o, lse, do, seq_len=T)
        check_backward(q, k, v, D ** -0.5, bounds, o, lse, do, grads, layout)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H,HK", [
    ([1], 2, 2), ([0, 5, 0, 0, 130, 1, 0], 4, 1), ([300, 128, 7, 256, 64], 2, 2), ([1] * 40, 8, 2), ([0, 0], 1, 1),
    ([129, 127, 511], 6, 3), ([1025, 3], 2, 1), ([37] * 12 + [400], 3, 1)])
def test_packed(lens, H, HK, D):
    rng = np.random.default_rng(sum(lens) + D)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = int(cu[-1]) + 45  # rows behind the last sequence
    q, k, v = make(rng, tokens, (H, HK, HK), D, "fused")
    do, = make(rng, tokens, (H,), D)
    for t in (q, k, v, do):
        t[cu[-1]:] = float("nan")
    bounds = [(a, b) for a, b in zip(cu, cu[1:]) if b > a]
    dcu, err = torch.from_numpy(cu).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((tokens, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, tokens), 7.0, device="cuda")
    lap.la_attn_prefill_fwd(q, k, v, 0.2, cu_seqlens=dcu, o=o, lse=lse, dev_error=err)
    check_forward(q, k, v, 0.2, bounds, o, lse)
    assert (o[cu[-1]:] == 7).all() and (lse[:, cu[-1]:] == 7).all() and err.item() == 0
    o2, lse2 = o.clone(), lse.clone()
    o2[cu[-1]:], lse2[:, cu[-1]:] = float("nan"), float("nan")
    grads = [torch.full((tokens, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (H, HK, HK)]
    lap.la_attn_prefill_bwd(q, k, v, 0.2, o2, lse2, do, cu_seqlens=dcu, dq=grads[0], dk=grads[1], dv=grads[2], dev_error=err)
    check_backward(q, k, v, 0.2, bounds, o, lse, do, grads)
    assert all((g[cu[-1]:] == 7).all() for g in grads) and err.item() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_a_sequence_of_non_finite_values_reaches_no_other(D):
    rng = np.random.default_rng(5)
    lens = [100, 60, 200]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    q, k, v = make(rng, 360, (2, 1, 1), D)
    do, = make(rng, 360, (2,), D)
    dcu = torch.from_numpy(cu).cuda()
    o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.3, cu_seqlens=dcu)
    grads = lap.la_attn_prefill_bwd(q, k, v, 0.3, o, lse, do, cu_seqlens=dcu)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t in (q, k, v, do):
            t[100:160] = bad
        o2, lse2 = lap.la_attn_prefill_fwd(q, k, v, 0.3, cu_seqlens=dcu)
        g2 = lap.la_attn_prefill_bwd(q, k, v, 0.3, o2, lse2, do, cu_seqlens=dcu)
        for a, b in ((o, o2), (lse.T, lse2.T), *zip(grads, g2)):
            assert torch.equal(a[:100], b[:100]) and torch.equal(a[160:], b[160:])


@pytest.mark.parametrize("D", [64, 128])
def test_large_scores_and_scales(D):
    rng = np.random.default_rng(6)
    for scale, size in ((1.0, 4.0), (-0.5, 1.0), (0.0, 1.0), (30.0, 1.0), (1e-3, 1.0)):
        q, k, v = make(rng, 300, (2, 1, 1), D, scale=size)
        o, lse = lap.la_attn_prefill_fwd(q, k, v, scale, seq_len=300)
        check_forward(q, k, v, scale, [(0, 300)], o, lse, f"scale {scale}")
        do, = make(rng, 300, (2,), D)
        grads = lap.la_attn_prefill_bwd(q, k, v, scale, o, lse, do, seq_len=300)
        check_backward(q, k, v, scale, [(0, 300)], o, lse, do, grads, f"scale {scale}")
    # scores that rise along the keys, so that the running maximum moves in every tile, and that fall
    for sign in (1.0, -1.0):
        q, k, v = make(rng, 700, (1, 1, 1), D)
        q[:] = 1.0
        k[:] = (sign * torch.arange(700, device="cuda") / 16)[:, None, None]
        o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.05, seq_len=700)
        check_forward(q, k, v, 0.05, [(0, 700)], o, lse, f"rising {sign}")


@pytest.mark.parametrize("D", [64, 128])
def test_long_sequence_against_single_rows(D):
    """A long sequence: chosen rows against the definition, in one head of a group."""
    rng = np.random.default_rng(7)
    T, H, HK = 9001, 4, 2
    q, k, v = make(rng, T, (H, HK, HK), D, "fused")
    o, lse = lap.la_attn_prefill_fwd(q, k, v, D ** -0.5, seq_len=T)
    K, V = f64(k), f64(v)
    for row in (0, 4095, 4096, 8191, 8500, 9000):
        for h in range(H):
            ro, rl, eo, el = attend(f64(q[row:row + 1, h]), K[:row + 1, h // 2], V[:row + 1, h // 2], np.ones((1, row + 1), bool), D ** -0.5)
            near(o[row:row + 1, h], ro, eo, f"row {row} head {h}")
            near(lse[h, row:row + 1], rl, el, f"lse row {row} head {h}", 2.0 ** -24)
    again = lap.la_attn_prefill_fwd(q, k, v, D ** -0.5, seq_len=T)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    do, = make(rng, T, (H,), D)
    g = lap.la_attn_prefill_bwd(q, k, v, D ** -0.5, o, lse, do, seq_len=T)
    g2 = lap.la_attn_prefill_bwd(q, k, v, D ** -0.5, o, lse, do, seq_len=T)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))
    # the last 700 keys' gradients and the first rows' depend on those rows alone
    sub = slice(T - 700, T)
    O, L, DO, Q = f64(o), f64(lse), f64(do), f64(q)
    for hk in range(HK):
        dk = dv = edk = edv = 0
        for h in (2 * hk, 2 * hk + 1):
            ref = attend_grad(Q[sub, h], K[sub, hk], V[sub, hk], D ** -0.5, O[sub, h], L[h, sub], DO[sub, h])
            dk, edk, dv, edv = dk + ref["dk"][0], edk + ref["dk"][1], dv + ref["dv"][0], edv + ref["dv"][1]
        near(g[1][sub, hk], dk, edk, "dk")
        near(g[2][sub, hk], dv, edv, "dv")


def test_bad_bounds_skip_their_sequence():
    rng = np.random.default_rng(8)
    q, k, v = make(rng, 300, (2, 2, 2), 64)
    do, = make(rng, 300, (2,), 64)
    for cu in ([0, 100, 90, 300], [-1, 100, 200, 300], [0, 100, 200, 301]):
        dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        good = [(a, b) for a, b in zip(cu, cu[1:]) if 0 <= a <= b <= 300]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full((300, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((2, 300), device="cuda")
        lap.la_attn_prefill_fwd(q, k, v, 0.1, cu_seqlens=dcu, o=o, lse=lse, dev_error=err)
        assert err.item() == lap.DEV_ERR_BAD_SEQLENS
        if cu[2] != 90:  # there two sequences overlap
            check_forward(q, k, v, 0.1, good, o, lse)
            seen = np.zeros(300, bool)
            for a, b in good:
                seen[a:b] = True
            assert (o[torch.from_numpy(~seen).cuda()] == 7).all()
            err.zero_()
            grads = lap.la_attn_prefill_bwd(q, k, v, 0.1, o, lse, do, cu_seqlens=dcu, dev_error=err)
            check_backward(q, k, v, 0.1, good, o, lse, do, grads)
            assert err.item() == lap.DEV_ERR_BAD_SEQLENS


def test_rows_past_32_bit_offsets():
    T, ld = 70000, 65536
    gen = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")  # 9 GB
    wide[:, -192:] = torch.randn((T, 192), generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (1, 64)) for t in wide[:, -192:].split(64, 1))
    cu = torch.tensor([0, 100, T - 300, T], dtype=torch.int32, device="cuda")
    o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.125, cu_seqlens=cu, o=wide[:, :64].unflatten(1, (1, 64)))
    dense = [t.contiguous() for t in (q, k, v)]
    o2, lse2 = lap.la_attn_prefill_fwd(*dense, 0.125, cu_seqlens=cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_forward(q, k, v, 0.125, [(T - 300, T)], o, lse)
    outs = [wide[:, 128 + 64 * i:192 + 64 * i].unflatten(1, (1, 64)) for i in range(3)]
    g = lap.la_attn_prefill_bwd(q, k, v, 0.125, o, lse, v, cu_seqlens=cu, dq=outs[0], dk=outs[1], dv=outs[2])
    g2 = lap.la_attn_prefill_bwd(*dense, 0.125, o2, lse2, dense[2], cu_seqlens=cu)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))


def test_captured_and_replayed_with_new_values_and_streams():
    rng = np.random.default_rng(9)
    T, H, HK, D = 333, 4, 2, 128
    q, k, v = make(rng, 2 * T, (H, HK, HK), D, "fused")
    do, = make(rng, 2 * T, (H,), D)

    def step(stream=None, ws=None):
        o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.1, seq_len=T, stream=stream)
        return o, lse, *lap.la_attn_prefill_bwd(q, k, v, 0.1, o, lse, do, seq_len=T, stream=stream, workspace=ws)
    want = step()
    torch.cuda.synchronize()
    ws = torch.full((lap.la_attn_prefill_bwd_workspace(2, T, H, HK, D),), 255, dtype=torch.uint8, device="cuda")  # NaN
    side = torch.cuda.Stream()
    got = step(side, ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):  # two graphs on one workspace, replayed in turn
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got = step(ws=ws)
    for g in graphs + graphs:
        q.copy_(torch.randn_like(q.float()))
        g.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_a_layer_of_the_operators_together():
    """Norm and rotation, prompt attention, and both gradients chained, against autograd in 64 bits."""
    rng = np.random.default_rng(10)
    lens, H, HK, D = [70, 1, 200], 4, 2, 64
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = int(cu[-1])
    q, k, v = make(rng, n, (H, HK, HK), D, "fused")
    do, = make(rng, n, (H,), D)
    wq, wk = (torch.rand(D, device="cuda") + 0.5 for _ in range(2))
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).cuda()
    freq = (10000.0 ** (-torch.arange(0, D, 2) / D)).cuda()
    dcu = torch.from_numpy(cu).cuda()
    qr, kr = lap.la_qk_norm_rope_fwd(q, k, wq, wk, 1e-6, pos, freq)
    o, lse = lap.la_attn_prefill_fwd(qr, kr, v, D ** -0.5, cu_seqlens=dcu)
    dqr, dkr, dv = lap.la_attn_prefill_bwd(qr, kr, v, D ** -0.5, o, lse, do, cu_seqlens=dcu)
    dq, dk, dwq, dwk = lap.la_qk_norm_rope_bwd(q, k, wq, wk, 1e-6, dqr, dkr, pos, freq)
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v, wq, wk)]
    Q, K, V, WQ, WK = leaves
    a = pos.double().cpu()[:, None, None] * freq.double().cpu()

    def rot(x, w):
        y = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        lo, hi = y.chunk(2, -1)
        return torch.cat([lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()], -1)
    qq, kk = rot(Q, WQ), rot(K, WK)
    outs = []
    for lo, hi in zip(cu, cu[1:]):
        z = torch.einsum("thgd,nhd->hgtn", qq[lo:hi].unflatten(1, (HK, -1)), kk[lo:hi]) * D ** -0.5
        z = z.masked_fill(~torch.tril(torch.ones(z.shape[-2:], dtype=torch.bool)), -torch.inf)
        outs.append(torch.einsum("hgtn,nhd->thgd", z.softmax(-1), V[lo:hi]).flatten(1, 2))
    ref = torch.cat(outs)
    (ref * do.double().cpu()).sum().backward()
    # five roundings to BF16 on the way to a gradient (rotated rows, P, dS, o in delta, the outputs),
    # each 2^-8 at most and spread evenly, so their RMS is 2^-8 / sqrt(3): sqrt(5 / 3) 2^-8 of the
    # terms; terms cancel to half their size at most times in these sums
    for got, want in ((o, ref), *zip((dq, dk, dv, dwq, dwk), (t.grad for t in leaves))):
        want = want.detach()
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= 2 * (5 / 3) ** 0.5 * 2.0 ** -8, err


def test_wrong_arguments_are_refused():
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for over, kind in ((dict(seq_len=None), ValueError), (dict(seq_len=3), ValueError), (dict(seq_len=0), ValueError),
                       (dict(k=q[:3]), ValueError), (dict(v=q[:, :1]), ValueError), (dict(q=q[:, :, :32]), ValueError),
                       (dict(o=q.float()), TypeError), (dict(lse=torch.zeros((2, 3), device="cuda")), ValueError),
                       (dict(cu_seqlens=torch.zeros(2, device="cuda")), TypeError), (dict(k=q.cpu()), ValueError),
                       (dict(q=q[:, :1].expand(4, 2, 64)), lap.LaError), (dict(o=q), lap.LaError),
                       (dict(q=torch.zeros((4, 2, 68), dtype=torch.bfloat16, device="cuda")[:, :, 4:]), lap.LaError)):
        a = dict(q=q, k=q, v=q, scale=1.0, seq_len=4)
        with pytest.raises(kind):
            lap.la_attn_prefill_fwd(**{**a, **over})


@pytest.mark.parametrize("D", [64, 128])
def test_a_value_that_is_not_finite_reaches_only_rows_that_see_it(D):
    """Masked places hold it too: rows before it, in its own tile of keys, keep their bits."""
    rng = np.random.default_rng(12)
    q, k, v = make(rng, 400, (4, 2, 2), D, "fused")
    o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.2, seq_len=400)
    for row in (0, 1, 63, 64, 127, 128, 200, 255, 300, 399):
        for bad in (float("nan"), float("inf"), -float("inf")):
            keep = v[row].clone()
            v[row, 1, D // 2 + 3] = bad
            o2, lse2 = lap.la_attn_prefill_fwd(q, k, v, 0.2, seq_len=400)
            v[row] = keep
            assert torch.equal(lse, lse2) and torch.equal(o[:row], o2[:row]) and torch.equal(o[:, :2], o2[:, :2])
            cols = [c for c in range(D) if c != D // 2 + 3]
            # other columns: the row's own values count in full, except that what is not finite is apart
            assert torch.equal(o[:, 2:, cols], o2[:, 2:, cols])
            assert not torch.isfinite(o2[row:, 2:, D // 2 + 3]).any()
        keepk, keepq = k[row].clone(), q[row].clone()
        k[row], q[row] = float("nan"), float("nan")
        o2, lse2 = lap.la_attn_prefill_fwd(q, k, v, 0.2, seq_len=400)
        k[row], q[row] = keepk, keepq
        assert torch.equal(o[:row], o2[:row]) and torch.equal(lse[:, :row], lse2[:, :row])
        assert torch.isnan(o2[row:]).all() and torch.isnan(lse2[:, row:]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1e-38, -1e-33, 1e-12])
def test_tiny_scales(scale, D):
    """Scores that are all but equal: lse stands far beyond them, in units of the scale."""
    rng = np.random.default_rng(41)
    q, k, v = make(rng, 200, (4, 2, 2), D)
    o, lse = lap.la_attn_prefill_fwd(q, k, v, scale, seq_len=200)
    check_forward(q, k, v, scale, [(0, 200)], o, lse)
    do, = make(rng, 200, (4,), D)
    check_backward(q, k, v, scale, [(0, 200)], o, lse, do, lap.la_attn_prefill_bwd(q, k, v, scale, o, lse, do, seq_len=200))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,HK", [(8, 1), (14, 2), (5, 1), (40, 1), (6, 6)])
def test_groups_of_heads_shared_out(H, HK, D):
    """Few key/value heads and tiles: a group's heads are summed in parts, on a workspace of NaN."""
    rng = np.random.default_rng(13)
    lens = [300, 0, 129, 5]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = int(cu[-1]) + 30
    q, k, v = make(rng, tokens, (H, HK, HK), D, "fused")
    do, = make(rng, tokens, (H,), D)
    dcu = torch.from_numpy(cu).cuda()
    o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.15, cu_seqlens=dcu)
    ws = torch.full((lap.la_attn_prefill_bwd_workspace(1, tokens, H, HK, D),), 255, dtype=torch.uint8, device="cuda")
    grads = [torch.full((tokens, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (H, HK, HK)]
    lap.la_attn_prefill_bwd(q, k, v, 0.15, o, lse, do, cu_seqlens=dcu, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
    check_backward(q, k, v, 0.15, [(a, b) for a, b in zip(cu, cu[1:]) if b > a], o, lse, do, grads)
    assert all((g[cu[-1]:] == 7).all() for g in grads)
    if H > HK:
        assert ws.numel() > 4 * H * tokens * 2


def test_calls_at_once_on_several_streams():
    """Whole layers on five streams at a time give the bits that they give one after the other."""
    rng = np.random.default_rng(61)
    jobs = []
    for D, H, HK, lens in ((64, 8, 1, [300, 0, 1]), (128, 6, 2, [129, 700]), (64, 4, 4, [257]), (128, 10, 1, [5, 64, 500]),
                           (64, 2, 1, [1500]), (128, 16, 4, [100, 128, 256]), (64, 6, 3, [90, 91])):
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        q, do, k, v = make(rng, sum(lens), (H, H, HK, HK), D)
        per = -(-max(lens) // 16)
        kc, vc = make(rng, len(lens) * per * 16, (HK, HK), D)
        kc, vc = kc.view(-1, 16, HK, D), vc.view(-1, 16, HK, D)
        table = torch.from_numpy(rng.permutation(len(lens) * per).reshape(len(lens), per).astype(np.int32)).cuda()
        held, pos = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.arange(sum(lens), dtype=torch.int32, device="cuda")
        freq, w, draft = 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D), torch.ones(D, device="cuda"), make(rng, 3 * len(lens), (H, HK, HK), D)

        def layer(q=q, k=k, v=v, do=do, cu=cu, D=D, w=w, pos=pos, freq=freq, draft=draft, kc=kc, vc=vc, held=held, table=table):
            qr, kr = lap.la_qk_norm_rope_fwd(q, k, w, w, 1e-6, pos, freq)
            o, lse = lap.la_attn_prefill_fwd(qr, kr, v, D ** -0.5, cu_seqlens=cu)
            g = lap.la_attn_prefill_bwd(qr, kr, v, D ** -0.5, o, lse, do, cu_seqlens=cu)
            back = lap.la_qk_norm_rope_bwd(q, k, w, w, 1e-6, g[0], g[1], pos, freq)
            return qr, kr, o, lse, *g, *back, lap.la_attn_verify(*draft, D ** -0.5, kc, vc, held, 3, page_table=table)

        jobs.append(layer)
    ref = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    for turn in range(4):
        out = []
        for i, job in enumerate(jobs):
            with torch.cuda.stream(streams[(i + turn) % 5]):
                out.append(job())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(ref, out) for a, b in zip(x, y))
