"""The norm and rotation of queries and keys and the softmax attention without a GPU: refusals of the
C entry points and of the binding, workspace sizes, and the 64-bit reference's gradients against
differences."""
import ctypes

import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_reference import attend, attend_grad, causal, norm_rope, norm_rope_grad

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
BUF = [(i + 1) << 42 for i in range(24)]  # fake buffers, never dereferenced
(Q, K, V, WQ, WK, POS, FREQ, O, KO, DQ, DK, DV, DWQ, DWK, WS, ERR, CU, LSE, DO, KC, VC, LENS, TAB, MASK) = BUF
ACC, PATH = 25 << 42, 26 << 42


def rope(**over):
    a = dict(q=Q, k=K, wq=WQ, wk=WK, eps=1e-6, pos=POS, freq=FREQ, qo=O, ko=KO, ldq=256, hsq=64, ldk=128, hsk=64,
             ldqo=256, hsqo=64, ldko=128, hsko=64, tokens=10, H=4, HK=2, D=64, R=64, inter=0, dt=0, stream=None)
    a.update(over)
    return lap.load_library().la_qk_norm_rope_fwd(*a.values())


def rope_back(**over):
    a = dict(q=Q, k=K, wq=WQ, wk=WK, eps=1e-6, pos=POS, freq=FREQ, gq=O, gk=KO, dq=DQ, dk=DK, dwq=DWQ, dwk=DWK, ldq=256,
             hsq=64, ldk=128, hsk=64, ldgq=256, hsgq=64, ldgk=128, hsgk=64, lddq=256, hsdq=64, lddk=128, hsdk=64,
             tokens=10, H=4, HK=2, D=64, R=64, inter=0, dt=0, ws=WS, wsb=1 << 30, stream=None)
    a.update(over)
    return lap.load_library().la_qk_norm_rope_bwd(*a.values())


def attn(**over):
    a = dict(q=Q, k=K, v=V, scale=0.1, cu=None, o=O, lse=LSE, ldq=256, hsq=64, ldk=128, hsk=64, ldv=128, hsv=64, ldo=256,
             hso=64, B=2, T=100, N=2, H=4, HK=2, D=64, err=None, stream=None)
    a.update(over)
    return lap.load_library().la_attn_prefill_fwd(*a.values())


def attn_back(**over):
    a = dict(q=Q, k=K, v=V, scale=0.1, o=O, lse=LSE, do=DO, cu=None, dq=DQ, dk=DK, dv=DV, ldq=256, hsq=64, ldk=128, hsk=64,
             ldv=128, hsv=64, ldo=256, hso=64, lddo=256, hsdo=64, lddq=256, hsdq=64, lddk=128, hsdk=64, lddv=128, hsdv=64,
             B=2, T=100, N=2, H=4, HK=2, D=64, ws=WS, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lap.load_library().la_attn_prefill_bwd(*a.values())


def verify(**over):
    a = dict(q=Q, k=K, v=V, scale=0.1, kc=KC, vc=VC, lens=LENS, tab=TAB, mask=None, o=O, ldq=256, hsq=64, ldk=128, hsk=64,
             ldv=128, hsv=64, ldo=256, hso=64, kp=2048, kt=128, kh=64, vp=2048, vt=128, vh=64, ldt=8, B=3, T=4, H=4, HK=2,
             D=64, pages=24, size=16, width=8, ws=WS, wsb=1 << 40, err=None, stream=None)
    a.update(over)
    return lap.load_library().la_attn_verify(*a.values())


def commit(**over):
    a = dict(k=K, v=V, kc=KC, vc=VC, lens=LENS, cu=None, acc=ACC, path=PATH, tab=TAB, ldk=128, hsk=64, ldv=128, hsv=64,
             kp=2048, kt=128, kh=64, vp=2048, vt=128, vh=64, ldt=8, B=3, T=4, HK=2, D=64, pages=24, size=16, width=8,
             err=None, stream=None)
    a.update(over)
    return lap.load_library().la_attn_commit(*a.values())


SIZES = [(dict(D=96), UNSUPPORTED), (dict(H=0), INVALID), (dict(HK=-1), INVALID)]
ROPE = SIZES + [
    (dict(tokens=-1), INVALID), (dict(R=3), INVALID), (dict(R=66), INVALID), (dict(R=-2), INVALID), (dict(dt=2), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(q=None), INVALID), (dict(dk=None, ko=None), INVALID), (dict(ldq=255), INVALID), (dict(hsq=63), INVALID),
    (dict(hsk=0), INVALID), (dict(ldk=1 << 50), INVALID), (dict(q=Q + 1), INVALID), (dict(dt=1, k=K + 2), INVALID),
    (dict(pos=POS + 2), INVALID), (dict(wk=WK + 1), INVALID), (dict(tokens=2 ** 31 - 1), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", ROPE)
def test_norm_rope_refusals(over, status):
    assert rope(**{k: v for k, v in over.items() if k != "dk"}) == status
    assert lap.load_library().la_last_error() != b""


@pytest.mark.parametrize("over,status", [(o, s) for o, s in ROPE if "ko" not in o] + [
    (dict(gq=None), INVALID), (dict(dk=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=16), INVALID),
    (dict(ws=WS + 8), INVALID), (dict(dwq=DWQ + 2), INVALID), (dict(lddk=64), INVALID)])
def test_norm_rope_gradient_refusals(over, status):
    assert rope_back(**over) == status
    assert lap.load_library().la_last_error() != b""


@pytest.mark.parametrize("fn,over", [
    (rope, dict(qo=K)), (rope, dict(qo=Q + 2)), (rope, dict(qo=Q, ldqo=512)), (rope, dict(ko=O + 64)),
    (rope, dict(qo=POS)), (rope, dict(ko=WQ)), (rope, dict(ko=FREQ)), (rope_back, dict(dq=Q)), (rope_back, dict(dq=KO)),
    (rope_back, dict(dwq=DQ)), (rope_back, dict(dwq=DWK)), (rope_back, dict(ws=DK)), (rope_back, dict(dk=POS)),
    (attn, dict(o=Q)), (attn, dict(lse=O)), (attn, dict(err=LSE)), (attn, dict(o=V + 512)),
    (attn, dict(o=CU, cu=CU, B=1, T=200)), (attn_back, dict(dq=Q)), (attn_back, dict(dk=DV)), (attn_back, dict(dv=DO)),
    (attn_back, dict(ws=LSE)), (attn_back, dict(dq=O)), (verify, dict(o=Q)), (verify, dict(o=KC + 4096)),
    (verify, dict(o=LENS)), (verify, dict(ws=VC)), (verify, dict(err=MASK, mask=MASK)), (commit, dict(kc=VC)),
    (commit, dict(kc=K)), (commit, dict(vc=TAB)), (commit, dict(vc=PATH)), (commit, dict(err=KC + 8)),
    (commit, dict(vc=KC + 128, kp=4096, vp=4096, kt=256, vt=192))])
def test_overlaps_are_refused(fn, over):
    assert fn(**over) == INVALID
    assert b"overlaps" in lap.load_library().la_last_error()


PROMPT = SIZES + [
    (dict(H=3), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(B=-1, N=-1), INVALID), (dict(N=3), INVALID),
    (dict(cu=CU), INVALID), (dict(cu=CU + 2, B=1), INVALID), (dict(T=1 << 30), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(o=None), INVALID), (dict(v=V + 8), INVALID), (dict(ldq=260), INVALID), (dict(hsk=68, ldk=200), INVALID),
    (dict(ldk=64), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(err=ERR + 1), INVALID), (dict(lse=LSE + 2), INVALID)]


@pytest.mark.parametrize("over,status", PROMPT)
def test_prompt_refusals(over, status):
    assert attn(**over) == status
    assert lap.load_library().la_last_error() != b""


@pytest.mark.parametrize("over,status", PROMPT + [
    (dict(lse=None), INVALID), (dict(do=None), INVALID), (dict(dk=None), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=100), INVALID), (dict(lddv=100), INVALID)])
def test_prompt_gradient_refusals(over, status):
    assert attn_back(**over) == status
    assert lap.load_library().la_last_error() != b""


CACHE = [
    (dict(D=32), UNSUPPORTED), (dict(HK=0), INVALID), (dict(B=-1), INVALID), (dict(pages=0), INVALID), (dict(size=0), INVALID),
    (dict(size=24), UNSUPPORTED), (dict(width=0), INVALID), (dict(ldt=7), INVALID), (dict(width=1 << 28, ldt=1 << 28), UNSUPPORTED),
    (dict(tab=None, pages=2), INVALID), (dict(lens=None), INVALID), (dict(lens=LENS + 2), INVALID), (dict(tab=TAB + 1), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(kc=KC + 8), INVALID), (dict(kt=120), INVALID), (dict(kt=132), INVALID),
    (dict(vp=2000), INVALID), (dict(vh=32), INVALID), (dict(kp=0), INVALID), (dict(k=None), INVALID), (dict(ldv=60), INVALID),
    (dict(err=ERR + 2), INVALID), (dict(T=1 << 30), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", CACHE + [
    (dict(H=3), UNSUPPORTED), (dict(H=258 * 2), UNSUPPORTED), (dict(T=0), INVALID), (dict(mask=MASK + 4), INVALID),
    (dict(mask=MASK, T=65), UNSUPPORTED), (dict(ws=None), INVALID), (dict(wsb=0), INVALID), (dict(q=Q + 4), INVALID),
    (dict(o=None), INVALID), (dict(scale=float("-inf")), INVALID)])
def test_verify_refusals(over, status):
    assert verify(**over) == status
    assert lap.load_library().la_last_error() != b""


@pytest.mark.parametrize("over,status", CACHE + [
    (dict(cu=CU), INVALID), (dict(cu=CU, path=None), INVALID), (dict(acc=ACC + 2), INVALID), (dict(path=PATH + 2), INVALID),
    (dict(T=-1), INVALID)])
def test_commit_refusals(over, status):
    assert commit(**over) == status
    assert lap.load_library().la_last_error() != b""


def test_nothing_to_do():
    assert rope(tokens=0, q=None) == OK and attn(B=0, N=0, q=None) == OK and attn_back(B=0, N=0, ws=None) == OK
    assert attn(cu=CU, B=1, T=0, N=3) == OK and verify(B=0, q=None) == OK and commit(B=0, k=None) == OK
    assert commit(T=0) == OK and rope_back(tokens=0, dwq=None, dwk=None, ws=None, wsb=0) == OK


def test_no_tokens_have_no_positions():
    """An empty tensor's pointer is null."""
    assert rope(tokens=0, pos=None) == rope_back(tokens=0, pos=None, dwq=None, dwk=None) == OK
    assert rope(tokens=0, freq=None) == rope(tokens=1, pos=None) == rope_back(tokens=1, pos=None) == INVALID


def test_allowed_layouts_pass_every_host_check():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    # past every host check: the device query fails
    assert rope() == rope_back() == attn() == attn_back() == verify() == commit() == CUDA
    assert rope(qo=Q, ko=K) == rope_back(dq=O, dk=KO) == CUDA
    # q, k, v and their gradients as column ranges of one matrix [tokens, (4 + 2 + 2) * 64]
    ld = dict(ldq=512, ldk=512, ldv=512)
    assert attn(k=Q + 512, v=Q + 768, **ld) == CUDA
    assert attn_back(dk=DQ + 512, dv=DQ + 768, lddq=512, lddk=512, lddv=512) == CUDA
    assert rope(k=Q + 512, qo=Q, ko=Q + 512, ldq=512, ldk=512, ldqo=512, ldko=512) == CUDA
    # heads first
    assert attn(ldq=64, hsq=6400 * 2, ldk=64, hsk=12800, ldo=64, hso=12800) == CUDA
    assert rope(ldq=64, hsq=640, ldqo=64, hsqo=640) == CUDA
    # keys and values in the same pages: token by token, and one after the other
    assert commit(vc=KC + 256, kt=256, vt=256, kp=4096, vp=4096) == CUDA
    assert commit(vc=KC + 4096, kp=4096, vp=4096) == CUDA
    assert commit(kt=64, kh=1024, vt=64, vh=1024) == CUDA  # head-major pages
    # one range per request, of any size
    assert verify(tab=None, pages=3, size=37, kp=37 * 128, vp=37 * 128) == CUDA
    assert verify(mask=MASK, T=64) == verify(T=1, B=1, ldt=0) == CUDA
    assert rope(R=0, pos=None, freq=None) == rope(wq=None, wk=None) == CUDA


def test_drafted_tokens_whose_tiles_pass_32_bits_are_refused():
    big = dict(B=1, tab=None, pages=1, H=128, HK=1, ldq=128 * 64, ldo=128 * 64, ldk=64, ldv=64, kt=64, vt=64, kp=1024, vp=1024)
    assert verify(T=(1 << 18) + 1, **big) == UNSUPPORTED
    assert lap.la_attn_verify_workspace(1, 1 << 18, 128, 1, 64) > 0
    with pytest.raises(lap.LaError):
        lap.la_attn_verify_workspace(1, (1 << 18) + 1, 128, 1, 64)


def test_workspace_queries():
    lib = lap.load_library()
    assert lap.la_qk_norm_rope_bwd_workspace(0, 4, 2, 64) == 0 and lap.la_qk_norm_rope_bwd_workspace(100, 4, 2, 64) % 256 == 0
    assert lap.la_attn_prefill_bwd_workspace(2, 100, 4, 2, 64) >= 3200 and lap.la_attn_verify_workspace(3, 4, 4, 2, 64) % 256 == 0
    for bad in ((lap.la_qk_norm_rope_bwd_workspace, (1, 4, 2, 100)), (lap.la_attn_prefill_bwd_workspace, (1, -1, 4, 2, 64)), (lap.la_attn_prefill_bwd_workspace, (1, 1, 4, 3, 64)),
                (lap.la_attn_verify_workspace, (1, 0, 4, 2, 64)), (lap.la_attn_verify_workspace, (1, 1, 4, 3, 64))):
        with pytest.raises(lap.LaError):
            bad[0](*bad[1])
    assert lib.la_attn_verify_workspace(1, 1, 4, 2, 64, None) == INVALID
    assert lib.la_attn_prefill_bwd_workspace(1, 1, 4, 2, 64, None) == INVALID
    assert lib.la_qk_norm_rope_bwd_workspace(1, 4, 2, 64, None) == INVALID


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros((8, 2, 64), dtype=torch.bfloat16)
    w, lens, cache = torch.zeros(64), torch.zeros(8, dtype=torch.int32), torch.zeros((8, 16, 2, 64), dtype=torch.bfloat16)
    calls = (lambda t: lap.la_qk_norm_rope_fwd(t, t, w, w, 1e-6), lambda t: lap.la_qk_norm_rope_bwd(t, t, w, w, 1e-6, t, t),
             lambda t: lap.la_attn_prefill_fwd(t, t, t, 1.0, seq_len=8), lambda t: lap.la_attn_commit(t, t, cache, cache, lens, T=1),
             lambda t: lap.la_attn_prefill_bwd(t, t, t, 1.0, t, w, t, seq_len=8),
             lambda t: lap.la_attn_verify(t, t, t, 1.0, cache, cache, lens, 1))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(x)
        with pytest.raises(ValueError, match="3 dims"):
            call(x[0])
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call([0])
    for call in calls[2:]:
        with pytest.raises(TypeError, match="bfloat16"):
            call(x.half())


def test_reference_norm_rope_gradients_against_differences():
    rng = np.random.default_rng(2)
    for interleaved, R in ((False, 4), (True, 6), (False, 0)):
        x, dout = rng.standard_normal((2, 3, 2, 6))
        w, pos, freq = rng.standard_normal(6), np.array([0, 3, 1000]), rng.random(R // 2)
        ref = norm_rope_grad(x, w, 1e-2, dout, pos, freq, interleaved)

        def loss(x, w):
            return (norm_rope(x, w, 1e-2, pos, freq, interleaved)[0] * dout).sum()
        for i in np.ndindex(*x.shape):
            d = np.zeros_like(x)
            d[i] = 1e-5
            assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-5 - ref["dx"][0][i]) <= 1e-8
        for i in range(6):
            d = np.zeros(6)
            d[i] = 1e-5
            assert abs((loss(x, w + d) - loss(x, w - d)) / 2e-5 - ref["dw"][0][i]) <= 1e-8


def test_reference_attention_gradients_against_differences():
    rng = np.random.default_rng(3)
    q, k, v, do = rng.standard_normal((4, 5, 3))
    args = dict(q=q, k=k, v=v)

    def forward(**over):
        a = {**args, **over}
        return attend(a["q"], a["k"], a["v"], causal(5, 5), 0.7)
    o, lse, _, _ = forward()
    ref = attend_grad(q, k, v, 0.7, o, lse, do)
    for name in args:
        for i in np.ndindex(5, 3):
            d = np.zeros((5, 3))
            d[i] = 1e-5
            diff = ((forward(**{name: args[name] + d})[0] - forward(**{name: args[name] - d})[0]) * do).sum() / 2e-5
            assert abs(diff - ref["d" + name][0][i]) <= 1e-8


def test_reference_special_cases():
    v = np.arange(12.0).reshape(4, 3)
    o, lse, _, _ = attend(np.zeros((4, 3)), np.ones((4, 3)), v, causal(4, 4), 1.0)
    np.testing.assert_allclose(o, np.cumsum(v, 0) / np.arange(1, 5)[:, None], rtol=1e-14)
    np.testing.assert_allclose(lse, np.log(np.arange(1, 5)), rtol=1e-14)
    o, lse, _, _ = attend(np.ones((2, 3)), np.ones((4, 3)), v, np.zeros((2, 4), dtype=bool), 1.0)
    assert not o.any() and np.all(lse == -np.inf)
    # a whole turn, and turns of neighbours and halves by a right angle
    x = np.array([[[3.0, 4.0]]])
    for interleaved in (False, True):
        y, _ = norm_rope(x, None, 0.0, [1], [np.pi / 2], interleaved)
        np.testing.assert_allclose(y[0, 0], np.array([-4.0, 3.0]) / np.sqrt(12.5), atol=1e-14)
