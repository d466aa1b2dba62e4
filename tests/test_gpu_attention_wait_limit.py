"""The timeout exit of the attention kernels, without hanging anything: a build with a 100 ns limit,
which ordinary waits for tiles and products exceed.  The calls return LA_OK, the error word carries the
timeout bit, the context stays usable, and the normal library gives the same bits as before."""
import ctypes

import pytest

import linear_attention_prefill_chunkwise_gb300 as lap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def short():
    from linear_attention_prefill_chunkwise_gb300 import build as b
    lib, real = ctypes.CDLL(b.build(wait_limit_ns=100, part="attention")), lap.load_library()
    for name in ("la_attn_prefill_fwd", "la_attn_prefill_bwd", "la_attn_verify"):
        getattr(lib, name).argtypes = getattr(real, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    return lib


def timed_out(call):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert call(err.data_ptr()) == 0
    torch.cuda.synchronize()  # raises if the kernel had faulted and the context were lost
    assert int(err) & lap.DEV_ERR_TIMEOUT, f"error word {int(err)}: the short limit never tripped"


@pytest.mark.parametrize("D", [64, 128])
def test_prompt(short, D):
    B, T, H, HK = 2, 4096, 8, 2
    q, do = (torch.randn(B * T, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(B * T, HK, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    want = lap.la_attn_prefill_fwd(q, k, v, 0.1, seq_len=T)
    grads = lap.la_attn_prefill_bwd(q, k, v, 0.1, *want, do, seq_len=T)
    o, lse = torch.empty_like(q), torch.empty_like(want[1])
    s = torch.cuda.current_stream().cuda_stream
    lq, lk = (H * D, D), (HK * D, D)
    timed_out(lambda err: short.la_attn_prefill_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), 0.1, None, o.data_ptr(),
                                                    lse.data_ptr(), *lq, *lk, *lk, *lq, B, T, B, H, HK, D, err, s))
    n = lap.la_attn_prefill_bwd_workspace(B, T, H, HK, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    timed_out(lambda err: short.la_attn_prefill_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), 0.1, want[0].data_ptr(), want[1].data_ptr(), do.data_ptr(), None,
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *lq, *lk, *lk, *lq, *lq, *lq, *lk, *lk, B, T, B, H, HK, D, ws.data_ptr(),
        n, err, s))
    again = lap.la_attn_prefill_fwd(q, k, v, 0.1, seq_len=T)
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    again = lap.la_attn_prefill_bwd(q, k, v, 0.1, *want, do, seq_len=T, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))


@pytest.mark.parametrize("D", [64, 128])
def test_verify(short, D):
    B, T, H, HK, S = 8, 4, 8, 2, 4096
    q = torch.randn(B * T, H, D, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(B * T, HK, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    kc, vc = (torch.randn(B, S, HK, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    want = lap.la_attn_verify(q, k, v, 0.1, kc, vc, lens, T)
    n = lap.la_attn_verify_workspace(B, T, H, HK, D)
    ws, o = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    s = torch.cuda.current_stream().cuda_stream
    lq, lk, c = (H * D, D), (HK * D, D), (S * HK * D, HK * D, D)
    timed_out(lambda err: short.la_attn_verify(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), 0.1, kc.data_ptr(), vc.data_ptr(), lens.data_ptr(), None, None, o.data_ptr(),
        *lq, *lk, *lk, *lq, *c, *c, 0, B, T, H, HK, D, B, S, 0, ws.data_ptr(), n, err, s))
    assert torch.equal(lap.la_attn_verify(q, k, v, 0.1, kc, vc, lens, T, workspace=ws), want)
