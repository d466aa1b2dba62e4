"""The timeout exit of the gated scan, without hanging anything: a build with a 100 ns limit, which
the ordinary waits of one block for another's words exceed.  The calls return LA_OK, the error word
carries the timeout bit, the context stays usable, and the normal library gives the same bits as
before.  (The waits for a block's own copies have the same exit, but the hardware's wait instruction
sits out ordinary latencies by itself, so a short limit does not reach them.)"""
import ctypes

import pytest

import linear_attention_prefill_chunkwise_gb300 as lap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def short():
    from linear_attention_prefill_chunkwise_gb300 import build as b
    lib, real = ctypes.CDLL(b.build(wait_limit_ns=100, part="gated")), lap.load_library()
    for name in ("la_gated_scan_fwd", "la_gated_scan_bwd"):
        getattr(lib, name).argtypes = getattr(real, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    return lib


def timed_out(call):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert call(err.data_ptr()) == 0
    torch.cuda.synchronize()  # raises if the kernel had faulted and the context were lost
    assert int(err) & lap.DEV_ERR_TIMEOUT, f"error word {int(err)}: the short limit never tripped"


@pytest.mark.parametrize("B,T,C", [(1, 20000, 64), (1, 20000, 65)])
def test_scan(short, B, T, C):
    """One long sequence, whose state passes from block to block; aligned and unaligned rows."""
    x, r, g, o, d, dx, dr, dg = (torch.randn(B * T, C, device="cuda").to(torch.bfloat16) for _ in range(8))
    slopes, ds = torch.rand(C, device="cuda"), torch.empty(C, device="cuda")
    want = lap.la_gated_scan_fwd(x, r, g, slopes, seq_len=T)
    n = lap.la_gated_scan_workspace(B, T, B, C, False, torch.bfloat16, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    p = [t.data_ptr() for t in (x, r, g, slopes)]
    timed_out(lambda err: short.la_gated_scan_fwd(*p, None, None, None, o.data_ptr(), None, C, C, C, C, B, T, B, C, 0, 0,
                                                  ws.data_ptr(), n, err, s))
    timed_out(lambda err: short.la_gated_scan_bwd(*p, None, o.data_ptr(), d.data_ptr(), None, None, None, dx.data_ptr(),
                                                  dr.data_ptr(), dg.data_ptr(), ds.data_ptr(), None, *[C] * 8, B, T, B, C, 0,
                                                  0, ws.data_ptr(), n, err, s))
    assert torch.equal(lap.la_gated_scan_fwd(x, r, g, slopes, seq_len=T, workspace=ws), want)

