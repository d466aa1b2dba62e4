"""The RMS norm's persistent kernels (8-bit output, gradients) where their ring of stages goes round
several times, against the 64-bit form."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from gated_reference import HALF_STEP, norm, norm_grad
from test_gpu_norm import EPS, f64, mat, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def weights(rng, C):
    return torch.from_numpy(rng.standard_normal(C).astype(np.float32)).cuda()


# More rows than eight per SM at once (the 8-bit form is then persistent), in more turns than a block
# has stages: wide rows, narrow ones of which a block takes many, rows that are not 16-byte aligned
FP8 = [(2600, 8192, 0), (160000, 64, 0), (12000, 1001, 1), (3000, 4100, 0), (2600, 4096, 8), (1500, 16384, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,C,off", FP8)
def test_many_rows_of_8_bits(rows, C, off, group, dtype):
    rng = np.random.default_rng(rows + C + group)
    x, res, w = mat(rng, rows, C, dtype, 1.0, off, off), mat(rng, rows, C, dtype, 2.0, off, off), weights(rng, C)
    y, scales, s = lap.la_rms_norm_fwd_fp8(x, w, EPS, residual=res, group=group)
    keep = res.clone()
    y2, scales2, s2 = lap.la_rms_norm_fwd_fp8(x, w, EPS, residual=keep, residual_out=keep, group=group)
    assert s2 is keep and torch.equal(keep, s) and torch.equal(y2.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(scales2, scales)
    ref, rs, _ = norm(f64(x), f64(res), f64(w), EPS)
    width = group or C
    sc = np.stack([np.abs(ref[:, k:k + width]).max(1) for k in range(0, C, width)], 1)
    rel = (0.5 * C + 4) * 2.0 ** -24 + 2.0 ** -20  # of y, of its maximum and of the quotient
    near(scales, np.maximum(sc, 2.0 ** -40) / 448, rel * sc / 448, "fp32", "scales")
    near(s, rs, 2.0 ** -24 * np.abs(rs), dtype, "residual_out")
    want = ref / np.repeat(f64(scales), width, axis=1)[:, :C]
    # half a step of e4m3 (2^-4 relative, 2^-10 below its normal range) beyond the quotient's error
    err = np.abs(f64(y) - want)
    assert np.all(err <= 2 * rel * np.abs(want) + np.maximum(HALF_STEP["e4m3"] * np.abs(want), 2.0 ** -10)
                  * (1 + 2.0 ** -10) + 1e-30)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C,off", [(1300, 8192, 0), (20000, 512, 0), (10000, 1001, 1), (160000, 64, 8), (1300, 9000, 0)])
def test_many_rows_of_gradients(rows, C, off, dtype):
    rng = np.random.default_rng(rows * 3 + C)
    s, dy, dres = (mat(rng, rows, C, dtype, k, off, off) for k in (2.0, 1.0, 1.0))
    w = weights(rng, C)
    dx, dw = lap.la_rms_norm_bwd(s, w, EPS, dy, dres=dres)
    ref = norm_grad(f64(s), f64(w), EPS, f64(dy), f64(dres))
    near(dx, *ref["dx"], dtype, "dx")
    near(dw, *ref["dweight"], "fp32", "dweight")
