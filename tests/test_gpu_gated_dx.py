"""GPU: dX of w4a16_gated_bwd is formed from dG and dU as they are before they are rounded to bf16: its
error is that of its own rounding and little else.

Relative to the result (Frobenius): the weights' rounding to fp16 and that of the gradients' fp16 rows are
2^-11 / sqrt(3) = 2.8e-4 in root mean square at most each, independent of each other and of dX's own
rounding: their squares add up. 1% is for what 50000 such products average to, the sums'
truncation (below 1e-4) included. From rounded gradients the error would be sqrt(2) of its own rounding's."""
import pytest
import torch

import gated_ref as R
import test_gpu_gated as T
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = T.DEV


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("M,H,K,group", [(100, 1536, 576, 32), (600, 2056, 640, 32), (300, 1000, 768, 128)])
def test_error_of_dx(M, H, K, group, ckpt, act):
    wg, wu = T.weights(H, K, group, "asym", M)
    x, dh = R.rows(M, K, 1, DEV), R.rows(M, H, 2, DEV, std=0.01)
    kw = dict(X=x)
    if ckpt:
        x8, xs = w4.alloc_ckpt(M, K)
        w4.fp8_ckpt_save(x, M, K, x8, xs)
        x, kw = R.restored(x8, xs).to(R.BF16), dict(ckpt=(x8, xs))
    got = T.run_bwd(dh, wg, wu, group, "asym", act, **kw)
    T.status_ok()
    T.check_bwd(got, x, dh, wg, wu, group, act)
    ref = R.gated_grads(x, dh, wg, wu, group, act)[2]
    error, own = R.rel(got[2], ref), R.rel(ref.to(R.BF16), ref)
    assert error ** 2 <= 1.01 * own ** 2 + 2 * 2.82e-4 ** 2, (error, own)


@pytest.mark.parametrize("M,H,K", [(3, 72, 64), (40, 264, 128)])
def test_gradients_of_every_size(M, H, K):
    """Gradients whose rounding carries into the next power of two, that round to infinity, are subnormal or
    zero: the rest of a rounding never changes what is finite or which sign it has."""
    g = 64
    wg, wu = T.weights(H, K, g, "asym", 5)
    x = R.rows(M, K, 1, DEV)
    for power in (-120, -60, 0, 100):
        dh = (R.rows(M, H, 2, DEV).double() * 2.0 ** power).to(R.BF16)
        dh[0] = 0.0
        got = T.run_bwd(dh, wg, wu, g, "asym", "silu", X=x)
        T.status_ok()
        rx = R.gated_grads(x, dh, wg, wu, g, "silu")[2]
        assert bool((got[2][0] == 0).all())
        # M H K terms: few elements carry the norm, so HALF bounds dX's rounding; 2^-11 twice as above
        assert R.rel(got[2][1:], rx[1:]) <= R.HALF + 2 * 2.0 ** -11
