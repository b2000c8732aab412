"""GPU: products whose tiles two CTAs share, with several tiles for each pair (accumulators, powers of
rows and the columns of dH change from tile to tile), odd counts of lane tiles, ragged columns, and
reductions that are split, across the two sources of dX too. Bounds and tolerances are those of
test_gpu_gated.py and test_gpu_ckpt.py; each call is repeated and has to give the same bits.

fp32 dW: products of random signs are truncated in both directions and that averages out (sqrt(2048) *
0.29 * 2^-25 = 4e-7 of the sum); the sum is truncated after each of the 128 steps of an accumulator's 2048
rows, 128 * 2^-23 = 1.53e-5 at most, and rounded where accumulators are added up: 1.6e-5."""
import pytest
import torch

import gated_ref as R
import test_gpu_gated as T
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = T.DEV


def again(run):
    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)
    T.status_ok()
    return first


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,K,group", [(1030, 3000, 768, 128), (600, 2056, 640, 32)])
def test_gated_and_its_gradients(M, H, K, group, act):
    wg, wu = T.weights(H, K, group, "asym", M)
    x, dh = R.rows(M, K, 1, DEV, outliers=4), R.rows(M, H, 2, DEV, std=0.01)
    again(lambda: [T.run_gated(x, wg, wu, group, "asym", act)])
    T.check_gated(x, wg, wu, group, "asym", act)
    T.check_bwd(again(lambda: T.run_bwd(dh, wg, wu, group, "asym", act, X=x)), x, dh, wg, wu, group, act)


@pytest.mark.parametrize("M,N,K,group", [(1100, 1000, 4224, 64), (300, 4096, 2112, 32)])
def test_dgrad(M, N, K, group):
    w, dy = R.weight(N, K, group, "asym", 4, DEV), R.rows(M, N, 5, DEV, std=0.01)
    dx = again(lambda: [T.run_dgrad(dy, w, group, "asym")])[0]
    a = R.dequant(w, group)
    ref = dy.double() @ a
    T.near(dx, ref, (2.0 ** -11 + 2.0 ** -12) * (dy.double().abs() @ a.abs()) + R.HALF * ref.abs() + 1e-30, 2.6e-3)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("M,N,K", [(8000, 520, 1056), (700, 1544, 4160), (5000, 1544, 4160)])
def test_wgrad(M, N, K, fp32):
    x = R.rows(M, K, 3, DEV, outliers=4)
    x8, xs = w4.alloc_ckpt(M, K)
    w4.fp8_ckpt_save(x, M, K, x8, xs)
    dy, ws = R.rows(M, N, 4, DEV, std=0.01), w4.alloc_ckpt_wgrad_workspace(M, N, K)

    def run():
        dw = torch.full((N, K), float("nan"), dtype=torch.float32 if fp32 else R.BF16, device=DEV)
        w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32 if fp32 else 0, ws)
        return [dw]

    dw = again(run)[0]
    ref = dy.double().t() @ R.restored(x8, xs)
    assert bool(torch.isfinite(dw).all())
    assert R.rel(dw, ref) <= (1.6e-5 if fp32 else 2.6e-3), R.rel(dw, ref)
