"""GPU: the gated block, its gradients, the input gradient and the checkpoint at the largest M, H (N) and K
that they accept, 2^24, against their 64-bit forms at the first and last rows and columns. Terms have
random signs; bounds are those of test_gpu_gated.py (the sums' share of them, 2^-12 of the sum of magnitudes,
is far above what sums of random signs lose)."""
import pytest
import torch

import gated_ref as R
import test_gpu_gated as T
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = T.DEV
MOST = 1 << 24
G = 32


def big_rows(M, K, seed, std=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(M, K, device=DEV, dtype=R.BF16, generator=gen).mul_(std)


def cut(w, sl):
    return tuple(t[sl].contiguous() for t in w)


ENDS = (slice(0, 48), slice(-48, None))


def check_y(y, x, wg, wu, act="silu"):
    """y [m, h] of the rows x [m, K] and the features of wg, wu."""
    g, u = x.double() @ R.dequant(wg, G).t(), x.double() @ R.dequant(wu, G).t()
    e = 2.0 ** -12 + 2.0 ** -11
    dg, du = e * T.magnitudes(x, wg, G), e * T.magnitudes(x, wu, G)
    ref = R.act(g, act) * u
    T.near(y, ref, 1.13 * dg * (u.abs() + du) + R.act(g, act).abs() * du + R.HALF * ref.abs() + 1e-30, 1.0)


def test_most_rows():
    M, H, K = MOST, 8, 32
    wg, wu = T.big_weight(H, K, G, 1), T.big_weight(H, K, G, 2)
    x, dh = big_rows(M, K, 3), big_rows(M, H, 4, 0.01)
    y = T.run_gated(x, wg, wu, G, "asym", "silu")
    x8, xs = w4.alloc_ckpt(M, K)
    w4.fp8_ckpt_save(x, M, K, x8, xs)
    got = T.run_bwd(dh, wg, wu, G, "asym", "silu", ckpt=(x8, xs))
    w = T.big_weight(H, 64, G, 5)
    dx = T.run_dgrad(dh, w, G, "asym")
    T.status_ok()
    for sl in ENDS:
        check_y(y[sl], x[sl], wg, wu)
        rs, rv = R.save(x[sl].cpu())
        assert torch.equal(xs[sl].cpu(), rs) and torch.equal(x8[sl].cpu().view(torch.float8_e4m3fn).double(), rv)
        T.check_bwd([t[sl] for t in got], R.restored(x8[sl], xs[sl]), dh[sl], wg, wu, G, "silu")
        a = R.dequant(w, G)
        ref = dh[sl].double() @ a
        T.near(dx[sl], ref, (2.0 ** -11 + 2.0 ** -12) * (dh[sl].double().abs() @ a.abs()) + R.HALF * ref.abs() + 1e-30, 1.0)
    del y, got, dx
    back = torch.empty_like(x)
    w4.fp8_ckpt_load(x8, xs, M, K, back)
    dws = []
    for flags, dtype in ((0, R.BF16), (w4.W4_OUT_FP32, torch.float32)):
        dw = torch.full((H, K), float("nan"), dtype=dtype, device=DEV)
        w4.fp8_ckpt_wgrad(dh, x8, xs, M, H, K, dw, flags, w4.alloc_ckpt_wgrad_workspace(M, H, K))
        dws.append(dw)
    T.status_ok()
    for sl in ENDS:
        assert torch.equal(back[sl].double(), R.restored(x8[sl], xs[sl]))
    ref = mag = 0.0
    for m in range(0, M, 1 << 21):
        sl = slice(m, m + (1 << 21))
        d, v = dh[sl].double(), back[sl].double()
        ref, mag = ref + d.t() @ v, mag + d.abs().t() @ v.abs()
    for dw, half in zip(dws, (R.HALF, 2.0 ** -24)):
        # An accumulator's sum of 2^15 terms is about 181 terms large and is truncated 2^11 times, by 2^-12 of
        # itself at most; 512 such losses have random signs: sqrt(512) * 181 * 2^-12 = 1 term (a product's own
        # truncation averages out). 2^-20 of the 2^24 * 0.6 magnitudes is ten.
        T.near(dw, ref, 2.0 ** -20 * mag + half * ref.abs(), 1.0)


@pytest.mark.parametrize("M", [1, 5, 17])
def test_most_features(M):
    H, K = MOST, 32
    wg, wu = T.big_weight(H, K, G, 1), T.big_weight(H, K, G, 2)
    x, dh = big_rows(M, K, 3), big_rows(M, H, 4, 0.01)
    y = T.run_gated(x, wg, wu, G, "asym", "gelu_tanh")
    T.status_ok()
    for sl in ENDS:
        check_y(y[:, sl], x, cut(wg, sl), cut(wu, sl), "gelu_tanh")
    dg, du, dx = T.run_bwd(dh, wg, wu, G, "asym", "silu", X=x)
    dx2 = T.run_dgrad(dh, wg, G, "asym")
    T.status_ok()
    rx = rx2 = mx = mx2 = 0.0
    for h in range(0, H, 1 << 21):
        sl = slice(h, h + (1 << 21))
        a, b = cut(wg, sl), cut(wu, sl)
        d, p, q = dh[:, sl].double(), dg[:, sl].double(), du[:, sl].double()
        T.check_bwd([dg[:, sl], du[:, sl], None], x, dh[:, sl], a, b, G, "silu")
        a, b = R.dequant(a, G), R.dequant(b, G)
        # Of the gradients as they are rounded, which dX is not formed from: their roundings are independent, so
        # these sums of random signs differ by 2^-8 / sqrt(3) of them in the mean at most
        rx, mx = rx + p @ a + q @ b, mx + p.abs() @ a.abs() + q.abs() @ b.abs()
        rx2, mx2 = rx2 + d @ a, mx2 + d.abs() @ a.abs()
    e = 2.0 ** -11 + 2.0 ** -12
    T.near(dx, rx, e * mx + R.HALF * rx.abs(), 1.0)
    T.near(dx2, rx2, e * mx2 + R.HALF * rx2.abs(), 1.0)
    # sums of random signs: the weights' roundings are off by 2^-11 of the result in the mean at most
    assert R.rel(dx, rx) <= R.HALF * (1 + 3 ** -0.5) + 2.0 ** -11 and R.rel(dx2, rx2) <= R.HALF + 2.0 ** -11


@pytest.mark.parametrize("M", [1, 2, 5, 17, 300])
def test_most_columns(M):
    H, K = 8, MOST
    wg, wu = T.big_weight(H, K, G, 1), T.big_weight(H, K, G, 2)
    x, dh = big_rows(M, K, 3, 2.0 ** -12), big_rows(M, H, 4, 0.01)
    y = T.run_gated(x, wg, wu, G, "asym", "silu")
    dx = T.run_dgrad(dh, wg, G, "asym")
    T.status_ok()
    a, b = R.dequant(wg, G), R.dequant(wu, G)
    refs = []
    for rows in torch.arange(M, device=DEV).split(16):
        v = x[rows].double()
        g, u, mg, mu = v @ a.t(), v @ b.t(), v.abs() @ a.abs().t(), v.abs() @ b.abs().t()
        e = 2.0 ** -11 + 2.0 ** -12
        ref = R.act(g, "silu") * u
        T.near(y[rows], ref, 1.13 * e * mg * (u.abs() + e * mu) + R.act(g, "silu").abs() * e * mu + R.HALF * ref.abs(), 1.0)
        refs.append(ref)
    # sums of random signs: the weights' roundings are off by 2^-11 of a projection in the mean at most
    assert R.rel(y, torch.cat(refs)) <= R.HALF + 2 * 2.0 ** -11
    for sl in ENDS:
        ref = dh.double() @ a[:, sl]
        T.near(dx[:, sl], ref, (2.0 ** -11 + 2.0 ** -12) * (dh.double().abs() @ a[:, sl].abs()) + R.HALF * ref.abs() + 1e-30, 1.0)


def test_most_columns_of_dw():
    M, N, K = 40, 8, MOST
    x8 = torch.randint(0, 0x7F, (M, K), dtype=torch.uint8, device=DEV)
    xs = torch.randint(120, 130, (M, K // 32), dtype=torch.uint8, device=DEV)
    dy = R.rows(M, N, 1, DEV)
    dw = torch.full((N, K), float("nan"), dtype=torch.float32, device=DEV)
    w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32, w4.alloc_ckpt_wgrad_workspace(M, N, K))
    T.status_ok()
    for lo, hi in ((0, 96), (K - 96, K)):
        v = R.restored(x8[:, lo:hi].contiguous(), xs[:, lo // 32:hi // 32].contiguous())
        ref, mag = dy.double().t() @ v, dy.double().abs().t() @ v.abs()
        T.near(dw[:, lo:hi], ref, 40 * 1.25 * 2.0 ** -25 * mag + 2.0 ** -24 * ref.abs(), 1.0)
    N, K = MOST, 32
    x8, xs = x8[:, :K].contiguous(), xs[:, :1].contiguous()
    dy = big_rows(M, N, 2)
    dw = torch.full((N, K), float("nan"), dtype=torch.float32, device=DEV)
    w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32, w4.alloc_ckpt_wgrad_workspace(M, N, K))
    T.status_ok()
    v = R.restored(x8, xs)
    for sl in ENDS:
        ref, mag = dy[:, sl].double().t() @ v, dy[:, sl].double().abs().t() @ v.abs()
        T.near(dw[sl], ref, 40 * 1.25 * 2.0 ** -25 * mag + 2.0 ** -24 * ref.abs(), 1.0)
