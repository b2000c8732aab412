"""GPU: the gated block, its gradients and the input gradient at the edges of their inputs: zero points
far outside the codes, infinities and NaN. The bounds are those of test_gpu_gated.py; a zero point
of any size costs a weight the same one rounding to fp16."""
import pytest
import torch

import gated_ref as R
import test_gpu_gated as T
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = T.DEV
FAR = [0, 15, 16, -1, 1022, 1023, 1024, 1025, -1023, -1024, -1025, 2047, 2049, -5000, 7001, 32767, -32768]


def far_weight(N, K, group, seed):
    """Random codes; each group's zero point is one of FAR, or all of a row's groups the same one (so
    that warps see them mixed and alone); scales such that no weight passes fp16's range."""
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=gen)
    z = torch.tensor(FAR, dtype=torch.int16)
    mixed = z[torch.randint(0, len(FAR), (N, K // group), generator=gen)]
    alone = z[torch.arange(N) % len(FAR)][:, None].expand(-1, K // group)
    zeros = torch.where(((torch.arange(N) // 64) % 2 == 0)[:, None], mixed, alone).contiguous()
    s = (torch.rand(N, K // group, generator=gen) * 0.01 + 0.001).half()
    return codes.to(DEV), s.to(DEV), zeros.to(DEV)


# one and two rows of a large layer (bytes), few rows, one CTA a tile, and pairs
@pytest.mark.parametrize("M,H,K,group", [(1, 8192, 4096, 128), (2, 4104, 8192, 32), (4, 200, 512, 64), (16, 136, 256, 256),
                                         (40, 264, 512, 32), (300, 520, 1088, 64), (600, 2056, 640, 32)])
def test_zero_points_of_any_size(M, H, K, group):
    wg, wu = far_weight(H, K, group, 1), far_weight(H, K, group, 2)
    x = R.rows(M, K, 3, DEV, std=0.01)
    T.check_gated(x, wg, wu, group, "asym", "silu")
    if M < 40:
        return
    dh = R.rows(M, H, 4, DEV, std=0.01)
    got = T.run_bwd(dh, wg, wu, group, "asym", "gelu_tanh", X=x)
    T.status_ok()
    T.check_bwd(got, x, dh, wg, wu, group, "gelu_tanh")


@pytest.mark.parametrize("M,N,K,group", [(3, 72, 128, 32), (64, 1000, 512, 256), (300, 520, 1088, 64), (300, 4096, 2112, 32)])
def test_dgrad_zero_points_of_any_size(M, N, K, group):
    w, dy = far_weight(N, K, group, 5), R.rows(M, N, 6, DEV, std=0.01)
    dx = T.run_dgrad(dy, w, group, "asym")
    T.status_ok()
    a = R.dequant(w, group)
    ref = dy.double() @ a
    T.near(dx, ref, (2.0 ** -11 + 2.0 ** -12) * (dy.double().abs() @ a.abs()) + R.HALF * ref.abs() + 1e-30, 2.6e-3)


def same_kind(got, ref):
    """NaN where the formula gives NaN, and the same infinities."""
    got, ref = got.double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.isposinf(got), torch.isposinf(ref)) and torch.equal(torch.isneginf(got), torch.isneginf(ref))


@pytest.mark.parametrize("M,N,K", [(12, 72, 128), (300, 328, 1088)])
def test_dgrad_infinities_and_nan(M, N, K):
    """Each row's own affair: an infinity gives infinities of the weights' signs (NaN where a weight is
    zero), two of opposite signs and a NaN give NaN; the other rows keep their bits."""
    g = 64 if K % 64 == 0 else 32
    w, dy = R.weight(N, K, g, "asym", 1, DEV), R.rows(M, N, 2, DEV)
    base, bad = T.run_dgrad(dy, w, g, "asym"), dy.clone()
    bad[1, 3], bad[4, N - 1], bad[5, 0], bad[7, 8], bad[7, 9], bad[9] = float("nan"), float("inf"), float("-inf"), float("inf"), float("-inf"), 0.0
    dx = T.run_dgrad(bad, w, g, "asym")
    T.status_ok()
    keep = [m for m in range(M) if m not in (1, 4, 5, 7, 9)]
    assert torch.equal(dx[keep], base[keep]) and bool((dx[9] == 0).all())
    a = R.dequant(w, g)
    # one infinity a row: the formula by hand (a library's sum may form inf - inf on the way)
    inf = float("inf")
    for m, n, v in ((4, N - 1, inf), (5, 0, -inf)):
        same_kind(dx[m], a[n] * v)
    assert bool(torch.isnan(dx[1]).all()) and not bool(torch.isfinite(dx[7]).any())


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("M,H,K", [(12, 72, 128), (300, 520, 384)])
def test_gated_bwd_infinities_and_nan(M, H, K, ckpt):
    g = 64
    wg, wu = R.weight(H, K, g, "asym", 1, DEV), R.weight(H, K, g, "asym", 2, DEV)
    x, dh = R.rows(M, K, 3, DEV), R.rows(M, H, 4, DEV)

    def run(x, dh):
        if not ckpt:
            return T.run_bwd(dh, wg, wu, g, "asym", "silu", X=x)
        x8, xs = w4.alloc_ckpt(M, K)
        w4.fp8_ckpt_save(x, M, K, x8, xs)
        return T.run_bwd(dh, wg, wu, g, "asym", "silu", ckpt=(x8, xs))

    base = run(x, dh)
    xb, db = x.clone(), dh.clone()
    xb[1, 40], xb[3, 7] = float("nan"), float("inf")
    db[5, 9], db[6, 10], db[8] = float("nan"), float("inf"), 0.0
    got = run(xb, db)
    T.status_ok()
    keep = [m for m in range(M) if m not in (1, 3, 5, 6, 8)]
    for a, b in zip(got, base):
        assert torch.equal(a[keep], b[keep])
        assert bool(torch.isnan(a[1]).all()) and not bool(torch.isfinite(a[3]).any()) and bool((a[8] == 0).all())
    for a, b in zip(got[:2], base[:2]):     # a gradient that is not finite touches its own feature only
        for m, h in ((5, 9), (6, 10)):
            others = [i for i in range(H) if i != h]
            assert torch.equal(a[m, others], b[m, others]) and not bool(torch.isfinite(a[m, h]))
    assert bool(torch.isnan(got[0][5, 9])) and bool(torch.isnan(got[2][5]).all()) and not bool(torch.isfinite(got[2][6]).any())


@pytest.mark.parametrize("M,H,K,power", [(2, 200, 256, 97), (9, 200, 256, 97), (1, 8192, 4096, 110), (20, 200, 256, 110)])
def test_huge_activations(M, H, K, power):
    """|G| of 2^90 and more: the product is infinite, of U's sign, or zero where the gate closes; no NaN."""
    g = 64
    wg, wu = T.weights(H, K, g, "asym", 9)
    x = (R.rows(M, K, 1, DEV).double() * 2.0 ** power).to(R.BF16)
    y = T.run_gated(x, wg, wu, g, "asym", "silu").double()
    T.status_ok()
    G, U = x.double() @ R.dequant(wg, g).t(), x.double() @ R.dequant(wu, g).t()
    e = 2.0 ** -11 + 2.0 ** -12
    sure = (G.abs() > e * T.magnitudes(x, wg, g)) & (U.abs() > e * T.magnitudes(x, wu, g))
    assert float(sure.double().mean()) > 0.95
    want = torch.where(G > 0, float("inf") * torch.sign(U), 0.0 * U)
    assert torch.equal(y[sure], want[sure]) and not bool(torch.isnan(y).any())
