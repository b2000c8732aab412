"""GPU: checkpoints whose bytes another program wrote. Every pair of a value byte and a scale byte means
value * 2^(scale - 127), E4M3's NaN (0x7F of either sign) under any scale and the scale byte 255 mean
NaN. The restored value is that one rounded once to bf16: exact for what fp8_ckpt_save writes, and
elsewhere but below bf16's smallest normal value (scale bytes 0 to 2) and past its largest (from 247
up, to infinity)."""
import pytest
import torch

import gated_ref as R
import test_gpu_gated as T
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = T.DEV


def load(x8, xs):
    x = torch.full(x8.shape, 77.0, dtype=R.BF16, device=DEV)
    w4.fp8_ckpt_load(x8, xs, x8.shape[0], x8.shape[1], x)
    T.status_ok()
    return x


def restored(x8, xs):
    """In bf16: a value has four bits, so fp32 holds it and is no second rounding."""
    return R.restored(x8, xs).to(torch.float32).to(R.BF16)


def same(got, ref):
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got.view(torch.int16)[~nan], ref.view(torch.int16)[~nan])


def every_byte():
    """[256, 512]: row s has scale byte s and every value byte twice, once with its block's others NaN-free."""
    v = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    w = v.clone()
    w[(w & 0x7F) == 0x7F] = 0x38
    x8 = torch.cat([v, w], 1).to(DEV)
    xs = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).contiguous().to(DEV)
    return x8, xs


def test_load_every_byte():
    x8, xs = every_byte()
    same(load(x8, xs), restored(x8, xs))
    f8, e8 = x8.view(torch.float8_e4m3fn), xs.view(torch.float8_e8m0fnu)
    same(load(f8, e8), restored(x8, xs))


@pytest.mark.parametrize("N", [8, 264])
def test_wgrad_every_byte(N):
    """One 1 a column of dY picks one row of the checkpoint: dW is that row."""
    x8, xs = every_byte()
    # a NaN would spread over its column of x (0 * NaN): rows of finite values first
    fin = x8.clone()
    fin[(fin & 0x7F) == 0x7F] = 0x38
    keep = xs.clone()
    keep[keep > 246] = 246      # an infinity likewise
    for lo in range(0, 256, N):
        dy = torch.zeros(256, N, dtype=R.BF16, device=DEV)
        n = min(N, 256 - lo)
        dy[lo:lo + n, :n] = torch.eye(n, dtype=R.BF16, device=DEV)
        dw = torch.full((N, 512), float("nan"), dtype=R.BF16, device=DEV)
        w4.fp8_ckpt_wgrad(dy, fin, keep, 256, N, 512, dw, 0, w4.alloc_ckpt_wgrad_workspace(256, N, 512))
        T.status_ok()
        # + 0: a sum of a negative zero and zeros is zero
        same(dw[:n] + 0, restored(fin, keep)[lo:lo + n] + 0)


@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("M,N,K,scale", [(5, 16, 96, 127), (300, 264, 1056, 127), (300, 264, 1056, 140), (300, 8, 1056, 3)])
def test_wgrad_nan_values(M, N, K, scale, code):
    """A NaN makes its column of x NaN in dW, wherever it stands, and leaves the others as they were."""
    gen = torch.Generator().manual_seed(M)
    x8 = torch.randint(0, 0x7F, (M, K), dtype=torch.uint8, generator=gen).to(DEV)
    xs = torch.full((M, K // 32), scale, dtype=torch.uint8, device=DEV)
    dy = R.rows(M, N, 2, DEV)
    ws = w4.alloc_ckpt_wgrad_workspace(M, N, K)

    def run():
        dw = torch.full((N, K), 77.0, dtype=torch.float32, device=DEV)
        w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32, ws)
        T.status_ok()
        return dw

    base = run()
    at = [(0, 0), (M - 1, 1), (M // 2, 2), (1, 35), (M - 2, 70), (M // 2, K - 1)]
    for m, k in at:
        x8[m, k] = code
    dw = run()
    cols = [k for _, k in at]
    rest = [k for k in range(K) if k not in cols]
    assert bool(torch.isnan(dw[:, cols]).all()) and torch.equal(dw[:, rest], base[:, rest])


@pytest.mark.parametrize("M,H,K", [(9, 72, 128), (300, 264, 384)])
def test_gated_bwd_from_any_bytes(M, H, K):
    """Bit for bit the gradients at the restored bf16 values."""
    g = 64
    wg, wu = R.weight(H, K, g, "asym", 1, DEV), R.weight(H, K, g, "asym", 2, DEV)
    gen = torch.Generator().manual_seed(M)
    x8 = torch.randint(0, 256, (M, K), dtype=torch.uint8, generator=gen)
    x8[(x8 & 0x7F) == 0x7F] = 0x38
    x8[3, 5], x8[4, K - 1] = 0x7F, 0xFF
    xs = torch.randint(118, 124, (M, K // 32), dtype=torch.uint8, generator=gen)
    xs[5], xs[6, 0] = 0, 1
    x8, xs = x8.to(DEV), xs.to(DEV)
    dh = R.rows(M, H, 2, DEV, std=0.01)
    got = T.run_bwd(dh, wg, wu, g, "asym", "silu", ckpt=(x8, xs))
    want = T.run_bwd(dh, wg, wu, g, "asym", "silu", X=restored(x8, xs))
    T.status_ok()
    for a, b in zip(got, want):
        same(a, b)
        assert bool(torch.isnan(a[3:5]).all()) and not bool(torch.isnan(a[5:]).any())
