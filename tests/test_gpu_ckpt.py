"""GPU fp8_ckpt_save, fp8_ckpt_load and fp8_ckpt_wgrad against their definitions, and one training
step of an adapter beside the gated feed-forward block.

The checkpoint's scales and codes and the restored values are exact: compared bit for bit. dW: the
products are exact; fp32 sums of M terms on the tensor cores, which truncate at 2^-23 of the
largest partial sum at each of M / 16 steps: M / 16 * 2^-23 relative at most for sums that do not
cancel, and these (random signs) have partial sums no larger than about their result:
1000 / 16 * 2^-23 = 7.5e-6 -> 1e-5 in fp32. bf16 adds its rounding, HALF / sqrt(3): 2.6e-3 with
margin."""
import pytest
import torch

import gated_ref as R
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def status_ok():
    torch.cuda.synchronize()
    assert w4.w4_device_status() == 0


def save(x):
    M, K = x.shape
    x8, xs = w4.alloc_ckpt(M, K)
    x8.fill_(0x55)
    xs.fill_(0x55)
    w4.fp8_ckpt_save(x, M, K, x8, xs)
    return x8, xs


def load(x8, xs):
    x = torch.full(x8.shape, 77.0, dtype=R.BF16, device=DEV)
    w4.fp8_ckpt_load(x8, xs, x8.shape[0], x8.shape[1], x)
    return x


def check_save(x):
    x8, xs = save(x)
    status_ok()
    rs, rv = R.save(x.cpu())
    assert torch.equal(xs.cpu(), rs)
    got = x8.cpu().view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(rv, nan=1e9))
    back = load(x8, xs)
    status_ok()
    ref = R.restored(x8, xs)
    assert torch.equal(torch.nan_to_num(back.double(), nan=1e300), torch.nan_to_num(ref, nan=1e300))
    return x8, xs


@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (3, 96), (7, 2880), (130, 160), (1000, 1056), (2, 65536)])
def test_save_and_load(M, K):
    check_save(R.rows(M, K, M + K, DEV, outliers=4))


def test_save_every_bf16_value():
    """Each bf16 value as a block's only value, as its largest beside ones of every smaller size,
    and as a small one beside 1: subnormals, the largest values, both zeros, infinities, NaN."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(R.BF16)
    x = torch.zeros(65536, 32, dtype=R.BF16)
    x[:, 0] = v
    check_save(x.to(DEV))
    x[:, 1] = 1.0
    check_save(x.to(DEV))
    x = (v.float()[:, None] * 2.0 ** -torch.arange(32.0)).to(R.BF16)
    check_save(x.to(DEV))


def test_save_blocks_are_independent():
    x = R.rows(4, 96, 1, DEV)
    x[1, 40], x[2, 0], x[3, 95] = float("nan"), float("-inf"), float("inf")
    x8, xs = check_save(x)
    assert xs[1, 1] == 255 and xs[2, 0] == 255 and xs[3, 2] == 255 and int((xs == 255).sum()) == 3


WGRAD = [(1, 8, 32), (5, 16, 96), (64, 8, 160), (130, 72, 320), (257, 264, 1056), (1000, 16, 4096), (1000, 512, 768), (300, 1000, 288), (900, 520, 1056)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("M,N,K", WGRAD)
def test_wgrad(M, N, K, fp32):
    x8, xs = save(R.rows(M, K, 3, DEV, outliers=4))
    dy = R.rows(M, N, 4, DEV, std=0.01)
    dw = torch.full((N, K), float("nan"), dtype=torch.float32 if fp32 else R.BF16, device=DEV)
    ws = w4.alloc_ckpt_wgrad_workspace(M, N, K)
    for _ in range(2):
        w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32 if fp32 else 0, ws)
        status_ok()
        ref = dy.double().t() @ R.restored(x8, xs)
        assert bool(torch.isfinite(dw).all())
        assert R.rel(dw, ref) <= (1e-5 if fp32 else 2.6e-3), R.rel(dw, ref)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("M,N,K", [(40, 4096, 8192), (8, 2056, 16384), (100, 8, 131072)])
def test_wgrad_of_few_rows_and_many_tiles(M, N, K, fp32):
    """Several tiles an SM, each of one or two stages: the results of the last tile must wait for its
    own products, not for those of a tile before. Tolerances as above (100 rows and fewer)."""
    x8, xs = save(R.rows(M, K, 3, DEV))
    dy = R.rows(M, N, 4, DEV, std=0.01)
    dw = torch.full((N, K), float("nan"), dtype=torch.float32 if fp32 else R.BF16, device=DEV)
    ws = w4.alloc_ckpt_wgrad_workspace(M, N, K)
    ref = dy.double().t() @ R.restored(x8, xs)
    for _ in range(3):
        dw.fill_(float("nan"))
        w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32 if fp32 else 0, ws)
        status_ok()
        assert bool(torch.isfinite(dw).all())
        assert R.rel(dw, ref) <= (1e-5 if fp32 else 2.6e-3), R.rel(dw, ref)


@pytest.mark.parametrize("M,N,K", [(5000, 24, 160), (4100, 1544, 4128), (2049, 8, 32), (9000, 264, 1056)])
def test_wgrad_of_many_rows(M, N, K):
    """fp32 results are added up from 2048 rows to the next: 2048 / 16 * 2^-23 = 1.53e-5 of a partial sum
    at most, and a rounding of 2^-24 for each of the five partial sums at most: 1.6e-5. bf16 sums
    truncate at M / 16 steps: 9000 / 16 * 2^-23 = 6.7e-5, with 2^-8 / sqrt(3) = 2.26e-3 below 2.6e-3."""
    x8, xs = save(R.rows(M, K, 3, DEV))
    dy = R.rows(M, N, 4, DEV, std=0.01)
    ref = dy.double().t() @ R.restored(x8, xs)
    ws = w4.alloc_ckpt_wgrad_workspace(M, N, K)
    for fp32 in (True, False, True):
        dw = torch.full((N, K), float("nan"), dtype=torch.float32 if fp32 else R.BF16, device=DEV)
        w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32 if fp32 else 0, ws)
        status_ok()
        assert bool(torch.isfinite(dw).all())
        assert R.rel(dw, ref) <= (1.6e-5 if fp32 else 2.6e-3), R.rel(dw, ref)


def test_wgrad_large_and_tiny_scales_and_nan_blocks():
    """Rows of magnitude 2^100 and 2^-100 in one checkpoint, and a block that was not finite."""
    M, N, K = 80, 16, 96
    x = R.rows(M, K, 5, "cpu").double()
    x[:40, :32] *= 2.0 ** 100
    x[40:, 32:64] *= 2.0 ** -100
    x = x.to(R.BF16)
    x[7, 70] = float("inf")
    x8, xs = save(x.to(DEV))
    dy = R.rows(M, N, 6, DEV)
    dw = torch.empty(N, K, dtype=torch.float32, device=DEV)
    w4.fp8_ckpt_wgrad(dy, x8, xs, M, N, K, dw, w4.W4_OUT_FP32, w4.alloc_ckpt_wgrad_workspace(M, N, K))
    status_ok()
    ref = dy.double().t() @ R.restored(x8, xs)
    assert bool(torch.isnan(dw[:, 64:]).all()) and bool(torch.isfinite(dw[:, :64]).all())
    assert R.rel(dw[:, :32], ref[:, :32]) <= 1e-5 and R.rel(dw[:, 32:64], ref[:, 32:64]) <= 1e-5


def test_training_step_of_an_adapter():
    """The operators as a training program uses them: the forward pass keeps x in 8 bits only; the
    backward pass takes the gradient through the 4-bit down projection, through the gated block
    and to the weight of an adapter that runs beside the gate projection. Each result against its
    64-bit form on the inputs that it was given (the checkpoint's value of x)."""
    M, H, K, g, r = 150, 264, 256, 64, 16
    wg, wu = R.weight(H, K, g, "asym", 1, DEV), R.weight(H, K, g, "asym", 2, DEV)
    wd = R.weight(K, H // 8 * 8 if H % g == 0 else 256, g, "asym", 3, DEV)  # down: [K, 256] of the first 256 features
    x = R.rows(M, K, 4, DEV)
    x8, xs = w4.alloc_ckpt(M, K)
    w4.fp8_ckpt_save(x, M, K, x8, xs)
    y = torch.empty(M, H, dtype=R.BF16, device=DEV)
    w4.w4a16_gated(x, M, wg, wu, H, K, g, "asym", "silu", y, w4.alloc_gated_workspace(M, H, K, g))
    dout = R.rows(M, K, 5, DEV, std=0.01)
    dh = torch.zeros(M, H, dtype=R.BF16, device=DEV)
    dh256 = torch.empty(M, 256, dtype=R.BF16, device=DEV)
    w4.w4a16_dgrad(dout, M, wd, K, 256, g, "asym", dh256, w4.alloc_dgrad_workspace(M, K, 256, g))
    dh[:, :256] = dh256
    dg, du = torch.empty_like(dh), torch.empty_like(dh)
    dx = torch.empty(M, K, dtype=R.BF16, device=DEV)
    w4.w4a16_gated_bwd(dh, M, wg, wu, H, K, g, "asym", "silu", dg, du, dx,
                       w4.alloc_gated_bwd_workspace(M, H, K, g, from_ckpt=True), X8=x8, x_scale=xs)
    b = R.rows(H, r, 6, DEV, std=0.1)                       # adapter: gate += (x A^T) B^T
    t = (dg.float() @ b.float()).to(R.BF16)                 # gradient of x A^T
    da = torch.empty(r, K, dtype=torch.float32, device=DEV)
    w4.fp8_ckpt_wgrad(t, x8, xs, M, r, K, da, w4.W4_OUT_FP32, w4.alloc_ckpt_wgrad_workspace(M, r, K))
    status_ok()
    xr = R.restored(x8, xs)
    # the tolerances of test_gpu_gated.py
    assert R.rel(y, R.gated(x, wg, wu, g, "silu")) <= 2.6e-3
    assert R.rel(dh256, dout.double() @ R.dequant(wd, g)) <= 2.6e-3
    rg, ru, rx = R.gated_grads(xr, dh, wg, wu, g, "silu")
    assert R.rel(dg, rg) <= 2.6e-3 and R.rel(du, ru) <= 2.6e-3 and R.rel(dx, rx) <= 3.5e-3
    assert R.rel(da, t.double().t() @ xr) <= 1e-5


@pytest.mark.parametrize("M,H,K", [(24, 264, 512), (300, 1032, 768)])
def test_a_captured_step_with_one_workspace(M, H, K):
    """Forward, checkpoint, backward and both kinds of weight product on a side stream and in a
    captured graph, all through one workspace, replayed on new inputs: bit for bit the separate
    calls' results."""
    g = 64
    wg, wu, wd = (R.weight(*s, g, "asym", i, DEV) for i, s in enumerate([(H, K), (H, K), (K, H // g * g)]))
    ins = [(R.rows(M, K, s, DEV), R.rows(M, H, s + 10, DEV, std=0.01), R.rows(M, K, s + 20, DEV, std=0.01)) for s in (1, 2, 3)]
    need = max(w4.w4a16_gated_workspace_bytes(M, H, K, g), w4.w4a16_gated_bwd_workspace_bytes(M, H, K, g, 1),
               w4.w4a16_dgrad_workspace_bytes(M, K, H // g * g, g), w4.fp8_ckpt_wgrad_workspace_bytes(M, H, K))

    def outputs():
        f = lambda *s, t=R.BF16: torch.full(s, float("nan"), dtype=t, device=DEV)
        return [f(M, H), f(M, H), f(M, H), f(M, K), f(M, H // g * g), f(H, K, t=torch.float32)]

    def step(x, dh, dy, o, ck, ws, **kw):
        x8, xs = ck
        w = (lambda n: ws) if ws is not None else (lambda n: torch.zeros(max(n, 16), dtype=torch.uint8, device=DEV))
        w4.w4a16_gated(x, M, wg, wu, H, K, g, "asym", "silu", o[0], w(w4.w4a16_gated_workspace_bytes(M, H, K, g)), **kw)
        w4.fp8_ckpt_save(x, M, K, x8, xs, **kw)
        w4.w4a16_dgrad(dy, M, wd, K, H // g * g, g, "asym", o[4], w(w4.w4a16_dgrad_workspace_bytes(M, K, H // g * g, g)), **kw)
        w4.w4a16_gated_bwd(dh, M, wg, wu, H, K, g, "asym", "silu", o[1], o[2], o[3],
                           w(w4.w4a16_gated_bwd_workspace_bytes(M, H, K, g, 1)), X8=x8, x_scale=xs, **kw)
        w4.fp8_ckpt_wgrad(o[1], x8, xs, M, H, K, o[5], w4.W4_OUT_FP32, w(w4.fp8_ckpt_wgrad_workspace_bytes(M, H, K)), **kw)

    want = []
    for i in ins:
        want.append(outputs())
        step(*i, want[-1], w4.alloc_ckpt(M, K), None)
    ws, o, ck = torch.zeros(need, dtype=torch.uint8, device=DEV), outputs(), w4.alloc_ckpt(M, K)
    buf = [t.clone() for t in ins[0]]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(2):  # what the first round leaves in the workspace, too
        step(*buf, o, ck, ws, stream=s)
        s.synchronize()
        assert [torch.equal(a, b) for a, b in zip(o, want[0])] == [True] * 6
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(*buf, o, ck, ws)
    for i in (1, 2, 0):
        for b, v in zip(buf, ins[i]):
            b.copy_(v)
        for t in o:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want[i]))
    status_ok()


def test_offsets_past_32_bits():
    """More than 2^31 values in the checkpoint, and in dW: the last rows."""
    M, K = 66000, 32768
    x = torch.randn(M, K, device=DEV, dtype=R.BF16, generator=torch.Generator(device=DEV).manual_seed(1))
    x8, xs = save(x)
    back = load(x8, xs)
    status_ok()
    for sl in (slice(0, 64), slice(M - 64, M)):
        rs, rv = R.save(x[sl].cpu())
        assert torch.equal(xs[sl].cpu(), rs) and torch.equal(x8[sl].cpu().view(torch.float8_e4m3fn).double(), rv)
        assert torch.equal(back[sl].double(), R.restored(x8[sl], xs[sl]))
    del x, back
    dy = R.rows(M, 8, 2, DEV, std=0.01)
    dw = torch.full((8, K), float("nan"), dtype=R.BF16, device=DEV)
    w4.fp8_ckpt_wgrad(dy, x8, xs, M, 8, K, dw, 0, w4.alloc_ckpt_wgrad_workspace(M, 8, K))
    status_ok()
    cols = slice(K - 96, K)
    ref = dy.double().t() @ R.restored(x8[:, cols].contiguous(), xs[:, K // 32 - 3:].contiguous())
    # truncation at 66000 / 16 steps, 2^-23 each: 4.9e-4, beside the output's 2.26e-3
    assert R.rel(dw[:, cols], ref) <= 2.9e-3
    n, m = 66000, 20
    x8, xs = x8[:m].contiguous(), xs[:m].contiguous()
    dy = R.rows(m, n, 3, DEV)
    dw = torch.full((n, K), float("nan"), dtype=torch.float32, device=DEV)
    w4.fp8_ckpt_wgrad(dy, x8, xs, m, n, K, dw, w4.W4_OUT_FP32, w4.alloc_ckpt_wgrad_workspace(m, n, K))
    status_ok()
    for sl in (slice(0, 100), slice(n - 200, n)):
        assert R.rel(dw[sl], dy[:, sl].double().t() @ R.restored(x8, xs)) <= 1e-5
