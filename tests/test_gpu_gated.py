"""GPU w4a16_gated, w4a16_gated_bwd and w4a16_dgrad against their 64-bit forms.

Tolerances. A value rounded to bf16 is off by at most 2^-8 of it (HALF), a weight dequantized to
fp16 by 2^-11. Element by element, with A = |X| |W|^T the sum of magnitudes of a projection:
  - the projections are off by at most D = (2^-11 + 2^-12) A (2^-12: fp32 accumulation, far above
    it); for M <= 16 the weights are exact integers and D = 2^-12 A;
  - an activation's slope is at most 1.13 in magnitude, its second derivative at most 1.2, so
    |dY| <= 1.13 Dg (|u| + Du) + |act(g)| Du + HALF |Y|, and the gradients likewise.
Over all elements the roundings are independent, so the relative Frobenius error is about
HALF / sqrt(3) = 2.3e-3 at most for each rounding to bf16 that enters: the output's for Y, dG, dU
and dgrad (2.6e-3 with those of the weights, an eighth each), and dG's and dU's too for dX:
sqrt(2 / 3) HALF = 3.2e-3 -> 3.5e-3. These are means over many roundings: with
fewer than 4096 outputs a few large ones carry the norm (a single one may be off by HALF = 3.9e-3
from its own rounding alone), so only the element bounds hold there."""
import pytest
import torch

import gated_ref as R
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def nan_like(*shape):
    return torch.full(shape, float("nan"), dtype=R.BF16, device=DEV)


def status_ok():
    torch.cuda.synchronize()
    assert w4.w4_device_status() == 0


def run_gated(x, wg, wu, group, mode, act, ws="new"):
    M, K, H = x.shape[0], x.shape[1], wg[0].shape[0]
    y = nan_like(M, H)
    if ws == "new":
        ws = w4.alloc_gated_workspace(M, H, K, group)
    w4.w4a16_gated(x, M, wg, wu, H, K, group, mode, act, y, ws)
    return y


def run_bwd(dh, wg, wu, group, mode, act, X=None, ckpt=None, want_dx=True):
    M, H, K = dh.shape[0], wg[0].shape[0], wg[0].shape[1] * 2
    dg, du, dx = nan_like(M, H), nan_like(M, H), nan_like(M, K) if want_dx else None
    x8, xs = ckpt if ckpt is not None else (None, None)
    ws = w4.alloc_gated_bwd_workspace(M, H, K, group, from_ckpt=ckpt is not None)
    w4.w4a16_gated_bwd(dh, M, wg, wu, H, K, group, mode, act, dg, du, dx, ws, X=X, X8=x8, x_scale=xs)
    return dg, du, dx


def run_dgrad(dy, w, group, mode):
    M, N, K = dy.shape[0], w[0].shape[0], w[0].shape[1] * 2
    dx = nan_like(M, K)
    w4.w4a16_dgrad(dy, M, w, N, K, group, mode, dx, w4.alloc_dgrad_workspace(M, N, K, group))
    return dx


def magnitudes(x, w, group):
    return x.double().abs() @ R.dequant(w, group).abs().t()


def near(got, ref, bound, frob):
    got, ref = got.double(), ref.double()
    assert bool(torch.isfinite(got).all()), "unwritten outputs"
    over = (got - ref).abs() > bound
    assert not bool(over.any()), (int(over.sum()), torch.nonzero(over)[:8].tolist())
    if ref.numel() >= 4096:
        assert R.rel(got, ref) <= frob, R.rel(got, ref)


def weights(H, K, group, mode, seed, shift=0.0):
    return (R.weight(H, K, group, mode, seed, DEV, shift), R.weight(H, K, group, mode, seed + 1, DEV, shift))


def check_gated(x, wg, wu, group, mode, act):
    y = run_gated(x, wg, wu, group, mode, act)
    status_ok()
    g, u = x.double() @ R.dequant(wg, group).t(), x.double() @ R.dequant(wu, group).t()
    few = x.shape[0] <= 16
    e = 2.0 ** -12 + (0 if few else 2.0 ** -11)
    dg, du = e * magnitudes(x, wg, group), e * magnitudes(x, wu, group)
    ref = R.act(g, act) * u
    bound = 1.13 * dg * (u.abs() + du) + R.act(g, act).abs() * du + R.HALF * ref.abs() + 1e-30
    near(y, ref, bound, 2.6e-3)


# rows from one token up, over and beside the kernels' tile sizes; odd H; K of whole and half
# blocks of 64, shorter than a block, and long
SHAPES = [
    (1, 64, 128, 128, "asym"), (1, 1, 32, 32, "sym"), (2, 7, 96, 32, "asym"), (5, 333, 320, 64, "sym"),
    (8, 65, 512, 256, "asym"), (9, 200, 576, 32, "sym"), (16, 129, 1056, 32, "asym"), (16, 40, 4096, 128, "sym"),
    (17, 64, 128, 128, "asym"), (17, 3, 32, 32, "asym"), (33, 100, 96, 32, "sym"), (64, 65, 256, 64, "asym"),
    (100, 333, 576, 64, "sym"), (129, 127, 1024, 256, "asym"), (255, 64, 160, 32, "asym"), (257, 193, 1088, 64, "asym"),
    (300, 1000, 2048, 128, "asym"), (520, 96, 8192, 256, "sym"), (1, 2049, 2048, 128, "asym"), (3, 515, 14336, 128, "asym"),
    # one and two rows of layers from 2^25 weights a matrix (their own kernel), and three beside them
    (1, 8200, 4096, 128, "asym"), (2, 4097, 8192, 32, "sym"), (2, 16391, 2048, 64, "asym"), (1, 2056, 16384, 256, "asym"),
    (1, 65536, 544, 32, "asym"), (3, 8192, 4096, 64, "sym"), (2, 1048577, 32, 32, "asym"), (1, 524289, 64, 64, "sym"),
]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,K,group,mode", SHAPES)
def test_gated(M, H, K, group, mode, act):
    wg, wu = weights(H, K, group, mode, M + H)
    check_gated(R.rows(M, K, K + M, DEV, outliers=4), wg, wu, group, mode, act)


@pytest.mark.parametrize("M", [4, 40])
@pytest.mark.parametrize("shift", [0.5, -3.0])
def test_gated_zero_points_outside_the_codes(M, shift):
    """Weights all of one sign have zero points far from 0..15 (here about -90 and 600)."""
    wg, wu = weights(72, 256, 64, "asym", 5, shift)
    assert int(wg[2].abs().max()) > 60
    check_gated(R.rows(M, 256, 7, DEV), wg, wu, 64, "asym", "silu")


def test_gated_two_large_rows_are_independent():
    """As below, for the kernel of one and two rows: rows of very different sizes, a NaN in one, and
    slices of zeros and of tiny values."""
    H, K = 4096, 8192
    wg, wu = weights(H, K, 128, "asym", 3)
    x = R.rows(2, K, 4, DEV)
    x[0, 256:512], x[0, 512:640], x[1] = 0.0, 2.0 ** -130, x[1] * 2.0 ** 20
    check_gated(x, wg, wu, 128, "asym", "gelu_tanh")
    base = run_gated(x, wg, wu, 128, "asym", "silu")
    x[1, 700] = float("nan")
    y = run_gated(x, wg, wu, 128, "asym", "silu")
    status_ok()
    assert torch.equal(y[0], base[0]) and bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("M", [6, 50])
def test_gated_rows_are_independent(M):
    """A NaN or an infinity in one row, or a row of zeros, leaves the other rows as they were."""
    wg, wu = weights(96, 256, 128, "asym", 9)
    x = R.rows(M, 256, 11, DEV)
    base = run_gated(x, wg, wu, 128, "asym", "silu")
    bad = x.clone()
    bad[1, 3], bad[3, 200], bad[4] = float("nan"), float("inf"), 0.0
    y = run_gated(bad, wg, wu, 128, "asym", "silu")
    status_ok()
    keep = [m for m in range(M) if m not in (1, 3, 4)]
    assert torch.equal(y[keep], base[keep])
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[3]).any()) and bool((y[4] == 0).all())


BWD = [(1, 8, 32, 32, "sym"), (3, 64, 128, 128, "asym"), (16, 72, 96, 32, "asym"), (65, 136, 320, 64, "sym"),
       (130, 64, 512, 256, "asym"), (257, 200, 1088, 64, "asym"), (300, 1000, 768, 128, "sym")]


def check_bwd(got, x, dh, wg, wu, group, act):
    a, b = R.dequant(wg, group), R.dequant(wu, group)
    g, u, d = x.double() @ a.t(), x.double() @ b.t(), dh.double()
    e = 2.0 ** -11 + 2.0 ** -12
    eg, eu = e * magnitudes(x, wg, group), e * magnitudes(x, wu, group)
    rg, ru, rx = R.gated_grads(x, dh, wg, wu, group, act)
    bg = d.abs() * (1.13 * eu + 1.2 * eg * (u.abs() + eu)) + R.HALF * rg.abs() + 1e-30
    bu = d.abs() * 1.13 * eg + R.HALF * ru.abs() + 1e-30
    near(got[0], rg, bg, 2.6e-3)
    near(got[1], ru, bu, 2.6e-3)
    if got[2] is not None:
        bx = (1 + e) * (bg @ a.abs() + bu @ b.abs()) + e * (rg.abs() @ a.abs() + ru.abs() @ b.abs()) + R.HALF * rx.abs()
        near(got[2], rx, bx + 1e-30, 3.5e-3)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,K,group,mode", BWD)
def test_gated_bwd(M, H, K, group, mode, act):
    wg, wu = weights(H, K, group, mode, M + H)
    x, dh = R.rows(M, K, 1, DEV, outliers=4), R.rows(M, H, 2, DEV, std=0.01)
    got = run_bwd(dh, wg, wu, group, mode, act, X=x)
    status_ok()
    check_bwd(got, x, dh, wg, wu, group, act)


@pytest.mark.parametrize("M,H,K,group,mode", BWD)
def test_gated_bwd_from_the_checkpoint(M, H, K, group, mode):
    """The gradients at the checkpoint's value of x, which is exact in bf16: bit for bit those
    from the bf16 tensor of that value."""
    wg, wu = weights(H, K, group, mode, M + H)
    x, dh = R.rows(M, K, 1, DEV, outliers=4), R.rows(M, H, 2, DEV, std=0.01)
    x8, xs = w4.alloc_ckpt(M, K)
    w4.fp8_ckpt_save(x, M, K, x8, xs)
    got = run_bwd(dh, wg, wu, group, mode, "silu", ckpt=(x8, xs))
    status_ok()
    xr = R.restored(x8, xs).to(R.BF16)
    check_bwd(got, xr, dh, wg, wu, group, "silu")
    for p, q in zip(got, run_bwd(dh, wg, wu, group, mode, "silu", X=xr)):
        assert torch.equal(p, q)


def test_gated_bwd_without_dx():
    wg, wu = weights(64, 128, 64, "asym", 3)
    x, dh = R.rows(20, 128, 1, DEV), R.rows(20, 64, 2, DEV)
    full, part = run_bwd(dh, wg, wu, 64, "asym", "silu", X=x), run_bwd(dh, wg, wu, 64, "asym", "silu", X=x, want_dx=False)
    status_ok()
    assert torch.equal(full[0], part[0]) and torch.equal(full[1], part[1])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_bwd_against_differences(act):
    """<dX, V> against the central difference of the 64-bit forward along V. The difference is
    exact to 1e-8; the kernel's dX is off by the roundings of bf16, 3.5e-3 of |dX| |V| at most by
    Cauchy's inequality."""
    M, H, K, g = 48, 136, 256, 64
    wg, wu = weights(H, K, g, "asym", 21)
    x, dh = R.rows(M, K, 1, DEV), R.rows(M, H, 2, DEV)
    _, _, dx = run_bwd(dh, wg, wu, g, "asym", act, X=x)
    status_ok()
    for seed in range(4):
        v = R.rows(M, K, 30 + seed, DEV).double()
        h = 1e-5
        num = ((R.gated(x.double() + h * v, wg, wu, g, act) - R.gated(x.double() - h * v, wg, wu, g, act)) * dh.double()).sum() / (2 * h)
        assert abs(float((dx.double() * v).sum() - num)) <= 3.5e-3 * float(dx.double().norm() * v.norm())


DGRAD = [(1, 8, 32, 32, "sym"), (2, 24, 96, 32, "asym"), (16, 200, 128, 128, "asym"), (17, 64, 320, 64, "sym"),
         (64, 1000, 512, 256, "asym"), (130, 328, 1088, 64, "asym"), (300, 2048, 384, 128, "sym"), (257, 72, 4096, 128, "asym")]


@pytest.mark.parametrize("M,N,K,group,mode", DGRAD)
def test_dgrad(M, N, K, group, mode):
    w = R.weight(N, K, group, mode, N + K, DEV)
    dy = R.rows(M, N, 5, DEV, std=0.01)
    dx = run_dgrad(dy, w, group, mode)
    status_ok()
    a = R.dequant(w, group)
    ref = dy.double() @ a
    bound = (2.0 ** -11 + 2.0 ** -12) * (dy.double().abs() @ a.abs()) + R.HALF * ref.abs() + 1e-30
    near(dx, ref, bound, 2.6e-3)


@pytest.mark.parametrize("M,H,K,group", [(20, 50000, 32, 32), (300, 20000, 96, 32), (40, 40008, 128, 64)])
def test_many_tiles_of_a_short_reduction(M, H, K, group):
    """Several tiles an SM, each of one or two stages, in every product."""
    wg, wu = weights(H, K, group, "asym", 3)
    x = R.rows(M, K, 1, DEV)
    check_gated(x, wg, wu, group, "asym", "silu")
    dh = R.rows(M, H, 2, DEV, std=0.01)
    got = run_bwd(dh, wg, wu, group, "asym", "gelu_tanh", X=x)
    status_ok()
    check_bwd(got, x, dh, wg, wu, group, "gelu_tanh")
    N, K = K, H // group * group  # a wide layer of few rows
    w = R.weight(N, K, group, "asym", 4, DEV)
    dy = R.rows(M, N, 5, DEV, std=0.01)
    dx = run_dgrad(dy, w, group, "asym")
    status_ok()
    a = R.dequant(w, group)
    ref = dy.double() @ a
    near(dx, ref, (2.0 ** -11 + 2.0 ** -12) * (dy.double().abs() @ a.abs()) + R.HALF * ref.abs() + 1e-30, 2.6e-3)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [2, 40])
def test_activations_far_outside_their_bend(act, M):
    """|G| around 1e20, whose square is not a float: act(g) is g or 0 there, its slope 1 or 0."""
    H, K, g = 200, 256, 64
    wg, wu = weights(H, K, g, "asym", 9)
    x, dh = (R.rows(M, K, 1, DEV).double() * 2.0 ** 68).to(R.BF16), (R.rows(M, H, 2, DEV).double() * 2.0 ** -90).to(R.BF16)
    G, U, d = x.double() @ R.dequant(wg, g).t(), x.double() @ R.dequant(wu, g).t(), dh.double()
    y = run_gated(x, wg, wu, g, "asym", act)
    dg, du, _ = run_bwd(dh, wg, wu, g, "asym", act, X=x, want_dx=False)
    status_ok()
    # the weights' and the sums' roundings, then the result's
    e = 2.0 ** -11 + 2.0 ** -12
    eg, eu = e * magnitudes(x, wg, g), e * magnitudes(x, wu, g)
    sure, on = G.abs() > eg, (G > 0).double()
    assert float(sure.double().mean()) > 0.95
    for got, ref, off in ((y, G * U * on, eg * (U.abs() + eu) + G.abs() * eu), (dg, d * U * on, d.abs() * eu), (du, d * G * on, d.abs() * eg)):
        got, bound = got.double(), off * on + (1 + R.HALF) * R.HALF * (ref.abs() + off * on)
        assert not bool(torch.isnan(got).any())
        # y is up to 1e40: past bf16's largest value, 3.39e38, it is infinite
        inside = sure & (ref.abs() + bound < 3.38e38)
        assert bool(inside.any()) and not bool((inside & ((got - ref).abs() > bound)).any())
        assert bool((got.abs() >= 3.38e38)[sure & (ref.abs() - bound > 3.4e38)].all())


def test_two_calls_at_once():
    """Two streams, each with its own workspace, many rows and few, none waiting for the other."""
    g = 64
    calls = []
    for M, H, K in [(300, 1024, 2048), (40, 4096, 1024), (2, 8192, 4096), (9, 4096, 1024)]:
        wg, wu = weights(H, K, g, "asym", M)
        x = R.rows(M, K, M, DEV)
        calls.append((x, wg, wu, w4.alloc_gated_workspace(M, H, K, g), nan_like(M, H), run_gated(x, wg, wu, g, "asym", "silu")))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (x, wg, wu, ws, y, _) in zip(streams, calls):
            w4.w4a16_gated(x, x.shape[0], wg, wu, y.shape[1], x.shape[1], g, "asym", "silu", y, ws, stream=s)
    status_ok()
    for x, wg, wu, ws, y, want in calls:
        assert torch.equal(y, want)


def big_weight(N, K, group, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gen)
    s = (torch.rand(N, K // group, device=DEV, generator=gen) * 0.01 + 0.001).half()
    return codes, s, torch.randint(0, 16, (N, K // group), dtype=torch.int16, device=DEV, generator=gen)


def test_offsets_past_32_bits():
    """Codes of more than 2^32 bytes and results of more than 2^31 values: the last features and rows."""
    g, H, K = 128, 1 << 21, 4160 // 128 * 128 + 128
    wg, wu = big_weight(H, K, g, 1), big_weight(H, K, g, 2)
    assert wg[0].numel() > 1 << 32
    cut = lambda w, sl: tuple(t[sl].contiguous() for t in w)
    for M in (1, 3, 20):
        x = R.rows(M, K, M, DEV)
        y = run_gated(x, wg, wu, g, "asym", "silu")
        status_ok()
        for sl in (slice(0, 64), slice(H - 200, H)):
            want = R.gated(x, cut(wg, sl), cut(wu, sl), g, "silu")
            assert R.rel(y[:, sl], want) <= 2.6e-3
    del wg, wu, y
    M, N, K = 70000, 8, 32768
    w = R.weight(N, K, g, "asym", 3, DEV)
    dy = R.rows(M, N, 4, DEV)
    dx = run_dgrad(dy, w, g, "asym")
    status_ok()
    for sl in (slice(0, 128), slice(M - 300, M)):
        assert R.rel(dx[sl], dy[sl].double() @ R.dequant(w, g)) <= 2.6e-3


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,K,group,mode", [(250, 264, 2112, 64, "asym"), (700, 328, 1088, 32, "sym"), (1100, 72, 4096, 128, "asym")])
def test_two_ctas_a_tile(M, H, K, group, mode, act):
    """Columns and reductions long enough for pairs of CTAs, with an odd count of lane tiles, ragged
    columns and both whole and split reductions, in every product."""
    wg, wu = weights(H, K, group, mode, M)
    x, dh = R.rows(M, K, 1, DEV, outliers=4), R.rows(M, H, 2, DEV, std=0.01)
    check_gated(x, wg, wu, group, mode, act)
    got = run_bwd(dh, wg, wu, group, mode, act, X=x)
    status_ok()
    check_bwd(got, x, dh, wg, wu, group, act)
    n = K // 8 * 8
    w = R.weight(n, 3 * group * 11, group, mode, 5, DEV)
    dy = R.rows(M, n, 5, DEV, std=0.01)
    dx = run_dgrad(dy, w, group, mode)
    status_ok()
    a = R.dequant(w, group)
    ref = dy.double() @ a
    near(dx, ref, (2.0 ** -11 + 2.0 ** -12) * (dy.double().abs() @ a.abs()) + R.HALF * ref.abs() + 1e-30, 2.6e-3)


def test_results_do_not_change_from_run_to_run_and_workspaces_serve_again():
    """One workspace of the largest need over several shapes, each twice: the same bits."""
    shapes = [(40, 64, 4096, 128), (300, 64, 2048, 128), (1, 8192, 4096, 128), (17, 200, 8192, 128)]
    n = max(w4.w4a16_gated_workspace_bytes(*s) for s in shapes)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=DEV)
    for M, H, K, g in shapes + shapes[::-1]:
        wg, wu = weights(H, K, g, "asym", H)
        x = R.rows(M, K, M, DEV)
        first = run_gated(x, wg, wu, g, "asym", "silu", ws)
        assert torch.equal(first, run_gated(x, wg, wu, g, "asym", "silu", ws))
        assert torch.equal(first, run_gated(x, wg, wu, g, "asym", "silu"))
    status_ok()


def test_another_stream_and_a_replayed_graph():
    """Calls on a side stream and in a captured graph, replayed on new inputs."""
    g, act = 64, "silu"
    for M, H, K in [(4, 200, 512), (2, 8192, 4096), (70, 72, 4096)]:
        wg, wu = weights(H, K, g, "asym", 2)
        x = [R.rows(M, K, s, DEV) for s in (1, 2, 3)]
        want = [run_gated(v, wg, wu, g, "asym", act) for v in x]
        ws = w4.alloc_gated_workspace(M, H, K, g)
        buf, y = x[0].clone(), nan_like(M, H)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        w4.w4a16_gated(buf, M, wg, wu, H, K, g, "asym", act, y, ws, stream=s)
        s.synchronize()
        assert torch.equal(y, want[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            w4.w4a16_gated(buf, M, wg, wu, H, K, g, "asym", act, y, ws)
        for i in (1, 2, 0):
            buf.copy_(x[i])
            y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i])
    status_ok()


def test_rows_of_very_different_sizes():
    """Rows of magnitude 2^-100 to 2^60 side by side, and values far below their row's largest:
    each row as exact as alone (its results scale with it while the activation is linear)."""
    M, N, K, g = 40, 64, 256, 64
    w = R.weight(N, K, g, "asym", 4, DEV)
    dy = R.rows(M, N, 5, DEV).double()
    dy[:, :8] *= 2.0 ** -20
    dy = (dy * 2.0 ** torch.linspace(-100, 60, M, device=DEV).round().double()[:, None]).to(R.BF16)
    dx = run_dgrad(dy, w, g, "asym")
    status_ok()
    a = R.dequant(w, g)
    ref = dy.double() @ a
    near(dx, ref, (2.0 ** -11 + 2.0 ** -12) * (dy.double().abs() @ a.abs()) + R.HALF * ref.abs(), 1.0)
    for m in range(M):
        assert R.rel(dx[m], ref[m]) <= R.HALF + 2.0 ** -11
