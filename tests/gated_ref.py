"""64-bit forms of the gated feed-forward block, its gradients and the 8-bit activation
checkpoint, and inputs for their tests (torch tensors, any device)."""
import math

import torch

BF16, F64 = torch.bfloat16, torch.float64
HALF = 2.0 ** -8   # half a bf16 step, relative


def weight(N, K, group, mode, seed, device, shift=0.0):
    """A canonical 4-bit weight of N(shift, 0.02): codes, fp16 scales, zeros (None for sym)."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(N, K // group, group, generator=g) * 0.02 + shift
    if mode == "asym":
        lo, hi = w.amin(-1), w.amax(-1)
        s = ((hi - lo) / 15).clamp(min=1e-6).half()
        z = torch.round(-lo / s.float())
        q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp(0, 15)
    else:
        s, z = (w.abs().amax(-1) / 7).clamp(min=1e-6).half(), None
        q = torch.round(w / s.float()[..., None]).clamp(-7, 7) + 8
    q = q.reshape(N, K).to(torch.uint8)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    return codes.contiguous().to(device), s.to(device), None if z is None else z.to(torch.int16).to(device)


def dequant(w, group):
    codes, s, z = w
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).double()
    z = 8.0 if z is None else z.double().repeat_interleave(group, 1)
    return (q - z) * s.double().repeat_interleave(group, 1)


def act(g, name):
    if name == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def slope(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return s + g * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def gated(x, wg, wu, group, name):
    return act(x.double() @ dequant(wg, group).t(), name) * (x.double() @ dequant(wu, group).t())


def gated_grads(x, dh, wg, wu, group, name):
    a, b = dequant(wg, group), dequant(wu, group)
    g, u, d = x.double() @ a.t(), x.double() @ b.t(), dh.double()
    dg, du = d * u * slope(g, name), d * act(g, name)
    return dg, du, dg @ a + du @ b


def rows(M, K, seed, device, std=1.0, outliers=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * std
    if outliers:
        x[:, torch.randperm(K, generator=g)[:outliers]] *= 20.0
    return x.to(BF16).to(device)


def two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def save(x):
    """The checkpoint's definition: scale bytes and the E4M3 values as float64."""
    M, K = x.shape
    b = x.double().reshape(M, K // 32, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(top)
    t = torch.where(bad, torch.ones_like(top), top)
    e = torch.full_like(t, -124, dtype=torch.int64)
    for v in range(-123, 121):     # the smallest e with top <= 448 * 2^e
        e = torch.where(t > 448.0 * two_to(torch.full_like(e, v - 1)), torch.full_like(e, v), e)
    y = b / two_to(e)[..., None]
    low = torch.full_like(y, -6.0)
    for v in range(-5, 9):
        low = torch.where(y.abs() >= 2.0 ** v, torch.full_like(y, float(v)), low)
    step = 2.0 ** (low - 3)
    y = torch.round(y / step) * step
    y = torch.where(e[..., None] == 120, y.clamp(-240, 240), y)  # 256 * 2^120 is past bf16's range
    y = torch.where(bad[..., None], torch.full_like(y, math.nan), y)
    return torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8), y.reshape(M, K)


def restored(x8, scale):
    """value * 2^e in 64 bits; x8: uint8 codes or E4M3 values."""
    v = x8.view(torch.float8_e4m3fn).double() if x8.dtype == torch.uint8 else x8.double()
    f = two_to(scale.to(torch.int64) - 127)
    f = torch.where(scale == 255, torch.full_like(f, math.nan), f)
    return v * f.repeat_interleave(32, 1)


def rel(got, ref):
    got, ref = got.double(), ref.double()
    return float((got - ref).norm() / ref.norm().clamp_min(1e-300))
