"""The gated feed-forward block over 4-bit weights, its backward pass and the 8-bit activation
checkpoints that feed it: cases, inputs, plain forms and exact values.

Operators (`op` of a case):
  gated       H = act(X Wg^T) * (X Wu^T), Wg and Wu [H, K] as 4-bit codes with group scales
  gated_bwd   from dH and X (bf16, or the 8-bit checkpoint of it): dG, dU (gradients of the two
              projections' outputs) and dX = dG Wg + dU Wu
  dgrad       dX = dY W of one 4-bit linear layer W [N, K]
  ckpt        an activation in 8 bits: E4M3 values with one power-of-two scale for each 32 of a
              row ("save"), and back to bf16 ("load")
  wgrad       dW = dY^T X of an activation X held as such a checkpoint

`own` false: elementary torch operations in 32 bits. `own` true: the framework's calls.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token through the feed-forward block of an 8B model
        dict(name="gated one token 8B", op="gated", M=1, H=14336, K=4096, group=128, mode="asym", act="silu"),
        # a decode batch of 16 in an expert-sized block with groups of 32
        dict(name="gated 16 rows expert", op="gated", M=16, H=2880, K=2880, group=32, mode="asym", act="silu"),
        # a short prompt (or a speculative batch) of ragged length, symmetric groups of 64
        dict(name="gated 77 rows", op="gated", M=77, H=5632, K=2048, group=64, mode="sym", act="silu"),
        # prefill, the widest layer of the repository's W4A8 workload
        dict(name="gated prefill 4096", op="gated", M=4096, H=15360, K=3840, group=128, mode="asym", act="gelu_tanh"),
        # backward of a small layer from the bf16 activation
        dict(name="gated_bwd small", op="gated_bwd", M=100, H=1536, K=576, group=32, mode="sym", act="gelu_tanh",
             ckpt=False),
        # backward of a training batch from the 8-bit checkpoint
        dict(name="gated_bwd 2048 ckpt", op="gated_bwd", M=2048, H=14336, K=4096, group=128, mode="asym", act="silu",
             ckpt=True),
        # gradient of a few rows through an attention projection
        dict(name="dgrad 64 rows", op="dgrad", M=64, N=4096, K=4096, group=64, mode="sym"),
        # gradient of a training batch through the down projection
        dict(name="dgrad down 4096", op="dgrad", M=4096, N=4096, K=14336, group=128, mode="asym"),
        # checkpoint of a long batch, and the restore of a ragged one
        dict(name="ckpt save 16384", op="ckpt", dir="save", M=16384, K=4096),
        dict(name="ckpt load 1000", op="ckpt", dir="load", M=1000, K=2880),
        # gradient of an adapter of rank 16 from the checkpoint, and of a full projection
        dict(name="wgrad rank 16", op="wgrad", M=8192, N=16, K=4096, out="fp32"),
        dict(name="wgrad 4096", op="wgrad", M=2048, N=4096, K=4096, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = 4096 * 15360 * 3840  # rows x features x columns of the largest listed product


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "dgrad", "ckpt", "wgrad"])
    if op == "ckpt":
        M = _log_int(rng, 1, 16384)
        return dict(op=op, dir=rng.choice(["save", "load"]), M=M, K=32 * _log_int(rng, 2, max(2, min(512, 16384 * 4096 // (32 * M)))))
    if op == "wgrad":
        N = 8 * _log_int(rng, 1, 640)
        K = 32 * _log_int(rng, 4, 448)
        M = _log_int(rng, 1, 8192)
        while M * N * K > MOST // 4:
            M = max(1, M // 2)
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "fp32"]))
    group = rng.choice([32, 64, 128, 256])
    K = group * _log_int(rng, max(1, 256 // group), 8192 // group)
    M = _log_int(rng, 1, 4096)
    case = dict(op=op, M=M, K=K, group=group, mode=rng.choice(["sym", "asym"]))
    if op == "dgrad":
        N = 8 * _log_int(rng, 8, 1280)
        while M * N * K > MOST:
            M = M // 2
        return dict(case, M=M, N=N)
    H = _log_int(rng, 64, 14336)
    if op == "gated_bwd":
        H = 8 * max(1, H // 8)
        case["ckpt"] = rng.random() < 0.5
    case["act"] = rng.choice(["silu", "gelu_tanh"])
    while M * H * K > MOST // (2 if op == "gated_bwd" else 1):
        M = M // 2
    return dict(case, M=M, H=H)


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV) * std


def _activation(gen, M, K):
    """N(0, 1) with eight columns 20 times as large, as the repository's prefill workload has."""
    x = _normal(gen, M, K)
    x[:, torch.randperm(K, generator=gen, device=DEV)[:8]] *= 20.0
    return x.to(BF16)


def _weight(gen, N, K, group, mode):
    """Codes [N, K/2] (two a byte, the even column low), fp16 scales and, where asymmetric,
    int16 zero points [N, K/group] of a weight of N(0, 0.02)."""
    w = _normal(gen, N, K // group, group, std=0.02)
    if mode == "asym":
        lo, hi = w.amin(-1), w.amax(-1)
        s = ((hi - lo) / 15).to(torch.float16)
        z = torch.round(-lo / s.float())
        q = (torch.round(w / s.float().unsqueeze(-1)) + z.unsqueeze(-1)).clamp_(0, 15)
        zeros = z.to(torch.int16)
    else:
        s = (w.abs().amax(-1) / 7).to(torch.float16)
        q = torch.round(w / s.float().unsqueeze(-1)).clamp_(-7, 7) + 8
        zeros = None
    q = q.reshape(N, K).to(torch.uint8)
    return q[:, 0::2] | (q[:, 1::2] << 4), s, zeros


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    st = {"case": case, "keep": {}}
    if op in ("gated", "gated_bwd"):
        st["gate"] = _weight(gen, case["H"], K, case["group"], case["mode"])
        st["up"] = _weight(gen, case["H"], K, case["group"], case["mode"])
        st["X"] = _activation(gen, M, K)
    if op == "gated_bwd":
        st["dH"] = _normal(gen, M, case["H"], std=0.01).to(BF16)
        if case["ckpt"]:
            st["X8"], st["scale"] = _save(st.pop("X"))
    if op == "dgrad":
        st["W"] = _weight(gen, case["N"], K, case["group"], case["mode"])
        st["dY"] = _normal(gen, M, case["N"], std=0.01).to(BF16)
    if op == "ckpt":
        st["X"] = _activation(gen, M, K)
        if case["dir"] == "load":
            st["X8"], st["scale"] = _save(st.pop("X"))
    if op == "wgrad":
        st["X8"], st["scale"] = _save(_activation(gen, M, K))
        st["dY"] = _normal(gen, M, case["N"], std=0.01).to(BF16)
    return st


# ------------------------------------------------------------------ plain forms

def _dequant(w, group):
    """(q - z) s in 32 bits; z is 8 where the weight is symmetric."""
    codes, s, z = w
    q = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1, group)
    z = 8.0 if z is None else z.float().unsqueeze(-1)
    return ((q.float() - z) * s.float().unsqueeze(-1)).reshape(codes.shape[0], -1)


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _pow2(e):
    """2^e for whole e in [-126, 127], exactly (a power function may be off in the last bit)."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def _save(x):
    """E4M3 values of x / 2^e and the biased exponents e + 127 for each 32 columns of a row:
    2^e is the smallest power of two, not below 2^-124, with max|x| / 2^e <= 448 (at e = 120 the
    values stop at 240, or 256 2^120 would leave bf16). A block with a value that is not finite
    has exponent 255 and NaN values."""
    M, K = x.shape
    xb = x.float().reshape(M, K // 32, 32)
    amax = xb.abs().amax(-1)
    m, p = torch.frexp(amax)  # amax = m 2^p with m in [0.5, 1): the bound 448 is 0.875 2^9
    e = (p - 9 + (m > 0.875)).clamp(min=-124)
    e = torch.where(amax == 0, torch.full_like(e, -124), e)
    bad = ~torch.isfinite(amax)
    e = torch.where(bad, torch.zeros_like(e), e)
    v = xb * _pow2(-e).unsqueeze(-1)
    v = torch.where(e.unsqueeze(-1) == 120, v.clamp(-240, 240), v)
    v = torch.where(bad.unsqueeze(-1), torch.full_like(v, math.nan), v)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return v.to(torch.float8_e4m3fn).reshape(M, K), scale


def _load(x8, scale):
    M, K = x8.shape
    f = _pow2(scale.to(torch.int32) - 127)
    f = torch.where(scale == 255, torch.full_like(f, math.nan), f)
    return (x8.float().reshape(M, K // 32, 32) * f.unsqueeze(-1)).reshape(M, K)


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    op = c["op"]
    if op == "gated":
        x = state["X"].float()
        g = x @ _dequant(state["gate"], c["group"]).t()
        u = x @ _dequant(state["up"], c["group"]).t()
        return (_act(g, c["act"]) * u).to(BF16)
    if op == "gated_bwd":
        x = _load(state["X8"], state["scale"]) if c["ckpt"] else state["X"].float()
        wg, wu = _dequant(state["gate"], c["group"]), _dequant(state["up"], c["group"])
        g, u, dh = x @ wg.t(), x @ wu.t(), state["dH"].float()
        dg, du = dh * u * _act_slope(g, c["act"]), dh * _act(g, c["act"])
        return {"dG": dg.to(BF16), "dU": du.to(BF16), "dX": (dg @ wg + du @ wu).to(BF16)}
    if op == "dgrad":
        return (state["dY"].float() @ _dequant(state["W"], c["group"])).to(BF16)
    if op == "ckpt":
        if c["dir"] == "save":
            x8, scale = _save(state["X"])
            return {"X8": x8, "scale": scale}
        return _load(state["X8"], state["scale"]).to(BF16)
    dw = state["dY"].float().t() @ _load(state["X8"], state["scale"])
    return dw if c["out"] == "fp32" else dw.to(BF16)


# ------------------------------------------------------------------ the framework's calls

def _run_own(state, c):
    from bit_gemm_wise_b200 import w4

    op, M, K, keep = c["op"], c["M"], c["K"], state["keep"]
    if op == "gated":
        if "ws" not in keep:
            keep["ws"] = w4.alloc_gated_workspace(M, c["H"], K, c["group"])
        y = torch.empty(M, c["H"], dtype=BF16, device=DEV)
        w4.w4a16_gated(state["X"], M, state["gate"], state["up"], c["H"], K, c["group"], c["mode"], c["act"], y,
                       keep["ws"])
        return y
    if op == "gated_bwd":
        if "ws" not in keep:
            keep["ws"] = w4.alloc_gated_bwd_workspace(M, c["H"], K, c["group"], from_ckpt=c["ckpt"])
        dg, du = (torch.empty(M, c["H"], dtype=BF16, device=DEV) for _ in range(2))
        dx = torch.empty(M, K, dtype=BF16, device=DEV)
        w4.w4a16_gated_bwd(state["dH"], M, state["gate"], state["up"], c["H"], K, c["group"], c["mode"], c["act"],
                           dg, du, dx, keep["ws"], X=state.get("X"), X8=state.get("X8"), x_scale=state.get("scale"))
        return {"dG": dg, "dU": du, "dX": dx}
    if op == "dgrad":
        if "ws" not in keep:
            keep["ws"] = w4.alloc_dgrad_workspace(M, c["N"], K, c["group"])
        dx = torch.empty(M, K, dtype=BF16, device=DEV)
        w4.w4a16_dgrad(state["dY"], M, state["W"], c["N"], K, c["group"], c["mode"], dx, keep["ws"])
        return dx
    if op == "ckpt":
        if c["dir"] == "save":
            x8 = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
            scale = torch.empty(M, K // 32, dtype=torch.uint8, device=DEV)
            w4.fp8_ckpt_save(state["X"], M, K, x8, scale)
            return {"X8": x8, "scale": scale}
        x = torch.empty(M, K, dtype=BF16, device=DEV)
        w4.fp8_ckpt_load(state["X8"], state["scale"], M, K, x)
        return x
    if "ws" not in keep:
        keep["ws"] = w4.alloc_ckpt_wgrad_workspace(M, c["N"], K)
    fp32 = c["out"] == "fp32"
    dw = torch.empty(c["N"], K, dtype=F32 if fp32 else BF16, device=DEV)
    w4.fp8_ckpt_wgrad(state["dY"], state["X8"], state["scale"], M, c["N"], K, dw, w4.W4_OUT_FP32 if fp32 else 0,
                      keep["ws"])
    return dw


# ------------------------------------------------------------------ work and exact values

def _weight_bytes(N, K, group, mode):
    return N * K // 2 + N * (K // group) * (4 if mode == "asym" else 2)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "gated":
        H = case["H"]
        return {"bytes": 2 * _weight_bytes(H, K, case["group"], case["mode"]) + 2 * M * (K + H),
                "flops": 4 * M * H * K}
    if op == "gated_bwd":
        H = case["H"]
        x = M * K + M * K // 32 if case["ckpt"] else 2 * M * K
        return {"bytes": 2 * _weight_bytes(H, K, case["group"], case["mode"]) + x + 2 * M * (3 * H + K),
                "flops": 8 * M * H * K}
    if op == "dgrad":
        N = case["N"]
        return {"bytes": _weight_bytes(N, K, case["group"], case["mode"]) + 2 * M * (N + K), "flops": 2 * M * N * K}
    if op == "ckpt":
        return {"bytes": 3 * M * K + M * K // 32, "flops": 2 * M * K}
    N = case["N"]
    return {"bytes": M * K + M * K // 32 + 2 * M * N + (4 if case["out"] == "fp32" else 2) * N * K,
            "flops": 2 * M * N * K}


def _weight64(w, group):
    codes, s, z = w
    N, half = codes.shape
    q = torch.empty(N, 2 * half, dtype=F64, device=codes.device)
    q[:, 0::2] = codes.bitwise_and(15).double()
    q[:, 1::2] = codes.div(16, rounding_mode="floor").double()
    q -= 8.0 if z is None else z.double().repeat_interleave(group, dim=1)
    return q.mul_(s.double().repeat_interleave(group, dim=1))


def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _restored64(x8, scale):
    p = _two_to(scale.to(torch.int64) - 127)
    return x8.double() * p.masked_fill_(scale == 255, math.nan).repeat_interleave(32, dim=1)


def _checkpoint64(x):
    """The checkpoint's definition in 64 bits: the exponent by logarithm, set right by comparison,
    and the nearest multiple of the E4M3 step, ties to even."""
    xd = x.double()
    blocks = xd.reshape(x.shape[0], -1, 32)
    top = blocks.abs().max(dim=-1).values
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(top > 448.0 * _two_to(e), e + 1, e)
    e = torch.where(top <= 448.0 * _two_to(e - 1), e - 1, e).clamp(min=-124.0)
    v = xd / _two_to(e).repeat_interleave(32, dim=1)
    low = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    low = torch.where(v.abs() >= _two_to(low + 1), low + 1, low)
    low = torch.where((v.abs() < _two_to(low)) & (low > -6), low - 1, low)
    step = _two_to(low - 3)
    v = torch.round(v / step) * step
    top = torch.where(e == 120, 240.0, 448.0).repeat_interleave(32, dim=1)
    return torch.minimum(torch.maximum(v, -top), top), e


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "ckpt":
        if case["dir"] == "load":
            return _restored64(st["X8"], st["scale"])
        return {"X8": _checkpoint64(st["X"])[0], "scale": None}
    if op == "wgrad":
        return st["dY"].double().t() @ _restored64(st["X8"], st["scale"])
    if op == "dgrad":
        return st["dY"].double() @ _weight64(st["W"], case["group"])
    x = _restored64(st["X8"], st["scale"]) if "X8" in st else st["X"].double()
    wg, wu = _weight64(st["gate"], case["group"]), _weight64(st["up"], case["group"])
    g, u = x @ wg.t(), x @ wu.t()
    if case["act"] == "silu":
        sig = torch.sigmoid(g)
        a, slope = g * sig, sig + g * sig * (1 - sig)
    else:
        k = math.sqrt(2 / math.pi)
        th = torch.tanh(k * g * (1 + 0.044715 * g ** 2))
        a = g * (1 + th) / 2
        slope = (1 + th) / 2 + g / 2 * (1 - th ** 2) * (k + 3 * 0.044715 * k * g ** 2)
    if op == "gated":
        return a * u
    dh = st["dH"].double()
    dg, du = dh * u * slope, dh * a
    return {"dG": dg, "dU": du, "dX": dg @ wg + du @ wu}
