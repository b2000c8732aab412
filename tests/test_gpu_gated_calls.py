"""GPU: how the gated block, its gradients and the checkpoint are called: buffers that are larger than the
call's shape keep what lies behind it, calls on several streams at once, and a process whose first call is
captured into a graph."""
import os
import subprocess
import sys

import pytest
import torch

import gated_ref as R
import test_gpu_gated as T
from bit_gemm_wise_b200 import w4

pytestmark = pytest.mark.gpu
DEV = T.DEV
G = 64


def problem(M, H, K, seed, more=0):
    """Inputs with `more` extra rows of NaN (activations) or of other weights behind the call's own."""
    nan = lambda t: torch.cat([t, torch.full((more, t.shape[1]), float("nan"), dtype=t.dtype, device=DEV)])
    return dict(M=M, H=H, K=K, gate=R.weight(H + more, K, G, "asym", seed, DEV), up=R.weight(H + more, K, G, "asym", seed + 1, DEV),
                x=nan(R.rows(M, K, seed + 2, DEV)), dh=nan(R.rows(M, H, seed + 3, DEV, std=0.01)))


def outputs(p, more=0):
    f = lambda r, c, t=R.BF16: torch.full((r + more, c), 77.0, dtype=torch.float32, device=DEV).to(t)
    M, H, K = p["M"], p["H"], p["K"]
    return dict(y=f(M, H), dg=f(M, H), du=f(M, H), dx=f(M, K), dx2=f(M, K), x8=f(M, K, torch.uint8), xs=f(M, K // 32, torch.uint8),
                back=f(M, K), dw=f(H, K, torch.float32), dwb=f(H, K))


def workspaces(p):
    M, H, K = p["M"], p["H"], p["K"]
    n = max(w4.w4a16_gated_workspace_bytes(M, H, K, G), w4.w4a16_gated_bwd_workspace_bytes(M, H, K, G, 1),
            w4.w4a16_dgrad_workspace_bytes(M, H, K, G), w4.fp8_ckpt_wgrad_workspace_bytes(M, H, K))
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


def every_call(p, o, ws, **kw):
    M, H, K = p["M"], p["H"], p["K"]
    w4.w4a16_gated(p["x"], M, p["gate"], p["up"], H, K, G, "asym", "silu", o["y"], ws, **kw)
    w4.fp8_ckpt_save(p["x"], M, K, o["x8"], o["xs"], **kw)
    w4.fp8_ckpt_load(o["x8"], o["xs"], M, K, o["back"], **kw)
    w4.w4a16_gated_bwd(p["dh"], M, p["gate"], p["up"], H, K, G, "asym", "silu", o["dg"], o["du"], o["dx"], ws, X8=o["x8"],
                       x_scale=o["xs"], **kw)
    w4.w4a16_dgrad(p["dh"], M, p["gate"], H, K, G, "asym", o["dx2"], ws, **kw)
    w4.fp8_ckpt_wgrad(p["dh"], o["x8"], o["xs"], M, H, K, o["dw"], w4.W4_OUT_FP32, ws, **kw)
    w4.fp8_ckpt_wgrad(p["dh"], o["x8"], o["xs"], M, H, K, o["dwb"], 0, ws, **kw)


# few rows, the kernel of one and two rows, one CTA a tile, pairs, split reductions
SHAPES = [(3, 72, 192), (2, 8200, 4160), (40, 136, 192), (150, 264, 2112), (600, 2056, 640), (1030, 3000, 768)]


@pytest.mark.parametrize("M,H,K", SHAPES)
def test_what_lies_behind_is_neither_read_nor_written(M, H, K):
    more = 5
    big, p = problem(M, H, K, 1, more), problem(M, H, K, 1)
    # the same weights and rows without the rest
    p["gate"], p["up"] = (tuple(t[:H].contiguous() for t in big[n]) for n in ("gate", "up"))
    p["x"], p["dh"] = big["x"][:M].contiguous(), big["dh"][:M].contiguous()
    a, b, ws = outputs(big, more), outputs(p), workspaces(p)
    every_call(big, a, ws)
    every_call(p, b, ws)
    T.status_ok()
    for n in b:
        rows = b[n].shape[0]
        assert torch.equal(a[n][:rows].view(torch.uint8), b[n].view(torch.uint8)), n
        assert bool((a[n][rows:].float() == 77.0).all()), n
        assert not bool(torch.isnan(b[n].float()).any()), n


def test_every_call_on_several_streams_at_once():
    ps = [problem(*s, seed=10 * i) for i, s in enumerate(SHAPES)]
    want = []
    for p in ps:
        want.append(outputs(p))
        every_call(p, want[-1], workspaces(p))
    got, wss, streams = [outputs(p) for p in ps], [workspaces(p) for p in ps], [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, o, ws, s in zip(ps, got, wss, streams):
            every_call(p, o, ws, stream=s)
    T.status_ok()
    for a, b in zip(got, want):
        for n in a:
            assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


CHILD = """
import sys
import torch
import test_gpu_gated_calls as C
from bit_gemm_wise_b200 import w4
p = C.problem(*map(int, sys.argv[1:4]), seed=1)
o, ws = C.outputs(p), C.workspaces(p)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    C.every_call(p, o, ws)
g.replay()
torch.cuda.synchronize()
want = C.outputs(p)
C.every_call(p, want, ws)
torch.cuda.synchronize()
assert w4.w4_device_status() == 0
assert all(torch.equal(o[n].view(torch.uint8), want[n].view(torch.uint8)) for n in o)
print("captured")
"""


@pytest.mark.parametrize("M,H,K", [(2, 8200, 4160), (1030, 3000, 768)])
def test_first_call_of_a_process_is_captured(M, H, K):
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", CHILD, str(M), str(H), str(K)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
