"""Edges of the norm, the choice of experts and the adapters on the GPU: rows far from
ordinary sizes, the adapters' dispatch on many rows, a row's bits whatever the others
name, the gradients of a layer's path.

u = 2^-24.  The bounds of a gradient of the norm are those of test_layer_gpu.py: r comes
from a sum of positive terms ((c / 2 + 4) u, c = H / 1024 + 50), c2 is off by (c + 2) u of
the sum of its terms' magnitudes, the second term has three factors r and ten more
roundings, each of them relative whatever the row's size."""

import pytest
import torch

import prefill_q8_mxfp4_amd as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, ref, tol, half=0.0, least=0.0):
    """|got - ref| <= tol + half |ref| + least everywhere (half covers tol's own part too)."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape
    off, bound = (got - ref).abs(), tol * (1 + half) + half * ref.abs() + least
    assert bool((off <= bound).all()), (off / bound.clamp_min(1e-300)).max().item()  # a NaN fails


# ------------------------------------------------------------------- norm

def grad_ref(dy, h, w, eps):
    d, hd, wd, H = dy.double(), h.double(), w.double(), h.shape[1]
    r = (hd.square().mean(1, keepdim=True) + eps) ** -0.5
    n, t = hd * r, (d * wd * hd).mean(1, keepdim=True) * r * r
    mt = (d * wd * hd).abs().mean(1, keepdim=True) * r * r
    c = H / 1024 + 50
    tol = U * ((c / 2 + 8) * (r * d * wd).abs() + (2.5 * c + 32) * n.abs() * mt + 3 * ((r * d * wd).abs() + n.abs() * mt))
    return r * d * wd - n * t, tol, (d * n).sum(0), U * (h.shape[0] + 88 + c / 2) * (d * n).abs().sum(0)


@pytest.mark.parametrize("size,eps", [(1e13, 1e-6), (1e14, 1e-6), (1e15, 1e-6), (1e16, 1e-6), (1e-13, 0.0), (1e-14, 1e-35),
                                      (1e-16, 0.0)])
@pytest.mark.parametrize("dt,rt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("B,H", [(3, 64), (5, 521), (2, 2600), (2, 24600)])
def test_rms_norm_grad_of_large_and_tiny_rows(B, H, dt, rt, size, eps):
    """Rows whose r^3 is not a number of fp32 though their squares add up in it: dx is of
    dy's size over the row's.  dy has a part along h, so that the second term counts."""
    g = gen(H)
    unit = torch.randn(B, H, generator=g)
    h = (unit * size).to(DT[rt])
    dy = (torch.randn(B, H, generator=g) + unit).to(DT[dt])
    w = 1 + 0.3 * torch.randn(H, generator=g)
    ref, tol, dwr, dwt = grad_ref(dy, h, w, eps)
    dx, dr, dw = q.rms_norm_grad(dy.to(DEV), h.to(DEV), w.to(DEV), eps)
    within(dx, ref, tol, HALF[DT[dt]])
    within(dr, ref, tol, HALF[DT[rt]])
    within(dw, dwr, dwt)
