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
from test_layer_gpu import DEV, DT, HALF, U, Adapters, gen, norm_rel, pick, rows, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- norm

def grad_ref(dy, h, w, eps):
    d, hd, wd, H = dy.double(), h.double(), w.double(), h.shape[1]
    r = (hd.square().mean(1, keepdim=True) + eps) ** -0.5
    n, t = hd * r, (d * wd * hd).mean(1, keepdim=True) * r * r
    mt = (d * wd * hd).abs().mean(1, keepdim=True) * r * r
    c = H / 1024 + 50
    tol = U * ((c / 2 + 8) * (r * d * wd).abs() + (2.5 * c + 32) * n.abs() * mt + 3 * ((r * d * wd).abs() + n.abs() * mt))
    return r * d * wd - n * t, tol, (d * n).sum(0), U * (h.shape[0] + 88 + c / 2) * (d * n).abs().sum(0)


@pytest.mark.parametrize("size,eps", [(1e16, 1e-6), (1e10, 0.0), (1e-18, 0.0), (1e-18, 1e-37)])
@pytest.mark.parametrize("B,H", [(3, 64), (5, 521), (2, 24600)])
def test_rms_norm_of_large_and_tiny_rows(B, H, size, eps):
    """Rows whose squares add up in fp32 and whose mean square with eps is above 2^-126."""
    g = gen(H)
    x, w = torch.randn(B, H, generator=g) * size, 1 + 0.3 * torch.randn(H, generator=g)
    r = (x.double().square().mean(1, keepdim=True) + eps) ** -0.5
    y = x.double() * r * w.double()
    within(q.rms_norm(x.to(DEV), w.to(DEV), eps), y, norm_rel(H) * y.abs())
    codes, scales = q.rms_norm_codes(x.to(DEV), w.to(DEV), eps)
    back = codes.double() * scales.double()[:, None]
    top = y.abs().amax(1, keepdim=True)
    within(back, y, (0.5 / 127 + 1e-4) * top)   # half a code, and the roundings of the scale


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


# --------------------------------------------------------------- adapters

@pytest.mark.parametrize("act,out", [("bf16", "bf16"), ("f32", "f32"), ("codes", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("K,rank,own", [(5120, 16, 16), (2000, 8, 8), (17408, 64, 64), (5120, 64, 40), (5120, 64, 24),
                                        (800, 48, 32), (5120, 128, 16)])
def test_adapt_row_alone_and_in_company(K, rank, own, act, out):
    """A row's bits are the same however many of the others name its adapter, wherever
    in a tile it stands, whatever ranks the others have."""
    g = gen(K + rank)
    B, N, E = 64, 80, 3
    ad = Adapters(E, K, N, rank, g, [own, rank, 8])
    x, base = rows(B, K, g), torch.randn(B, N, generator=g).to(DT[out]).to(DEV)
    if act == "codes":
        cod, sc = q.quantize_rows(x.to(DEV))
    else:
        x = x.to(DT[act]).to(DEV)
    want = None
    for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64):
        for at in (0, B - 1, 20):
            ids = torch.full((B,), -1, dtype=torch.int32)
            free = [i for i in range(B) if i != at]
            ids[free[:n - 1] if at else free[64 - n:]] = 0   # rows before and after it
            ids[[i for i in free if ids[i] < 0][::3]] = 1
            ids[at] = 0
            assert (ids == 0).sum() == n
            plan = q.adapter_rows(ids.to(DEV), E)
            # the row that is looked at, moved to its place
            order = torch.tensor([0 if i == at else at if i == 0 else i for i in range(B)], device=DEV)
            if act == "codes":
                c = torch.empty(B, q.code_stride(K), dtype=torch.int8, device=DEV)
                c[:, :K] = cod[order]
                y = q.adapt_codes(c[:, :K], sc[order], ad.at, ad.bt, rank, plan, base[order], ranks=ad.gr, factors=ad.gf)
            else:
                y = ad.run(x[order], plan, base[order])
            want = y[at].clone() if want is None else want
            assert torch.equal(y[at], want), (n, at)
    assert q.device_status(clear=True) == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["f32", "bf16", "codes"])
@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("B", [1024, 1025, 2100])
def test_adapt_many_rows(B, rank, act, out):
    """Rows of a prompt, on both sides of 1024, from where a launch between the two
    products adds the pieces of K (three of them here); ranks up to the largest, one of 0."""
    g = gen(B + rank)
    K, N, E = 1700, 81, 5
    sizes = [rank, 8, 0, max(8, rank // 16 * 8), rank]
    ad = Adapters(E, K, N, rank, g, sizes)
    ad.at[2] = ad.bt[2] = 0
    ids = pick(B, E, g)
    plan = q.adapter_rows(ids.to(DEV), E)
    x, base = rows(B, K, g), torch.randn(B, N, generator=g).to(DT[out])
    over = base.to(DEV)
    if act == "codes":
        c, s = q.quantize_rows(x.to(DEV))
        x = c.cpu().double() * s.cpu().double()[:, None]
        args = (c, s, ad.at, ad.bt, rank, plan)
        y = q.adapt_codes(*args, base.to(DEV), ranks=ad.gr, factors=ad.gf)
        q.adapt_codes(*args, over, y=over, ranks=ad.gr, factors=ad.gf)
    else:
        x = x.to(DT[act])
        y = ad.run(x.to(DEV), plan, base.to(DEV))
        ad.run(x.to(DEV), plan, over, y=over)
    ref, tol = ad.ref(x, ids, base, DT[out])
    within(y, ref, tol, HALF[DT[out]])
    still = (ids < 0) | (ids == 2)
    assert torch.equal(y.cpu()[still], base[still]) and torch.equal(over, y)
    assert q.device_status(clear=True) == 0


@pytest.mark.parametrize("act,out", [("bf16", "bf16"), ("f32", "f32")])
def test_adapt_one_piece(act, out):
    """So many rows that K stays in one piece, ten turns of every wave and an odd end."""
    g = gen(31)
    B, K, N, E = 12300, 5123, 40, 3
    ad = Adapters(E, K, N, 16, g, [16, 8, 16])
    ids = pick(B, E, g)
    x, base = rows(B, K, g, DT[act]), torch.randn(B, N, generator=g).to(DT[out])
    y = ad.run(x.to(DEV), q.adapter_rows(ids.to(DEV), E), base.to(DEV))
    ref, tol = ad.ref(x, ids, base, DT[out])
    within(y, ref, tol, HALF[DT[out]])
    add = ref - base.double()
    if out == "f32":   # the products' own bound, which does not grow with K
        assert ((y.cpu().double() - ref).norm(dim=1) <= 1e-5 * add.norm(dim=1) + 1e-6 * base.double().norm(dim=1)).all()
