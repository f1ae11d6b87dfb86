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
from test_layer_gpu import (DEV, DT, EPS, HALF, U, Adapters, choose_ref, gen, grad_choose_ref, norm_ref, norm_rel, pick,
                            rows, within)
from test_layer_gpu import grad_ref as ordinary_grad_ref

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


# -------------------------------------------------------- as they are used

def experts_path(s):
    """A layer's expert part and its gradients: residual and norm, the choice, rows to
    their experts and back, each expert a factor of its own on its rows, and all the way
    back to the norm's input.  Everything that a step gave."""
    n, h = q.rms_norm(s["x"], s["w"], EPS, residual=s["res"])
    logits = n.float() @ s["gate"]
    ids, w = q.choose(logits, 4, score="sigmoid", bias=s["bias"], groups=4, keep=2, best=2, scale=2.5)
    off, pos = q.route(ids, s["gate"].shape[1])
    xs = torch.zeros(pos.numel(), n.shape[1], dtype=n.dtype, device=DEV)
    q.dispatch(n, pos, xs)
    of_row = torch.bucketize(torch.arange(pos.numel(), device=DEV, dtype=torch.int32), off[1:], right=True)
    f = s["f"][of_row.clamp_max(s["f"].numel() - 1)][:, None]
    ys = (xs.float() * f).to(xs.dtype)
    out = torch.empty_like(n)
    q.combine(ys, pos, w, out)
    dys, dw = torch.zeros_like(ys), torch.empty_like(w)
    q.combine_grad(s["dy"], ys, pos, w, dys, dw)
    dl = q.choose_grad(logits, ids, dw, score="sigmoid", scale=2.5)
    dxs = (dys.float() * f).to(dys.dtype)
    back = torch.empty_like(n)
    q.dispatch_grad(dxs, pos, back)
    dn = back + (dl @ s["gate"].t()).to(back.dtype)
    dx, _, dwn = q.rms_norm_grad(dn, h, s["w"], EPS, dh=s["dy"])
    return {"n": n, "h": h, "logits": logits, "ids": ids, "w": w, "off": off, "pos": pos, "xs": xs, "ys": ys, "out": out,
            "dys": dys, "dw": dw, "dl": dl, "dxs": dxs, "back": back, "dn": dn, "dx": dx, "dwn": dwn}


def test_layer_gradients_end_to_end():
    """Each step against 64 bits from what the steps before it stored, forward and back.
    The experts differ, so that a token's dweights do, and the logits have a gradient."""
    g = gen(91)
    B, H, E = 70, 512, 16
    s = {"x": rows(B, H, g, torch.bfloat16), "res": rows(B, H, g, torch.bfloat16),
         "w": (1 + 0.1 * torch.randn(H, generator=g)).bfloat16(), "gate": torch.randn(H, E, generator=g) * H ** -0.5,
         "bias": 0.05 * torch.randn(E, generator=g), "dy": torch.randn(B, H, generator=g).bfloat16(),
         "f": 0.25 + 1.5 * torch.rand(E, generator=g)}
    o = {k: v.cpu() for k, v in experts_path({k: v.to(DEV) for k, v in s.items()}).items()}
    half = HALF[torch.bfloat16]
    h, _, n = norm_ref(s["x"], s["res"], s["w"])
    assert torch.equal(o["h"], h)
    within(o["n"], n, norm_rel(H) * n.abs(), half)
    ids, w = choose_ref(o["logits"], 4, "sigmoid", s["bias"], 4, 2, 2, True, 2.5)
    assert torch.equal(o["ids"], ids)
    args = (2 * o["logits"].double().abs().amax(1, keepdim=True) + 80) * U
    within(o["w"], w, args * w)
    pos = o["pos"].long()
    assert sorted(pos.flatten().tolist()) == list(range(4 * B))
    for t in range(B):
        assert torch.equal(o["xs"][pos[t]], o["n"][t].expand(4, H))
        assert ((pos[t] >= o["off"][ids[t].long()]) & (pos[t] < o["off"][ids[t].long() + 1])).all()
    w, dy, ys = o["w"].double(), s["dy"].double(), o["ys"].double()[pos]     # [B][4][H]
    sums = lambda m: (m * w[:, :, None]).sum(1)  # noqa: E731
    within(o["out"], sums(ys), 8 * U * sums(ys.abs()), half)
    # back: products and sums in fp32, H of them for dw
    within(o["dys"][pos], w[:, :, None] * dy[:, None], 2 * U * (w[:, :, None] * dy[:, None]).abs(), half)
    dot = ys * dy[:, None]
    within(o["dw"], dot.sum(2), (H + 8) * U * dot.abs().sum(2))
    dl, mag, own = grad_choose_ref(o["logits"], o["ids"], o["dw"], "sigmoid", True, 2.5)
    tol = (200 + 2 * o["logits"].double().abs().amax(1, keepdim=True)) * U * mag + own
    within(o["dl"], dl, tol)
    assert (dl.abs() > 100 * tol).any(1).all()      # zeros would not pass
    dxs = o["dxs"].double()[pos]
    within(o["back"], dxs.sum(1), 8 * U * dxs.abs().sum(1), half)
    dx, dxt, dwn, dwt = ordinary_grad_ref(o["dn"], o["h"], s["w"], s["dy"])
    within(o["dx"], dx, dxt, half)
    within(o["dwn"], dwn, dwt)
    assert (dx - dy).abs().max() > 0.1 and dwn.abs().max() > 0.1
