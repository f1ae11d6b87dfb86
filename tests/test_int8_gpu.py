"""The 8-bit integer products and the row movements on the GPU, against plain
forms in 64 bits (numpy and torch on the CPU).

Tolerances, u = 2^-24 (half a step of fp32): an output is fp32(acc) * s * t, an
exact whole number rounded three times, so 3 u relative, written 3.01 u for the
products of those factors.  SwiGLU of G and U, each 3 u off: SiLU'(G) G / SiLU(G)
is at most 1 + |G|, the exponential's argument is rounded twice (2 |G| u) and
its value by 2 u, 1 + e, the quotient and the two products once each: together
under (12 + 6 |G|) u.  bf16 outputs add half a step of bf16, 2^-8.  Sums of
fp32 products (combine, gradients) of n terms: n + 1 roundings at most, each u
of the sum of magnitudes.  Codes, scales, sorted places and copies are exact."""

import numpy as np
import pytest
import torch

import prefill_q8_mxfp4_amd as q
import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def code_rows(B, K, g, pitch=None):
    """int8 codes on the CPU and on the GPU (at a pitch), scales of both."""
    c = torch.randint(-128, 128, (B, K), generator=g, dtype=torch.int64).to(torch.int8)
    buf = torch.full((B, pitch or q.code_stride(K)), 77, dtype=torch.int8, device=DEV)
    buf[:, :K] = c.to(DEV)
    s = (torch.rand(B, generator=g) + 0.1) * 0.02
    return c, s, buf[:, :K], s.to(DEV)


def weight(N, K, g):
    c = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int64).to(torch.int8)
    s = (torch.rand(N, generator=g) + 0.1) * 1e-3
    return c, s, q.pack_int8(c.to(DEV), s.to(DEV))


def exact_product(cx, sx, cw, sw):
    """64-bit floats hold the whole sum exactly (below 2^53)."""
    return (cx.double() @ cw.double().t()) * sx.double()[:, None] * sw.double()[None, :]


def check_product(y, ref, swiglu, dt):
    y, nh = y.double().cpu(), ref.shape[1] // 2
    if swiglu:
        gate, up = ref[:, :nh], ref[:, nh:]
        ref = gate * torch.sigmoid(gate) * up
        tol = (12 + 6 * gate.abs()) * U
    else:
        tol = torch.full_like(ref, 3.01 * U)
    tol = tol + HALF[dt] * (1 + tol)
    off = (y - ref).abs()
    worst = (off / (tol * ref.abs() + 1e-36)).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, worst


# ------------------------------------------------------------------- rows

def quantize_ref(x, ldc):
    """x fp32 numpy -> codes [B][ldc], scales; numpy's fp32 quotients are correctly rounded."""
    B, K = x.shape
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(axis=1)
        s = (amax / np.float32(127)).astype(np.float32)
        r = np.rint((x / s[:, None]).astype(np.float32))
        c = np.clip(np.nan_to_num(r, nan=0.0, posinf=127, neginf=-127), -127, 127)
    fine = np.isfinite(amax) & (s > 0)
    s = np.where(np.isfinite(amax), s, np.float32("nan"))
    out = np.zeros((B, ldc), np.int8)
    out[:, :K] = np.where(fine[:, None], c, 0)
    return out, s


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("B,K", [(1, 1), (3, 7), (5, 16), (130, 63), (7, 512), (4, 1023), (4, 1024), (6, 1025), (2, 2729),
                                 (3, 8192), (3, 8200), (2, 18432), (2, 18433), (1, 40001), (1000, 256), (300, 2500),
                                 (4096, 512), (4101, 509), (5000, 1)])
def test_quantize_rows(act, B, K):
    g = gen(B * 7919 + K)
    x = torch.randn(B, K, generator=g) * torch.exp(torch.randn(B, 1, generator=g))
    x = x.to(DT[act])
    ldc = q.code_stride(K) + 32
    codes = torch.full((B, ldc), 99, dtype=torch.int8, device=DEV)
    cv, sv = q.quantize_rows(x.to(DEV), codes[:, :K], torch.empty(B, device=DEV))
    rc, rs = quantize_ref(x.float().numpy(), ldc)
    assert np.array_equal(sv.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), rc)
    c2, s2 = q.quantize_rows(x.to(DEV))             # allocated outputs
    assert torch.equal(c2, cv) and torch.equal(s2, sv)


@pytest.mark.parametrize("K", [40, 1400, 20000])
def test_quantize_special_rows(K):
    """Zeros, ties, subnormal rows and scales, the largest values, NaN and inf."""
    tiny = np.float32(1.4e-45)
    x = np.zeros((12, K), np.float32)
    x[1, :] = -0.0
    x[2, 5] = tiny                        # the scale underflows to zero
    x[3, :] = np.arange(K) % 200 * tiny   # subnormal values, a subnormal scale
    x[4, :] = np.where(np.arange(K) % 2, 1e-38, -3e-39)
    x[5, :] = np.float32(3.4028235e38)
    x[6, :] = (np.arange(K) % 255 - 127) + 0.5
    x[6, 0] = 127.0                       # scale 1: every other value a tie
    x[7, K - 1] = np.inf
    x[8, 3] = np.nan
    x[9, :] = -np.inf
    x[10, :] = np.linspace(-1, 1, K, dtype=np.float32)
    x[11, K // 2] = -np.nan
    rc, rs = quantize_ref(x, q.code_stride(K))
    c, s = q.quantize_rows(torch.from_numpy(x).to(DEV))
    s = s.cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(rs)) and np.array_equal(np.isnan(s), [False] * 7 + [True] * 3 + [False, True])
    assert np.array_equal(s[~np.isnan(s)].view(np.uint32), rs[~np.isnan(rs)].view(np.uint32))
    assert np.array_equal(c.cpu().numpy(), rc[:, :K])


@pytest.mark.parametrize("N,K", [(1, 1), (37, 131), (256, 512), (50, 1000)])
def test_pack_device_and_dequantize(N, K):
    g = gen(N + K)
    c, s, packed = weight(N, K, g)
    host = q.pack("int8", N, K, c.numpy(), s.numpy())
    assert np.array_equal(packed.cpu().numpy(), host)
    w = q.dequantize("int8", packed, N, K).cpu().numpy()
    assert np.array_equal(w, c.numpy().astype(np.float32) * s.numpy()[:, None])


# --------------------------------------------------------------- products

SHAPES = [(1, 16, 1), (1, 5, 64), (2, 48, 128), (15, 100, 131), (16, 64, 1000), (17, 33, 2729), (33, 272, 640),
          (64, 513, 127), (65, 130, 129), (70, 256, 512), (129, 257, 1152), (256, 128, 65), (257, 300, 333),
          (300, 1000, 2048), (1000, 515, 96)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,K", SHAPES)
def test_product(B, N, K, out):
    """Both tiers, with and without a K split: within three roundings of the
    exact sum, and the same bits from all."""
    g = gen(B + 31 * N + 977 * K)
    cx, sx, dx, dsx = code_rows(B, K, g, q.code_stride(K) + 16 * (B % 3))
    cw, sw, packed = weight(N, K, g)
    ref = exact_product(cx, sx, cw, sw)
    first = None
    for tier in (None, "skinny", "tiled"):
        plan = q.Plan("int8", N, K, act="bf16", out=out, tier=tier)
        for ws in ("auto", None):
            y = torch.full((B, N), float("nan"), dtype=DT[out], device=DEV)
            plan.run_codes(dx, dsx, packed, y, workspace=ws)
            if first is None:
                first = y
                check_product(y, ref, False, DT[out])
            assert torch.equal(y, first), (tier, ws)


@pytest.mark.parametrize("shape", range(1, 9))
@pytest.mark.parametrize("B,N,K", [(5, 70, 200), (130, 300, 700), (300, 544, 2100)])
def test_product_tile_shapes(B, N, K, shape, monkeypatch):
    """Every tile shape of the large-batch tier, its K in one, two and five
    pieces, plain and fused: the same bits as the small-batch tier."""
    g = gen(B + shape)
    _, _, dx, dsx = code_rows(B, K, g)
    cw, sw, packed = weight(N, K, g)
    for epi, n in (("none", N), ("swiglu", N // 32 * 32)):
        w = packed if epi == "none" else q.pack_int8(cw[:n].contiguous().to(DEV), sw[:n].contiguous().to(DEV))
        cols = n if epi == "none" else n // 2
        monkeypatch.delenv("QGEMM_I8_SHAPE", raising=False)
        monkeypatch.delenv("QGEMM_TI_SPLIT", raising=False)
        small = q.Plan("int8", n, K, act="bf16", out="f32", epilogue=epi, tier="skinny")
        want = small.run_codes(dx, dsx, w, torch.empty(B, cols, device=DEV))
        monkeypatch.setenv("QGEMM_I8_SHAPE", str(shape))
        for pieces in (1, 2, 5):
            monkeypatch.setenv("QGEMM_TI_SPLIT", str(pieces))
            plan = q.Plan("int8", n, K, act="bf16", out="f32", epilogue=epi, tier="tiled")
            y = plan.run_codes(dx, dsx, w, torch.full((B, cols), float("nan"), device=DEV))
            assert torch.equal(y, want), (epi, pieces)


@pytest.mark.parametrize("B,N,K,swiglu", [(520, 25 * 256 * 4 + 40, 96, False), (1030, 2 * 128 * 90, 80, True),
                                          (300, 160 * 256, 64, False)])
def test_product_last_round_in_pieces(B, N, K, swiglu, monkeypatch):
    """More 256 x 256 tiles than a round: the last round's cut in 4, 1 and 2."""
    g = gen(B)
    _, _, dx, dsx = code_rows(B, K, g)
    cw = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int64).to(torch.int8).to(DEV)
    w = q.pack_int8(cw, torch.rand(N, generator=g).to(DEV))
    epi, cols = ("swiglu", N // 2) if swiglu else ("none", N)
    monkeypatch.setenv("QGEMM_I8_SHAPE", "8")
    ys = [q.Plan("int8", N, K, act="bf16", out="bf16", epilogue=epi, tier=t).run_codes(
        dx, dsx, w, torch.full((B, cols), float("nan"), dtype=torch.bfloat16, device=DEV))
        for t in ("skinny", "tiled")]
    assert torch.equal(*ys)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("B,nh,K", [(1, 16, 64), (3, 48, 131), (16, 272, 512), (40, 80, 1000), (70, 144, 2729),
                                    (200, 528, 640), (513, 160, 256)])
def test_product_swiglu(B, nh, K, out):
    g = gen(B + 31 * nh + 977 * K)
    cx, sx, dx, dsx = code_rows(B, K, g)
    cw, sw, packed = weight(2 * nh, K, g)
    sw[: nh // 2] *= 20                   # gates that saturate
    packed = q.pack_int8(cw.to(DEV), sw.to(DEV))
    ref = exact_product(cx, sx, cw, sw)
    first = None
    for tier in ("skinny", "tiled"):
        plan = q.Plan("int8", 2 * nh, K, act="bf16", out=out, epilogue="swiglu", tier=tier)
        for ws in ("auto", None):
            y = torch.full((B, nh), float("nan"), dtype=DT[out], device=DEV)
            plan.run_codes(dx, dsx, packed, y, workspace=ws)
            if first is None:
                first = y
                check_product(y, ref, True, DT[out])
            assert torch.equal(y, first), (tier, ws)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,K", [(1, 64, 100), (1, 50, 1), (2, 37, 2048), (2, 33, 4096), (2, 33, 4104), (2, 33, 1001),
                                   (1, 8200, 328), (1, 8200, 333),
                                   (1, 20, 8192), (1, 20, 8200), (2, 9000, 96), (70, 272, 1000), (300, 513, 640)])
def test_product_of_float_rows(B, N, K, act):
    """run() quantises as quantize_rows does: the same bits as run_codes of its
    codes, by the workspace and by the library's own scratch."""
    g = gen(B + N)
    x = torch.randn(B, K, generator=g).to(DT[act]).to(DEV)
    _, _, packed = weight(N, K, g)
    plan = q.Plan("int8", N, K, act=act, out="f32")
    codes, scales = q.quantize_rows(x)
    want = plan.run_codes(codes, scales, packed, torch.empty(B, N, device=DEV))
    assert torch.equal(plan.run(x, packed, torch.empty(B, N, device=DEV)), want)
    assert torch.equal(plan.run_noalloc(x, packed, torch.empty(B, N, device=DEV)), want)
    ws = torch.full((plan.workspace_bytes(B),), 255, dtype=torch.uint8, device=DEV)  # need not be zeroed
    assert torch.equal(plan.run(x, packed, torch.empty(B, N, device=DEV), workspace=ws), want)
    small = torch.zeros(plan.workspace_bytes(B) // 2, dtype=torch.uint8, device=DEV)
    for bad in (None, small[: 1024]):
        with pytest.raises(q.QgemmError) as e:
            plan.run(x, packed, torch.empty(B, N, device=DEV), workspace=bad)
        assert e.value.status == q.ENOTSUP


def test_largest_sums():
    """K = 131071 with every code -128: the sum 2^31 - 2^14 fits."""
    N, K = 32, 131071
    cw = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    packed = q.pack_int8(cw, torch.ones(N, device=DEV))
    for B in (3, 70):
        codes = torch.full((B, q.code_stride(K)), -128, dtype=torch.int8, device=DEV)[:, :K]
        for tier in ("skinny", "tiled"):
            y = torch.empty(B, N, device=DEV)
            q.Plan("int8", N, K, act="f32", out="f32", tier=tier).run_codes(codes, torch.ones(B, device=DEV), packed, y)
            assert (y == float(np.float32(16384 * K))).all()


def test_row_depends_on_itself_alone():
    """A row's bits are the same at any batch width, in any place, beside NaN rows."""
    g = gen(5)
    N, K = 200, 700
    x = torch.randn(300, K, generator=g).to(DEV)
    _, _, packed = weight(N, K, g)
    plan = q.Plan("int8", N, K, act="f32", out="f32")
    y = plan.run(x, packed, torch.empty(300, N, device=DEV))
    for B in (1, 16, 17, 64, 65, 128, 299):
        assert torch.equal(plan.run(x[:B], packed, torch.empty(B, N, device=DEV)), y[:B])
        z = plan.run(x[300 - B:].contiguous(), packed, torch.empty(B, N, device=DEV))
        assert torch.equal(z, y[300 - B:])
    x[::3] = float("nan")
    x[1, 5] = float("inf")
    z = plan.run(x, packed, torch.empty(300, N, device=DEV))
    gone = torch.zeros(300, dtype=torch.bool, device=DEV)
    gone[::3] = True
    gone[1] = True
    assert z[gone].isnan().all() and torch.equal(z[~gone], y[~gone])


# ---------------------------------------------------------------- experts

def experts(E, N, K, g):
    parts = [weight(N, K, g) for _ in range(E)]
    table = torch.tensor([p[2].data_ptr() for p in parts], dtype=torch.int64, device=DEV)
    return parts, table


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,K,behind", [
    ([1], 16 * 2, 64, 0), ([0, 3, 0, 0, 17, 1, 0], 96, 131, 5), ([64, 65, 0, 16, 33], 160, 640, 0),
    ([0, 0, 0], 64, 64, 4), ([200, 0, 129, 128, 1, 300], 288, 333, 70), ([5] * 70, 64, 200, 1),
    ([1000], 96, 100, 0)])
def test_experts(counts, N, K, behind, swiglu, monkeypatch):
    """Each expert's rows are those of a dense call, for each tile shape; rows
    behind the last expert's are neither read (they would be NaN) nor written."""
    E, T = len(counts), sum(counts) + behind
    g = gen(T + N)
    cx, sx, dx, dsx = code_rows(T, K, g, q.code_stride(K) + 16)
    dsx[T - behind:] = float("nan")
    parts, table = experts(E, N, K, g)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    epi, ncols = ("swiglu", N // 2) if swiglu else ("none", N)
    for out in ("f32", "bf16"):
        for tier in (None, 4, 9, 10):      # by the mean count, and each of its tile shapes
            if tier is not None:
                monkeypatch.setenv("QGEMM_I8_SHAPE", str(tier))
            plan = q.Plan("int8", N, K, act="bf16", out=out, epilogue=epi)
            monkeypatch.delenv("QGEMM_I8_SHAPE", raising=False)
            y = torch.full((T, ncols), 7.0, dtype=DT[out], device=DEV)
            plan.run_grouped_codes(dx, dsx, table, off, y)
            assert (y[T - behind:] == 7.0).all()
            a = 0
            for e, n in enumerate(counts):
                if n:
                    cw, sw, packed = parts[e]
                    one = plan.run_codes(dx[a:a + n], dsx[a:a + n].clone(), packed,
                                         torch.empty(n, ncols, dtype=DT[out], device=DEV))
                    assert torch.equal(y[a:a + n], one), (out, tier, e)
                    if tier is None:
                        check_product(one, exact_product(cx[a:a + n], sx[a:a + n], cw, sw), swiglu, DT[out])
                a += n
    assert q.device_status() & q.DEV_BAD_OFFSETS == 0


@pytest.mark.parametrize("shape", [4, 9, 10])
def test_experts_bad_offsets(shape, monkeypatch):
    """An expert whose offsets break the rules is left out and reported."""
    N, K, T, E = 64, 128, 40, 4
    g = gen(1)
    _, _, dx, dsx = code_rows(T, K, g)
    _, table = experts(E, N, K, g)
    monkeypatch.setenv("QGEMM_I8_SHAPE", str(shape))
    plan = q.Plan("int8", N, K, act="bf16", out="f32")
    q.device_status(clear=True)
    for off in ([0, 10, 5, 20, 40], [0, 10, 20, 30, 41], [1, 10, 20, 30, 40], [0, -1, 20, 30, 40],
                [0, 10, 2 ** 31 - 1, 30, 40]):
        y = torch.full((T, N), 7.0, device=DEV)
        plan.run_grouped_codes(dx, dsx, table, torch.tensor(off, dtype=torch.int32, device=DEV), y)
        assert q.device_status(clear=True) == q.DEV_BAD_OFFSETS, off
    many = torch.full((3001,), 40, dtype=torch.int32)   # expert 0 has all rows, a late one breaks the rules
    many[0], many[2500] = 0, 39
    y = torch.full((T, N), 7.0, device=DEV)
    plan.run_grouped_codes(dx, dsx, table[:1].expand(3000).contiguous(), many.to(DEV), y)
    assert q.device_status(clear=True) == q.DEV_BAD_OFFSETS
    y = torch.full((T, N), 7.0, device=DEV)
    plan.run_grouped_codes(dx, dsx, table, torch.zeros(E + 1, dtype=torch.int32, device=DEV), y)
    assert q.device_status() == 0 and (y == 7.0).all()


# ------------------------------------------------------- rows by expert

def route_ref(ids, E):
    flat = ids.reshape(-1)
    kept = (flat >= 0) & (flat < E)
    off = np.zeros(E + 1, np.int64)
    off[1:] = np.cumsum(np.bincount(flat[kept], minlength=E))
    pos = np.full(flat.size, -1, np.int64)
    order = np.argsort(flat[kept], kind="stable")
    pos[np.flatnonzero(kept)[order]] = np.arange(order.size)
    return off, pos.reshape(ids.shape)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 10, 512), (16, 10, 512), (3, 64, 7), (63, 1, 2), (65, 3, 37),
                                   (777, 3, 37), (2048, 10, 512), (1024, 1, 300), (1000, 2, 16384), (5000, 8, 64),
                                   (20000, 8, 129)])
@pytest.mark.parametrize("how", ["even", "dropped", "one", "wild"])
def test_route(T, k, E, how):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k))
    if how == "dropped":
        ids[rng.random((T, k)) < 0.4] = -1
    elif how == "one":
        ids[rng.random((T, k)) < 0.9] = E - 1       # one expert has nearly all
    elif how == "wild":
        ids = rng.choice([-2 ** 31, -7, -1, 0, E - 1, E, E + 1, 2 ** 31 - 1], (T, k))
    off, pos = route_ref(ids, E)
    o, p = q.route(torch.from_numpy(ids.astype(np.int32)).to(DEV), E)
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(p.cpu().numpy(), pos)


def test_route_of_no_tokens():
    o, p = q.route(torch.empty((0, 4), dtype=torch.int32, device=DEV), 9,
                   torch.full((10,), 5, dtype=torch.int32, device=DEV))
    assert (o == 0).all() and p.shape == (0, 4)


MOVES = [(1, 1, 1, 1, 0.0), (3, 2, 4, 7, 0.3), (16, 10, 512, 2048, 0.0), (65, 3, 5, 1021, 0.25), (200, 4, 9, 512, 0.5),
         (33, 64, 64, 40, 0.1), (50, 2, 8, 5120, 1.0), (9, 3, 6, 8200, 0.2), (129, 1, 3, 255, 0.0)]


def moved(T, k, E, H, drop, dt, seed=0):
    g = gen(seed + T + H)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    R = T * k
    pos = torch.from_numpy(route_ref(ids.numpy(), E)[1].astype(np.int32))
    x, ys = (torch.randn(n, H, generator=g).to(dt) for n in (T, R))
    return pos, x, ys, torch.randn(T, k, generator=g), R


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,E,H,drop", MOVES)
def test_moves(T, k, E, H, drop, act):
    """dispatch, combine and the gradients of both; rows no choice names stay."""
    dt = DT[act]
    pos, x, ys, w, R = moved(T, k, E, H, drop, dt)
    named = pos[pos >= 0].long()
    at = torch.nonzero(pos.reshape(-1) >= 0).reshape(-1)
    tok = at // k
    dpos, dw_in = pos.to(DEV), w.to(DEV)
    # dispatch: copies
    xs = torch.full((R, H), 7.0, dtype=dt)
    want = xs.clone()
    want[named] = x[tok]
    assert torch.equal(q.dispatch(x.to(DEV), dpos, xs.to(DEV)).cpu(), want)
    # combine
    wf, yd = w.double().reshape(-1), ys.double()
    ref = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, wf[at][:, None] * yd[named])
    mag = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, (wf[at][:, None] * yd[named]).abs())
    poisoned = ys.clone()                           # rows no choice names must not matter
    unnamed = torch.ones(R, dtype=torch.bool)
    unnamed[named] = False
    poisoned[unnamed] = float("nan")
    y = q.combine(poisoned.to(DEV), dpos, dw_in, torch.full((T, H), 9.0, dtype=dt, device=DEV)).double().cpu()
    tol = (k + 1) * U * mag
    assert ((y - ref).abs() <= tol + HALF[dt] * (ref.abs() + tol)).all()
    # the gradient of dispatch: the same with ones
    ref1 = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, yd[named])
    mag1 = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, yd[named].abs())
    dx = q.dispatch_grad(poisoned.to(DEV), dpos, torch.empty(T, H, dtype=dt, device=DEV)).double().cpu()
    tol = (k + 1) * U * mag1
    assert ((dx - ref1).abs() <= tol + HALF[dt] * (ref1.abs() + tol)).all()
    # the gradient of combine, dy = x
    dys, dw = q.combine_grad(x.to(DEV), poisoned.to(DEV), dpos, dw_in, torch.full((R, H), 7.0, dtype=dt, device=DEV),
                             torch.full((T, k), 9.0, device=DEV))
    dys, dw = dys.double().cpu(), dw.double().cpu().reshape(-1)
    rdys = wf[at][:, None] * x.double()[tok]
    assert ((dys[named] - rdys).abs() <= (U + HALF[dt] * (1 + U)) * rdys.abs()).all()
    assert (dys[unnamed] == 7.0).all()
    prod = x.double()[tok] * yd[named]
    assert ((dw[at] - prod.sum(1)).abs() <= (H + 1) * U * prod.abs().sum(1)).all()
    gone = torch.ones(T * k, dtype=torch.bool)
    gone[at] = False
    assert (dw[gone] == 0).all()
    assert q.device_status() & q.DEV_BAD_ROUTE == 0


def test_gradients_against_differences():
    """combine and dispatch are linear in their rows and weights: a difference
    quotient is the derivative up to the roundings of both values."""
    T, k, E, H = 11, 3, 5, 37
    pos, x, ys, w, R = moved(T, k, E, H, 0.2, torch.float32, 9)
    g = gen(3)
    dy = torch.randn(T, H, generator=g)
    d = [t.to(DEV) for t in (pos, x, ys, w, dy)]
    dys, dw = q.combine_grad(d[4], d[2], d[0], d[3], torch.zeros(R, H, device=DEV), torch.zeros(T, k, device=DEV))
    dxs = torch.randn(R, H, generator=g).to(DEV)
    dx = q.dispatch_grad(dxs, d[0], torch.zeros(T, H, device=DEV))

    def comb(ys_, w_):
        y = q.combine(ys_, d[0], w_, torch.zeros(T, H, device=DEV))
        return (y.double() * d[4].double()).sum().item()

    def disp(x_):
        xs = q.dispatch(x_, d[0], torch.zeros(R, H, device=DEV))
        return (xs.double() * dxs.double()).sum().item()

    # sums of at most k terms of size <= 6 * 5, T * H outputs of |dy| <= 6
    eps, noise = 1.0, 2 * T * H * 6 * (k + 1) * U * k * 30
    for f in range(0, T * k, 4):
        v = w.clone().reshape(-1)
        v[f] += eps
        got = (comb(d[2], v.reshape(T, k).to(DEV)) - comb(d[2], d[3])) / eps
        assert abs(got - dw.reshape(-1)[f].item()) <= noise
    for i in range(0, R * H, 97):
        v = ys.clone().reshape(-1)
        v[i] += eps
        got = (comb(v.reshape(R, H).to(DEV), d[3]) - comb(d[2], d[3])) / eps
        assert abs(got - dys.reshape(-1)[i].item()) <= noise
    for i in range(0, T * H, 29):
        v = x.clone().reshape(-1)
        v[i] += eps
        got = (disp(v.reshape(T, H).to(DEV)) - disp(d[1])) / eps
        assert abs(got - dx.reshape(-1)[i].item()) <= noise


def test_bad_positions():
    """A position of R or more names nothing and is reported."""
    T, k, R, H = 6, 2, 8, 48
    x = torch.randn(T, H, device=DEV)
    good = torch.full((T, k), -1, dtype=torch.int32)
    good.reshape(-1)[:4] = torch.tensor([3, 0, 7, 1])
    bad = good.clone()
    bad[4, 0], bad[4, 1], bad[5, 0] = R, 2 ** 31 - 1, -2 ** 31
    good, bad = good.to(DEV), bad.to(DEV)
    w = torch.rand(T, k, device=DEV)
    ys = torch.randn(R, H, device=DEV)

    def outs(pos):
        codes, scales = torch.full((R, H), 5, dtype=torch.int8, device=DEV), torch.full((R,), 5.0, device=DEV)
        q.device_status(clear=True)
        got, bits = [], []
        for f in (lambda: q.dispatch(x, pos, torch.full((R, H), 7.0, device=DEV)),
                  lambda: q.combine(ys, pos, w, torch.empty(T, H, device=DEV)),
                  lambda: q.combine_grad(x, ys, pos, w, torch.full((R, H), 7.0, device=DEV),
                                         torch.empty(T, k, device=DEV)),
                  lambda: q.dispatch_codes(x, pos, codes, scales)):
            r = f()
            got += list(r) if isinstance(r, tuple) else [r]
            bits.append(q.device_status(clear=True))
        return got, bits

    a, bits = outs(good)
    assert bits == [0] * 4
    b, bits = outs(bad)
    assert bits == [q.DEV_BAD_ROUTE] * 4
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,E,K,drop", [(1, 1, 1, 5, 0.0), (16, 10, 512, 2048, 0.0), (70, 3, 9, 1021, 0.3),
                                          (5, 4, 4, 9000, 0.2), (3, 2, 4, 20000, 0.0), (300, 2, 7, 96, 0.1)])
def test_dispatch_codes(T, k, E, K, drop, act):
    """The same bits as quantize_rows and a copy of its rows."""
    pos, x, _, _, R = moved(T, k, E, K, drop, DT[act])
    x = x.to(DEV)
    c, s = q.quantize_rows(x)
    buf = torch.full((R, q.code_stride(K)), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((R,), 5.0, device=DEV)
    q.dispatch_codes(x, pos.to(DEV), buf[:, :K], scales)
    named, tok = pos[pos >= 0].long(), torch.nonzero(pos.reshape(-1) >= 0).reshape(-1) // k
    wc = torch.full((R, q.code_stride(K)), 99, dtype=torch.int8)
    ws = torch.full((R,), 5.0)
    wc[named] = 0
    wc[named, :K] = c.cpu()[tok]
    ws[named] = s.cpu()[tok]
    assert torch.equal(buf.cpu(), wc) and torch.equal(scales.cpu(), ws)


# ------------------------------------------------------------ a whole layer

def layer(x, ids, weights, E, gu_plan, gu_table, dn_plan, dn_table, st=None):
    """One expert layer as a program would call it."""
    T, k = ids.shape
    R, H, nh = T * k, x.shape[1], gu_plan.out_cols
    off, pos = q.route(ids, E, stream=st)
    codes, scales = torch.empty((R, q.code_stride(H)), dtype=torch.int8, device=x.device)[:, :H], torch.empty(R, device=x.device)
    q.dispatch_codes(x, pos, codes, scales, stream=st)
    h = torch.zeros(R, nh, dtype=torch.bfloat16, device=x.device)
    gu_plan.run_grouped_codes(codes, scales, gu_table, off, h, stream=st)
    hc, hs = q.quantize_rows(h, stream=st)
    ys = torch.empty(R, H, dtype=x.dtype, device=x.device)
    dn_plan.run_grouped_codes(hc, hs, dn_table, off, ys, stream=st)
    return q.combine(ys, pos, weights, torch.empty_like(x), stream=st)


def make_layer(T, k, E, H, nh, drop, seed):
    g = gen(seed)
    gu, gt = experts(E, 2 * nh, H, g)
    dn, dt = experts(E, H, nh, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    gp = q.Plan("int8", 2 * nh, H, act="bf16", out="bf16", epilogue="swiglu")
    dp = q.Plan("int8", H, nh, act="bf16", out="bf16")
    return gu, gt, dn, dt, x, ids, w, gp, dp


@pytest.mark.parametrize("T,k,E,H,nh,drop", [(1, 2, 4, 128, 32, 0.0), (16, 4, 24, 256, 48, 0.0), (70, 3, 8, 200, 80, 0.3),
                                             (300, 2, 3, 96, 16, 0.1)])
def test_layer(T, k, E, H, nh, drop):
    gu, gt, dn, dt, x, ids, w, gp, dp = make_layer(T, k, E, H, nh, drop, 11)
    y = layer(x.to(DEV), ids.to(DEV), w.to(DEV), E, gp, gt, dp, dt).double().cpu()
    ref, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    c, s = quantize_ref(x.float().numpy(), H)
    c, s = torch.from_numpy(c), torch.from_numpy(s)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                continue
            go = exact_product(c[t:t + 1], s[t:t + 1], gu[e][0], gu[e][1])
            h = (go[:, :nh] * torch.sigmoid(go[:, :nh]) * go[:, nh:]).to(torch.bfloat16)
            hc, hs = quantize_ref(h.float().numpy(), nh)
            z = exact_product(torch.from_numpy(hc), torch.from_numpy(hs), dn[e][0], dn[e][1])[0] * w[t, j].double()
            # at worst every value of h rounds to its other bf16 neighbour (a step, 2^-7 of its
            # size) and every code to the next one (a step of the row's scale)
            slack = ((2.0 ** -7 * h.double().abs() + torch.from_numpy(hs).double()[:, None])
                     @ (dn[e][0].double().abs() * dn[e][1].double()[:, None]).t())[0] * w[t, j].double()
            ref[t] += z
            mag[t] += slack + 2.0 ** -8 * (slack + z.abs())
    assert ((y - ref).abs() <= mag * (1 + (k + 1) * U) + 2.0 ** -8 * (ref.abs() + mag) + 1e-30).all()
    # only values within a few u of a border do so (a share of some 2^-14 of them), which
    # leaves the roundings of ys and y to bf16: 2^-8 each at most, 2^-7 in all
    assert (y - ref).norm() <= 2.0 ** -7 * ref.norm()


def test_layer_captured():
    """Captured once, replayed three times with eager work between, on another
    stream than the current one: the eager bits each time."""
    gu, gt, dn, dt, x, ids, w, gp, dp = make_layer(33, 4, 16, 256, 48, 0.2, 12)
    x, ids, w = x.to(DEV), ids.to(DEV), w.to(DEV)
    xb = x.flip(0).contiguous()
    want, wantb = (layer(v, ids, w, 16, gp, gt, dp, dt) for v in (x, xb))
    st = torch.cuda.Stream()
    buf, graph = x.clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        got = layer(buf, ids, w, 16, gp, gt, dp, dt)
    for rep in range(3):
        buf.copy_(xb if rep == 1 else x)
        other = layer(xb, ids, w, 16, gp, gt, dp, dt)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, wantb if rep == 1 else want) and torch.equal(other, wantb)
    with torch.cuda.stream(st):
        again = layer(x, ids, w, 16, gp, gt, dp, dt)
    torch.cuda.synchronize()
    assert torch.equal(again, want)
    st.wait_stream(torch.cuda.current_stream())
    again = layer(x, ids, w, 16, gp, gt, dp, dt, st)
    torch.cuda.synchronize()
    assert torch.equal(again, want)


def test_sorted_rows_feed_the_block_formats():
    """route and dispatch make the offsets and rows that run_grouped takes."""
    E, T, k, K, N = 6, 40, 2, 256, 64
    g = gen(2)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).to(DEV)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
    bufs = [torch.from_numpy(q.pack_logical(synth.gen_expert_weights("mxfp4", N, K, e))).to(DEV) for e in range(E)]
    table = torch.tensor([b.data_ptr() for b in bufs], dtype=torch.int64, device=DEV)
    plan = q.Plan("mxfp4", N, K, act="bf16", out="f32")
    off, pos = q.route(ids, E)
    xs = q.dispatch(x, pos, torch.empty(T * k, K, dtype=torch.bfloat16, device=DEV))
    ys = plan.run_grouped(xs, table, off, torch.empty(T * k, N, device=DEV))
    y = q.combine(ys, pos, None, torch.empty(T, N, device=DEV))
    dense = torch.stack([q.dequantize("mxfp4", b, N, K) for b in bufs]).double()
    ref = torch.zeros(T, N, dtype=torch.float64, device=DEV)
    for j in range(k):
        ref += (dense[ids[:, j].long()] @ x.double()[:, :, None])[:, :, 0]
    assert ((y - ref).norm() / ref.norm()).item() <= 1e-5  # exact products, fp32 sums
    assert q.device_status() & q.DEV_BAD_OFFSETS == 0


def test_workspace_of_two_graphs():
    """Two graphs captured with one plan's workspace keep it when a wider eager
    call makes the plan take a larger one."""
    g = gen(8)
    N, K = 512, 640
    _, _, packed = weight(N, K, g)
    plan = q.Plan("int8", N, K, act="f32", out="f32")
    xs = [torch.randn(B, K, generator=g).to(DEV) for B in (20, 100)]
    want = [plan.run(x, packed, torch.empty(x.shape[0], N, device=DEV)) for x in xs]
    graphs, ys = [], []
    for x in xs:
        y = torch.empty(x.shape[0], N, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run(x, packed, y)
        graphs.append(graph)
        ys.append(y)
    big = torch.randn(6000, K, generator=g).to(DEV)
    plan.run(big, packed, torch.empty(6000, N, device=DEV))
    trash = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    for rep in range(3):
        for graph, y, w in zip(graphs, ys, want):
            y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, w), rep
    assert all((t == 255).all() for t in trash)
