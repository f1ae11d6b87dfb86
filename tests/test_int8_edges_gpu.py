"""Edges of the INT8 products and the row movements on the GPU: rows of experts that
break the rules, experts far down a long table, ids at any address, many choices,
counters at the border of 64 KB, calls on another stream, a row of codes at a row
of its own.  All results are exact: compared bit for bit."""

import numpy as np
import pytest
import torch

import prefill_q8_mxfp4_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def code_rows(B, K, g):
    c = torch.randint(-128, 128, (B, K), generator=g, dtype=torch.int64).to(torch.int8)
    buf = torch.zeros((B, q.code_stride(K)), dtype=torch.int8, device=DEV)
    buf[:, :K] = c.to(DEV)
    return buf[:, :K], ((torch.rand(B, generator=g) + 0.1) * 0.02).to(DEV)


def weight(N, K, g):
    c = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int64).to(torch.int8)
    return q.pack_int8(c.to(DEV), ((torch.rand(N, generator=g) + 0.1) * 1e-3).to(DEV))


def route_ref(ids, E):
    flat = ids.reshape(-1)
    kept = (flat >= 0) & (flat < E)
    off = np.zeros(E + 1, np.int64)
    off[1:] = np.cumsum(np.bincount(flat[kept], minlength=E))
    pos = np.full(flat.size, -1, np.int64)
    order = np.argsort(flat[kept], kind="stable")
    pos[np.flatnonzero(kept)[order]] = np.arange(order.size)
    return off, pos.reshape(ids.shape)


def check_route(ids, E, dids):
    off, pos = route_ref(ids, E)
    o, p = q.route(dids, E)
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(p.cpu().numpy(), pos)


# 4, 9, 10: the tile shapes of routed rows, 64, 32 and 128 rows high
@pytest.mark.parametrize("shape", [4, 9, 10])
@pytest.mark.parametrize("off,bad", [([0, 10, 5, 20, 40], {1}), ([0, 10, 20, 30, 41], {3}), ([1, 10, 20, 30, 40], {0}),
                                     ([0, -1, 20, 30, 40], {0, 1}), ([0, 10, 2 ** 31 - 1, 30, 40], {1, 2})])
def test_rows_of_an_expert_left_out(off, bad, shape, monkeypatch):
    """A bad expert's rows stay as they were, the others' are those of a dense call
    where only one expert names them."""
    N, K, T, E = 64, 128, 40, 4
    g = gen(1)
    dx, ds = code_rows(T, K, g)
    parts = [weight(N, K, g) for _ in range(E)]
    table = torch.tensor([w.data_ptr() for w in parts], dtype=torch.int64, device=DEV)
    monkeypatch.setenv("QGEMM_I8_SHAPE", str(shape))
    plan = q.Plan("int8", N, K, act="bf16", out="f32")
    q.device_status(clear=True)
    y = torch.full((T, N), 7.0, device=DEV)
    plan.run_grouped_codes(dx, ds, table, torch.tensor(off, dtype=torch.int32, device=DEV), y)
    assert q.device_status(clear=True) == q.DEV_BAD_OFFSETS
    names = [[e for e in range(E) if e not in bad and off[e] <= t < off[e + 1]] for t in range(T)]
    for t, n in enumerate(names):
        if not n:
            assert (y[t] == 7.0).all(), t
        elif len(n) == 1:
            one = plan.run_codes(dx[t:t + 1], ds[t:t + 1].clone(), parts[n[0]], torch.empty(1, N, device=DEV))
            assert torch.equal(y[t:t + 1], one), t


@pytest.mark.parametrize("shape", [None, 4, 9, 10])
@pytest.mark.parametrize("E", [1023, 1024, 1025, 2048, 2500, 4097])
def test_experts_far_down_the_table(E, shape, monkeypatch):
    """Rows of experts on both sides of every step of the scan over the offsets."""
    N, K = 32, 64
    g = gen(E)
    counts = np.zeros(E, np.int64)
    for e, n in ((0, 3), (511, 1), (512, 2), (1022, 1), (1023, 70), (1024, 1), (1025, 33), (2047, 2), (2048, 5),
                 (2499, 130), (4095, 1), (4096, 4), (E - 1, 9)):
        if e < E:
            counts[e] = n
    T = int(counts.sum())
    off = np.concatenate([[0], np.cumsum(counts)])
    dx, ds = code_rows(T, K, g)
    parts = [weight(N, K, g) for _ in range(5)]
    table = torch.tensor([parts[e % 5].data_ptr() for e in range(E)], dtype=torch.int64, device=DEV)
    if shape is not None:
        monkeypatch.setenv("QGEMM_I8_SHAPE", str(shape))
    plan = q.Plan("int8", N, K, act="bf16", out="f32")
    y = plan.run_grouped_codes(dx, ds, table, torch.tensor(off, dtype=torch.int32, device=DEV),
                               torch.full((T, N), 7.0, device=DEV))
    assert q.device_status() & q.DEV_BAD_OFFSETS == 0
    for e in np.flatnonzero(counts):
        a, b = int(off[e]), int(off[e + 1])
        one = plan.run_codes(dx[a:b], ds[a:b].clone(), parts[e % 5], torch.empty(b - a, N, device=DEV))
        assert torch.equal(y[a:b], one), e


@pytest.mark.parametrize("T,k,E", [(1, 1, 3), (63, 3, 37), (2048, 10, 512), (20000, 8, 129)])
def test_route_of_ids_at_any_address(T, k, E):
    """ids that begin 4, 8 or 12 bytes past a multiple of 16."""
    ids = np.random.default_rng(T).integers(-1, E + 1, (T, k))
    for shift in (1, 2, 3):
        buf = torch.zeros(T * k + shift, dtype=torch.int32, device=DEV)
        view = buf[shift:].view(T, k)
        view.copy_(torch.from_numpy(ids.astype(np.int32)))
        assert view.is_contiguous() and view.data_ptr() % 16 == 4 * shift
        check_route(ids, E, view)


@pytest.mark.parametrize("T,k,E,one", [(32768, 8, 64, False), (40000, 8, 64, False), (40000, 8, 64, True),
                                       (70001, 5, 300, False)])
def test_route_of_many_choices(T, k, E, one):
    """More than 262144 choices: a workgroup places more than 1024 of them, in turns."""
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E, (T, k))
    if one:
        ids[rng.random((T, k)) < 0.9] = 3
    check_route(ids, E, torch.from_numpy(ids.astype(np.int32)).to(DEV))


@pytest.mark.parametrize("E", [8184, 8185, 8191, 8192, 8193])
def test_route_counters_at_64_kilobytes(E):
    ids = np.random.default_rng(E).integers(0, E, (500, 2))
    ids[0, 0], ids[1, 1] = 0, E - 1
    check_route(ids, E, torch.from_numpy(ids.astype(np.int32)).to(DEV))


def test_layer_on_an_explicit_stream():
    """One expert layer on a stream that is not the current one, every buffer made
    before that stream waits for the current one, the others by the binding."""
    T, k, E, H, nh = 70, 3, 8, 256, 48
    R, g = T * k, gen(4)
    gu, dn = [weight(2 * nh, H, g) for _ in range(E)], [weight(H, nh, g) for _ in range(E)]
    gt, dt = (torch.tensor([w.data_ptr() for w in ws], dtype=torch.int64, device=DEV) for ws in (gu, dn))
    gp = q.Plan("int8", 2 * nh, H, act="bf16", out="bf16", epilogue="swiglu")
    dp = q.Plan("int8", H, nh, act="bf16", out="bf16")
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32).to(DEV)
    wts = torch.rand(T, k, generator=g).to(DEV)

    def run(st):
        codes, scales = torch.zeros((R, H), dtype=torch.int8, device=DEV), torch.zeros(R, device=DEV)
        h = torch.zeros(R, nh, dtype=torch.bfloat16, device=DEV)
        ys, y = torch.zeros(R, H, dtype=torch.bfloat16, device=DEV), torch.zeros_like(x)
        if st is not None:
            st.wait_stream(torch.cuda.current_stream())
        off, pos = q.route(ids, E, stream=st)
        q.dispatch_codes(x, pos, codes, scales, stream=st)
        gp.run_grouped_codes(codes, scales, gt, off, h, stream=st)
        hc, hs = q.quantize_rows(h, stream=st)
        dp.run_grouped_codes(hc, hs, dt, off, ys, stream=st)
        q.combine(ys, pos, wts, y, stream=st)
        dense = gp.run(x, gu[0], torch.empty(T, nh, dtype=torch.bfloat16, device=DEV) if st is None else keep, stream=st)
        if st is not None:
            torch.cuda.current_stream().wait_stream(st)
        for t in (off, pos, hc, hs):
            t.record_stream(torch.cuda.current_stream())
        return off, pos, hc.clone(), hs, y, dense

    want = run(None)
    side, keep = torch.cuda.Stream(), torch.zeros(T, nh, dtype=torch.bfloat16, device=DEV)
    for _ in range(3):
        got = run(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_one_row_leaves_the_next_alone():
    """The padding of a single row of codes is its own."""
    K = 20
    buf = torch.full((4, 48), 9, dtype=torch.int8, device=DEV)
    x = torch.randn(1, K, generator=gen(2)).to(DEV)
    c, s = q.quantize_rows(x)
    q.quantize_rows(x, buf[1:2, :K], torch.empty(1, device=DEV))
    want = torch.full((4, 48), 9, dtype=torch.int8, device=DEV)
    want[1] = 0
    want[1, :K] = c[0]
    assert torch.equal(buf, want)
    dense = torch.full((4, K), 9, dtype=torch.int8, device=DEV)
    with pytest.raises(ValueError, match="pitch"):
        q.quantize_rows(x, dense[:1], s)
    torch.cuda.synchronize()
    assert (dense == 9).all()


def test_weights_past_four_gigabytes():
    """2^20 channels of 8192: the last channels lie 8 GB into the packed weights."""
    N, K, tail = 1 << 20, 8192, 512
    g = torch.Generator(device=DEV).manual_seed(6)
    cw = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=DEV, generator=g)
    sw = torch.rand(N, device=DEV, generator=g) * 1e-3
    w, last = q.pack_int8(cw, sw), q.pack_int8(cw[-tail:], sw[-tail:])
    del cw
    wide, narrow = q.Plan("int8", N, K, act="bf16", out="bf16"), q.Plan("int8", tail, K, act="bf16", out="bf16")
    for B in (1, 4, 70, 300):
        x = torch.randn(B, K, device=DEV, generator=g).to(torch.bfloat16)
        y = wide.run(x, w, torch.empty(B, N, dtype=torch.bfloat16, device=DEV))
        want = narrow.run(x, last, torch.empty(B, tail, dtype=torch.bfloat16, device=DEV))
        assert torch.equal(y[:, -tail:], want), B


def test_rows_past_four_gigabytes():
    """140000 sorted rows of 8192 fp32, 4.6 GB: the ends of both sides of each move."""
    T, k, H = 70000, 2, 8192
    R = T * k
    g = torch.Generator(device=DEV).manual_seed(7)
    pos = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=DEV).view(T, k)  # backwards: token 0 goes last
    x = torch.randn(T, H, device=DEV, generator=g)
    xs = q.dispatch(x, pos, torch.empty(R, H, device=DEV))
    tokens = [0, 1, T // 2, T - 1]
    for t in tokens:
        for j in range(k):
            assert torch.equal(xs[R - 1 - (t * k + j)], x[t]), (t, j)
    wts = torch.full((T, k), 0.5, device=DEV)
    y = q.combine(xs, pos, wts, torch.empty(T, H, device=DEV))       # 0.5 x + 0.5 x, exact
    assert torch.equal(y, x)
    dys, dw = q.combine_grad(x, xs, pos, wts, torch.zeros(R, H, device=DEV), torch.empty(T, k, device=DEV))
    for t in tokens:
        for j in range(k):
            assert torch.equal(dys[R - 1 - (t * k + j)], 0.5 * x[t]), (t, j)
    assert torch.equal(dw[:, 0], dw[:, 1])
    del dys, xs, y
    codes, scales = torch.empty((R, H), dtype=torch.int8, device=DEV), torch.empty(R, device=DEV)
    q.dispatch_codes(x, pos, codes, scales)
    for t in tokens:
        c, s = q.quantize_rows(x[t:t + 1])
        for j in range(k):
            r = R - 1 - (t * k + j)
            assert torch.equal(codes[r], c[0]) and scales[r] == s[0], (t, j)
    big = x.repeat(2, 1)                                            # 4.6 GB of rows
    c, s = q.quantize_rows(big)
    assert torch.equal(c[:T], c[T:]) and torch.equal(s[:T], s[T:])
    assert torch.equal(c[0], codes[R - 1]) and s[-1] == scales[0]
    assert q.device_status() & q.DEV_BAD_ROUTE == 0
