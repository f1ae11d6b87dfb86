"""The 8-bit integer format and the row movements without a GPU: packed
layout, plans and their tiers, and the refusals, all before any HIP call."""

import ctypes

import numpy as np
import pytest
import torch

import prefill_q8_mxfp4_amd as q

P16 = 0x10000  # stands for a 16-byte aligned device address; never followed


def test_pack_layout_roundtrip():
    rng = np.random.default_rng(3)
    for n, k in ((37, 96), (16, 128), (1, 1), (50, 131), (33, 1000)):
        codes = rng.integers(-128, 128, (n, k)).astype(np.int8)
        scales = rng.standard_normal(n).astype(np.float32)
        buf = q.pack("int8", n, k, codes, scales)
        npad, kpad = -(-n // 16) * 16, -(-k // 256) * 256
        soff = -(-npad * kpad // 256) * 256
        assert buf.size == q.weight_bytes("int8", n, k) == soff + -(-npad * 4 // 256) * 256
        # [row tile][slab][k group][row][16 codes]
        body = buf[:npad * kpad].view(np.int8).reshape(npad // 16, kpad // 64, 4, 16, 16)
        full = body.transpose(0, 3, 1, 2, 4).reshape(npad, kpad)
        assert np.array_equal(full[:n, :k], codes)
        assert not full[n:].any() and not full[:, k:].any()
        sc = buf[soff:soff + npad * 4].view(np.float32)
        assert np.array_equal(sc[:n], scales) and not sc[n:].any()


def test_pack_refusals():
    codes, scales = np.zeros((16, 32), np.int8), np.ones(16, np.float32)
    for bad in (np.ones((16, 1), np.float32), np.ones(16, np.float64), np.ones(15, np.float32)):
        with pytest.raises(q.QgemmError):
            q.pack("int8", 16, 32, codes, bad)
    with pytest.raises(q.QgemmError):
        q.pack("int8", 16, 32, codes, scales, np.ones(1, np.float32))  # tensor scales are NVFP4's
    assert q.weight_bytes("int8", 0, 32) == 0 and q.weight_bytes("int8", 16, 0) == 0


def _create(*args):
    h = ctypes.c_void_p()
    return q.lib().qgemm_create(ctypes.byref(h), *args), h


@pytest.mark.parametrize("args,status", [
    # fmt, act, out, epilogue, math, N, K, flags
    ((4, 0, 0, 0, 2, 256, 512, 0), q.OK),
    ((4, 1, 1, 0, 2, 7, 1, 0), q.OK),                  # any K
    ((4, 1, 1, 1, 2, 64, 513, 0), q.OK),               # fused gate+up
    ((4, 1, 1, 1, 2, 40, 512, 0), q.ENOTSUP),          # N/2 % 16
    ((4, 1, 1, 1, 2, 33, 512, 0), q.EINVAL),           # odd N
    ((4, 0, 0, 0, 0, 256, 512, 0), q.EINVAL),          # fp32 math
    ((4, 1, 0, 0, 1, 256, 512, 0), q.EINVAL),          # bf16 math
    ((0, 0, 0, 0, 2, 256, 512, 0), q.EINVAL),          # int8 math of other weights
    ((5, 0, 0, 0, 2, 256, 512, 0), q.EINVAL),          # unknown format
    ((4, 0, 0, 0, 3, 256, 512, 0), q.EINVAL),          # unknown math
    ((4, 0, 0, 0, 2, 256, 131071, 0), q.OK),           # largest K
    ((4, 0, 0, 0, 2, 256, 131072, 0), q.EINVAL),       # 2^31 does not fit
    ((4, 0, 0, 0, 2, 256, 512, 1), q.OK),
    ((4, 0, 0, 0, 2, 256, 512, 2), q.OK),
    ((4, 0, 0, 0, 2, 256, 512, 4), q.ENOTSUP),         # no GEMV tier
])
def test_create(args, status):
    st, h = _create(*args)
    assert st == status, q.lib().qgemm_last_error()
    if st == q.OK:
        assert q.lib().qgemm_destroy(h) == q.OK


def test_tiers():
    p = q.Plan("int8", 5120, 5120, act="bf16")
    assert p.math == "int8"
    assert p.tier(1) == "skinny" and p.tier(4096) == "tiled"
    assert p.grouped_tier(512, 160) == "tiled" and p.grouped_tier(4, 4096) == "tiled"
    assert q.Plan("int8", 64, 64, tier="tiled").tier(1) == "tiled"
    assert q.Plan("int8", 64, 64, tier="tiled").grouped_tier(8, 8) == "tiled"
    assert q.Plan("int8", 64, 64, tier="skinny").tier(4096) == "skinny"
    assert p.workspace_bytes(0) == 0
    # the quantised rows at least: codes and a scale each
    for B in (1, 64, 65, 2048):
        assert p.workspace_bytes(B) >= B * (5120 + 4)


def test_run_refusals():
    L = q.lib()
    st, h = _create(4, 1, 1, 0, 2, 256, 512, 0)
    assert st == q.OK
    run, codes = L.qgemm_run, L.qgemm_run_codes
    assert run(h, 0, None, None, None, None) == q.OK
    assert run(h, 4, P16, P16, P16, None) == q.ENOTSUP          # needs a workspace
    assert L.qgemm_run_ws(h, 4, P16, P16, P16, P16, 64, None) == q.ENOTSUP
    assert L.qgemm_run_grouped(h, 4, 4, P16, P16, P16, P16, None) == q.ENOTSUP
    good = [h, 4, P16, P16, 512, P16, P16, None, 0, None]

    def but(i, v):
        a = list(good)
        a[i] = v
        return codes(*a)

    assert codes(h, 0, None, None, 512, None, None, None, 0, None) == q.OK
    assert but(0, None) == q.EINVAL
    for i in (2, 3, 5, 6):
        assert but(i, None) == q.EINVAL, i
    for i in (2, 3, 6):
        assert but(i, P16 + 8) == q.EINVAL, i
    assert but(5, P16 + 2) == q.EINVAL
    for ldc in (0, 496, 511, 520, 1 << 22):
        assert but(4, ldc) == q.EINVAL, ldc
    assert but(1, -1) == q.EINVAL and but(1, (1 << 30) + 1) == q.EINVAL
    assert but(1, 1 << 22) == q.EINVAL                          # 2^31 bytes of codes
    st, small = _create(4, 1, 1, 0, 2, 16, 16, 1)               # forced to the small-batch tier
    assert codes(small, 16 * 65535 + 1, P16, P16, 16, P16, P16, None, 0, None) == q.EINVAL
    L.qgemm_destroy(small)
    st, wide = _create(4, 1, 1, 0, 2, 1 << 28, 16, 0)           # workgroups of one launch
    for B in (1, 4):
        assert codes(wide, B, P16, P16, 16, P16, P16, None, 0, None) == q.EINVAL
        assert L.qgemm_run_ws(wide, B, P16, P16, P16, P16, 1 << 40, None) == q.EINVAL
    L.qgemm_destroy(wide)
    st, short = _create(4, 1, 1, 0, 2, 1, 1, 0)                 # rows of one element, 16 bytes of codes
    for B in (1 << 27, 1 << 30):
        assert L.qgemm_run_ws(short, B, P16, P16, P16, P16, 1 << 40, None) == q.EINVAL
    L.qgemm_destroy(short)
    assert but(7, P16 + 128) == q.EINVAL                        # workspace alignment
    L.qgemm_destroy(h)
    st, h = _create(0, 0, 0, 0, 0, 256, 512, 0)
    assert codes(h, 4, P16, P16, 512, P16, P16, None, 0, None) == q.ENOTSUP
    assert L.qgemm_run_grouped_codes(h, 4, 4, P16, P16, P16, 512, P16, P16, None) == q.ENOTSUP
    L.qgemm_destroy(h)


def test_grouped_refusals():
    L = q.lib()
    st, h = _create(4, 1, 1, 0, 2, 256, 512, 0)
    good = [h, 4, 10, P16, P16, P16, 512, P16, P16, None]

    def but(i, v):
        a = list(good)
        a[i] = v
        return L.qgemm_run_grouped_codes(*a)

    assert L.qgemm_run_grouped_codes(h, 4, 0, None, None, None, 512, None, None, None) == q.OK
    assert but(1, 0) == q.EINVAL and but(1, (1 << 16) + 1) == q.EINVAL and but(2, -1) == q.EINVAL
    for i in (0, 3, 4, 5, 7, 8):
        assert but(i, None) == q.EINVAL, i
    assert but(3, P16 + 4) == q.EINVAL and but(4, P16 + 2) == q.EINVAL and but(5, P16 + 8) == q.EINVAL
    assert but(6, 511) == q.EINVAL
    L.qgemm_destroy(h)


def test_row_refusals():
    L = q.lib()
    good = [1, 4, 512, P16, P16, 512, P16, None]

    def but(i, v):
        a = list(good)
        a[i] = v
        return L.qgemm_quantize_rows(*a)

    assert L.qgemm_quantize_rows(1, 0, 512, None, None, 512, None, None) == q.OK
    assert but(0, 2) == q.EINVAL and but(1, -1) == q.EINVAL and but(2, 0) == q.EINVAL
    assert but(1, 1 << 26) == q.EINVAL                          # threads of one launch
    assert but(2, (1 << 20) + 1) == q.EINVAL and but(5, 510) == q.EINVAL and but(5, 496) == q.EINVAL
    for i in (3, 4, 6):
        assert but(i, None) == q.EINVAL, i
    assert but(3, P16 + 4) == q.EINVAL and but(4, P16 + 8) == q.EINVAL and but(6, P16 + 1) == q.EINVAL
    pd = [4, 256, 512, P16, P16, P16, 1 << 20, None]

    def pbut(i, v):
        a = list(pd)
        a[i] = v
        return L.qgemm_pack_device(*a)

    assert pbut(0, 0) == q.ENOTSUP and pbut(0, 9) == q.EINVAL and pbut(1, 0) == q.EINVAL
    assert pbut(2, 1 << 17) == q.EINVAL and pbut(6, 1000) == q.EINVAL
    for i in (3, 4, 5):
        assert pbut(i, None) == q.EINVAL, i
    assert pbut(5, P16 + 8) == q.EINVAL and pbut(4, P16 + 2) == q.EINVAL


def test_route_refusals():
    L = q.lib()
    assert L.qgemm_route(0, 4, 2, P16, P16, P16, None) == q.EINVAL
    assert L.qgemm_route((1 << 16) + 1, 4, 2, P16, P16, P16, None) == q.EINVAL
    assert L.qgemm_route(16385, 4, 2, P16, P16, P16, None) == q.ENOTSUP
    assert L.qgemm_route(8, -1, 2, P16, P16, P16, None) == q.EINVAL
    assert L.qgemm_route(8, 4, 0, P16, P16, P16, None) == q.EINVAL
    assert L.qgemm_route(8, 4, q.MAX_TOPK + 1, P16, P16, P16, None) == q.EINVAL
    assert L.qgemm_route(8, 1 << 25, 64, P16, P16, P16, None) == q.EINVAL
    assert L.qgemm_route(8, 4, 2, None, P16, P16, None) == q.EINVAL
    assert L.qgemm_route(8, 4, 2, P16, None, P16, None) == q.EINVAL
    assert L.qgemm_route(8, 4, 2, P16, P16, None, None) == q.EINVAL
    assert L.qgemm_route(8, 4, 2, P16, P16 + 2, P16, None) == q.EINVAL


MOVES = {  # name: (arguments, indexes of the pointers that may not be null, 16-byte aligned ones)
    "qgemm_dispatch": ([0, 4, 2, 64, 8, P16, P16, P16, None], (5, 6, 7), (5, 7)),
    "qgemm_combine": ([0, 4, 2, 64, 8, P16, P16, None, P16, None], (5, 6, 8), (5, 8)),
    "qgemm_combine_grad": ([0, 4, 2, 64, 8, P16, P16, P16, P16, P16, P16, None], (5, 6, 7, 8, 9, 10), (5, 6, 9)),
    "qgemm_dispatch_codes": ([0, 4, 2, 64, 8, P16, P16, P16, 64, P16, None], (5, 6, 7, 9), (5, 7)),
}


@pytest.mark.parametrize("name", sorted(MOVES))
def test_move_refusals(name):
    good, pointers, aligned = MOVES[name]
    f = getattr(q.lib(), name)

    def but(i, v):
        a = list(good)
        a[i] = v
        return f(*a)

    assert but(1, 0) == q.OK                                    # no tokens: nothing enqueued
    assert but(0, 2) == q.EINVAL
    for i, v in ((1, -1), (1, (1 << 30) + 1), (2, 0), (2, 65), (3, 0), (3, (1 << 20) + 1), (4, -1), (4, (1 << 30) + 1)):
        assert but(i, v) == q.EINVAL, (i, v)
    assert but(1, 1 << 26) == q.EINVAL                          # threads of one launch
    for i in pointers:
        assert but(i, None) == q.EINVAL, i
        assert but(i, P16 + 2) == q.EINVAL, i
    for i in aligned:
        assert but(i, P16 + 8) == q.EINVAL, i
    assert q.lib().qgemm_last_error().decode().startswith(name)


def test_binding_refusals():
    """Types, shapes and devices are checked before the library is called."""
    f32, bf16, i8, i32 = torch.float32, torch.bfloat16, torch.int8, torch.int32
    z = torch.zeros
    plan = q.Plan("int8", 32, 48, act="bf16", out="bf16")
    w, y, s = z(q.weight_bytes("int8", 32, 48), dtype=torch.uint8), z(4, 32, dtype=bf16), z(4)
    for codes, exc in ((z(4, 48), TypeError), (z(4, 47, dtype=i8), ValueError), (z(4, 2, 48, dtype=i8), ValueError),
                       (z(4, 49, dtype=i8)[:, :48], ValueError),          # pitch 49
                       (z(48, 4, dtype=i8).t(), ValueError)):             # columns apart
        with pytest.raises(exc):
            plan.run_codes(codes, s, w, y)
    with pytest.raises(ValueError):
        plan.run_codes(z(4 * 64 - 16, dtype=i8).as_strided((4, 48), (64, 1)), s, w, y)  # the last row's pitch
    with pytest.raises(ValueError):
        plan.run_codes(z(4, 48, dtype=i8), z(3), w, y)
    with pytest.raises(ValueError, match="CUDA"):
        plan.run_codes(z(4, 48, dtype=i8), s, w, y)                       # host tensors
    with pytest.raises(TypeError):
        q.quantize_rows(z(4, 48, dtype=torch.float16))
    with pytest.raises(ValueError):
        q.quantize_rows(z(48))
    with pytest.raises(ValueError):
        q.quantize_rows(z(4, 48), z(3, 48, dtype=i8), z(4))
    with pytest.raises(TypeError):
        q.route(z(4, 2, dtype=torch.int64), 8)
    with pytest.raises(ValueError):
        q.route(z(4, 2, dtype=i32), 8, z(8, dtype=i32))
    with pytest.raises(ValueError):
        q.route(z(4, 2, dtype=i32), 8, z(9, dtype=i32), z(2, 4, dtype=i32))
    pos = z(4, 2, dtype=i32)
    with pytest.raises(TypeError):
        q.dispatch(z(4, 64), pos, z(8, 64, dtype=bf16))
    with pytest.raises(ValueError):
        q.dispatch(z(4, 64), pos, z(8, 63))
    with pytest.raises(TypeError):
        q.dispatch(z(5, 64), pos, z(8, 64))
    with pytest.raises(TypeError):
        q.combine(z(8, 64), pos, z(4, 2, dtype=bf16), z(4, 64))
    with pytest.raises(TypeError):
        q.combine(z(8, 64), pos, z(2, 4), z(4, 64))
    with pytest.raises(ValueError):
        q.combine_grad(z(4, 64), z(8, 64), pos, z(4, 2), z(7, 64), z(4, 2))
    with pytest.raises(ValueError):
        q.pack_int8(z(16, 32, dtype=i8), z(15))
    with pytest.raises(ValueError):
        q.pack_int8(z(16, 32, dtype=i8), z(16), z(8, dtype=torch.uint8))


def test_knobs_that_name_nothing(monkeypatch):
    """A number of K pieces below one, or a tile shape there is not, leaves the
    choice as it is (a negative number of pieces would be a negative grid)."""
    def sizes():
        return [q.Plan("int8", N, K, tier="tiled").workspace_bytes(B)
                for B, N, K in ((20, 64, 17408), (64, 128, 8192), (17, 32, 100000), (70, 5120, 17408))]

    own = sizes()
    for knob, values in (("QGEMM_TI_SPLIT", ("-1", "-3", "0", "-100000")), ("QGEMM_I8_SHAPE", ("-1", "0", "11", "99"))):
        for v in values:
            monkeypatch.setenv(knob, v)
            assert sizes() == own, (knob, v)
            monkeypatch.delenv(knob)


def test_no_room_in_the_scratch_names_what_takes_the_rows():
    """Beyond the library's scratch the error names entry points of the format."""
    L = q.lib()
    st, h = _create(4, 1, 1, 0, 2, 5120, 17408, 0)
    assert L.qgemm_run_noalloc(h, 4096, P16, P16, P16, None) == q.EINVAL
    text = L.qgemm_last_error().decode()
    assert "qgemm_run_ws" in text and "qgemm_run_codes" in text and "qgemm_run " not in text + " "
    L.qgemm_destroy(h)
    st, h = _create(0, 0, 0, 0, 0, 1 << 20, 17408, 0)
    assert L.qgemm_run_noalloc(h, 16, P16, P16, P16, None) == q.EINVAL
    assert "qgemm_run " in L.qgemm_last_error().decode() + " "
    L.qgemm_destroy(h)
