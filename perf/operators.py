"""The 8-bit integer operators, as cases that can be timed and compared.

Kinds of case:

* ``product``: rows times an int8 weight with one scale a channel.  Rows come
  as fp32 or bf16 and are quantised in the call, one scale a token, or as
  codes that an earlier call made (``codes``).  ``swiglu`` fuses gate and up.
* ``experts``: the same product for rows sorted by expert.
* ``sort``: expert ids to sorted positions, rows to their experts and back
  with the router's weights.
* ``backward``: the gradients of the two row movements and of the weights.
* ``layer``: a whole expert layer: sort, quantise on the way, gate and up,
  quantise, down, back with weights.

With ``own`` false, ``run`` computes plain torch forms in fp32; with it true,
the library's entry points.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ESZ = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token through an attention projection: latency
        {"name": "product decode", "kind": "product", "B": 1, "N": 5120, "K": 5120, "act": "bf16", "out": "bf16",
         "swiglu": False, "codes": False},
        # draft tokens verified in the down projection, fp32 rows
        {"name": "product verify", "kind": "product", "B": 70, "N": 5120, "K": 17408, "act": "f32", "out": "f32",
         "swiglu": False, "codes": False},
        # a prompt chunk through the fused gate and up projection
        {"name": "product prompt", "kind": "product", "B": 2048, "N": 34816, "K": 5120, "act": "bf16", "out": "bf16",
         "swiglu": True, "codes": False},
        # an odd batch of codes from an earlier call, odd sizes throughout
        {"name": "product ragged", "kind": "product", "B": 301, "N": 4999, "K": 2729, "act": "bf16", "out": "f32",
         "swiglu": False, "codes": True},
        # sixteen sequences, one token each: few rows for each of a few experts
        {"name": "experts decode", "kind": "experts", "T": 16, "topk": 10, "E": 512, "N": 1024, "K": 2048,
         "out": "bf16", "swiglu": True, "drop": 0.0},
        # a prompt chunk through all experts, a share of the choices on another device
        {"name": "experts prompt", "kind": "experts", "T": 2048, "topk": 10, "E": 512, "N": 1024, "K": 2048,
         "out": "bf16", "swiglu": True, "drop": 0.1},
        # a prompt chunk's rows to their experts and back
        {"name": "sort prompt", "kind": "sort", "T": 2048, "topk": 10, "E": 512, "H": 2048, "act": "bf16",
         "drop": 0.0},
        # odd sizes, fp32, choices on another device
        {"name": "sort ragged", "kind": "sort", "T": 777, "topk": 3, "E": 37, "H": 1021, "act": "f32", "drop": 0.25},
        # the gradients of a training batch
        {"name": "backward prompt", "kind": "backward", "T": 2048, "topk": 10, "E": 512, "H": 2048, "act": "bf16",
         "drop": 0.0},
        {"name": "backward ragged", "kind": "backward", "T": 777, "topk": 3, "E": 37, "H": 1021, "act": "f32",
         "drop": 0.25},
        # the whole layer, for one token of each of sixteen sequences and for a prompt chunk
        {"name": "layer decode", "kind": "layer", "T": 16, "topk": 10, "E": 512, "H": 2048, "nh": 512, "act": "bf16",
         "drop": 0.0},
        {"name": "layer prompt", "kind": "layer", "T": 2048, "topk": 10, "E": 512, "H": 2048, "nh": 512,
         "act": "bf16", "drop": 0.0},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["product", "product", "experts", "sort", "backward", "layer"])
    act, out, swiglu = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]), rng.random() < 0.4
    drop = rng.choice([0.0, 0.0, 0.05, 0.3, 0.6])
    if kind == "product":
        while True:
            B, N, K = _log(rng, 1, 4096), _log(rng, 48, 34816), _log(rng, 33, 17408)
            if B * N * K <= 2048 * 34816 * 5120 and N * K <= 34816 * 5120:
                break
        if swiglu:
            N = max(32, N // 32 * 32)
        return {"kind": kind, "B": B, "N": N, "K": K, "act": act, "out": out, "swiglu": swiglu,
                "codes": rng.random() < 0.3}
    E = _log(rng, 2, 512)
    topk = rng.randint(1, min(10, E))
    if kind == "experts":
        while True:
            T, N, K = _log(rng, 1, 2048), _log(rng, 48, 2048), _log(rng, 33, 4096)
            if E * N * K <= 512 * 1024 * 2048 and T * topk <= 20480 and T * topk * N * K <= 20480 * 1024 * 2048:
                break
        if swiglu:
            N = max(32, N // 32 * 32)
        return {"kind": kind, "T": T, "topk": topk, "E": E, "N": N, "K": K, "out": out, "swiglu": swiglu,
                "drop": drop}
    if kind == "layer":
        while True:
            T, H, nh = _log(rng, 1, 2048), _log(rng, 64, 2048), _log(rng, 16, 1024) // 16 * 16
            if E * H * nh <= 512 * 512 * 2048 and T * topk * H * nh <= 20480 * 512 * 2048:
                break
        # fp32 outputs would hang on which way a bf16 value between the two products is rounded
        return {"kind": kind, "T": T, "topk": topk, "E": E, "H": H, "nh": nh, "act": "bf16", "drop": drop}
    while True:
        T, H = _log(rng, 1, 8192), _log(rng, 16, 5120)
        if T * topk * H <= 20480 * 2048:
            break
    return {"kind": kind, "T": T, "topk": topk, "E": E, "H": H, "act": act, "drop": drop}


# ------------------------------------------------------------------ inputs

def _rows(g, B, K, dtype):
    """Activation rows: tokens of different size, a few large channels."""
    x = torch.randn(B, K, device="cuda", generator=g)
    x *= torch.exp(torch.randn(B, 1, device="cuda", generator=g) * 0.5)
    x *= 1.0 + 15.0 * (torch.rand(1, K, device="cuda", generator=g) < 0.002)
    return x.to(dtype)


def _weight_codes(g, *shape):
    return (torch.randn(*shape, device="cuda", generator=g) * 33.0).round_().clamp_(-127, 127).to(torch.int8)


def _weight_scales(g, *shape):
    return (0.5 + torch.rand(*shape, device="cuda", generator=g)) * 6e-4


def _ids(g, c):
    """topk distinct experts for each token, some experts liked more than
    others; a share `drop` of the choices is -1 (an expert held elsewhere)."""
    liked = torch.randn(c["E"], device="cuda", generator=g) * 0.3
    key = torch.rand(c["T"], c["E"], device="cuda", generator=g) + 0.3 * liked
    ids = torch.topk(key, c["topk"], dim=1).indices.to(torch.int32)
    gone = torch.rand(c["T"], c["topk"], device="cuda", generator=g) < c["drop"]
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def _router_weights(g, c):
    return torch.softmax(torch.randn(c["T"], c["topk"], device="cuda", generator=g), dim=1).contiguous()


def _experts_packed(codes, scales):
    """Packed weights of every expert in one buffer, and the address table."""
    import prefill_q8_mxfp4_amd as q

    E, N, K = codes.shape
    nb = q.weight_bytes("int8", N, K)
    buf = torch.empty(E, nb, dtype=torch.uint8, device="cuda")
    for e in range(E):
        q.pack_int8(codes[e], scales[e], buf[e])
    table = torch.arange(E, dtype=torch.int64, device="cuda") * nb + buf.data_ptr()
    return buf, table


def _codes_buffer(R, K):
    """Room for R rows of K codes, rows 16-byte aligned."""
    return torch.zeros(R, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["kind"] == "product":
        B, N, K = c["B"], c["N"], c["K"]
        s["x"] = _rows(g, B, K, DT[c["act"]])
        wq, wsc = _weight_codes(g, N, K), _weight_scales(g, N)
        if c["codes"]:
            xs = s["x"].float().abs().amax(1) / torch.full((B,), 127.0, device="cuda")
            cod = (s.pop("x").float() / xs[:, None]).round().clamp(-127, 127).to(torch.int8)
            s["codes"], s["scales"] = _codes_buffer(B, K), xs
            s["codes"].copy_(cod)
        if own:
            import prefill_q8_mxfp4_amd as q

            s["w"] = q.pack_int8(wq, wsc)
            s["plan"] = q.Plan("int8", N, K, act=c["act"], out=c["out"],
                               epilogue="swiglu" if c["swiglu"] else "none")
            s["y"] = torch.empty(B, N // 2 if c["swiglu"] else N, dtype=DT[c["out"]], device="cuda")
        else:
            s["wq"], s["ws"] = wq, wsc
        return s
    T, k, E = c["T"], c["topk"], c["E"]
    R = T * k
    ids = _ids(g, c)
    if c["kind"] == "experts":
        N, K = c["N"], c["K"]
        counts = torch.bincount(ids[ids >= 0].long(), minlength=E)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.cumsum(counts, 0)
        s["offsets"], s["most"] = off, max(1, int(counts.max()))
        x = _rows(g, R, K, torch.bfloat16).float()
        xs = x.abs().amax(1) / torch.full((R,), 127.0, device="cuda")
        s["codes"], s["scales"] = _codes_buffer(R, K), xs
        s["codes"].copy_((x / xs[:, None]).round().clamp(-127, 127).to(torch.int8))
        wq, wsc = _weight_codes(g, E, N, K), _weight_scales(g, E, N)
        nout = N // 2 if c["swiglu"] else N
        if own:
            import prefill_q8_mxfp4_amd as q

            s["w"], s["table"] = _experts_packed(wq, wsc)
            s["plan"] = q.Plan("int8", N, K, act="bf16", out=c["out"],
                               epilogue="swiglu" if c["swiglu"] else "none")
            s["y"] = torch.zeros(R, nout, dtype=DT[c["out"]], device="cuda")
        else:
            s["wq"], s["ws"] = wq, wsc
        return s
    H, dt = c["H"], DT[c["act"]]
    s["ids"], s["weights"] = ids, _router_weights(g, c)
    if c["kind"] == "sort":
        s["x"] = _rows(g, T, H, dt)
        s["ys"] = _rows(g, R, H, dt)
        if own:
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            s["pos"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["xs"] = torch.zeros(R, H, dtype=dt, device="cuda")
            s["y"] = torch.empty(T, H, dtype=dt, device="cuda")
        return s
    if c["kind"] == "backward":
        s["pos"] = _plain_route(ids, E)[1]
        s["dy"] = torch.randn(T, H, device="cuda", generator=g).to(dt)
        s["ys"] = _rows(g, R, H, dt)
        s["dxs"] = torch.randn(R, H, device="cuda", generator=g).to(dt)
        if own:
            s["dys"] = torch.zeros(R, H, dtype=dt, device="cuda")
            s["dw"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
            s["dx"] = torch.empty(T, H, dtype=dt, device="cuda")
        return s
    nh = c["nh"]
    s["x"] = _rows(g, T, H, dt)
    s["most"] = max(1, int(torch.bincount(ids[ids >= 0].long(), minlength=E).max()))
    gu, gus = _weight_codes(g, E, 2 * nh, H), _weight_scales(g, E, 2 * nh)
    dn, dns = _weight_codes(g, E, H, nh), _weight_scales(g, E, H)
    if own:
        import prefill_q8_mxfp4_amd as q

        s["gu"], s["gu_table"] = _experts_packed(gu, gus)
        s["dn"], s["dn_table"] = _experts_packed(dn, dns)
        s["gu_plan"] = q.Plan("int8", 2 * nh, H, act=c["act"], out="bf16", epilogue="swiglu")
        s["dn_plan"] = q.Plan("int8", H, nh, act="bf16", out=c["act"])
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["pos"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["codes"], s["scales"] = _codes_buffer(R, H), torch.zeros(R, device="cuda")
        s["h"] = torch.zeros(R, nh, dtype=torch.bfloat16, device="cuda")
        s["hcodes"], s["hscales"] = _codes_buffer(R, nh), torch.zeros(R, device="cuda")
        s["ys"] = torch.zeros(R, H, dtype=dt, device="cuda")
        s["y"] = torch.empty(T, H, dtype=dt, device="cuda")
    else:
        s["gu"], s["gus"], s["dn"], s["dns"] = gu, gus, dn, dns
    return s


# ------------------------------------------------------------- plain forms

def _plain_quantize(x):
    """Codes (as fp32) and the scale of each row."""
    x = x.float()
    amax = x.abs().amax(1)
    sc = amax / torch.full_like(amax, 127.0)
    cod = (x / sc[:, None]).round().clamp(-127, 127)
    return torch.where(sc[:, None] > 0, cod, torch.zeros_like(cod)), sc


def _plain_swiglu(y):
    nh = y.shape[-1] // 2
    gate, up = y[..., :nh], y[..., nh:]
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_route(ids, E):
    """Offsets and positions: a stable sort of the kept choices by expert."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    pos = torch.where(kept, place, torch.full_like(place, -1)).to(torch.int32).reshape(ids.shape)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))
    off = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    off[1:] = torch.cumsum(counts[:E], 0)
    return off, pos


def _plain_experts(cod, xs, wq, ws, off, most):
    """acc * scales in fp32 for rows sorted by expert; rows behind the last are zero.
    Few rows: each with its own copy of its expert's weight; else rows padded
    to the fullest expert and one batched product."""
    R, (E, N, K) = cod.shape[0], wq.shape
    r = torch.arange(R, device=cod.device)
    e = torch.searchsorted(off[1:].long().contiguous(), r, right=True)
    valid, e = e < E, e.clamp(max=E - 1)
    if 2 * R <= E:
        acc = torch.bmm(wq[e].float(), cod.float()[:, :, None]).squeeze(2)
    else:
        slot = (r - off.long()[e]).clamp(max=most)
        slot = torch.where(valid, slot, torch.full_like(slot, most))
        xp = torch.zeros(E, most + 1, K, device=cod.device)
        xp[e, slot] = cod.float()
        acc = torch.bmm(wq.float(), xp.transpose(1, 2).contiguous()).transpose(1, 2)[e, slot]
    return torch.where(valid[:, None], acc * xs[:, None] * ws[e], torch.zeros_like(acc))


def _plain_gather(rows, pos):
    """rows[pos] as fp32 [T, k, H], zero where a choice was dropped."""
    got = rows[pos.long().clamp(min=0)].float()
    return torch.where((pos >= 0)[:, :, None], got, torch.zeros_like(got))


def _plain_scatter(values, pos, R):
    """out[pos[t, j]] = values[t, j]; rows no choice names are zero."""
    out = torch.zeros(R + 1, values.shape[-1], dtype=values.dtype, device=values.device)
    at = torch.where(pos >= 0, pos.long(), torch.full_like(pos, R, dtype=torch.int64))
    out[at.reshape(-1)] = values.reshape(-1, values.shape[-1])
    return out[:R]


def _run_plain(s):
    c = s["case"]
    if c["kind"] == "product":
        cod, xs = (s["codes"].float(), s["scales"]) if c["codes"] else _plain_quantize(s["x"])
        y = (cod @ s["wq"].float().t()) * xs[:, None] * s["ws"][None, :]
        return (_plain_swiglu(y) if c["swiglu"] else y).to(DT[c["out"]])
    if c["kind"] == "experts":
        y = _plain_experts(s["codes"], s["scales"], s["wq"], s["ws"], s["offsets"], s["most"])
        return (_plain_swiglu(y) if c["swiglu"] else y).to(DT[c["out"]])
    T, k, dt = c["T"], c["topk"], DT[c["act"]]
    if c["kind"] == "sort":
        off, pos = _plain_route(s["ids"], c["E"])
        xs = _plain_scatter(s["x"][:, None, :].expand(T, k, c["H"]), pos, T * k)
        y = (s["weights"][:, :, None] * _plain_gather(s["ys"], pos)).sum(1).to(dt)
        return {"offsets": off, "pos": pos, "xs": xs, "y": y}
    if c["kind"] == "backward":
        pos, dy = s["pos"], s["dy"].float()
        dys = _plain_scatter((s["weights"][:, :, None] * dy[:, None, :]).to(dt), pos, T * k)
        dw = (dy[:, None, :] * _plain_gather(s["ys"], pos)).sum(2)
        return {"dys": dys, "dw": dw, "dx": _plain_gather(s["dxs"], pos).sum(1).to(dt)}
    off, pos = _plain_route(s["ids"], c["E"])
    cod, xs = _plain_quantize(s["x"])
    cods = _plain_scatter(cod[:, None, :].expand(T, k, c["H"]), pos, T * k)
    xss = _plain_scatter(xs[:, None, None].expand(T, k, 1), pos, T * k)[:, 0]
    h = _plain_swiglu(_plain_experts(cods, xss, s["gu"], s["gus"], off, s["most"])).to(torch.bfloat16)
    hc, hs = _plain_quantize(h)
    ys = _plain_experts(hc, hs, s["dn"], s["dns"], off, s["most"]).to(dt)
    y = (s["weights"][:, :, None] * _plain_gather(ys, pos)).sum(1).to(dt)
    return {"offsets": off, "pos": pos, "y": y}


def _run_own(s):
    import prefill_q8_mxfp4_amd as q

    c = s["case"]
    if c["kind"] == "product":
        if c["codes"]:
            return s["plan"].run_codes(s["codes"], s["scales"], s["w"], s["y"])
        return s["plan"].run(s["x"], s["w"], s["y"])
    if c["kind"] == "experts":
        return s["plan"].run_grouped_codes(s["codes"], s["scales"], s["table"], s["offsets"], s["y"])
    if c["kind"] == "sort":
        q.route(s["ids"], c["E"], s["offsets"], s["pos"])
        q.dispatch(s["x"], s["pos"], s["xs"])
        q.combine(s["ys"], s["pos"], s["weights"], s["y"])
        return {n: s[n] for n in ("offsets", "pos", "xs", "y")}
    if c["kind"] == "backward":
        q.combine_grad(s["dy"], s["ys"], s["pos"], s["weights"], s["dys"], s["dw"])
        q.dispatch_grad(s["dxs"], s["pos"], s["dx"])
        return {n: s[n] for n in ("dys", "dw", "dx")}
    q.route(s["ids"], c["E"], s["offsets"], s["pos"])
    q.dispatch_codes(s["x"], s["pos"], s["codes"], s["scales"])
    s["gu_plan"].run_grouped_codes(s["codes"], s["scales"], s["gu_table"], s["offsets"], s["h"])
    q.quantize_rows(s["h"], s["hcodes"], s["hscales"])
    s["dn_plan"].run_grouped_codes(s["hcodes"], s["hscales"], s["dn_table"], s["offsets"], s["ys"])
    q.combine(s["ys"], s["pos"], s["weights"], s["y"])
    return {n: s[n] for n in ("offsets", "pos", "y")}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------- work

def _used(c):
    """Experts that some kept choice names, as expected of even choices."""
    return c["E"] * (1.0 - (1.0 - c["topk"] * (1.0 - c["drop"]) / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["kind"] == "product":
        B, N, K = c["B"], c["N"], c["K"]
        nout = N // 2 if c["swiglu"] else N
        rows = B * K + 4 * B if c["codes"] else B * K * ESZ[c["act"]]
        return {"bytes": N * K + 4 * N + rows + B * nout * ESZ[c["out"]], "flops": 2.0 * B * N * K}
    T, k = c["T"], c["topk"]
    R = T * k * (1.0 - c["drop"])
    if c["kind"] == "experts":
        N, K = c["N"], c["K"]
        nout = N // 2 if c["swiglu"] else N
        return {"bytes": _used(c) * N * (K + 4) + R * (K + 4) + R * nout * ESZ[c["out"]] + 4 * c["E"],
                "flops": 2.0 * R * N * K}
    H, e = c["H"], ESZ[c["act"]]
    if c["kind"] == "sort":
        return {"bytes": 12.0 * T * k + 4 * c["E"] + 2 * e * H * (T + R), "flops": 2.0 * R * H}
    if c["kind"] == "backward":
        return {"bytes": 12.0 * T * k + e * H * (2 * T + 3 * R), "flops": 4.0 * R * H}
    return {"bytes": 12.0 * T * k + 4 * c["E"] + 2 * e * H * T + _used(c) * 3 * c["nh"] * H,
            "flops": 6.0 * R * c["nh"] * H}


# ------------------------------------------------- the definition, in 64 bits

def _exact_codes(x):
    x = x.double()
    sc = (x.abs().amax(1) / 127.0).float().double()  # the scale is held in fp32
    safe = torch.where(sc > 0, sc, torch.ones_like(sc))
    quotient = (x / safe[:, None]).float().double()  # and so is the quotient that is rounded
    return torch.round(quotient).clamp(-127, 127) * (sc > 0)[:, None], sc


def _exact_act(y, swiglu):
    if not swiglu:
        return y
    half = y.shape[-1] // 2
    return y[..., :half] * torch.sigmoid(y[..., :half]) * y[..., half:]


def _exact_order(ids, E):
    """For each expert the flat choices that name it, in order."""
    flat = ids.reshape(-1).cpu().tolist()
    lists = [[] for _ in range(E)]
    for f, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(f)
    return lists


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["kind"] == "product":
        if c["codes"]:
            cod, xs = s["codes"].double(), s["scales"].double()
        else:
            cod, xs = _exact_codes(s["x"])
        w = s["wq"].double() * s["ws"].double()[:, None]
        return _exact_act(torch.mm(cod * xs[:, None], w.t()), c["swiglu"])
    if c["kind"] == "experts":
        off = s["offsets"].cpu().tolist()
        nout = c["N"] // 2 if c["swiglu"] else c["N"]
        y = torch.zeros(s["codes"].shape[0], nout, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            if b > a:
                w = s["wq"][e].double() * s["ws"][e].double()[:, None]
                y[a:b] = _exact_act((s["codes"][a:b].double() * s["scales"][a:b].double()[:, None]) @ w.t(),
                                    c["swiglu"])
        return y
    T, k, H = c["T"], c["topk"], c["H"]
    lists = _exact_order(s["ids"], c["E"])
    order = torch.tensor([f for one in lists for f in one], dtype=torch.int64, device="cuda")
    kept = order.numel()
    wflat = s["weights"].double().reshape(-1)
    if c["kind"] == "sort":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        y.index_add_(0, order // k, wflat[order][:, None] * s["ys"][:kept].double())
        xs = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        xs[:kept] = s["x"].double()[order // k]
        return {"offsets": None, "pos": None, "xs": xs, "y": y}
    if c["kind"] == "backward":
        dys = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        dys[:kept] = wflat[order][:, None] * s["dy"].double()[order // k]
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dw[order] = (s["dy"].double()[order // k] * s["ys"][:kept].double()).sum(1)
        dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        dx.index_add_(0, order // k, s["dxs"][:kept].double())
        return {"dys": dys, "dw": dw.reshape(T, k), "dx": dx}
    cod, xs = _exact_codes(s["x"])
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e, one in enumerate(lists):
        if one:
            f = torch.tensor(one, dtype=torch.int64, device="cuda")
            gate_up = (cod[f // k] @ s["gu"][e].double().t()) * xs[f // k][:, None] * s["gus"][e].double()
            hc, hs = _exact_codes(_exact_act(gate_up, True).to(torch.bfloat16))
            down = (hc @ s["dn"][e].double().t()) * hs[:, None] * s["dns"][e].double()
            y.index_add_(0, f // k, wflat[f][:, None] * down)
    return {"offsets": None, "pos": None, "y": y}
