"""Cases of the experts' step between the dispatch and the combine: microscaled 4-bit (MXFP4)
quantization and the grouped product on it, the whole expert step for a few tokens, and SwiGLU with
its gradient from an 8-bit checkpoint.

Each case is one call of one operator.  With `own` false, run() computes it in plain torch
operations (32 bits, one rounding at the end); with `own` true it calls the library.  exact()
computes it again from the definitions, in 64 bits.  Codes are returned as the values they stand
for.  Conventions are the library's: expert id -1 is "no expert", the rows of expert e are
packed_off[e] .. packed_off[e] + packed_cnt[e], and rows outside every segment stay as they were.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2.0, "f32": 4.0, "fp8": 1.0 + 4.0 / 128, "mxfp4": 0.5 + 1.0 / 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the 256 packed rows of a decode step (32 tokens, top 8), on the way to a 4-bit product
        {"name": "quantize_decode", "op": "quantize", "rows": 256, "H": 7168, "dt": "bf16"},
        # eight experts' f32 master weights, quantized once
        {"name": "quantize_weights", "op": "quantize", "rows": 32768, "H": 7168, "dt": "f32"},
        # first product of a decode step over 128 experts, about two rows each, with SwiGLU
        {"name": "product_decode", "op": "product", "rows": 256, "E": 128, "N": 4096, "H": 4096,
         "cap": False, "swiglu": True, "out": "bf16"},
        # odd sizes, padded segments, f32 sums
        {"name": "product_odd", "op": "product", "rows": 3001, "E": 60, "N": 1000, "H": 1056,
         "cap": True, "swiglu": False, "out": "f32"},
        # first product of a 4096-token prefill, top 8 of 64 experts
        {"name": "product_prefill", "op": "product", "rows": 32768, "E": 64, "N": 4096, "H": 7168,
         "cap": False, "swiglu": True, "out": "bf16"},
        # one token of one sequence: the weights of 8 experts are read and nothing else counts
        {"name": "layer_one_token", "op": "layer", "T": 1, "H": 6144, "I": 1024, "E": 128, "K": 8,
         "wt": "bf16", "out": "bf16", "none": False},
        # a few tokens, odd sizes, tokens without experts, f32 result
        {"name": "layer_odd", "op": "layer", "T": 7, "H": 1000, "I": 264, "E": 10, "K": 3,
         "wt": "bf16", "out": "f32", "none": True},
        # a decode step of 32 sequences with 4-bit weights
        {"name": "layer_decode", "op": "layer", "T": 32, "H": 7168, "I": 1024, "E": 128, "K": 8,
         "wt": "mxfp4", "out": "bf16", "none": False},
        # fine-tuning on a short odd batch: padded segments, f32 activations
        {"name": "swiglu_short", "op": "swiglu", "rows": 4008, "I": 1408, "dt": "f32", "cap": True},
        # one training micro-batch: 8192 tokens, top 8
        {"name": "swiglu_train", "op": "swiglu", "rows": 65536, "I": 2048, "dt": "bf16",
         "cap": False},
        # the gradient of a short batch that kept its activations in f32
        {"name": "swiglu_backward_short", "op": "swiglu_backward", "rows": 2003, "I": 776,
         "dt": "f32", "gu": "f32", "cap": False},
        # the gradient of the training micro-batch, from the 8-bit checkpoint
        {"name": "swiglu_backward_train", "op": "swiglu_backward", "rows": 65536, "I": 2048,
         "dt": "bf16", "gu": "fp8", "cap": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "layer", "swiglu", "swiglu_backward"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 32768), "H": 32 * _log_int(rng, 1, 224),
                "dt": rng.choice(["bf16", "f32"])}
    if op == "product":
        swiglu = rng.random() < 0.5
        return {"op": op, "rows": _log_int(rng, 1, 16384), "E": _log_int(rng, 1, 64),
                "N": (16 if swiglu else 8) * _log_int(rng, 2, 256),
                "H": 32 * _log_int(rng, 1, 224), "cap": rng.random() < 0.5, "swiglu": swiglu,
                "out": rng.choice(["bf16", "f32"])}
    if op == "layer":
        wt = rng.choice(["bf16", "mxfp4"])
        step = 8 if wt == "bf16" else 32
        H, inner = step * _log_int(rng, 2, 7168 // step), step * _log_int(rng, 2, 2048 // step)
        E = _log_int(rng, 1, max(1, min(256, 2700000000 // (3 * H * inner))))
        K = rng.randint(1, min(8, E))
        return {"op": op, "T": _log_int(rng, 1, 1024 // K if H * inner < 4000000 else 64), "H": H,
                "I": inner, "E": E, "K": K, "wt": wt, "out": rng.choice(["bf16", "f32"]),
                "none": rng.random() < 0.5}
    gu = rng.choice(["bf16", "f32", "fp8"]) if op == "swiglu_backward" else "fp8"
    inner = 128 * _log_int(rng, 1, 16) if gu == "fp8" else 8 * _log_int(rng, 2, 256)
    case = {"op": op, "rows": _log_int(rng, 1, 32768), "I": inner,
            "dt": rng.choice(["bf16", "f32"]), "cap": rng.random() < 0.5}
    if op == "swiglu_backward":
        case["gu"] = gu
    return case


# ---------------------------------------------------------------------------
# the formats, in 32 bits (every step but a rounding to codes is exact)
# ---------------------------------------------------------------------------

def _pow2(e):
    """2^e in 64 bits, from its bits (exp2 and pow are not exact there)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mxfp4(x):
    """x f32 [..., H] -> (e2m1 magnitudes with sign, in units of the block scale; exponents of the
    block scales).  The exponent e puts the block's largest magnitude into [3.5, 7) * 2^e."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = ((amax.view(torch.int32) + 0x200000) >> 23) - 129
    e = torch.where(amax == 0, 0, e.clamp(min=-127))
    v = b * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)
    a = v.abs()
    q = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a),
                                                               (torch.round(a / 2) * 2).clamp(max=6.0)))
    return torch.copysign(q, v), e


def _mxfp4_codes(x):
    """x f32 [..., H] -> uint8 codes [..., H/2], uint8 scales [..., H/32]."""
    q, e = _mxfp4(x)
    mag = torch.bucketize(q.abs(), torch.tensor(E2M1[:8], device=x.device))
    code = (mag + 8 * torch.signbit(q)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _mxfp4_widen(codes, scales):
    """The values of MXFP4 codes, f32 [..., H]."""
    t = torch.tensor(E2M1, device=codes.device)
    pairs = torch.stack((t.repeat(16), t.repeat_interleave(16)), -1)
    v = pairs.index_select(0, codes.reshape(-1).int()).view(*scales.shape, 32)
    s = _pow2(scales.int() - 127).float()
    return v.mul_(s.unsqueeze(-1)).flatten(-2)


def _e4m3(x):
    """x f32 [R, 2I] -> (e4m3 codes, f32 scale per 128 elements: the smallest power of two that
    keeps the block's largest magnitude within 448)."""
    b = x.unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1)
    k = ((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 135
    k = torch.where(amax == 0, 0, k.clamp(min=-126))
    s = ((127 + k) << 23).view(torch.float32)
    inv = ((127 - k) << 23).view(torch.float32)
    return (b * inv.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2), s


def _e4m3_widen(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128))
    return (v * scales.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dt, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(DTYPES[dt])


def _segments(g, rows, E, cap):
    """Experts of uneven load (a few of many have none): packed_cnt, packed_off, the number of rows
    of the buffer and the largest segment.  Compact segments leave a few rows behind the last one,
    padded ones the tails of all."""
    load = torch.softmax(0.4 * torch.randn(E, generator=g, device=DEV), 0)
    at = torch.multinomial(load, rows, replacement=True, generator=g)
    cnt = torch.bincount(at, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    if cap:
        room = max(1, int(1.3 * rows / E))
        cnt = cnt.clamp(max=room)
        off = torch.arange(E + 1, device=DEV) * room
        total = E * room
    else:
        off[1:] = torch.cumsum(cnt, 0)
        total = rows + rows // 16
    return cnt.int(), off.int(), total, int(cnt.max())


def _weights(g, E, rows, cols, wt):
    """Expert weights [E, rows, cols] of about unit gain, expert by expert."""
    w = torch.empty((E, rows, cols if wt == "bf16" else cols // 2), device=DEV,
                    dtype=torch.bfloat16 if wt == "bf16" else torch.uint8)
    s = None if wt == "bf16" else torch.empty((E, rows, cols // 32), dtype=torch.uint8, device=DEV)
    for e in range(E):
        v = _normal(g, (rows, cols), "f32", cols ** -0.5)
        if wt == "bf16":
            w[e] = v.to(torch.bfloat16)
        else:
            w[e], s[e] = _mxfp4_codes(v)
    return w, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        # rows of very different size, a few outliers
        x = _normal(g, (case["rows"], case["H"]), "f32")
        x *= torch.exp2(4.0 * torch.randn((case["rows"], 1), generator=g, device=DEV))
        x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.001, x * 64, x)
        s["x"] = x.to(DTYPES[case["dt"]])
    elif op == "product":
        s["cnt"], s["off"], total, s["most"] = _segments(g, case["rows"], case["E"], case["cap"])
        s["a"], s["as"] = _mxfp4_codes(_normal(g, (total, case["H"]), "f32"))
        s["w"], s["ws"] = _weights(g, case["E"], case["N"], case["H"], "mxfp4")
        s["y"] = torch.zeros((total, case["N"] // (2 if case["swiglu"] else 1)), device=DEV,
                             dtype=DTYPES[case["out"]])
    elif op == "layer":
        T, H, I, E, K = (case[k] for k in ("T", "H", "I", "E", "K"))
        s["x"] = _normal(g, (T, H), "bf16")
        idx = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :K].int()
        if case["none"]:     # a fifth of the entries has no expert
            idx[torch.rand((T, K), generator=g, device=DEV) < 0.2] = -1
        s["idx"] = idx.contiguous()
        s["w"] = torch.softmax(_normal(g, (T, K), "f32"), -1)
        s["w13"], s["s13"] = _weights(g, E, 2 * I, H, case["wt"])
        s["w2"], s["s2"] = _weights(g, E, H, I, case["wt"])
        s["out"] = torch.empty((T, H), dtype=DTYPES[case["out"]], device=DEV)
    else:
        rows, I = case["rows"], case["I"]
        s["cnt"] = s["off"] = None
        if case["cap"]:
            s["cnt"], s["off"], rows, _ = _segments(g, rows, min(32, rows), True)
        s["rows"] = rows
        gu = _normal(g, (rows, 2 * I), "f32", 1.5)
        h_dt = DTYPES[case["dt"]]
        if op == "swiglu":
            s["gu"] = gu.to(h_dt)
            s["h"] = torch.zeros((rows, I), dtype=h_dt, device=DEV)
            s["codes"] = torch.zeros((rows, 2 * I), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.ones((rows, 2 * I // 128), dtype=torch.float32, device=DEV)
        else:
            s["dh"] = _normal(g, (rows, I), case["dt"], 0.1)
            s["dgu"] = torch.zeros((rows, 2 * I), dtype=h_dt, device=DEV)
            s["h"] = torch.zeros((rows, I), dtype=h_dt, device=DEV)
            if case["gu"] == "fp8":
                q, s["scales"] = _e4m3(gu)
                s["gu"] = q.view(torch.uint8)
            else:
                s["gu"], s["scales"] = gu.to(DTYPES[case["gu"]]), None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_RUN_OWN if own else _RUN_PLAIN)[state["case"]["op"]](state)


def _plain_quantize(s):
    q, e = _mxfp4(s["x"].float())
    return (q * _pow2(e).float().unsqueeze(-1)).flatten(-2).to(s["x"].dtype)


def _rows_of(cnt, off, total):
    """(expert, slot, whether the expert owns it) of every row."""
    r = torch.arange(total, device=cnt.device)
    e = torch.searchsorted(off.long(), r, right=True).sub_(1).clamp_(max=cnt.numel() - 1)
    slot = r - off.long()[e]
    return e, slot, slot < cnt.long()[e]


def _plain_product(s):
    total, most = s["a"].shape[0], max(1, s["most"])
    e, slot, owned = _rows_of(s["cnt"], s["off"], total)
    a = _mxfp4_widen(s["a"], s["as"])
    at = s["off"][:-1].long().unsqueeze(1) + torch.arange(most, device=a.device)
    y = torch.bmm(a[at.clamp(max=total - 1)], _mxfp4_widen(s["w"], s["ws"]).transpose(1, 2))
    if s["case"]["swiglu"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return torch.where(owned.unsqueeze(1), y[e, slot.clamp(max=most - 1)], 0.0).to(s["y"].dtype)


def _widen(w, scales):
    return w.float() if scales is None else _mxfp4_widen(w, scales)


def _pick(w, scales, at):
    return _widen(w[at], None if scales is None else scales[at])


def _plain_layer(s):
    T, K = s["idx"].shape
    E, H, _ = s["w2"].shape
    x, idx = s["x"].float(), s["idx"].long()
    weight = torch.where(idx >= 0, s["w"], 0.0)
    if T * K <= E:      # the experts of the entries, one by one
        at = idx.clamp(min=0).flatten()
        gate, up = torch.bmm(_pick(s["w13"], s["s13"], at),
                             x.repeat_interleave(K, 0).unsqueeze(-1)).chunk(2, 1)
        h = gate / (1.0 + torch.exp(-gate)) * up
        y = torch.bmm(_pick(s["w2"], s["s2"], at), h).view(T, K, H)
        return (y * weight.unsqueeze(-1)).sum(1).to(s["out"].dtype)
    # every expert on every token, weighted with 0 where the token has not chosen it
    share = torch.zeros((T, E), device=x.device)
    share.scatter_add_(1, idx.clamp(min=0), weight)
    gate, up = (_widen(s["w13"], s["s13"]).flatten(0, 1) @ x.t()).view(E, -1, T).chunk(2, 1)
    h = gate / (1.0 + torch.exp(-gate)) * up * share.t().unsqueeze(1)
    return torch.bmm(_widen(s["w2"], s["s2"]), h).sum(0).t().to(s["out"].dtype).contiguous()


def _owned(s):
    """Which rows a segment owns: [rows, 1], or None for all."""
    return None if s["cnt"] is None else _rows_of(s["cnt"], s["off"], s["rows"])[2].unsqueeze(1)


def _keep(owned, v, was=0.0):
    return v if owned is None else torch.where(owned, v, was)


def _plain_swiglu(s):
    owned = _owned(s)
    gu = s["gu"].float()
    gate, up = gu.chunk(2, -1)
    h = gate / (1.0 + torch.exp(-gate)) * up
    kept = _e4m3_widen(*_e4m3(gu))
    return _keep(owned, h).to(s["h"].dtype), _keep(owned, kept).to(torch.bfloat16)


def _plain_swiglu_backward(s):
    owned = _owned(s)
    gu = s["gu"].float() if s["scales"] is None else _e4m3_widen(s["gu"], s["scales"])
    gate, up = gu.chunk(2, -1)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig
    dgu = torch.cat((dh * up * (sig * (1.0 + gate * (1.0 - sig))), dh * act), -1)
    return _keep(owned, dgu).to(s["dgu"].dtype), _keep(owned, act * up).to(s["h"].dtype)


_RUN_PLAIN = {"quantize": _plain_quantize, "product": _plain_product, "layer": _plain_layer,
              "swiglu": _plain_swiglu, "swiglu_backward": _plain_swiglu_backward}


def _own_quantize(s):
    import combine_moe_route_count_amd as moe
    codes, scales = moe.mxfp4_quantize(s["x"])
    return moe.mxfp4_dequantize(codes, scales, out_dtype=s["x"].dtype)


def _own_product(s):
    import combine_moe_route_count_amd as moe
    return moe.expert_product_mxfp4(s["a"], s["as"], s["w"], s["ws"], s["cnt"], s["off"],
                                    swiglu=s["case"]["swiglu"], y=s["y"])


def _own_layer(s):
    import combine_moe_route_count_amd as moe
    c = s["case"]
    if "work" not in s:   # a program keeps one workspace for its batch size
        s["work"] = moe.experts_decode_workspace(c["T"], c["K"], c["I"])
    return moe.experts_decode(s["x"], s["idx"], s["w"], s["w13"], s["w2"], w13_scales=s["s13"],
                              w2_scales=s["s2"], out=s["out"], ws=s["work"])


def _own_swiglu(s):
    import combine_moe_route_count_amd as moe
    h, codes, scales = moe.swiglu(s["gu"], packed_cnt=s["cnt"], packed_off=s["off"], save=True,
                                  h=s["h"], codes=s["codes"], scales=s["scales"])
    return h, moe.fp8_dequant(codes, scales)


def _own_swiglu_backward(s):
    import combine_moe_route_count_amd as moe
    return moe.swiglu_backward(s["dh"], s["gu"], scales=s["scales"], packed_cnt=s["cnt"],
                               packed_off=s["off"], dgu=s["dgu"], h=s["h"])


_RUN_OWN = {"quantize": _own_quantize, "product": _own_product, "layer": _own_layer,
            "swiglu": _own_swiglu, "swiglu_backward": _own_swiglu_backward}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        n = float(case["rows"] * case["H"])
        return {"bytes": n * (2 * BYTES[case["dt"]] + BYTES["mxfp4"]), "flops": 4.0 * n}
    if op == "product":
        rows, E, N, H = (float(case[k]) for k in ("rows", "E", "N", "H"))
        if case["cap"]:
            rows *= 0.95                                     # about what finds room
        used = E * (1.0 - (1.0 - 1.0 / E) ** rows)           # experts with a row
        out = N / (2 if case["swiglu"] else 1) * BYTES[case["out"]]
        return {"bytes": (rows + used * N) * H * BYTES["mxfp4"] + rows * out,
                "flops": 2.0 * rows * N * H}
    if op == "layer":
        T, H, I, E, K = (float(case[k]) for k in ("T", "H", "I", "E", "K"))
        live = K * (0.8 if case["none"] else 1.0)
        used = E * (1.0 - (1.0 - live / E) ** T)
        return {"bytes": used * 3 * H * I * BYTES[case["wt"]] + T * H * (2.0 + BYTES[case["out"]])
                + T * K * 8.0, "flops": 6.0 * T * live * H * I}
    n = float(case["rows"] * case["I"])
    if op == "swiglu":   # the checkpoint is written, and its values are returned
        return {"bytes": n * (3 * BYTES[case["dt"]] + 2 * BYTES["fp8"] + 4.0), "flops": 6.0 * n}
    return {"bytes": n * (4 * BYTES[case["dt"]] + 2 * BYTES[case["gu"]]), "flops": 12.0 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_mxfp4(x):
    """MXFP4 values of x, by comparison with the midpoints of the code values (ties to even)."""
    b = x.double().unflatten(-1, (-1, 32))
    m, ex = torch.frexp(b.abs().amax(-1))                    # amax = m * 2^ex, m in [1/2, 1)
    e = torch.where(m == 0, 0, torch.where(m < 0.875, ex - 3, ex - 2)).clamp(min=-127)
    scale = _pow2(e).unsqueeze(-1)
    v = (b / scale).abs()
    out = torch.zeros_like(v)
    for i in range(7):
        lo, hi = E2M1[i], E2M1[i + 1]
        mid = (lo + hi) / 2
        out += (hi - lo) * ((v > mid) | ((v == mid) & (i % 2 == 1)))
    return (torch.sign(b) * out * scale).flatten(-2)


def _exact_values(codes, scales):
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    mag = (code & 7).double()
    v = torch.where(mag < 2, mag * 0.5, _pow2(torch.floor(mag / 2) - 1) * (1 + 0.5 * (mag % 2)))
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, 32))
    return (v * _pow2(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return torch.cat([_exact_mxfp4(b) for b in s["x"].split(4096)])
    if op == "product":
        out = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        cnt, off = s["cnt"].tolist(), s["off"].tolist()
        for e in range(case["E"]):
            r = slice(off[e], off[e] + cnt[e])
            y = _exact_values(s["a"][r], s["as"][r]) @ _exact_values(s["w"][e], s["ws"][e]).t()
            if case["swiglu"]:
                y = y[:, :case["N"] // 2] * torch.sigmoid(y[:, :case["N"] // 2]) * y[:, case["N"] // 2:]
            out[r] = y
        return out
    if op == "layer":
        I = case["I"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        wide = lambda w, sc, e: w[e].double() if sc is None else _exact_values(w[e], sc[e])
        for e in s["idx"].unique().tolist():
            if e < 0:
                continue
            t, k = torch.nonzero(s["idx"] == e, as_tuple=True)
            y = s["x"][t].double() @ wide(s["w13"], s["s13"], e).t()
            h = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
            y = h @ wide(s["w2"], s["s2"], e).t()
            out.index_add_(0, t, y * s["w"][t, k].double().unsqueeze(1))
        return out
    rows, I = s["rows"], case["I"]
    owned = torch.ones((rows, 1), dtype=torch.bool, device=DEV)
    if s["cnt"] is not None:
        owned.zero_()
        for c, o in zip(s["cnt"].tolist(), s["off"].tolist()):
            owned[o:o + c] = True
    gu = s["gu"]
    if op == "swiglu":
        z = gu.double()
        b = z.unflatten(-1, (-1, 128))
        amax = b.abs().amax(-1, keepdim=True)
        k = torch.ceil(torch.log2(amax / 448.0)).clamp(min=-126.0)
        k = torch.where(amax == 0, 0.0, k + 1.0 * (amax > 448.0 * _pow2(k))
                        - 1.0 * (amax <= 224.0 * _pow2(k)))
        sc = _pow2(k)
        v = b / sc
        # e4m3: steps of 2^(exponent - 3), the exponent at least -6; halves to even
        step = _pow2((torch.frexp(v)[1] - 1).clamp(min=-6) - 3)
        kept = (torch.round(v / step) * step * sc).flatten(-2)
        h = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
        return torch.where(owned, h, 0.0), torch.where(owned, kept, 0.0)
    if s["scales"] is not None:
        z = gu.view(torch.float8_e4m3fn).double() * s["scales"].double().repeat_interleave(128, 1)
    else:
        z = gu.double()
    gate, up, dh = z[:, :I], z[:, I:], s["dh"].double()
    sig = torch.sigmoid(gate)
    dgu = torch.cat((dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig), 1)
    return torch.where(owned, dgu, 0.0), torch.where(owned, gate * sig * up, 0.0)
