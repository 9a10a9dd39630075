"""Cases of the training-side operators next to the dispatch and the combine: the top-k gate, the
gradients of gate, dispatch and combine, the embedding lookup and its gradient.

Each case is one call of one operator.  With `own` false, run() computes it in plain torch
operations (32 bits, one rounding at the end); with `own` true it calls the library.  exact()
computes it again from the definitions, in 64 bits.  Conventions are the library's: expert id -1
is "no expert", tok_map -1 is "no row", token id -1 is "no token".
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2.0, "f32": 4.0, "fp8": 1.0, "fp4": 0.5}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 32 sequences: the gate is on the latency path
        {"name": "gate_decode", "op": "gate", "T": 32, "E": 128, "K": 8, "dt": "f32",
         "renorm": True, "scale": 1.0, "masked": False},
        # a long prefill, bf16 logits (many exact ties), some experts masked out with -inf
        {"name": "gate_prefill", "op": "gate", "T": 16384, "E": 256, "K": 8, "dt": "bf16",
         "renorm": False, "scale": 2.5, "masked": True},
        # fine-tuning on a short odd batch, expert count not a power of two
        {"name": "gate_backward_short", "op": "gate_backward", "T": 1001, "E": 60, "K": 6,
         "dt": "bf16", "renorm": True, "scale": 1.0, "masked": True},
        # one training micro-batch of the 256-expert configuration
        {"name": "gate_backward_train", "op": "gate_backward", "T": 8192, "E": 256, "K": 8,
         "dt": "f32", "renorm": False, "scale": 2.5, "masked": False},
        # a small odd batch whose experts answered in e4m3, padded expert segments
        {"name": "combine_backward_fp8", "op": "combine_backward", "T": 501, "H": 6144, "E": 128,
         "K": 8, "zipf": False, "cap": 40, "y": "fp8", "dt": "bf16", "dow": True},
        # the combine of the 8192-token skewed configuration, trained in bf16
        {"name": "combine_backward_train", "op": "combine_backward", "T": 8192, "H": 7168, "E": 256,
         "K": 8, "zipf": True, "cap": 0, "y": "bf16", "dt": "bf16", "dow": False},
        # the smallest configuration
        {"name": "dispatch_backward_tiny", "op": "dispatch_backward", "T": 64, "H": 256, "E": 8,
         "K": 2, "zipf": False, "cap": 0, "dt": "bf16", "out": "bf16", "residual": False},
        # f32 training of the 64-expert configuration, added to the residual stream's gradient
        {"name": "dispatch_backward_train", "op": "dispatch_backward", "T": 16384, "H": 4096,
         "E": 64, "K": 6, "zipf": False, "cap": 0, "dt": "f32", "out": "f32", "residual": True},
        # token rows of one decode step
        {"name": "embedding_decode", "op": "embedding", "N": 32, "H": 6144, "V": 65536,
         "dt": "bf16", "out": "bf16", "wide": False, "scale": 1.0, "pad": False},
        # a training batch read from an f32 master table, scaled by sqrt(H), 5% padding
        {"name": "embedding_train", "op": "embedding", "N": 16384, "H": 7168, "V": 131072,
         "dt": "f32", "out": "bf16", "wide": True, "scale": math.sqrt(7168.0), "pad": True},
        # a short odd batch on a small vocabulary, bf16 gradients
        {"name": "embedding_backward_short", "op": "embedding_backward", "N": 777, "H": 1000,
         "V": 5003, "dt": "bf16", "out": "bf16", "wide": False, "scale": 1.0, "pad": True},
        # 65536 tokens into the f32 gradient of a 131072-row table, Zipf tokens (long runs)
        {"name": "embedding_backward_train", "op": "embedding_backward", "N": 65536, "H": 4096,
         "V": 131072, "dt": "bf16", "out": "f32", "wide": True, "scale": 64.0, "pad": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate_backward", "combine_backward", "dispatch_backward",
                     "embedding", "embedding_backward"])
    dt = rng.choice(["bf16", "f32"])
    if op in ("gate", "gate_backward"):
        E = _log_int(rng, 4, 1024)
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "K": rng.randint(1, min(16, E)),
                "dt": dt, "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "masked": rng.random() < 0.5}
    if op in ("combine_backward", "dispatch_backward"):
        E = _log_int(rng, 4, 256)
        K = rng.randint(1, min(8, E))
        y = rng.choice(["bf16", "f32", "fp8", "fp4"]) if op == "combine_backward" else dt
        H = 128 * _log_int(rng, 1, 56) if y in ("fp8", "fp4") else 8 * _log_int(rng, 8, 896)
        T = _log_int(rng, 1, 8192 if "f32" not in (y, dt) else 4096)
        # half of the layouts are padded to about 1.3 times the mean load, so some entries drop
        cap = max(1, int(1.3 * T * K / E)) if rng.random() < 0.5 else 0
        case = {"op": op, "T": T, "H": H, "E": E, "K": K, "zipf": rng.random() < 0.5, "cap": cap}
        if op == "combine_backward":
            case.update(y=y, dt=dt, dow=rng.random() < 0.5)
        else:
            case.update(dt=dt, out=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.5)
        return case
    V = _log_int(rng, 100, 131072)
    return {"op": op, "N": _log_int(rng, 1, 16384 if op == "embedding" else 65536),
            "H": 8 * _log_int(rng, 8, 512), "V": V, "dt": dt, "out": rng.choice(["bf16", "f32"]),
            "wide": rng.random() < 0.5, "scale": rng.choice([1.0, 32.0]), "pad": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dt, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(DTYPES[dt])


def _experts(g, T, E, K, zipf):
    """K distinct experts per token, uniform or Zipf(1.2) over a random order of the experts."""
    u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-7, 1.0 - 1e-7)
    keys = -torch.log(-torch.log(u))
    if zipf:
        rank = torch.randperm(E, generator=g, device=DEV).float()
        keys -= 1.2 * torch.log1p(rank)
    idx = torch.topk(keys, K, dim=1).indices.to(torch.int32)
    # the last tokens of the batch are padding: they have no expert
    idx[T - T // 50:] = -1
    return idx


def _route(idx, E, cap):
    """The dispatch's slots: stable by expert, compact (cap 0) or padded segments."""
    T, K = idx.shape
    flat = idx.reshape(-1).long()
    n = flat.numel()
    key = torch.where(flat < 0, E, flat)
    cnt = torch.bincount(key, minlength=E + 1)[:E]
    off = torch.zeros(E + 2, dtype=torch.int64, device=DEV)
    off[1:E + 1] = torch.cumsum(cnt, 0)
    off[E + 1] = n
    order = torch.sort(key, stable=True).indices
    skey = key[order]
    slot = torch.arange(n, device=DEV) - off[skey]
    if cap > 0:
        row = torch.where((skey < E) & (slot < cap), skey * cap + slot, -1)
        rows, packed_cnt = E * cap, cnt.clamp(max=cap)
        packed_off = torch.arange(E + 1, device=DEV) * cap
    else:
        row = torch.where(skey < E, off[skey] + slot, -1)
        rows, packed_cnt, packed_off = n, cnt, off[:E + 1]
    tok_map = torch.empty(n, dtype=torch.int64, device=DEV)
    tok_map[order] = row
    return tok_map.view(T, K), packed_cnt.int(), packed_off.int(), rows


def _token_ids(g, N, V, wide, pad):
    """Zipf(1) token ids (frequent tokens have low ids); with pad, about 5% are -1."""
    cdf = torch.cumsum(1.0 / torch.arange(1, V + 1, dtype=torch.float64, device=DEV), 0)
    u = torch.rand(N, generator=g, device=DEV, dtype=torch.float64) * cdf[-1]
    ids = torch.searchsorted(cdf, u).clamp_(max=V - 1)
    if pad:
        ids[torch.rand(N, generator=g, device=DEV) < 0.05] = -1
    return ids if wide else ids.int()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("gate", "gate_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        logits = _normal(g, (T, E), case["dt"], 1.5)
        if case["masked"]:   # a tenth of the experts are out, and every 97th token has none at all
            logits[:, torch.rand(E, generator=g, device=DEV) < 0.1] = -math.inf
            logits[5::97] = -math.inf
        s["logits"] = logits
        if op == "gate":
            s["idx_out"] = torch.empty((T, K), dtype=torch.int32, device=DEV)
            s["w_out"] = torch.empty((T, K), dtype=torch.float32, device=DEV)
        else:
            s["idx"] = _plain_choice(logits.float(), K)
            s["dw"] = _normal(g, (T, K), "f32")
            s["dlogits_out"] = torch.empty_like(logits)
    elif op in ("combine_backward", "dispatch_backward"):
        T, H, E, K = case["T"], case["H"], case["E"], case["K"]
        idx = _experts(g, T, E, K, case["zipf"])
        s["tok_map"], s["packed_cnt"], s["packed_off"], rows = _route(idx, E, case["cap"])
        if op == "combine_backward":
            s["w"] = torch.softmax(_normal(g, (T, K), "f32"), -1)
            s["dout"] = _normal(g, (T, H), case["dt"], 0.1)
            s["dow"] = _normal(g, (T,), "f32", 0.1) if case["dow"] else None
            s["scales"] = None
            if case["y"] in ("fp8", "fp4"):
                s["scales"] = torch.rand((rows, H // 128), generator=g, device=DEV) + 0.5
            if case["y"] == "fp8":
                s["y"] = _normal(g, (rows, H), "f32").to(torch.float8_e4m3fn).view(torch.uint8)
            elif case["y"] == "fp4":
                s["y"] = torch.randint(0, 256, (rows, H // 2), generator=g, device=DEV,
                                       dtype=torch.uint8)
            else:
                s["y"] = _normal(g, (rows, H), case["y"])
            s["dy_out"] = torch.empty((rows, H), dtype=DTYPES[case["dt"]], device=DEV)
            s["dw_out"] = torch.empty((T, K), dtype=torch.float32, device=DEV)
        else:
            s["dpacked"] = _normal(g, (rows, H), case["dt"], 0.1)
            s["residual"] = _normal(g, (T, H), case["out"], 0.1) if case["residual"] else None
            s["dx_out"] = torch.empty((T, H), dtype=DTYPES[case["out"]], device=DEV)
    else:
        N, H, V = case["N"], case["H"], case["V"]
        s["ids"] = _token_ids(g, N, V, case["wide"], case["pad"])
        if op == "embedding":
            s["table"] = _normal(g, (V, H), case["dt"], 0.02)
            s["out"] = torch.empty((N, H), dtype=DTYPES[case["out"]], device=DEV)
        else:
            s["dout"] = _normal(g, (N, H), case["dt"], 0.1)
            s["dtable_out"] = torch.empty((V, H), dtype=DTYPES[case["out"]], device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_RUN_OWN if own else _RUN_PLAIN)[state["case"]["op"]](state)


def _plain_choice(l, K):
    """The K largest logits of each token, ties to the lowest index; -1 where none is left."""
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    return torch.where(torch.isneginf(v[:, :K]), -1, i[:, :K]).int()


def _plain_probs(l, idx, renorm):
    """(p over the chosen, p over all): softmax over the chosen logits, or over all of them."""
    at = idx.clamp(min=0).long()
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isneginf(top), 0.0, top))
    chosen = torch.where(idx >= 0, e.gather(1, at), 0.0)
    total = (chosen if renorm else e).sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    return chosen / total, e / total


def _plain_gate(s):
    c = s["case"]
    l = s["logits"].float()
    idx = _plain_choice(l, c["K"])
    return idx, _plain_probs(l, idx, c["renorm"])[0] * c["scale"]


def _plain_gate_backward(s):
    c = s["case"]
    l, idx = s["logits"].float(), s["idx"]
    p, p_all = _plain_probs(l, idx, c["renorm"])
    d = p * s["dw"] * c["scale"]                       # zero where idx is -1
    dot = d.sum(1, keepdim=True)
    if c["renorm"]:
        grad, d = torch.zeros_like(l), d - p * dot
    else:
        grad = -p_all * dot
    grad.scatter_add_(1, idx.clamp(min=0).long(), d)
    return grad.to(s["logits"].dtype)


def _widen(y, kind, scales):
    """Expert rows in 32 bits: bf16 / f32 as they are, e4m3 / e2m1 codes times their block scale."""
    if kind in DTYPES:
        return y.float()
    if kind == "fp8":
        v = y.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1, device=y.device)
        v = torch.stack((table[(y & 15).long()], table[(y >> 4).long()]), -1).view(y.shape[0], -1)
    return (v.view(v.shape[0], -1, 128) * scales.unsqueeze(-1)).view(v.shape)


def _plain_combine_backward(s):
    c = s["case"]
    T, K = s["tok_map"].shape
    dout = s["dout"].float()
    rows = s["tok_map"].reshape(-1)
    has = rows >= 0
    y = _widen(s["y"], c["y"], s["scales"])
    dw = (y[rows.clamp(min=0)].view(T, K, -1) * dout.unsqueeze(1)).sum(-1)
    if s["dow"] is not None:
        dw = dw + s["dow"].unsqueeze(1)
    dw = torch.where(has.view(T, K), dw, 0.0)
    part = (s["w"].unsqueeze(-1) * dout.unsqueeze(1)).view(T * K, -1)
    dy = torch.zeros((y.shape[0] + 1, y.shape[1]), device=y.device)
    dy[torch.where(has, rows, y.shape[0])] = part
    return dy[:-1].to(s["dout"].dtype), dw


def _plain_dispatch_backward(s):
    T, K = s["tok_map"].shape
    rows = s["tok_map"].reshape(-1)
    d = s["dpacked"].float()[rows.clamp(min=0)]
    dx = torch.where((rows >= 0).unsqueeze(1), d, 0.0).view(T, K, -1).sum(1)
    if s["residual"] is not None:
        dx = s["residual"].float() + dx
    return dx.to(s["dx_out"].dtype)


def _plain_embedding(s):
    ids = s["ids"].long()
    rows = s["table"][ids.clamp(min=0)].float() * s["case"]["scale"]
    return torch.where((ids >= 0).unsqueeze(1), rows, 0.0).to(s["out"].dtype)


def _plain_embedding_backward(s):
    c = s["case"]
    ids = s["ids"].long()
    grad = torch.zeros((c["V"] + 1, c["H"]), device=ids.device)
    grad.index_add_(0, torch.where(ids < 0, c["V"], ids), s["dout"].float())
    return (grad[:-1] * c["scale"]).to(s["dtable_out"].dtype)


_RUN_PLAIN = {"gate": _plain_gate, "gate_backward": _plain_gate_backward,
              "combine_backward": _plain_combine_backward,
              "dispatch_backward": _plain_dispatch_backward, "embedding": _plain_embedding,
              "embedding_backward": _plain_embedding_backward}


def _own_gate(s):
    import combine_moe_route_count_amd as moe
    c = s["case"]
    return moe.gate(s["logits"], c["K"], renormalize=c["renorm"], scale=c["scale"],
                    idx=s["idx_out"], w=s["w_out"])


def _own_gate_backward(s):
    import combine_moe_route_count_amd as moe
    c = s["case"]
    return moe.gate_backward(s["logits"], s["idx"], s["dw"], renormalize=c["renorm"],
                             scale=c["scale"], dlogits=s["dlogits_out"])


def _own_combine_backward(s):
    import combine_moe_route_count_amd as moe
    return moe.combine_backward(s["dout"], s["y"], s["tok_map"], s["w"], y_scales=s["scales"],
                                fp4=s["case"]["y"] == "fp4", dout_weights=s["dow"],
                                packed_cnt=s["packed_cnt"], packed_off=s["packed_off"],
                                dy=s["dy_out"], dw=s["dw_out"])


def _own_dispatch_backward(s):
    import combine_moe_route_count_amd as moe
    return moe.dispatch_backward(s["dpacked"], s["tok_map"], residual=s["residual"],
                                 dx=s["dx_out"])


def _own_embedding(s):
    import combine_moe_route_count_amd as moe
    return moe.embedding(s["ids"], s["table"], scale=s["case"]["scale"], out=s["out"])


def _own_embedding_backward(s):
    import combine_moe_route_count_amd as moe
    c = s["case"]
    if "ws" not in s:   # a program keeps one workspace for its batch size
        s["ws"] = moe.embedding_workspace(c["N"], c["V"], c["H"])
    return moe.embedding_backward(s["dout"], s["ids"], c["V"], scale=c["scale"],
                                  dtable=s["dtable_out"], ws=s["ws"])


_RUN_OWN = {"gate": _own_gate, "gate_backward": _own_gate_backward,
            "combine_backward": _own_combine_backward,
            "dispatch_backward": _own_dispatch_backward, "embedding": _own_embedding,
            "embedding_backward": _own_embedding_backward}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _distinct(N, V, pad):
    """Expected number of distinct Zipf(1) ids among N draws."""
    p = 1.0 / torch.arange(1, V + 1, dtype=torch.float64)
    p /= p.sum()
    n = N * (0.95 if pad else 1.0)
    return float((1.0 - torch.exp(n * torch.log1p(-p.clamp(max=1.0 - 1e-12)))).sum())


def work(case):
    op = case["op"]
    if op in ("gate", "gate_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        read = T * E * BYTES[case["dt"]]
        if op == "gate":
            return {"bytes": read + T * K * 8.0, "flops": 4.0 * T * E}
        return {"bytes": 2 * read + T * K * 8.0, "flops": 6.0 * T * E}
    if op in ("combine_backward", "dispatch_backward"):
        T, H, E, K, cap = case["T"], case["H"], case["E"], case["K"], case["cap"]
        rows = E * cap if cap else T * K
        full = min(rows, (T - T // 50) * K)    # rows that an entry owns, at most
        if op == "combine_backward":
            scales = full * H / 128 * 4.0 if case["y"] in ("fp8", "fp4") else 0.0
            b = (T * H * BYTES[case["dt"]] + full * H * BYTES[case["y"]] + scales
                 + rows * H * BYTES[case["dt"]] + T * K * 16.0)
            return {"bytes": b, "flops": 3.0 * full * H}
        b = (full * H * BYTES[case["dt"]] + T * K * 8.0
             + T * H * BYTES[case["out"]] * (2 if case["residual"] else 1))
        return {"bytes": b, "flops": 1.0 * full * H}
    N, H, V = case["N"], case["H"], case["V"]
    ids = N * (8.0 if case["wide"] else 4.0)
    if op == "embedding":
        rows = _distinct(N, V, case["pad"])
        return {"bytes": ids + rows * H * BYTES[case["dt"]] + N * H * BYTES[case["out"]],
                "flops": 1.0 * N * H}
    n = N * (0.95 if case["pad"] else 1.0)
    return {"bytes": ids + n * H * BYTES[case["dt"]] + V * H * BYTES[case["out"]],
            "flops": 1.0 * n * H}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gate", "gate_backward"):
        z = s["logits"].double()
        T, E = z.shape
        K = case["K"]
        # expert j's place: how many experts come before it (larger, or equal with a lower index);
        # in blocks of tokens, since it compares every pair of a token's experts
        idx = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
        lower = torch.ones((E, E), dtype=torch.bool, device=DEV).tril(-1)     # [j, i]: i < j
        step = max(1, (1 << 27) // (E * E))
        for t in range(0, T, step):
            b = z[t:t + step]
            before = (b.unsqueeze(1) > b.unsqueeze(2)) | ((b.unsqueeze(1) == b.unsqueeze(2)) & lower)
            place = before.sum(2)
            tt, j = torch.nonzero((place < K) & (b > -math.inf), as_tuple=True)
            idx[t + tt, place[tt, j]] = j.int()
        chosen = torch.zeros((T, E + 1), dtype=torch.bool, device=DEV)
        chosen.scatter_(1, torch.where(idx < 0, E, idx).long(), True)
        chosen = chosen[:, :E]
        live = z.masked_fill(~chosen, -math.inf) if case["renorm"] else z
        p = torch.nan_to_num(torch.softmax(live, 1), nan=0.0)     # NaN: a token with no expert at all
        at = idx.clamp(min=0).long()
        if op == "gate":
            return idx, torch.where(idx >= 0, p.gather(1, at), 0.0) * case["scale"]
        dp = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        dp.scatter_add_(1, at, torch.where(idx >= 0, s["dw"].double() * case["scale"], 0.0))
        return p * (dp - (p * dp).sum(1, keepdim=True))
    if op == "combine_backward":
        T, K = s["tok_map"].shape
        dout, w = s["dout"].double(), s["w"].double()
        scales = None if s["scales"] is None else s["scales"].double()
        if case["y"] == "fp4":
            code = torch.stack((s["y"] & 15, s["y"] >> 4), -1).view(s["y"].shape[0], -1).long()
            mag = code & 7
            v = torch.where(mag < 2, mag * 0.5, torch.exp2((mag // 2 - 1).double()) * (1 + 0.5 * (mag % 2)))
            y = torch.where(code >= 8, -v, v).double()
        elif case["y"] == "fp8":
            y = s["y"].view(torch.float8_e4m3fn).double()
        else:
            y = s["y"].double()
        if scales is not None:
            y = y * scales.repeat_interleave(128, dim=1)
        dy = torch.zeros_like(y)
        dw = torch.zeros((T, K), dtype=torch.float64, device=DEV)
        for k in range(K):
            t = torch.nonzero(s["tok_map"][:, k] >= 0).flatten()
            r = s["tok_map"][t, k]
            dy[r] = w[t, k].unsqueeze(1) * dout[t]
            dw[t, k] = (y[r] * dout[t]).sum(1) + (s["dow"].double()[t] if case["dow"] else 0.0)
        return dy, dw
    if op == "dispatch_backward":
        T, K = s["tok_map"].shape
        dx = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV)
        if s["residual"] is not None:
            dx += s["residual"].double()
        for k in range(K):
            t = torch.nonzero(s["tok_map"][:, k] >= 0).flatten()
            dx[t] += s["dpacked"][s["tok_map"][t, k]].double()
        return dx
    ids = s["ids"].long()
    n = torch.nonzero(ids >= 0).flatten()
    if op == "embedding":
        out = torch.zeros((case["N"], case["H"]), dtype=torch.float64, device=DEV)
        out[n] = s["table"][ids[n]].double() * case["scale"]
        return out
    grad = torch.zeros((case["V"], case["H"]), dtype=torch.float64, device=DEV)
    grad.index_put_((ids[n],), s["dout"][n].double() * case["scale"], accumulate=True)
    return grad
