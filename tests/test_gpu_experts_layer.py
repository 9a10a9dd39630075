"""GPU tests of the experts' step inside its layer: gate, dispatch, MXFP4 products and
combine as a server runs them, SwiGLU and its gradient as a training step runs them,
the whole in graphs and on several streams, and the calls that are refused.

Tolerances are those of each operator's own tests where a stage is compared on the
inputs it really had.  A block's MXFP4 rounding is off by at most its scale 2^e (half
the step between 4 and 6, or 7 saturated to 6), and 2^e <= amax / 3.5: that bounds how
far a layer with quantized activations may be from one without.  For the training step
every sum of the chain is carried once in values and once in magnitudes; a result is
off by at most (steps that round) * 2^-24 of its magnitude."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note
from test_gpu_expert_product import _check as _check_product
from test_gpu_expert_product import _ref as _product_ref
from test_gpu_experts_decode import BF16, F32, U, _gen, _values
from test_gpu_experts_decode import _check as _check_decode
from test_gpu_experts_decode import _ref as _decode_ref

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _quant(v):
    """(codes, scales) of v on the GPU, by the framework."""
    return moe.mxfp4_quantize(v.to(DEV))


def _weights(g, E, rows, cols):
    c, s = _quant((torch.randn((E * rows, cols), generator=g) * cols ** -0.5))
    return c.view(E, rows, cols // 2), s.view(E, rows, cols // 32)


def _cpu(*ts):
    return [t.cpu() for t in ts]


def _block_max(v):
    return v.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).expand(
        *v.shape[:-1], -1, 32).flatten(-2)


def _serve(x, logits, K, weights, cap, out_dtype, **buf):
    """One layer: (every stage's result)."""
    w13, s13, w2, s2 = weights
    E = w13.shape[0]
    idx, w = moe.gate(logits, K, **{k: buf[k] for k in ("idx", "w") if k in buf})
    d = moe.dispatch(x, idx, E, cap=cap, out=buf.get("d"), ws=buf.get("ws"))
    qa, sa = moe.mxfp4_quantize(d.packed, buf.get("qa"), buf.get("sa"))
    h = moe.expert_product_mxfp4(qa, sa, w13, s13, d.packed_cnt, d.packed_off, swiglu=True,
                                 y=buf.get("h"))
    qh, sh = moe.mxfp4_quantize(h, buf.get("qh"), buf.get("sh"))
    y = moe.expert_product_mxfp4(qh, sh, w2, s2, d.packed_cnt, d.packed_off, y=buf.get("y"),
                                 out_dtype=out_dtype)
    out, _ = moe.combine(y, d.tok_map, w, out_dtype=out_dtype, out=buf.get("out"),
                         out_weights=buf.get("out_w"))
    return dict(idx=idx, w=w, d=d, qa=qa, sa=sa, h=h, qh=qh, sh=sh, y=y, out=out)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,I,E,K,cap", [
    (1, 128, 96, 4, 2, 0), (19, 160, 32, 7, 3, 0), (45, 256, 160, 5, 2, 45), (130, 96, 64, 3, 3, 130),
    (300, 64, 96, 40, 4, 0)])
def test_serving_layer(T, H, I, E, K, cap, out_dtype):
    note(f"layer T={T} H={H} I={I} E={E} K={K} cap={cap} {out_dtype}")
    g = _gen(T + H)
    codes, scales = _quant(torch.randn((T, H), generator=g))
    x = moe.mxfp4_dequantize(codes, scales)             # rows that MXFP4 holds exactly
    logits = torch.randn((T, E), generator=g)
    logits[:, E // 2] = -float("inf")                    # an expert that is never chosen
    weights = _weights(g, E, 2 * I, H) + _weights(g, E, H, I)
    r = _serve(x, logits.to(DEV), K, weights, cap, out_dtype)
    torch.cuda.synchronize()
    d = r["d"]
    cnt, off, src, tok = _cpu(d.packed_cnt, d.packed_off, d.packed_src, d.tok_map)
    rows = d.packed.shape[0]
    v13, v2 = (_values(c.cpu(), s.cpu()) for c, s in (weights[:2], weights[2:]))

    mine = torch.zeros(rows, dtype=torch.bool)
    for e in range(E):
        mine[int(off[e]):int(off[e]) + int(cnt[e])] = True
    xs = x.cpu().double()
    va = _values(*_cpu(r["qa"], r["sa"]))
    assert torch.equal(va[mine], xs[src[mine].long()]), "rows that MXFP4 holds have changed"

    def stage(got, ref):
        y, tol, owned = ref
        assert torch.equal(owned, mine)
        keep = got.cpu().clone()
        keep[~mine] = 7.0                                # _check wants rows without an owner to hold 7
        _check_product(keep, (y, tol, owned), "layer")
    stage(r["h"], _product_ref(va, v13, cnt, off, rows, True))
    hs = r["h"].cpu().double()
    vh = _values(*_cpu(r["qh"], r["sh"]))
    assert ((vh - hs).abs() <= _block_max(hs) / 3.5)[mine].all()
    stage(r["y"], _product_ref(vh, v2, cnt, off, rows, False))
    ys, w, idx = r["y"].cpu().double(), r["w"].cpu().double(), r["idx"].cpu()
    terms = torch.where((tok >= 0).unsqueeze(-1), ys[tok.clamp(min=0)] * w.unsqueeze(-1), 0.0)
    want = terms.sum(1)
    lim = terms.abs().sum(1) * (K + 1) * U + want.abs() * torch.finfo(out_dtype).eps / 2
    assert ((r["out"].cpu().double() - want).abs() <= lim * (1 + 2.0 ** -7) + 1e-37).all()

    # the same layer for a few tokens in one call, which quantizes no activation
    if T * K > 1024:
        return
    got = moe.experts_decode(x, r["idx"], r["w"], weights[0], weights[2], weights[1], weights[3],
                             out_dtype=out_dtype)
    torch.cuda.synchronize()
    ref = _decode_ref(xs, idx, r["w"].cpu(), v13, v2, 3 if out_dtype == F32 else 2)
    _check_decode(got, ref, "decode in the layer")
    near = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            if tok[t, k] < 0:
                continue
            row, e = int(tok[t, k]), int(idx[t, k])
            dh = _block_max(hs[row]) / 3.5 + hs[row].abs() * 2.0 ** -7 + 2.0 ** -20
            near[t] += w[t, k] * (v2[e].abs() @ dh + ys[row].abs() * 2.0 ** -7)
    assert ((r["out"].cpu().double() - ref[0]).abs() <= near + ref[1] + ref[0].abs() * 2.0 ** -7).all()


def _grouped(rows, cnt, off, cols, fn):
    """The caller's products, in 64 bits, rounded to f32 once; NaN in rows without an owner."""
    out = torch.full((rows, cols), NAN, dtype=F32)
    for e, (c, o) in enumerate(zip(cnt.tolist(), off.tolist())):
        out[o:o + c] = fn(e, slice(o, o + c)).float()
    return out


@pytest.mark.parametrize("T,H,I,E,K,cap", [(1, 32, 128, 3, 2, 0), (37, 64, 256, 5, 2, 0),
                                           (50, 32, 128, 4, 3, 50)])
def test_training_step(T, H, I, E, K, cap):
    """Token rows with a single 1 and first weights that are multiples of 1/4 up to 2: the
    8-bit checkpoint then holds gate and up values exactly, and every gradient of the step
    can be compared with that of the layer in 64 bits."""
    note(f"training step T={T} H={H} I={I} E={E} K={K} cap={cap}")
    g = _gen(T + I)
    x = torch.zeros((T, H))
    x[torch.arange(T), torch.randint(0, H, (T,), generator=g)] = 1.0
    w13 = torch.randint(-8, 9, (E, 2 * I, H), generator=g).double() / 4
    w2 = torch.randn((E, H, I), generator=g).double() * I ** -0.5
    logits = torch.randn((T, E), generator=g)
    dout = torch.randn((T, H), generator=g)

    idx, w = moe.gate(logits.to(DEV), K)
    d = moe.dispatch(x.to(DEV), idx, E, cap=cap)
    cnt, off, tok = _cpu(d.packed_cnt, d.packed_off, d.tok_map)
    rows, seg = d.packed.shape[0], dict(packed_cnt=d.packed_cnt, packed_off=d.packed_off)
    packed = d.packed.cpu().double()
    gu = _grouped(rows, cnt, off, 2 * I, lambda e, s: packed[s] @ w13[e].t())
    h, codes, scales = moe.swiglu(gu.to(DEV), save=True, **seg)
    h_cpu = h.cpu().double()
    y = _grouped(rows, cnt, off, H, lambda e, s: h_cpu[s] @ w2[e].t()).to(DEV)
    out, _ = moe.combine(y, d.tok_map, w, out_dtype=F32)
    dy, dw = moe.combine_backward(dout.to(DEV), y, d.tok_map, w, **seg)
    dy_cpu = dy.cpu().double()
    dh = _grouped(rows, cnt, off, I, lambda e, s: dy_cpu[s] @ w2[e])
    dgu, h2 = moe.swiglu_backward(dh.to(DEV), codes, scales=scales, **seg)
    dgu_cpu, h2 = dgu.cpu().double(), h2.cpu().double()
    dpacked = _grouped(rows, cnt, off, H, lambda e, s: dgu_cpu[s] @ w13[e])
    dlogits = moe.gate_backward(logits.to(DEV), idx, dw)
    dx = moe.dispatch_backward(dpacked.to(DEV), d.tok_map)
    torch.cuda.synchronize()
    dw13, dw2 = torch.zeros_like(w13), torch.zeros_like(w2)
    for e in range(E):
        s = slice(int(off[e]), int(off[e]) + int(cnt[e]))
        dw13[e], dw2[e] = dgu_cpu[s].t() @ packed[s], dy_cpu[s].t() @ h2[s]

    # the layer in 64 bits, and the magnitudes of its sums
    leaf = [t.double().requires_grad_() for t in (x, w13, w2, logits)]
    ids, (xr, w13r, w2r, lr) = idx.cpu().long(), leaf
    wr = torch.softmax(lr.gather(1, ids), 1)
    outs, mags = [], dict(x=torch.zeros((T, H)).double(), w13=torch.zeros_like(w13), w2=torch.zeros_like(w2),
                          out=torch.zeros((T, H)).double(), dw=torch.zeros((T, K)).double())
    for t in range(T):
        acc = 0
        for k in range(K):
            e = int(ids[t, k])
            gate, up = (w13r[e] @ xr[t]).chunk(2)
            yt = w2r[e] @ (torch.nn.functional.silu(gate) * up)
            acc = acc + wr[t, k] * yt
            with torch.no_grad():
                s, wk = torch.sigmoid(gate), wr[t, k]
                hm = (gate * s * up).abs()
                ym, dym = w2r[e].abs() @ hm, wk * dout[t].double().abs()
                dhm = dym @ w2r[e].abs()
                dgum = torch.cat((dhm * up.abs() * s * (1 + gate.abs() * (1 - s)), dhm * gate.abs() * s))
                mags["out"][t] += wk * ym
                mags["dw"][t, k] = dout[t].double().abs() @ ym
                mags["w2"][e] += torch.outer(dym, hm)
                mags["w13"][e] += torch.outer(dgum, xr[t].abs())
                mags["x"][t] += dgum @ w13r[e].abs()
        outs.append(acc)
    want = torch.stack(outs)
    (want * dout.double()).sum().backward()

    # steps that round: those of an activation (20 and its argument, at most 2 here), of the
    # weights' softmax (logits below 5), casts, and K or H additions
    act, soft = 20 + 2, 20 + 2 * 5
    n = 2 * act + soft + 4 * 2 + 2 * K + 20

    def near(name, got, ref, mag, steps):
        over = (got.cpu().double() - ref).abs() > mag * (steps * U) + 1e-37
        assert not over.any(), f"{name}: {over.sum().item()} of {over.numel()} past the bound"
    wd = wr.detach()
    near("out", out, want.detach(), mags["out"], n)
    near("dx", dx, xr.grad, mags["x"], n)
    near("dw13", dw13, w13r.grad, mags["w13"], n)
    near("dw2", dw2, w2r.grad, mags["w2"], n)
    dw_err = mags["dw"] * (n + 2 * H)
    near("dlogits", dlogits.cpu().gather(1, ids), lr.grad.gather(1, ids),
         wd * (dw_err + (wd * dw_err).sum(1, True)) + wd * (mags["dw"] + (wd * mags["dw"]).sum(1, True)) * (soft + K), 1)


def _buffers(T, H, I, E, K, cap, out_dtype):
    rows = E * cap if cap else T * K
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)
    return dict(idx=torch.empty((T, K), dtype=torch.int32, device=DEV),
                w=torch.empty((T, K), dtype=F32, device=DEV),
                d=moe._lib.alloc_dispatch(T, H, K, E, rows, BF16, False, DEV), ws=moe.workspace(T, K, E),
                qa=u8(rows, H // 2), sa=u8(rows, H // 32),
                h=torch.empty((rows, I), dtype=BF16, device=DEV),
                qh=u8(rows, I // 2), sh=u8(rows, I // 32),
                y=torch.empty((rows, H), dtype=out_dtype, device=DEV),
                out=torch.empty((T, H), dtype=out_dtype, device=DEV),
                out_w=torch.empty(T, dtype=F32, device=DEV))


@pytest.mark.parametrize("cap", [0, 64])
def test_layer_in_a_graph(cap):
    """Everything of a serving layer and of the training side in one graph, replayed with new
    tokens and new routes (other segment sizes), with eager work in between."""
    T, H, I, E, K = 64, 256, 128, 6, 2
    g = _gen(3)
    weights = _weights(g, E, 2 * I, H) + _weights(g, E, H, I)
    batches = [(torch.randn((T, H), generator=g).to(BF16).to(DEV),
                (torch.randn((T, E), generator=g) * (1 + 4 * i)).to(DEV)) for i in range(3)]
    buf = _buffers(T, H, I, E, K, cap, BF16)
    x, logits = batches[0][0].clone(), batches[0][1].clone()
    ws = moe.experts_decode_workspace(T, K, I, H)
    rows = buf["h"].shape[0]
    new = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device=DEV)
    o = dict(dec=new(T, H), act=new(rows, I // 2), codes=new(rows, I, dt=torch.uint8),
             scales=new(rows, I // 128, dt=F32), dgu=new(rows, I, dt=F32), again=new(rows, I // 2, dt=F32),
             deq=new(rows, H))
    dh = torch.randn((rows, I // 2), generator=g).to(DEV)

    def step():
        r = _serve(x, logits, K, weights, cap, BF16, **buf)
        seg = dict(packed_cnt=r["d"].packed_cnt, packed_off=r["d"].packed_off)
        moe.experts_decode(x, r["idx"], r["w"], weights[0], weights[2], weights[1], weights[3],
                           out=o["dec"], ws=ws)
        # (h, of I = 128 columns, stands in for gate and up rows of 64)
        moe.swiglu(r["h"], h=o["act"], **seg)
        moe.swiglu_backward(dh, r["h"], dgu=o["dgu"], h=o["again"], **seg)
        moe.mxfp4_dequantize(r["qa"], r["sa"], y=o["deq"])

    def results():
        d = buf["d"]
        mine = torch.zeros(rows, dtype=torch.bool, device=DEV)
        for c, f in zip(d.packed_cnt.tolist(), d.packed_off.tolist()):
            mine[f:f + c] = True
        return [buf["out"].clone(), o["dec"].clone(), buf["h"][mine], buf["y"][mine],
                *(o[k][mine] for k in ("act", "dgu", "again", "deq"))]
    eager = []
    for b in batches:
        x.copy_(b[0])
        logits.copy_(b[1])
        step()
        eager.append(results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 2, 1, 1, 2, 0):
        for t in (buf["out"], buf["y"], buf["h"], *o.values()):
            t.view(torch.uint8).fill_(0x7f)
        x.copy_(batches[i][0])
        logits.copy_(batches[i][1])
        graph.replay()
        for got, want in zip(results(), eager[i]):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), i
        step()
        assert torch.equal(buf["out"], eager[i][0]) and torch.equal(o["dec"], eager[i][1])


def test_two_streams_at_once():
    """The same calls on two streams, each with its own outputs and workspace."""
    T, H, I, E, K = 96, 512, 256, 16, 4
    g = _gen(11)
    weights = _weights(g, E, 2 * I, H) + _weights(g, E, H, I)
    ins = [(torch.randn((T, H), generator=g).to(BF16).to(DEV), torch.randn((T, E), generator=g).to(DEV))
           for _ in range(2)]
    bufs = [_buffers(T, H, I, E, K, 0, F32) for _ in range(2)]
    ws = [moe.experts_decode_workspace(T, K, I, H) for _ in range(2)]
    outs = [torch.empty((T, H), dtype=F32, device=DEV) for _ in range(2)]

    def run(i):
        r = _serve(*ins[i], K, weights, 0, F32, **bufs[i])
        moe.experts_decode(ins[i][0], r["idx"], r["w"], weights[0], weights[2], weights[1], weights[3],
                           out=outs[i], ws=ws[i])
    want = []
    for i in range(2):
        run(i)
        torch.cuda.synchronize()
        want.append((bufs[i]["out"].clone(), outs[i].clone()))
    assert not torch.equal(want[0][0], want[1][0])
    for t in (*outs, bufs[0]["out"], bufs[1]["out"]):
        t.fill_(NAN)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(bufs[i]["out"], want[i][0]) and torch.equal(outs[i], want[i][1])


def _refused(kind, match, call):
    with pytest.raises(kind, match=match):
        call()


def test_refusals():
    """Wrong tensors raise before anything is enqueued, and the outputs keep what they held."""
    E, N, H, rows = 3, 64, 128, 10
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    bf = lambda *s: torch.zeros(s, dtype=BF16, device=DEV)
    V, M = ValueError, moe.MoeError
    x = bf(rows, H)
    keep = torch.full((rows, H), 7.0, dtype=BF16, device=DEV)

    _refused(V, "type", lambda: moe.mxfp4_quantize(x.half()))
    _refused(V, "dimensions", lambda: moe.mxfp4_quantize(x[0]))
    _refused(V, "contiguous", lambda: moe.mxfp4_quantize(bf(H, rows).t()))
    _refused(V, "shape", lambda: moe.mxfp4_quantize(x, codes=u8(rows, H)))
    _refused(V, "type", lambda: moe.mxfp4_quantize(x, scales=torch.zeros((rows, H // 32), device=DEV)))
    _refused(M, "multiple of 32", lambda: moe.mxfp4_quantize(bf(rows, 48)))
    _refused(M, "aligned", lambda: moe.mxfp4_quantize(bf(rows * H + 1)[1:].view(rows, H)))
    _refused(V, "shape", lambda: moe.mxfp4_dequantize(u8(rows, 64), u8(rows, 3)))
    _refused(V, "on cpu", lambda: moe.mxfp4_dequantize(u8(rows, 64), u8(rows, 4).cpu()))
    _refused(V, "type", lambda: moe.mxfp4_dequantize(u8(rows, 64), u8(rows, 4), out_dtype=torch.float16))

    a, sa, w, sw = u8(rows, H // 2), u8(rows, H // 32), u8(E, N, H // 2), u8(E, N, H // 32)
    cnt, off = i32(E), i32(E + 1)
    prod = moe.expert_product_mxfp4
    _refused(V, "w has shape", lambda: prod(a, sa, u8(E, N, H), sw, cnt, off))
    _refused(V, "w_scales has shape", lambda: prod(a, sa, w, u8(E, N, 3), cnt, off))
    _refused(V, "packed_off has shape", lambda: prod(a, sa, w, sw, cnt, cnt))
    _refused(V, "packed_cnt has type", lambda: prod(a, sa, w, sw, cnt.long(), off))
    _refused(V, "packed_cnt has shape", lambda: prod(a, sa, w, sw, i32(E + 1), off))
    _refused(V, "y has shape", lambda: prod(a, sa, w, sw, cnt, off, swiglu=True, y=bf(rows, N)))
    _refused(V, "y has type", lambda: prod(a, sa, w, sw, cnt, off, out_dtype=torch.float16))
    _refused(M, "multiple of 16", lambda: prod(a, sa, u8(E, 24, H // 2), u8(E, 24, H // 32), cnt, off, swiglu=True))
    _refused(M, "multiple of 8", lambda: prod(a, sa, u8(E, 12, H // 2), u8(E, 12, H // 32), cnt, off))
    whole = u8(rows * H * 2)
    _refused(M, "overlaps", lambda: prod(whole[:rows * H // 2].view(rows, H // 2), sa, w, sw, cnt, off,
                                         y=whole[:rows * N * 2].view(BF16).view(rows, N)))

    idx, gw = i32(rows, 2), torch.zeros((rows, 2), device=DEV)
    w13, w2 = bf(E, 2 * N, H), bf(E, H, N)
    dec = moe.experts_decode
    _refused(V, "x has type", lambda: dec(x.float(), idx, gw, w13, w2, out=keep))
    _refused(V, "idx has type", lambda: dec(x, idx.long(), gw, w13, w2, out=keep))
    _refused(V, "w has shape", lambda: dec(x, idx, gw[:, :1].contiguous(), w13, w2, out=keep))
    _refused(V, "w2 has shape", lambda: dec(x, idx, gw, w13, w2.transpose(1, 2).contiguous(), out=keep))
    _refused(V, "w13 has shape", lambda: dec(x, idx, gw, bf(E, 2 * N + 1, H), w2, out=keep))
    _refused(V, "go together", lambda: dec(x, idx, gw, w13, w2, w13_scales=sw, out=keep))
    _refused(V, "w13 has type", lambda: dec(x, idx, gw, w13, w2, sw, sw, out=keep))
    _refused(V, "out has shape", lambda: dec(x, idx, gw, w13, w2, out=keep[1:]))
    _refused(M, "workspace|ws", lambda: dec(x, idx, gw, w13, w2, out=keep, ws=u8(256)))
    _refused(V, "ws must be", lambda: dec(x, idx, gw, w13, w2, out=keep, ws=bf(1 << 20)))
    _refused(M, "overlaps", lambda: dec(keep, idx, gw, w13, w2, out=keep))
    _refused(M, "T\\*K", lambda: dec(bf(1025, H), i32(1025, 1), torch.zeros((1025, 1), device=DEV), w13, w2))
    _refused(M, "K=17", lambda: dec(x, i32(rows, 17), torch.zeros((rows, 17), device=DEV), w13, w2))
    _refused(M, "multiple of 8", lambda: dec(bf(rows, 12), idx, gw, bf(E, 16, 12), bf(E, 12, 8)))

    gu = bf(rows, 2 * H)
    _refused(V, "gu has shape", lambda: moe.swiglu(bf(rows, 17)))
    _refused(V, "go together", lambda: moe.swiglu(gu, packed_cnt=cnt))
    _refused(V, "need save", lambda: moe.swiglu(gu, codes=u8(rows, 2 * H)))
    _refused(V, "h has shape", lambda: moe.swiglu(gu, h=gu))
    _refused(M, "multiple of 128", lambda: moe.swiglu(bf(rows, 128), save=True))
    _refused(V, "scales go with", lambda: moe.swiglu_backward(x, u8(rows, 2 * H)))
    _refused(V, "scales go with", lambda: moe.swiglu_backward(x, gu, scales=torch.zeros((rows, 2), device=DEV)))
    _refused(V, "gu has shape", lambda: moe.swiglu_backward(x, x))
    _refused(V, "h has type", lambda: moe.swiglu_backward(x, gu, h=x.float()))
    _refused(V, "want_h", lambda: moe.swiglu_backward(x, gu, h=keep, want_h=False))
    torch.cuda.synchronize()
    assert (keep == 7).all()
