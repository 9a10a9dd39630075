"""Host-only checks of the training side of the C ABI (include/moe_train.h): the
library exports every function the header declares, sizes its workspace, and
rejects bad arguments with the documented status before enqueueing anything.

The calls run in a child process that sees no GPU (ROCR_VISIBLE_DEVICES=-1), with
stand-in pointers that nothing dereferences: every case fails a check.  The same
child runs once more against the library's host side built with AddressSanitizer
and UndefinedBehaviorSanitizer."""
import json
import os
import re
import subprocess
import sys
import textwrap

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "moe_train.h")
CSRC = os.path.join(ROOT, "combine_moe_route_count_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"

INVALID, WORKSPACE = -1, -3


def _declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


CHILD = textwrap.dedent(r"""
import ctypes, json, sys
sys.path.insert(0, ROOT)
from combine_moe_route_count_amd import _train as L
lib = L._lib()
P = ctypes.c_void_p
NEXT = [0x1000000]
def buf(off=0):            # a stand-in buffer of its own, 1 GiB apart from the others
    NEXT[0] += 1 << 30
    return NEXT[0] + off
B = {n: buf() for n in "logits idx w dw dlogits dout dow y ys tm dy pc po dp res dx table ids out st dt ws".split()}
res = {"exports": {n: hasattr(lib, n) for n in NAMES}}

def case(fn, order, base):
    def call(**kw):
        a = dict(base)
        a.update(kw)
        st = fn(*[a[k] for k in order], None)
        return [st, lib.moe_last_error().decode()]
    return call

gate = case(lib.moe_gate, "x dt T E K rn sc idx w".split(),
            dict(x=B["logits"], dt=1, T=5, E=16, K=4, rn=1, sc=1.0, idx=B["idx"], w=B["w"]))
res["gate"] = {
    "Tneg": gate(T=-1), "Thuge": gate(T=1 << 31), "E0": gate(E=0), "E1025": gate(E=1025),
    "K0": gate(K=0), "K17": gate(K=17, E=64), "K_over_E": gate(K=5, E=4), "dt_fp8": gate(dt=2),
    "dt_unknown": gate(dt=9), "x_null": gate(x=None), "x_odd": gate(x=B["logits"] + 2),
    "bf16_odd": gate(dt=0, x=B["logits"] + 1), "idx_null": gate(idx=None),
    "idx_odd": gate(idx=B["idx"] + 2), "w_null": gate(w=None), "w_odd": gate(w=B["w"] + 1),
    "idx_on_logits": gate(idx=B["logits"] + 16), "w_on_logits": gate(w=B["logits"]),
    "w_on_idx": gate(w=B["idx"] + 4), "TK": gate(T=(1 << 31) - 1, K=2),
}
gateb = case(lib.moe_gate_backward, "x dt T E K rn sc idx dw dl".split(),
             dict(x=B["logits"], dt=0, T=5, E=16, K=4, rn=0, sc=1.0, idx=B["idx"], dw=B["dw"],
                  dl=B["dlogits"]))
res["gate_backward"] = {
    "E0": gateb(E=0), "K_over_E": gateb(K=8, E=7), "dt": gateb(dt=3), "idx_null": gateb(idx=None),
    "dw_null": gateb(dw=None), "dl_null": gateb(dl=None), "dl_odd": gateb(dl=B["dlogits"] + 1),
    "in_place": gateb(dl=B["logits"]), "dl_on_idx": gateb(dl=B["idx"]), "dl_on_dw": gateb(dl=B["dw"]),
    "Tneg": gateb(T=-1),
}
comb = case(lib.moe_combine_backward,
            "dout ddt dow T H y ydt ys rows tm w K dy dydt pc po E dw".split(),
            dict(dout=B["dout"], ddt=0, dow=B["dow"], T=5, H=128, y=B["y"], ydt=0, ys=None, rows=10,
                 tm=B["tm"], w=B["w"], K=2, dy=B["dy"], dydt=0, pc=B["pc"], po=B["po"], E=8,
                 dw=B["dw"]))
res["combine_backward"] = {
    "Tneg": comb(T=-1), "Thuge": comb(T=1 << 62), "K0": comb(K=0), "K17": comb(K=17),
    "TK": comb(T=1 << 30, K=2), "H0": comb(H=0), "H12": comb(H=12), "Hhuge": comb(H=(1 << 24) + 8),
    "fp8_H64": comb(ydt=2, H=64), "ddt": comb(ddt=2), "dydt": comb(dydt=3), "ydt": comb(ydt=7),
    "dout_null": comb(dout=None), "dout_odd": comb(dout=B["dout"] + 8), "dow_odd": comb(dow=B["dow"] + 2),
    "y_null": comb(y=None), "y_odd": comb(y=B["y"] + 4), "scales_on_bf16": comb(ys=B["ys"]),
    "scales_odd": comb(ydt=2, ys=B["ys"] + 1), "rows_neg": comb(rows=-1), "rows_huge": comb(rows=1 << 31),
    "tm_null": comb(tm=None), "tm_odd": comb(tm=B["tm"] + 4), "w_null": comb(w=None), "w_odd": comb(w=B["w"] + 2),
    "dy_odd": comb(dy=B["dy"] + 8), "nothing": comb(dy=None, dw=None), "dw_odd": comb(dw=B["dw"] + 1),
    "pc_alone": comb(po=None), "po_alone": comb(pc=None), "E0": comb(E=0), "E1025": comb(E=1025),
    "pc_odd": comb(pc=B["pc"] + 2), "dy_on_y": comb(dy=B["y"]), "dy_on_dout": comb(dy=B["dout"]),
    "dy_on_w": comb(dy=B["w"] & ~15), "dy_on_tm": comb(dy=B["tm"]), "dw_on_y": comb(dw=B["y"] + 64),
    "dw_on_dy": comb(dw=B["dy"] + 64), "dw_on_w": comb(dw=B["w"]), "dw_on_tm": comb(dw=B["tm"]),
    "dw_on_dout": comb(dw=B["dout"]), "dw_on_dow": comb(dw=B["dow"]), "dy_on_dow": comb(dy=B["dow"]),
    "dw_on_scales": comb(ydt=2, ys=B["ys"], dw=B["ys"] + 8), "dy_on_scales": comb(ydt=3, ys=B["ys"], dy=B["ys"]),
    "dy_on_pc": comb(dy=B["pc"]), "dy_on_po": comb(dy=B["po"]), "dw_on_po": comb(dw=B["po"] + 32),
}
disp = case(lib.moe_dispatch_backward, "dp ddt rows H tm T K res dx dxdt".split(),
            dict(dp=B["dp"], ddt=0, rows=10, H=64, tm=B["tm"], T=5, K=2, res=B["res"], dx=B["dx"], dxdt=0))
res["dispatch_backward"] = {
    "Tneg": disp(T=-1), "K0": disp(K=0), "K17": disp(K=17), "H12": disp(H=12), "ddt": disp(ddt=2),
    "dxdt": disp(dxdt=4), "rows_neg": disp(rows=-1), "rows_huge": disp(rows=1 << 31),
    "dp_null": disp(dp=None), "dp_odd": disp(dp=B["dp"] + 8), "tm_null": disp(tm=None),
    "tm_odd": disp(tm=B["tm"] + 4), "dx_null": disp(dx=None), "dx_odd": disp(dx=B["dx"] + 4),
    "res_odd": disp(res=B["res"] + 8), "dx_on_dp": disp(dx=B["dp"]), "dx_on_tm": disp(dx=B["tm"]),
    "res_shifted": disp(res=B["dx"] + 16),
}
emb = case(lib.moe_embedding, "tb tdt V H ids ib N sc out odt st".split(),
           dict(tb=B["table"], tdt=0, V=100, H=64, ids=B["ids"], ib=4, N=5, sc=1.0, out=B["out"], odt=0,
                st=B["st"]))
res["embedding"] = {
    "tdt": emb(tdt=2), "odt": emb(odt=2), "V0": emb(V=0), "Vhuge": emb(V=1 << 31), "H12": emb(H=12),
    "Nneg": emb(N=-1), "Nhuge": emb(N=1 << 31), "ib": emb(ib=2), "ids_null": emb(ids=None),
    "ids_odd": emb(ids=B["ids"] + 2), "ids64_odd": emb(ib=8, ids=B["ids"] + 4), "tb_null": emb(tb=None),
    "tb_odd": emb(tb=B["table"] + 8), "out_null": emb(out=None), "out_odd": emb(out=B["out"] + 2),
    "st_odd": emb(st=B["st"] + 1), "out_on_tb": emb(out=B["table"] + 1024), "out_on_ids": emb(out=B["ids"]),
    "st_on_out": emb(st=B["out"]), "st_on_ids": emb(st=B["ids"]), "st_on_tb": emb(st=B["table"]),
}
need = lib.moe_embedding_workspace_size(5, 100, 64)
embb = case(lib.moe_embedding_backward, "do ddt ids ib N V H sc acc dt dtdt ws wsb".split(),
            dict(do=B["dout"], ddt=0, ids=B["ids"], ib=8, N=5, V=100, H=64, sc=1.0, acc=0, dt=B["dt"], dtdt=1,
                 ws=B["ws"], wsb=need))
res["embedding_backward"] = {
    "ddt": embb(ddt=3), "dtdt": embb(dtdt=2), "V0": embb(V=0), "Vhuge": embb(V=1 << 31), "H12": embb(H=12),
    "Nneg": embb(N=-1), "Nhuge": embb(N=1 << 31), "ib": embb(ib=3), "ids_null": embb(ids=None),
    "ids_odd": embb(ids=B["ids"] + 4), "do_null": embb(do=None), "do_odd": embb(do=B["dout"] + 8),
    "dt_null": embb(dt=None), "dt_odd": embb(dt=B["dt"] + 8), "dt_on_do": embb(dt=B["dout"]),
    "dt_on_ids": embb(dt=B["ids"]), "ws_on_do": embb(ws=B["dout"]), "ws_on_ids": embb(ws=B["ids"]),
    "ws_on_dt": embb(ws=B["dt"]),
}
res["embedding_ws"] = {"small": embb(wsb=need - 1), "null": embb(ws=None), "odd": embb(ws=B["ws"] + 16)}
sz = lib.moe_embedding_workspace_size
res["sizes"] = [sz(0, 1, 8), sz(1, 1, 8), sz(65536, 131072, 4096), sz((1 << 31) - 1, (1 << 31) - 1, 8)]
res["no_size"] = [sz(-1, 1, 8), sz(1 << 31, 1, 8), sz(1, 0, 8), sz(1, 1 << 31, 8), sz(1, 1, 12),
                  sz(1, 1, 0), sz(1, 1, (1 << 24) + 8)]
# nothing to do is not an error: no rows, no launch
res["empty"] = [gate(T=0, x=None, idx=None, w=None)[0], gateb(T=0, x=None, idx=None, dw=None, dl=None)[0],
                disp(T=0, tm=None, dx=None, res=None)[0], emb(N=0, ids=None, out=None, st=None)[0],
                embb(N=0, ids=None, do=None, acc=1)[0], comb(T=0, dout=None, tm=None, w=None, dw=None,
                                                             pc=None, po=None)[0]]
print(json.dumps(res))
""")


def _run_child(**extra):
    env = dict(os.environ, ROCR_VISIBLE_DEVICES="-1", HIP_VISIBLE_DEVICES="-1", **extra)
    code = f"ROOT = {ROOT!r}\nNAMES = {_declared_functions()!r}\n" + CHILD
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env,
                       timeout=150)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.fixture(scope="module")
def res():
    return _run_child()


def _check(res):
    assert res["exports"] and all(res["exports"].values()), res["exports"]
    for op in ("gate", "gate_backward", "combine_backward", "dispatch_backward", "embedding",
               "embedding_backward"):
        for name, (st, msg) in res[op].items():
            assert st == INVALID and msg, (op, name, st, msg)
    for name, (st, msg) in res["embedding_ws"].items():
        assert st == WORKSPACE and msg, (name, st, msg)
    assert res["empty"] == [0] * len(res["empty"])


def test_exports_and_argument_errors(res):
    _check(res)


def test_workspace_sizes(res):
    assert all(s > 0 and s % 256 == 0 for s in res["sizes"]), res["sizes"]
    assert res["no_size"] == [0] * len(res["no_size"])


def test_messages_name_the_argument(res):
    assert "K=5" in res["gate"]["K_over_E"][1]
    assert "dy overlaps y" in res["combine_backward"]["dy_on_y"][1]
    assert "dx overlaps residual" in res["dispatch_backward"]["res_shifted"][1]
    assert "id_bytes=2" in res["embedding"]["ib"][1]


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    import combine_moe_route_count_amd as moe
    f, i, m = torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int64)
    for call in (lambda: moe.gate(f, 2), lambda: moe.gate_backward(f, m.int(), torch.zeros((4, 2))),
                 lambda: moe.combine_backward(f, f, m, torch.zeros((4, 2))),
                 lambda: moe.dispatch_backward(f, m), lambda: moe.embedding(i, f),
                 lambda: moe.embedding_backward(f, i, 8)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_host_code_under_asan_ubsan(tmp_path):
    from combine_moe_route_count_amd import build
    san_src = [s for s in build.SOURCES if s.startswith("api")]
    objs = [os.path.join(ROOT, "_build", s + ".o") for s in build.SOURCES if s not in san_src]
    if not os.path.exists(CLANG) or not all(os.path.exists(o) for o in objs):
        pytest.skip("needs the ROCm clang and the objects of a prior build()")
    rt = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"],
                        capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(rt) or not os.path.exists(rt):
        pytest.skip("clang sanitizer runtime not installed")
    rocm = os.path.dirname(os.path.dirname(os.path.dirname(CLANG)))
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"]
    built = []
    for s in san_src:
        o = str(tmp_path / (s + ".o"))
        subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fPIC", "-fvisibility=hidden", *san,
                        "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"),
                        "-c", os.path.join(CSRC, s), "-o", o], check=True)
        built.append(o)
    lib = str(tmp_path / "libmoe_route_san.so")
    subprocess.run([CLANG, "-shared", "-fPIC", *san, "-shared-libsan", "-o", lib, *built, *objs,
                    "-L", os.path.join(rocm, "lib"), "-lamdhip64",
                    "-Wl,-rpath," + os.path.join(rocm, "lib")], check=True)
    _check(_run_child(MOE_ROUTE_LIB=lib, LD_PRELOAD=rt,
                      LD_LIBRARY_PATH=os.path.dirname(rt) + ":" + os.environ.get("LD_LIBRARY_PATH", ""),
                      ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1"))
