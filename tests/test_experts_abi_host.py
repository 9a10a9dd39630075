"""Host-only checks of the experts' step of the C ABI (include/moe_experts.h): the library
exports every function the header declares, sizes its workspace, and rejects bad
arguments with the documented status before enqueueing anything.

The calls run in a child process that sees no GPU (ROCR_VISIBLE_DEVICES=-1), with stand-in
pointers that nothing dereferences: every case fails a check.  The same child runs once
more against the library's host side built with AddressSanitizer and
UndefinedBehaviorSanitizer."""
import json
import os
import re
import subprocess
import sys
import textwrap

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "moe_experts.h")
CSRC = os.path.join(ROOT, "combine_moe_route_count_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"

INVALID, WORKSPACE = -1, -3


def _declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


CHILD = textwrap.dedent(r"""
import ctypes, json, sys
sys.path.insert(0, ROOT)
from combine_moe_route_count_amd import _experts as L
lib = L._lib()
NEXT = [0x1000000]
def buf(off=0):            # a stand-in buffer of its own, 1 GiB apart from the others
    NEXT[0] += 1 << 30
    return NEXT[0] + off
B = {n: buf() for n in "x q s y a as_ w ws_ pc po gu h dh dgu c sc idx wt w13 s13 w2 s2 out ws".split()}
res = {"exports": {n: hasattr(lib, n) for n in NAMES}}

def case(fn, order, base):
    def call(**kw):
        a = dict(base)
        assert all(k in a for k in kw), kw
        a.update(kw)
        st = fn(*[a[k] for k in order], None)
        return [st, lib.moe_last_error().decode()]
    return call

q = case(lib.moe_mxfp4_quantize, "x dt rows H q s".split(),
         dict(x=B["x"], dt=0, rows=5, H=64, q=B["q"], s=B["s"]))
res["mxfp4_quantize"] = {
    "dt": q(dt=2), "dt_unknown": q(dt=17), "H0": q(H=0), "H48": q(H=48), "Hneg": q(H=-32),
    "Hhuge": q(H=(1 << 24) + 32), "rows_neg": q(rows=-1), "rows_huge": q(rows=1 << 31),
    "x_null": q(x=None), "x_odd": q(x=B["x"] + 8), "q_null": q(q=None), "q_odd": q(q=B["q"] + 4),
    "s_null": q(s=None), "q_on_x": q(q=B["x"] + 16), "s_on_x": q(s=B["x"]), "s_on_q": q(s=B["q"] + 3),
}
dq = case(lib.moe_mxfp4_dequantize, "q s rows H y dt".split(),
          dict(q=B["q"], s=B["s"], rows=5, H=64, y=B["y"], dt=1))
res["mxfp4_dequantize"] = {
    "dt": dq(dt=3), "H": dq(H=16), "rows": dq(rows=-2), "q_null": dq(q=None), "q_odd": dq(q=B["q"] + 2),
    "s_null": dq(s=None), "y_null": dq(y=None), "y_odd": dq(y=B["y"] + 4), "y_on_q": dq(y=B["q"]),
    "y_on_s": dq(y=B["s"] & ~15),
}
pr = case(lib.moe_expert_product_mxfp4, "a sa rows H w sw N pc po E sg y dt".split(),
          dict(a=B["a"], sa=B["as_"], rows=9, H=64, w=B["w"], sw=B["ws_"], N=32, pc=B["pc"],
               po=B["po"], E=4, sg=0, y=B["y"], dt=0))
res["expert_product"] = {
    "dt": pr(dt=2), "H": pr(H=40), "N12": pr(N=12), "N0": pr(N=0), "N24_swiglu": pr(N=24, sg=1),
    "N_huge": pr(N=(1 << 24) + 16), "rows": pr(rows=-1), "rows_huge": pr(rows=1 << 31), "E0": pr(E=0),
    "E1025": pr(E=1025), "pc_null": pr(pc=None), "po_null": pr(po=None), "none": pr(pc=None, po=None),
    "pc_odd": pr(pc=B["pc"] + 2), "po_odd": pr(po=B["po"] + 1), "a_null": pr(a=None), "a_odd": pr(a=B["a"] + 8),
    "sa_null": pr(sa=None), "w_null": pr(w=None), "w_odd": pr(w=B["w"] + 1), "sw_null": pr(sw=None),
    "y_null": pr(y=None), "y_odd": pr(y=B["y"] + 2), "y_on_a": pr(y=B["a"]), "y_on_w": pr(y=B["w"] + 16),
    "y_on_sa": pr(y=B["as_"] & ~15), "y_on_sw": pr(y=B["ws_"] & ~15), "y_on_pc": pr(y=B["pc"] & ~15),
    "y_on_po": pr(y=B["po"] & ~15),
}
sw = case(lib.moe_swiglu, "gu dt rows I pc po E h hdt c sc".split(),
          dict(gu=B["gu"], dt=0, rows=5, I=128, pc=B["pc"], po=B["po"], E=4, h=B["h"], hdt=1,
               c=B["c"], sc=B["sc"]))
res["swiglu"] = {
    "dt": sw(dt=2), "hdt": sw(hdt=3), "I0": sw(I=0), "I64_save": sw(I=64), "I12": sw(I=12, c=None, sc=None),
    "Ihuge": sw(I=(1 << 24) + 128), "rows": sw(rows=-1), "gu_null": sw(gu=None), "gu_odd": sw(gu=B["gu"] + 8),
    "h_null": sw(h=None), "h_odd": sw(h=B["h"] + 4), "c_alone": sw(sc=None), "sc_alone": sw(c=None),
    "c_odd": sw(c=B["c"] + 8), "sc_odd": sw(sc=B["sc"] + 2), "pc_alone": sw(po=None), "po_alone": sw(pc=None),
    "E": sw(E=0), "pc_odd": sw(pc=B["pc"] + 1), "h_on_gu": sw(h=B["gu"]), "c_on_gu": sw(c=B["gu"]),
    "sc_on_gu": sw(sc=B["gu"] + 4), "c_on_h": sw(c=B["h"]), "sc_on_c": sw(sc=B["c"]), "h_on_pc": sw(h=B["pc"]),
}
sb = case(lib.moe_swiglu_backward, "dh ddt gu dt sc rows I pc po E dgu h odt".split(),
          dict(dh=B["dh"], ddt=0, gu=B["gu"], dt=2, sc=B["sc"], rows=5, I=128, pc=B["pc"], po=B["po"],
               E=4, dgu=B["dgu"], h=B["h"], odt=0))
res["swiglu_backward"] = {
    "ddt": sb(ddt=2), "dt_fp4": sb(dt=3), "odt": sb(odt=2), "I64_fp8": sb(I=64), "I4": sb(dt=0, sc=None, I=4),
    "rows": sb(rows=1 << 31), "dh_null": sb(dh=None), "dh_odd": sb(dh=B["dh"] + 2), "gu_null": sb(gu=None),
    "gu_odd": sb(gu=B["gu"] + 8), "sc_null": sb(sc=None), "sc_on_bf16": sb(dt=0), "sc_odd": sb(sc=B["sc"] + 1),
    "dgu_null": sb(dgu=None), "dgu_odd": sb(dgu=B["dgu"] + 8), "h_odd": sb(h=B["h"] + 8), "E": sb(E=1 << 20),
    "pc_alone": sb(po=None), "in_place": sb(dgu=B["gu"]), "dgu_on_dh": sb(dgu=B["dh"]),
    "h_on_dh": sb(h=B["dh"]), "h_on_dgu": sb(h=B["dgu"]), "dgu_on_sc": sb(dgu=B["sc"]),
}
need = lib.moe_experts_decode_workspace_size(5, 4, 64, 32)
de = case(lib.moe_experts_decode, "x T H idx w K E I w13 s13 w2 s2 wdt out odt ws n".split(),
          dict(x=B["x"], T=5, H=64, idx=B["idx"], w=B["wt"], K=4, E=8, I=32, w13=B["w13"], s13=B["s13"],
               w2=B["w2"], s2=B["s2"], wdt=3, out=B["out"], odt=0, ws=B["ws"], n=need))
res["experts_decode"] = {
    "odt": de(odt=2), "wdt_f32": de(wdt=1), "wdt_fp8": de(wdt=2), "H40": de(H=40), "I40": de(I=40),
    "H12_bf16": de(H=12, wdt=0, s13=None, s2=None), "H0": de(H=0), "I_huge": de(I=(1 << 20) + 32), "H_huge": de(H=(1 << 20) + 32),
    "K0": de(K=0), "K17": de(K=17), "Tneg": de(T=-1), "TK1025": de(T=1025, K=1), "TK_over": de(T=65, K=16),
    "Thuge": de(T=1 << 62), "E0": de(E=0), "E1025": de(E=1025), "x_null": de(x=None), "x_odd": de(x=B["x"] + 8),
    "idx_null": de(idx=None), "idx_odd": de(idx=B["idx"] + 2), "w_null": de(w=None), "w_odd": de(w=B["wt"] + 1),
    "w13_null": de(w13=None), "w13_odd": de(w13=B["w13"] + 8), "w2_null": de(w2=None), "w2_odd": de(w2=B["w2"] + 4),
    "s13_null": de(s13=None), "s2_null": de(s2=None), "scales_on_bf16": de(wdt=0), "one_scale": de(wdt=0, s2=None),
    "out_null": de(out=None), "out_odd": de(out=B["out"] + 2), "out_on_x": de(out=B["x"]),
    "out_on_w13": de(out=B["w13"]), "out_on_w2": de(out=B["w2"] + 64), "out_on_idx": de(out=B["idx"]),
    "out_on_wt": de(out=B["wt"]), "out_on_s13": de(out=B["s13"]), "out_on_s2": de(out=B["s2"]),
    "ws_on_x": de(ws=B["x"] & ~255), "ws_on_out": de(ws=B["out"] & ~255), "ws_on_w2": de(ws=B["w2"] & ~255),
}
res["decode_ws"] = {"null": de(ws=None), "small": de(n=need - 1), "odd": de(ws=B["ws"] + 128)}
size = lib.moe_experts_decode_workspace_size
res["grows"] = all(size(T, K, H, I) <= size(T + 1, K, H, I) <= size(T + 1, K + 1, H, I)
                   <= size(T + 1, K + 1, H + 8, I) <= size(T + 1, K + 1, H + 8, I + 8)
                   for T in (0, 1, 31, 59) for K in (1, 7, 15) for H in (8, 4096) for I in (8, 2048))
res["no_size"] = [size(-1, 1, 8, 8), size(1025, 1, 8, 8), size(65, 16, 8, 8), size(1, 0, 8, 8),
                  size(1, 17, 8, 8), size(1, 1, 8, 0), size(1, 1, 8, 12), size(1, 1, 12, 8),
                  size(1, 1, 8, (1 << 20) + 8), size(1, 1, (1 << 20) + 8, 8), size(1 << 62, 16, 8, 8)]
n = None
res["empty"] = [q(rows=0, x=n, q=n, s=n)[0], dq(rows=0, q=n, s=n, y=n)[0],
                pr(rows=0, a=n, sa=n, y=n)[0], sw(rows=0, gu=n, h=n)[0],
                sb(rows=0, dh=n, gu=n, sc=n, dgu=n)[0], de(T=0, x=n, idx=n, w=n, out=n)[0]]
print(json.dumps(res))
""")


def _run_child(**env):
    code = f"ROOT = {ROOT!r}\nNAMES = {_declared_functions()!r}\n" + CHILD
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=170,
                       env=dict(os.environ, ROCR_VISIBLE_DEVICES="-1", **env))
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
    return json.loads(r.stdout.splitlines()[-1])


@pytest.fixture(scope="module")
def res():
    return _run_child()


def _check(res):
    assert res["exports"] and all(res["exports"].values()), res["exports"]
    for op in ("mxfp4_quantize", "mxfp4_dequantize", "expert_product", "swiglu", "swiglu_backward",
               "experts_decode"):
        for name, (st, msg) in res[op].items():
            assert st == INVALID and msg, (op, name, st, msg)
    for name, (st, msg) in res["decode_ws"].items():
        assert st in (INVALID, WORKSPACE) and msg, (name, st, msg)
    assert res["decode_ws"]["small"][0] == WORKSPACE
    assert res["grows"]
    assert res["no_size"] == [0] * len(res["no_size"])
    assert res["empty"] == [0] * len(res["empty"])


def test_exports_and_argument_errors(res):
    _check(res)


def test_messages_name_the_argument(res):
    assert "H=48" in res["mxfp4_quantize"]["H48"][1]
    assert "y overlaps w" in res["expert_product"]["y_on_w"][1]
    assert "dgu overlaps gu" in res["swiglu_backward"]["in_place"][1]
    assert "T*K" in res["experts_decode"]["TK_over"][1]


def test_binding_refuses_tensors():
    """Off the GPU, and before anything about them is used."""
    import torch
    import combine_moe_route_count_amd as moe
    f, u, i = torch.zeros((4, 64)), torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(4, dtype=torch.int32)
    b = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: moe.mxfp4_quantize(f), lambda: moe.mxfp4_dequantize(u, u),
                 lambda: moe.expert_product_mxfp4(u, u, u.view(4, 1, 32), u, i, i),
                 lambda: moe.swiglu(f), lambda: moe.swiglu_backward(f, f),
                 lambda: moe.experts_decode(b, i.view(4, 1), f, b.view(4, 1, 64), b.view(4, 64, 1))):
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
