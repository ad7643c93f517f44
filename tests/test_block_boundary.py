"""Refusals of the operators of a residual block (ssd_block.h): host checks in the documented
order, none of which reaches a kernel launch, so they run without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import state_space_sequence_03_amd as lib
from state_space_sequence_03_amd import block, layer
from test_boundary import LLVM, device_disassembly, device_functions
from test_host_asan import CLANG_RT, HIPCC, _instrumented, _run_child

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssd_block.h")
OK, NULLP, SHAPE, DTYPE, MISAL, WS, UNSUP, BADVAL = 0, 1, 2, 4, 5, 6, 7, 10
PTR = 1 << 20      # 16-byte aligned, never dereferenced: a check fails first
ODD = PTR + 2
BIG = 2 ** 60


@pytest.fixture(scope="module", autouse=True)
def so():
    if not os.path.exists(lib.lib_path()):
        from state_space_sequence_03_amd import build
        build.build()
    return lib.load_library()


def test_exports_every_declared_symbol(so):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ssd_[a-z_0-9]+)\s*\(", text))
    assert names == {"ssd_block_abi_version", "ssd_add_norm_fwd", "ssd_add_norm_bwd", "ssd_add_norm_bwd_workspace_size",
                     "ssd_gated_norm_fwd_8bit", "ssd_quant8", "ssd_matmul8", "ssd_matmul8_workspace_size", "ssd_clip_grads",
                     "ssd_clip_grads_workspace_size"}
    for n in names:
        assert hasattr(so, n) and n in lib.__all__ and hasattr(lib, n), n
    assert lib.ssd_block_abi_version() == 1


def test_struct_sizes(tmp_path):
    # the C compiler's own sizes, from a small program that includes the header
    names = ["ssd_add_norm_problem", "ssd_quant8_problem", "ssd_matmul8_problem", "ssd_grad", "ssd_clip_options"]
    src = '#include <stdio.h>\n#include "%s"\nint main(void) { printf("%s", %s); return 0; }' % (
        HEADER, " ".join(["%zu"] * len(names)), ", ".join("sizeof(%s)" % n for n in names))
    exe = str(tmp_path / "struct_sizes")
    subprocess.run(["gcc", "-x", "c", "-", "-o", exe], input=src, text=True, check=True)
    sizes = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in sizes] == [ctypes.sizeof(getattr(block, n)) for n in names]


def p(v):
    return ctypes.c_void_p(v) if v else None


def st(batch, token):
    return ctypes.byref(layer.ssd_strides(batch, token))


def ref(prob):
    return None if prob is None else ctypes.byref(prob)


def size_of(name, prob):
    n = ctypes.c_size_t(7)
    return getattr(lib.load_library(), name)(ref(prob), ctypes.byref(n)), n.value


# ---- residual and norm ----

def AP(batch=2, seqlen=10, channels=64, eps=1e-5, io=1, res=0, reserved=0):
    return block.ssd_add_norm_problem(batch, seqlen, channels, eps, io, res, reserved)


def add_fwd(prob, x=PTR, xs=None, r=PTR, w=PTR, h=PTR, y=PTR, q=PTR, s=PTR):
    return lib.load_library().ssd_add_norm_fwd(ref(prob), p(x), xs, p(r), p(w), p(h), p(y), p(q), p(s), None)


def add_bwd(prob, h=PTR, w=PTR, dy=PTR, dh=PTR, dx=PTR, dr=PTR, dw=PTR, ws=PTR, n=0):
    return lib.load_library().ssd_add_norm_bwd(ref(prob), p(h), p(w), p(dy), p(dh), p(dx), p(dr), p(dw), p(ws), n, None)


BAD_ADD = [(dict(batch=0), SHAPE), (dict(seqlen=-1), SHAPE), (dict(channels=0), SHAPE), (dict(batch=2 ** 40, seqlen=2 ** 40), SHAPE),
           (dict(io=2), DTYPE), (dict(res=2), DTYPE), (dict(io=0, res=1), DTYPE), (dict(reserved=1), DTYPE),
           (dict(eps=-1.0), BADVAL), (dict(eps=float("nan")), BADVAL), (dict(eps=float("inf")), BADVAL),
           (dict(channels=8193), UNSUP), (dict(seqlen=2 ** 40), UNSUP)]


@pytest.mark.parametrize("kw,code", BAD_ADD)
def test_add_norm_bad_problem(kw, code):
    assert add_fwd(AP(**kw)) == code and lib.ssd_last_error_message()
    assert add_bwd(AP(**kw), n=BIG) == code
    assert size_of("ssd_add_norm_bwd_workspace_size", AP(**kw)) == (code, 7)


def test_add_norm_pointers():
    assert add_fwd(None) == NULLP and add_bwd(None) == NULLP
    for kw in (dict(x=0), dict(w=0), dict(y=0, q=0, s=0), dict(q=0), dict(s=0)):
        assert add_fwd(AP(), **kw) == NULLP, kw
    assert add_fwd(AP(batch=0), x=0) == NULLP
    for k in ("r", "w", "h", "y", "q", "s"):
        assert add_fwd(AP(), **{k: ODD}) == MISAL, k
    assert add_fwd(AP(), x=PTR + 1) == MISAL and add_fwd(AP(io=0), x=ODD) == MISAL
    assert add_fwd(AP(), xs=st(-1, 64)) == BADVAL and add_fwd(AP(), xs=st(2 ** 62, 64)) == SHAPE
    assert add_fwd(AP(), x=PTR + 1, xs=st(0, -1)) == BADVAL          # strides before alignment
    for kw in (dict(h=0), dict(w=0), dict(dy=0), dict(dx=0, dr=0), dict(dw=0), dict(ws=0)):
        assert add_bwd(AP(), **kw) == NULLP, kw
    for k in ("h", "w", "dy", "dh", "dx", "dr", "dw", "ws"):
        assert add_bwd(AP(), n=BIG, **{k: ODD}) == MISAL, k
    code, need = size_of("ssd_add_norm_bwd_workspace_size", AP())
    assert code == OK and need > 0 and add_bwd(AP(), n=need - 1) == WS
    assert size_of("ssd_add_norm_bwd_workspace_size", None)[0] == NULLP


def test_gated_norm_8bit():
    def call(x=PTR, z=PTR, zs=None, w=PTR, q=PTR, s=PTR, batch=2, seqlen=10, channels=256, groups=2, eps=1e-5, before=0, io=1, reserved=0):
        prob = layer.ssd_gated_norm_problem(batch, seqlen, channels, groups, eps, before, io, reserved)
        return lib.load_library().ssd_gated_norm_fwd_8bit(ref(prob), p(x), p(z), zs, p(w), p(q), p(s), None)
    for k in ("x", "w", "q", "s"):
        assert call(**{k: 0}) == NULLP and call(**{k: ODD}) == MISAL, k
    assert call(z=PTR + 1) == MISAL and call(zs=st(-1, 0)) == BADVAL and call(groups=3) == SHAPE and call(io=7) == DTYPE
    assert call(before=2) == BADVAL and call(eps=-1.0) == BADVAL and call(reserved=1) == DTYPE
    assert call(channels=200, groups=2) == UNSUP and call(channels=2 * 8193, groups=2) == UNSUP
    assert call(seqlen=2 ** 40) == UNSUP


def test_norms_refuse_what_their_own_launch_cannot_hold():
    # forwards 16 threads for a token of up to 128 channels, 512 for one of 4096; backwards any number of tokens
    for n, C in ((2 ** 28, 128), (2 ** 27, 129), (2 ** 23, 4096)):
        assert add_fwd(AP(batch=1, seqlen=n, channels=C)) == UNSUP, (n, C)
    for kw in (dict(batch=1, seqlen=2 ** 31), dict(batch=2 ** 16, seqlen=2 ** 15)):
        assert add_fwd(AP(channels=1, **kw)) == UNSUP and add_bwd(AP(channels=1, **kw), n=BIG) == UNSUP, kw
        assert size_of("ssd_add_norm_bwd_workspace_size", AP(channels=1, **kw)) == (UNSUP, 7)
    for kw in (dict(batch=1, seqlen=2 ** 23), dict(batch=1, seqlen=2 ** 31 - 1), dict(batch=2 ** 15, seqlen=2 ** 15)):
        code, need = size_of("ssd_add_norm_bwd_workspace_size", AP(**kw))
        assert code == OK and 0 < need < 2 ** 24 and add_bwd(AP(**kw), n=need - 1) == WS, kw


# ---- quantising ----

def QP(batch=2, seqlen=10, channels=64, io=1, tile=0, reserved=0):
    return block.ssd_quant8_problem(batch, seqlen, channels, io, tile, reserved)


def quant(prob, x=PTR, xs=None, q=PTR, s=PTR, qt=PTR, t=PTR):
    return lib.load_library().ssd_quant8(ref(prob), p(x), xs, p(q), p(s), p(qt), p(t), None)


def test_quant8():
    assert quant(None) == NULLP
    for kw in (dict(x=0), dict(q=0), dict(s=0), dict(qt=0), dict(t=0), dict(q=0, s=0, qt=0, t=0)):
        assert quant(QP(), **kw) == NULLP, kw
    for kw, code in ((dict(batch=0), SHAPE), (dict(channels=-3), SHAPE), (dict(batch=2 ** 40, seqlen=2 ** 40), SHAPE),
                     (dict(seqlen=2 ** 62), SHAPE), (dict(io=3), DTYPE), (dict(reserved=9), DTYPE), (dict(tile=2), BADVAL),
                     (dict(tile=-1), BADVAL), (dict(seqlen=2 ** 31), UNSUP), (dict(channels=2 ** 31, seqlen=1, batch=1), UNSUP),
                     (dict(seqlen=2 ** 24, channels=2 ** 16), UNSUP)):
        assert quant(QP(**kw)) == code, kw
    for k in ("q", "s", "qt", "t"):
        assert quant(QP(), **{k: ODD}) == MISAL, k
    assert quant(QP(), x=PTR + 1) == MISAL and quant(QP(), xs=st(0, -1)) == BADVAL and quant(QP(), xs=st(2 ** 62, 0)) == SHAPE


def test_quant8_refuses_what_its_own_launch_cannot_hold():
    # rows alone: 16 threads for each 128 of a row; tiles: 256 for each 128 x 128
    assert quant(QP(batch=1, seqlen=2 ** 28, channels=128), qt=0, t=0) == UNSUP
    for kw in (dict(tile=1), dict(tile=0)):
        assert quant(QP(batch=1, seqlen=2 ** 28, channels=1024, **kw)) == UNSUP, kw
        assert quant(QP(batch=1, seqlen=2 ** 28, channels=1024, **kw), q=0, s=0) == UNSUP, kw
    assert quant(QP(batch=1, seqlen=2 ** 28, channels=1024, tile=1), qt=0, t=0) == UNSUP


# ---- matrix product ----

def MP(rows=20, cols=30, depth=256, tile=1, out=1, reserved=0):
    return block.ssd_matmul8_problem(rows, cols, depth, tile, out, reserved)


def matmul(prob, x=PTR, xs=PTR, w=PTR, ws=PTR, y=PTR, mem=PTR, n=BIG):
    return lib.load_library().ssd_matmul8(ref(prob), p(x), p(xs), p(w), p(ws), p(y), p(mem), n, None)


BAD_MM = [(dict(rows=0), SHAPE), (dict(cols=-1), SHAPE), (dict(depth=0), SHAPE), (dict(depth=130), SHAPE),
          (dict(rows=2 ** 40, cols=2 ** 40), SHAPE), (dict(out=2), DTYPE), (dict(reserved=1), DTYPE), (dict(tile=2), BADVAL),
          (dict(rows=2 ** 31), UNSUP), (dict(cols=2 ** 33), UNSUP), (dict(depth=2 ** 31), UNSUP), (dict(rows=2 ** 22, cols=2 ** 22), UNSUP)]


@pytest.mark.parametrize("kw,code", BAD_MM)
def test_matmul8_bad_problem(kw, code):
    assert matmul(MP(**kw)) == code and lib.ssd_last_error_message()
    assert size_of("ssd_matmul8_workspace_size", MP(**kw)) == (code, 7)


def test_matmul8_pointers():
    assert matmul(None) == NULLP and size_of("ssd_matmul8_workspace_size", None)[0] == NULLP
    for k in ("x", "xs", "w", "ws", "y"):
        assert matmul(MP(), **{k: 0}) == NULLP and matmul(MP(), **{k: ODD}) == MISAL, k
    assert matmul(MP(), mem=ODD) == MISAL
    assert size_of("ssd_matmul8_workspace_size", MP())[0] == OK


def test_matmul8_refuses_what_its_own_launch_cannot_hold():
    # 512 threads for 16 columns of up to 16 rows, 256 for tiles of 64 x 64 and 128 x 128, 512 for 256 x 256
    size = "ssd_matmul8_workspace_size"
    for rows, cols, out in ((16, 2 ** 27 - 16, 1), (17, 2 ** 30 - 64, 0), (2 ** 30 - 64, 64, 1), (131077, 262147, 1), (131077, 262147, 0),
                            (2 ** 22, 10576, 1)):
        assert size_of(size, MP(rows, cols, 128, out=out)) == (OK, 0), (rows, cols, out)
    for rows, cols, out in ((16, 2 ** 27, 1), (17, 2 ** 30, 0), (2 ** 30, 64, 1), (2 ** 20, 2 ** 20, 1), (2 ** 20, 2 ** 20, 0)):
        assert size_of(size, MP(rows, cols, 128, out=out)) == (UNSUP, 7) and matmul(MP(rows, cols, 128, out=out)) == UNSUP


def test_products_of_every_form_are_tested(tmp_path):
    # every form of the plan, its depth whole and split, for results in bf16 and in fp32, has sizes among those that
    # the GPU tests run (by tile and by row each)
    from test_gpu_block import PRODUCT, PRODUCT_128
    src = tmp_path / "plan.cpp"
    src.write_text('#include <cstdio>\n#include "matmul8_plan.hpp"\n'
                   'int main() {\n  long long m, n, k;\n  int bf16;\n'
                   '  while (std::scanf("%lld %lld %lld %d", &m, &n, &k, &bf16) == 4) {\n'
                   '    const ssd::Matmul8Plan p = ssd::matmul8_plan(m, n, k, bf16);\n'
                   '    std::printf("%d %d %d\\n", (int)p.form, p.parts, p.each);\n  }\n}\n')
    exe = str(tmp_path / "plan")
    csrc = os.path.join(ROOT, "state_space_sequence_03_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I" + csrc, str(src), "-o", exe], check=True)
    cases = [(size, bf16) for size in PRODUCT + PRODUCT_128 for bf16 in (0, 1)]
    text = "".join("%d %d %d %d\n" % (size + (bf16,)) for size, bf16 in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    seen = {}
    for (size, bf16), line in zip(cases, out):
        form, parts, each = (int(v) for v in line.split())
        blocks = size[2] // 128
        assert (parts - 1) * each < blocks <= parts * each, (size, line)
        # the library's own plan: its workspace holds the parts
        need = 4 * parts * size[0] * size[1] if parts > 1 else 0
        assert size_of("ssd_matmul8_workspace_size", MP(*size, out=bf16)) == (OK, need), (size, line)
        seen.setdefault((["few", 64, 128, 256][form], parts > 1, bf16), []).append(size)
    want = {("few", False, b) for b in (0, 1)} | {(t, split, b) for t in (64, 128) for split in (False, True) for b in (0, 1)}
    assert set(seen) == want | {(256, False, 1)}, sorted(seen, key=str)
    # more than one block of the depth, and ends of both sides inside a tile, in every one of the tiled forms
    for (form, split, _), sizes in seen.items():
        if form != "few":
            assert any(k > 128 for _, _, k in sizes) and any(m % form and n % form for m, n, _ in sizes), (form, split, sizes)


# ---- clipping ----

def clip(items, n=None, most=1.0, eps=1e-6, scale=1.0, reserved=0, norm=PTR << 8, ws=PTR << 9, ws_bytes=BIG, none=None):
    arr = (block.ssd_grad * max(1, len(items)))(*[block.ssd_grad(*i) for i in items])
    opt = block.ssd_clip_options(most, eps, scale, reserved)
    return lib.load_library().ssd_clip_grads(None if none == "grads" else ctypes.addressof(arr), len(items) if n is None else n,
                                             None if none == "opt" else ctypes.byref(opt), p(norm), p(ws), ws_bytes, None)


def test_clip_grads():
    A, B, C = PTR, PTR + 4096, PTR + 8192
    ok = [(A, A, 1000, 0, 0), (B, C, 500, 1, 0)]
    assert clip(ok, none="grads") == NULLP and clip(ok, none="opt") == NULLP and clip(ok, norm=0) == NULLP and clip(ok, ws=0) == NULLP
    assert clip([(None, A, 3, 0, 0)]) == NULLP and clip([(A, None, 3, 0, 0)]) == NULLP
    assert clip(ok, n=0) == SHAPE and clip(ok, n=-4) == SHAPE and clip([(A, A, -1, 0, 0)]) == SHAPE
    assert clip([(A, A, 4, 2, 0)]) == DTYPE and clip([(A, A, 4, 0, -1)]) == DTYPE and clip(ok, reserved=1) == DTYPE
    nan, inf = float("nan"), float("inf")
    for kw in (dict(most=0.0), dict(most=-1.0), dict(most=nan), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(scale=0.0),
               dict(scale=nan), dict(scale=inf)):
        assert clip(ok, **kw) == BADVAL, kw
    assert clip([(A, B, 2 ** 41, 0, 0)]) == UNSUP
    # overlaps: out over another tensor's grad or out, over a part of its own, over its own of another type, over norm
    for items in ([(A, A, 1000, 0, 0), (A, C, 10, 0, 0)], [(A, C, 10, 0, 0), (A, A, 1000, 0, 0)], [(A, A, 10, 0, 0), (A, A, 10, 0, 0)],
                  [(A, C, 10, 0, 0), (B, C + 36, 10, 0, 0)], [(A, A + 4, 10, 0, 0)], [(A, A, 10, 1, 0)], [(A, A, 10, 0, 1)]):
        assert clip(items) == BADVAL, items
    assert clip(ok, norm=A + 8) == BADVAL and clip(ok, norm=B) == BADVAL
    # side by side, read twice, empty ones anywhere: past the checks, to the workspace's
    for items in (ok, [(A, C, 10, 0, 0), (A, C + 40, 10, 0, 0)], [(A, A, 0, 0, 0), (A, A, 10, 0, 0), (0, 0, 0, 1, 1)]):
        assert clip(items, ws_bytes=4) == WS, items
    assert clip([(A + 1, C, 4, 1, 0)]) == MISAL and clip([(A, C + 2, 4, 1, 0)]) == MISAL and clip([(A + 2, C, 4, 1, 0)], ws_bytes=4) == WS
    assert clip(ok, norm=(PTR << 8) + 2) == MISAL and clip(ok, ws=(PTR << 9) + 8) == MISAL
    n = ctypes.c_size_t(7)
    size = lib.load_library().ssd_clip_grads_workspace_size
    arr = (block.ssd_grad * 2)(*[block.ssd_grad(*i) for i in ok])
    assert size(ctypes.addressof(arr), 2, ctypes.byref(n)) == OK and n.value >= 16
    assert size(None, 2, ctypes.byref(n)) == NULLP and size(ctypes.addressof(arr), 0, ctypes.byref(n)) == SHAPE


# ---- the Python binding ----

def test_binding_rejects_cpu_tensors():
    x, w = torch.zeros(1, 2, 128), torch.zeros(128)
    t8 = lib.Tensor8(torch.zeros(2, 128).to(torch.float8_e4m3fn), torch.zeros(1, 2))
    for call in (lambda: lib.ssd_add_norm_fwd(x, None, w), lambda: lib.ssd_add_norm_bwd(x, w, x), lambda: lib.ssd_quant8(x),
                 lambda: lib.ssd_gated_norm_fwd_8bit(x, None, w), lambda: lib.ssd_matmul8(t8, t8), lambda: lib.ssd_clip_grads([x], 1.0)):
        with pytest.raises(lib.SsdArgumentError):
            call()


@pytest.mark.skipif(not CLANG_RT or not os.path.exists(HIPCC), reason="ROCm clang ASan runtime missing")
@pytest.mark.skipif("SSD_LIBRARY" in os.environ, reason="this is the instrumented run")
def test_host_code_under_asan(tmp_path):
    from state_space_sequence_03_amd import build as b
    objs = {os.path.splitext(s)[0]: os.path.join(b.BUILD_DIR, os.path.splitext(s)[0] + ".o") for s in b.SOURCES}
    if not all(os.path.exists(o) for o in objs.values()):
        b.build()
    asan = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]
    for src in ("ssd_api.cpp", "block_api.cpp"):
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        subprocess.run([HIPCC] + b.COMMON_FLAGS + asan + ["-x", "hip", "-c", os.path.join(b.CSRC, src), "-o", obj],
                       check=True, capture_output=True, text=True)
        objs[os.path.splitext(src)[0]] = obj
    so = str(tmp_path / "libssd_asan.so")
    subprocess.run([HIPCC, "--offload-arch=" + b.ARCH, "-shared", "-fPIC", "-shared-libasan",
                    "-Xarch_host", "-fsanitize=address", "-o", so] + list(objs.values()), check=True,
                   capture_output=True, text=True)
    assert _instrumented(so)
    _run_child(["tests/test_block_boundary.py"], {"LD_PRELOAD": CLANG_RT[-1], "SSD_LIBRARY": so})


# ---- the built device code ----

@pytest.mark.skipif(not os.path.exists("%s/llvm-objdump" % LLVM), reason="ROCm LLVM tools not installed")
@pytest.mark.parametrize("obj", ["add_norm.o", "quant8.o", "matmul8.o", "clip.o"])
def test_device_code(so, obj, tmp_path):
    # M0 is written for the direct-to-LDS loads alone, each write followed by its load; nothing is written
    # through the scalar data cache, no packed fp32 operation is there, and no register goes to memory
    # (spilled ones would be vector memory operations that the products' waits do not count)
    insts = device_disassembly(obj, tmp_path)
    assert insts, "no device code found"
    for k, ins in enumerate(insts):
        op = ins.split()[0] if ins else ""
        assert not re.match(r"s_(store|atomic|buffer_store|buffer_atomic|scratch_store|dcache_wb|dcache_discard)", op), ins
        assert not re.match(r"v_pk_(add|mul|fma)_f32", op) and not op.startswith("scratch_"), ins
        fields = [f.strip() for f in ins[len(op):].split(",")]
        if fields and fields[0] == "m0" and op.startswith("s_"):
            nxt = [i for i in insts[k + 1:k + 3] if not i.startswith("s_nop")]
            assert nxt and nxt[0].startswith("global_load_lds"), (obj, ins, insts[k + 1:k + 3])
    if obj == "matmul8.o":
        assert any(i.startswith("global_load_lds_dwordx4") for i in insts) and not any(i.startswith("s_bfe_i64") for i in insts)


@pytest.mark.skipif(not os.path.exists("%s/llvm-objdump" % LLVM), reason="ROCm LLVM tools not installed")
def test_products_wait_for_counted_loads(so, tmp_path):
    # The loop of the tiled products waits for all but a counted number of its latest loads: two waits in a
    # block of the depth, with kFirst + kHalfN loads between two of the same kind.  Every other vector memory
    # operation of the kernel lies behind the loop (the stores of y), so that the counts hold.
    funcs = {f: i for f, i in device_functions("matmul8.o", tmp_path).items() if "14matmul8_kernel" in f}
    # <results, y, NT, MT, WN, WM, by tile>: loads of a block for one wave
    loads = {"Li8ELi4ELi2ELi4E": 2 * 4 // 2 + 1 + 2 * (8 // 4), "Li4ELi4ELi2ELi2E": 2 * 4 // 2 + 1 + 2 * (4 // 2),
             "Li2ELi2ELi2ELi2E": 2 * 2 // 2 + 1 + 2 * (2 // 2)}
    seen = set()
    for name, insts in funcs.items():
        kind = next(k for k in loads if k in name)
        seen.add(kind)
        waits = [k for k, i in enumerate(insts) if re.match(r"s_waitcnt vmcnt\(%d\) lgkmcnt\(0\)" % loads[kind], i)]
        assert len(waits) == 3, (name, len(waits))          # in front of the loop, and two in it
        lds = [k for k, i in enumerate(insts) if i.startswith("global_load_lds")]
        others = [k for k, i in enumerate(insts) if re.match(r"(global|flat|buffer)_(load|store)", i) and k not in lds]
        assert min(others) > max(lds), name
        in_loop = [k for k in lds if k > waits[0]]
        assert len(in_loop) == loads[kind], (name, len(in_loop))
    assert seen == set(loads)
