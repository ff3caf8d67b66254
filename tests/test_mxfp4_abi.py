"""Refusals of the dense MXFP4 and the router's training entry points (no GPU
needed: every call here returns before any launch; the pointers are never
dereferenced), scratch sizes, and the binding's own checks."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import test_abi  # noqa: F401  (builds the library where none is there)
import mxfp4_quantized_weights_amd as M

FAKE = ctypes.c_void_p(0x10000)
ODD2, ODD8 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10008)
ODD1 = ctypes.c_void_p(0x10001)
OK, NULL, SHAPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 6
BF16, F32 = M.MOE_DTYPE_BF16, M.MOE_DTYPE_F32
BIG = 1 << 40
MAXD = 1 << 24


def test_quant_refusals():
    f = M.lib().moe_mxfp4_quant
    ok = [FAKE, BF16, 4, 100, 100, FAKE, FAKE, FAKE, FAKE, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_1=3) == UNSUP and call(_1=0) == UNSUP
    assert call(_2=-1) == SHAPE and call(_3=-1) == SHAPE and call(_4=99) == SHAPE and call(_2=MAXD + 1) == SHAPE
    assert call(_2=MAXD, _3=MAXD, _4=MAXD) == SHAPE
    assert call(_0=None) == NULL and call(_5=None) == NULL and call(_6=None) == NULL
    assert call(_7=None) == NULL and call(_8=None) == NULL
    assert call(_5=None, _6=None, _7=None, _8=None) == NULL
    assert call(_0=ODD1) == ALIGN and call(_0=ODD2, _1=F32) == ALIGN
    assert call(_5=ODD8) == ALIGN and call(_6=ODD2) == ALIGN and call(_7=ODD8) == ALIGN and call(_8=ODD2) == ALIGN
    assert call(_2=0, _0=None) == OK and call(_3=0, _0=None) == OK
    assert f(None, BF16, 0, 0, 0, None, None, None, None, None) == OK


def test_dequant_refusals():
    f = M.lib().moe_mxfp4_dequant
    assert f(FAKE, FAKE, 4, 100, 7, FAKE, 100, None) == UNSUP
    assert f(FAKE, FAKE, -4, 100, F32, FAKE, 100, None) == SHAPE
    assert f(FAKE, FAKE, 4, 100, F32, FAKE, 99, None) == SHAPE
    for i in (0, 1, 5):
        a = [FAKE, FAKE, 4, 100, F32, FAKE, 100, None]
        a[i] = None
        assert f(*a) == NULL
        a[i] = ODD2
        assert f(*a) == ALIGN
    assert f(None, None, 0, 100, F32, None, 100, None) == OK


def test_matmul_refusals():
    f = M.lib().moe_mxfp4_matmul
    ok = [40, 50, 256, FAKE, FAKE, FAKE, FAKE, F32, FAKE, 50, 0, FAKE, BIG, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_7=9) == UNSUP and call(_7=BF16, _10=1) == UNSUP
    for i in (0, 1, 2):
        assert call(**{f"_{i}": -1}) == SHAPE and call(**{f"_{i}": MAXD + 1, "_9": BIG}) == SHAPE
    assert call(_9=49) == SHAPE and call(_0=MAXD, _1=MAXD, _9=MAXD) == SHAPE
    for i in (3, 4, 5, 6, 8):
        assert call(**{f"_{i}": None}) == NULL
    for i in (3, 5):
        assert call(**{f"_{i}": ODD8}) == ALIGN
    for i in (4, 6, 8):
        assert call(**{f"_{i}": ODD2}) == ALIGN
    assert call(_0=0, _3=None, _8=None) == OK and call(_1=0, _9=0) == OK


def test_linear_refusals():
    f = M.lib().moe_mxfp4_linear
    need = M.lib().moe_mxfp4_linear_bytes(40, 50, 200)
    ok = [40, 50, 200, FAKE, BF16, 200, FAKE, FAKE, BF16, FAKE, 50, FAKE, need, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert need > 0
    assert call(_4=5) == UNSUP and call(_8=5) == UNSUP
    assert call(_0=-1) == SHAPE and call(_5=199) == SHAPE and call(_10=49) == SHAPE and call(_2=MAXD + 1, _5=BIG) == SHAPE
    for i in (3, 6, 7, 9, 11):
        assert call(**{f"_{i}": None}) == NULL
    assert call(_3=ODD1) == ALIGN and call(_6=ODD8) == ALIGN and call(_7=ODD2) == ALIGN and call(_9=ODD1) == ALIGN
    assert call(_11=ODD8) == ALIGN and call(_12=need - 1) == WS
    assert call(_0=0) == OK and call(_1=0) == OK


def test_linear_bwd_refusals():
    f = M.lib().moe_mxfp4_linear_bwd
    need = M.lib().moe_mxfp4_linear_bwd_bytes(40, 50, 200)
    # M N K dy dt ld_dy x_col xs w_col ws dx_dt dx ld_dx dw ld_dw acc ws bytes stream
    ok = [40, 50, 200, FAKE, BF16, 50, FAKE, FAKE, FAKE, FAKE, BF16, FAKE, 200, FAKE, 200, 0, FAKE, need, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_4=5) == UNSUP and call(_10=5) == UNSUP
    assert call(_0=-1) == SHAPE and call(_5=49) == SHAPE and call(_12=199) == SHAPE and call(_14=199) == SHAPE
    for i in (3, 6, 7, 8, 9, 16):
        assert call(**{f"_{i}": None}) == NULL
    assert call(_11=None, _13=None) == NULL
    for i in (3, 11):
        assert call(**{f"_{i}": ODD1}) == ALIGN
    for i in (6, 8, 16):
        assert call(**{f"_{i}": ODD8}) == ALIGN
    for i in (7, 9, 13):
        assert call(**{f"_{i}": ODD2}) == ALIGN
    assert call(_17=need - 1) == WS
    assert call(_2=0) == OK and call(_0=0, _1=0, _12=BIG, _14=BIG) == OK


def test_product_scratch_sizes():
    lib = M.lib()
    assert lib.moe_mxfp4_matmul_bytes(-1, 2, 3) == 0 and lib.moe_mxfp4_linear_bytes(2, MAXD + 1, 3) == 0
    for m in (1, 16, 17, 300, 4096):
        for n in (1, 288, 4096):
            for k in (1, 33, 4096, 16384):
                kp = (k + 127) // 128 * 128
                mm = lib.moe_mxfp4_matmul_bytes(m, n, k)
                assert mm <= 64 << 20                     # a split product is a small one
                assert lib.moe_mxfp4_linear_bytes(m, n, k) <= m * kp * 17 // 32 + 512 + mm
    assert lib.moe_mxfp4_matmul_bytes(4096, 8192, 4096) == 0


def test_balance_refusals():
    f = M.lib().moe_balance_loss
    need = M.lib().moe_balance_bytes(100, 288, 3)
    # logits ids T E k mask off S loss counts seq_tokens lse ws bytes stream
    ok = [FAKE, FAKE, 100, 288, 8, FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE, FAKE, need, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert need > 0 and M.lib().moe_balance_bytes(-1, 288, 1) == 0 and M.lib().moe_balance_bytes(1, 1025, 1) == 0
    assert M.lib().moe_balance_bytes(64, 288, 3) == 0 and M.lib().moe_balance_bytes(65, 288, 3) > 0
    assert M.lib().moe_balance_bytes(1, 8, 0) == 0 and M.lib().moe_balance_bytes(1, 8, 65537) == 0
    for i, bad in ((2, (-1, 1 << 22)), (3, (0, 7, 1025)), (4, (0, 17)), (7, (0, 65537))):
        for v in bad:
            assert call(**{f"_{i}": v}) == SHAPE
    assert call(_6=None) == SHAPE                          # several sequences without offsets
    for i in (0, 1, 8, 9, 10, 11, 12):
        assert call(**{f"_{i}": None}) == NULL
    for i in (0, 1, 6, 8, 9, 10, 11):
        assert call(**{f"_{i}": ODD2}) == ALIGN
    assert call(_12=ODD8) == ALIGN and call(_13=need - 1) == WS


def test_router_bwd_refusals():
    f = M.lib().moe_router_bwd
    # logits ids w dw T E k mask off S lse counts seq_tokens d_loss d_logits stream
    ok = [FAKE, FAKE, FAKE, FAKE, 100, 288, 8, FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE, FAKE, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for i, bad in ((4, (-1, 1 << 22)), (5, (0, 7, 1025)), (6, (0, 17)), (9, (0, 65537))):
        for v in bad:
            assert call(**{f"_{i}": v}) == SHAPE
    assert call(_8=None) == SHAPE
    for i in (0, 1, 2, 10, 11, 12, 14):
        assert call(**{f"_{i}": None}) == NULL
    assert call(_3=None, _13=None) == NULL
    for i in (0, 1, 2, 3, 8, 10, 11, 12, 13, 14):
        assert call(**{f"_{i}": ODD2}) == ALIGN
    assert call(_4=0, _0=None, _14=None) == OK


def test_binding_refuses_host_tensors_and_bad_arguments():
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    for call in (lambda: M.moe_mxfp4_quant(x), lambda: M.moe_mxfp4_dequant(q, s, 128),
                 lambda: M.moe_mxfp4_matmul(q, s, q, s), lambda: M.moe_mxfp4_linear(x, q, s),
                 lambda: M.moe_mxfp4_linear_bwd(x, (q, s), (q, s)), lambda: M.moe_mxfp4_linear_bwd(x),
                 lambda: M.moe_mxfp4_quant(x.half()), lambda: M.moe_mxfp4_quant(x[0]),
                 lambda: M.moe_balance_loss(x, q.int()), lambda: M.moe_router_bwd(x, q.int()),
                 lambda: M.moe_router_bwd(x, q.int(), d_weights=x), lambda: M.moe_router_bwd(x, q.int(), d_loss=x)):
        with pytest.raises(ValueError):
            call()


def _device_code(tmp_path):
    """Instructions of each function of the built gfx950 code objects."""
    objdump = "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("LLVM tools of the ROCm install not found")
    lib = tmp_path / "libmoe.so"
    shutil.copy(M.LIB_PATH, lib)
    subprocess.run([objdump, "--offloading", str(lib)], cwd=tmp_path, check=True, capture_output=True)
    for o in sorted(p for p in tmp_path.iterdir() if "gfx950" in p.name):
        dis = subprocess.run([objdump, "-d", "--mcpu=gfx950", str(o)], check=True, capture_output=True, text=True).stdout
        for name, body in re.findall(r"\n[0-9a-f]+ <([^>]+)>:\n(.*?)(?=\n[0-9a-f]+ <|\Z)", dis, flags=re.S):
            insts = [x.split("//")[0].strip() for x in body.splitlines()]
            yield name, [x for x in insts if x and not x.endswith(":")]


def test_direct_loads_of_the_dense_products(tmp_path):
    """The dense products' direct loads are inline assembly the compiler cannot
    see into.  Their scalar base must not have been written by a vector
    instruction within the five wait states before the load, and the lanes that
    some of them switch off are all switched on again right after."""
    seen = masked = 0
    for name, insts in _device_code(tmp_path):
        for i, ins in enumerate(insts):
            m = re.match(r"global_load_lds_dwordx4 v\d+, s\[(\d+):(\d+)\]", ins)
            if not m:
                continue
            seen += 1
            base = {int(m.group(1)), int(m.group(2))}
            if "exec_hi" in insts[i - 3]:
                masked += 1
                assert re.match(r"s_mov_b32 exec_lo, s\d+", insts[i - 4]) and re.match(r"s_mov_b32 exec_hi, s\d+", insts[i - 3])
                assert insts[i + 1] == "s_mov_b64 exec, -1", insts[i:i + 2]
            states, j = 0, i - 1
            while states < 5 and j >= 0:
                if insts[j].startswith("s_nop"):
                    states += int(insts[j].split()[1]) + 1
                else:
                    states += 1
                    w = re.match(r"v_\w+ s(\d+),|v_\w+ s\[(\d+):(\d+)\],", insts[j])
                    if w:
                        lo = int(w.group(1) or w.group(2))
                        assert not base & set(range(lo, int(w.group(3) or lo) + 1)), (name, insts[j:i + 1])
                j -= 1
    assert seen > 2 * masked > 100


def test_tile_results_read_after_their_wait_states(tmp_path):
    """Reads of a register that a 32x32x64 FP4 product (8 passes) has written
    come at least 16 wait states later, or after another product; the products
    of its own accumulator chain are interlocked."""
    def regs(spec):
        m = re.match(r"([av])\[(\d+):(\d+)\]", spec)
        if m:
            return {f"{m.group(1)}{k}" for k in range(int(m.group(2)), int(m.group(3)) + 1)}
        return {spec} if re.match(r"[av]\d+$", spec) else set()

    checked = 0
    for name, insts in _device_code(tmp_path):
        for i, ins in enumerate(insts):
            if not ins.startswith("v_mfma_scale_f32_32x32x64"):
                continue
            dst, states = regs(ins.replace(",", " ").split()[1]), 0
            for t in insts[i + 1:i + 60]:
                f = t.replace(",", " ").split()
                if f[0] == "s_nop":
                    states += int(f[1]) + 1
                    continue
                if f[0].startswith("v_mfma") or f[0] in ("s_endpgm", "s_branch") or f[0].startswith("s_cbranch"):
                    if not f[0].startswith("s_cbranch"):
                        break
                if len(f) > 2 and dst & set().union(*[regs(x) for x in f[2:]]):
                    assert states >= 16, (name, ins, t, states)
                    break
                states += 1
                if states >= 16:
                    break
            checked += 1
    assert checked > 300
