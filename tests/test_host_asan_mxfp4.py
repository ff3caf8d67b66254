"""The host code of the dense MXFP4 and the router's training entry points
(argument checks and size arithmetic) under the address and
undefined-behaviour checks of the host compiler.  Every call is refused, or
has nothing to do, before any launch.  Host only."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_quantized_weights_amd", "csrc")

ASAN_DRIVER = textwrap.dedent(r'''
    import ctypes, random, sys
    lib = ctypes.CDLL(sys.argv[1])
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    for n in ("matmul", "linear", "linear_bwd"):
        getattr(lib, f"moe_mxfp4_{n}_bytes").restype = SZ
    lib.moe_balance_bytes.restype = SZ
    F = P(1 << 40)
    rng = random.Random(5)
    dims = [-(2**31), -1, 0, 1, 31, 128, 4097, 2**20, 2**24, 2**24 + 1, 2**31 - 1]
    for _ in range(20000):
        m, n, k = rng.choice(dims), rng.choice(dims), rng.choice(dims)
        need = [getattr(lib, f"moe_mxfp4_{x}_bytes")(m, n, k) for x in ("matmul", "linear", "linear_bwd")]
        lib.moe_balance_bytes(m, n, k)
        # every call lacks its output, has a type of no meaning, or a workspace too short
        lib.moe_mxfp4_quant(F, rng.choice([0, 3]), m, n, I64(n), F, F, F, F, None)
        lib.moe_mxfp4_quant(None, 1, m, n, I64(n), F, F, F, F, None)
        lib.moe_mxfp4_dequant(F, F, m, n, 2, None, I64(n), None)
        lib.moe_mxfp4_matmul(m, n, k, F, F, F, F, 2, None, I64(n), 0, F, SZ(1 << 60), None)
        lib.moe_mxfp4_linear(m, n, k, F, 1, I64(k), F, F, 1, None, I64(n), F, SZ(1 << 60), None)
        if need[1]:
            assert lib.moe_mxfp4_linear(m, n, k, F, 1, I64(k), F, F, 1, F, I64(n), F, SZ(need[1] - 1), None) in (0, 6)
        if need[2]:
            assert lib.moe_mxfp4_linear_bwd(m, n, k, F, 1, I64(n), F, F, F, F, 1, F, I64(k), F, I64(k), 0, F,
                                            SZ(need[2] - 1), None) in (0, 6)
        lib.moe_balance_loss(F, F, m, n, k, F, F, rng.choice(dims), None, F, F, F, F, SZ(1 << 60), None)
        lib.moe_router_bwd(F, F, F, F, m, n, k, F, F, rng.choice(dims), F, F, F, F, None, None)
    print("done")
''')


def test_host_code_under_asan(tmp_path):
    """Argument checks and size arithmetic of these entry points under the
    address and undefined-behaviour checks of the host compiler."""
    hipcc, clang = "/opt/rocm/bin/hipcc", "/opt/rocm/llvm/bin/clang"
    if not (os.path.exists(hipcc) and os.path.exists(clang)) or torch.cuda.is_available():
        pytest.skip("needs the ROCm compilers and a host without a GPU")
    host = [w for f in ("address", "signed-integer-overflow,pointer-overflow") for w in ("-Xarch_host", "-fsanitize=" + f)]
    so = tmp_path / "lib.so"
    objs = []
    for src in ("mx_quant", "mx_matmul", "balance"):
        objs.append(str(tmp_path / (src + ".o")))
        r = subprocess.run([hipcc, "--offload-arch=gfx950", "-O1", "-std=c++20", "-fPIC", "-Xarch_host", "-g", *host,
                            "-Xarch_host", "-fno-sanitize-recover=all", "-Xclang", "-target-feature", "-Xclang",
                            "-packed-fp32-ops", "-c", os.path.join(CSRC, src + ".hip"), "-o", objs[-1]],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    r = subprocess.run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *host, *objs, "-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rt = subprocess.run([clang, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True).stdout.strip()
    drv = tmp_path / "drive.py"
    drv.write_text(ASAN_DRIVER)
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               HIP_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, str(drv), str(so)], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
