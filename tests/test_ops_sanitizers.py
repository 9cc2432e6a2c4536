"""Host code of the decode-step operators' entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): tests/sanitize/ops_driver.c walks the refusals and the sizing
functions."""
import os

import pytest

from test_sanitizers import CLANG, HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang not installed")
def test_ops_validation_under_asan_ubsan(tmp_path):
    from sparse_moe_transformer_wave_amd import build as b
    names = ("api", "route", "permute", "gemv", "gemm", "decode1", "decode_few")
    units = ("ops_api", "linear", "kv_append", "attn_decode", "logprobs")  # their host code sizes and checks
    objs = [os.path.join(b.BUILD_DIR, "moe_%s.o" % n) for n in names]
    if not all(os.path.exists(o) for o in objs):
        b.build_moe()
    for n in units:
        o = str(tmp_path / (n + "_san.o"))
        # the sanitizers instrument the host code only (-Xarch_host); the device code is as shipped
        _run([HIPCC] + [f for f in b.HIP_FLAGS if f != "-O3"] +
             ["-O1", "-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-sanitize-recover=all",
              "-c", os.path.join(ROOT, "sparse_moe_transformer_wave_amd", "csrc", n + ".hip"), "-o", o])
        objs.append(o)
    drv, exe = str(tmp_path / "ops_driver.o"), str(tmp_path / "ops_san")
    _run([CLANG, "-std=c11", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-c",
          os.path.join(SAN, "ops_driver.c"), "-o", drv])
    _run([CLANG + "++", "-fsanitize=address,undefined", drv] + objs +
         ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    out = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "ops driver: ok" in out
