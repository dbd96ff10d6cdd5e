"""Host sanitizer run (no GPU) of the argument checks, plans and workspace sizes of the
fused MXFP4 entry points: the library's host code with AddressSanitizer and
UndefinedBehaviorSanitizer (every -fsanitize follows -Xarch_host, device code is built as
usual), driven with sizes around and far beyond every limit."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, ENV, HERE, HIPCC, ROOT, _run


def test_fused_validation_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    exe = str(tmp_path / "fused_abi_asan")
    srcs = [os.path.join(CSRC, f) for f in (
        "api.hip", "pack.hip", "gemv.hip", "gemm_mfma.hip", "gemm_prefill.hip", "embed.hip",
        "mx_gemm.hip", "mx_grad.hip", "mx_linear.hip", "mx_loss.hip", "moe_mlp.hip")]
    srcs.append(os.path.join(HERE, "fused_abi_driver.cpp"))
    flags = ["--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include")]
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]

    def compile_one(so):
        s, o = so
        lang = ["-x", "hip"] if s.endswith(".cpp") else []
        return _run([HIPCC] + flags + ["-c"] + lang + [s, "-o", o], timeout=600)
    with ThreadPoolExecutor(min(len(srcs), os.cpu_count() or 1)) as ex:
        for rc, out in ex.map(compile_one, zip(srcs, objs)):
            assert rc == 0, out
    rc, out = _run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
                    "-Xarch_host", "-fsanitize=undefined"] + objs + ["-o", exe], timeout=600)
    assert rc == 0, out
    env = dict(ENV, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    rc, out = _run([exe], env=env, timeout=600)
    assert rc == 0 and "fused abi sanitizer run: ok" in out, out
