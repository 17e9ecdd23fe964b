"""Sanitizer build of the block operators' host code (no GPU needed): argument validation and workspace queries of the C ABI
(tests/sanitize/block_abi_validation.cpp against the library's sources), with AddressSanitizer and UndefinedBehaviorSanitizer on
the host pass only, required to run clean."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else "hipcc"


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="no hipcc")
def test_block_abi_validation_runs_clean_under_host_sanitizers(tmp_path):
    # host code only: what the queries and checks return does not depend on the kernels
    csrc = os.path.join(ROOT, "nonlinear_rnn_solve_amd", "csrc")
    flags = ["--offload-arch=gfx950", "-O1", "-std=c++17", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include")]
    sources = [os.path.join(csrc, f) for f in ("block_ssm.hip", "block_conv.hip", "block_ffn.hip", "block_adamw.hip")]
    sources.append(os.path.join(ROOT, "tests", "sanitize", "block_abi_validation.cpp"))
    jobs = [subprocess.Popen([HIPCC, *flags, "-c", src, "-o", str(tmp_path / ("%d.o" % k))], stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
            for k, src in enumerate(sources)]
    outs = [j.communicate(timeout=900)[0] for j in jobs]
    assert all(j.returncode == 0 for j in jobs), b"".join(outs)[-3000:]
    exe = str(tmp_path / "block_abi_validation")
    subprocess.run([HIPCC, *flags, *(str(tmp_path / ("%d.o" % k)) for k in range(len(sources))), "-o", exe], check=True, capture_output=True,
                   timeout=300)
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    out = p.stdout + p.stderr
    assert p.returncode == 0, out[-3000:]
    assert "checks passed" in out and "runtime error" not in out and "AddressSanitizer" not in out
