"""The host side of the paged cache's entry points under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: tests/host_sanitize_cache.cpp calls the sizing and plan
entry points over a grid of sizes, extremes included, and the others with arguments they must
refuse before any HIP call.  Sanitizers on the host pass only."""
import os
import subprocess
from pathlib import Path

ROOT = Path(__file__).resolve().parents[1]


def test_host_code_of_the_cache_clean_under_sanitizers(tmp_path):
    exe = tmp_path / "host_sanitize_cache"
    csrc = ROOT / "rejection_sampling_verify_02_amd" / "csrc"
    cmd = ["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
           "-I", str(ROOT / "include"), "-I", str(csrc), str(ROOT / "tests" / "host_sanitize_cache.cpp"),
           str(csrc / "spec_attention.hip"), str(csrc / "spec_cache.hip"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    got = dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())
    assert got["scale"] == "8" and got["stride"] == "6" and got["small"] == "5" and got["append"] == "6"
    assert got["commit"] == "8" and got["resize"] == "2" and got["fork"] == "2"
