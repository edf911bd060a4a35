"""The host-side checks of the dispatch, adapter and draft-verification entry
points under AddressSanitizer and UndefinedBehaviorSanitizer, built as
test_abi_sanitized.py builds the other entry points' (host code only; no call
reaches a device), with abi_sanitize/requests_host_checks.cpp as the program:
refused arguments at extreme sizes, and the workspace queries."""
import concurrent.futures as cf
import glob
import os
import subprocess

from test_abi_sanitized import CSRC, FLAGS, ROOT, SAN, _hipcc, _run

DRIVER = os.path.join(ROOT, "tests", "abi_sanitize", "requests_host_checks.cpp")


def test_requests_host_checks_under_asan_and_ubsan(tmp_path):
    hipcc = _hipcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + [DRIVER]
    objs = [str(tmp_path / (os.path.basename(s).rsplit(".", 1)[0] + ".o")) for s in srcs]
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        list(ex.map(lambda so: _run([hipcc, *FLAGS, *SAN, "-c", so[0], "-o", so[1]]),
                    zip(srcs, objs)))
    exe = str(tmp_path / "requests_host_checks")
    _run([hipcc, "--offload-arch=gfx950", *SAN, *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300, cwd=str(tmp_path))
    out = res.stdout + res.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert res.returncode == 0, out[-4000:]
    assert int(out.split("abi host checks:")[1].split("passed")[0]) >= 100 and ", 0 failed" in out, out
