"""The host code of the gated recurrent layer's entry points under AddressSanitizer and UndefinedBehaviorSanitizer:
test_abi_gated.py in a child process against the host-sanitized library (built if it is older than its sources).
No GPU needed."""
import glob
import os

import pytest

from test_sanitize import _run, pytestmark  # noqa: F401  (the same skip: fake device addresses)


def test_gated_host_code_under_sanitizers():
    from chunked_scan_amd import build

    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc is not installed")
    srcs = glob.glob(os.path.join(build.CSRC, "*")) + glob.glob(os.path.join(build.INCLUDE, "*.h"))
    newest = max(os.path.getmtime(f) for f in srcs)
    if not os.path.exists(build.SAN_LIB) or os.path.getmtime(build.SAN_LIB) < newest:
        build.build_sanitized(verbose=False)
    _run({"LACHUNK_LIB": build.SAN_LIB, "LD_PRELOAD": build.asan_runtime()}, ["tests/test_abi_gated.py"])
