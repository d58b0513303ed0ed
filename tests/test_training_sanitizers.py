"""The training operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): the C ABI's checks, built and preloaded
as in test_sanitizers.py, run the refusal tests, which launch nothing."""
import os

import pytest

from test_sanitizers import _run


def test_training_checks_under_sanitizers(tmp_path):
    from delta_rule_linear_gdn2_amd import build as lb

    lib = lb.build_sanitized(str(tmp_path))
    rt = lb.sanitizer_runtime_dir()
    runtime = os.path.join(rt, lb.SAN_RUNTIME)
    if not os.path.exists(runtime):
        pytest.fail(f"{runtime} missing")
    out = _run({"GDN2_LIBRARY": lib, "LD_PRELOAD": runtime,
                "LD_LIBRARY_PATH": rt + os.pathsep + os.environ.get("LD_LIBRARY_PATH", "")},
               ["tests/test_training_cpu.py", "-k", "rejects or workspace"], str(tmp_path))
    assert "passed" in out
