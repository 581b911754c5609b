"""The fine-tuning calls' host code (argument checks, size arithmetic) under
AddressSanitizer and UndefinedBehaviorSanitizer, as test_abi_sanitized.py runs
the other calls'."""
import os
import subprocess
import sys

from test_abi_sanitized import HERE, ROOT, _env, sanitized  # noqa: F401  (a fixture)

FILES = ["test_finetune_cpu.py", "test_distill_desc_cpu.py", "test_finetune_precise_cpu.py"]


def test_refusals_pass_under_sanitizers(sanitized):  # noqa: F811
    lib, runtime = sanitized
    cmd = [sys.executable, "-m", "pytest", *(os.path.join(HERE, f) for f in FILES), "-x", "-q",
           "-p", "no:cacheprovider", "-m", "not gpu"]
    r = subprocess.run(cmd, cwd=ROOT, env=_env(lib, runtime), capture_output=True, text=True,
                       timeout=900)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out
