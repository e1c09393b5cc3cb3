"""Host code of prompt and prefix attention, rotation and pages under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): every launch covers its
work once and writes inside its workspace, and no size overflows."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "sanitize"))


def test_serving_host_code_under_sanitizers(tmp_path):
    import serving_build

    exe = serving_build.build_serving_selftest(str(tmp_path))
    proc = subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"), timeout=600)
    out = proc.stdout + proc.stderr
    assert proc.returncode == 0 and "runtime error" not in out and "ERROR: AddressSanitizer" not in out, out
    assert "every launch covers its work" in out
