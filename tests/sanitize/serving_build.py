"""Build the host-sanitizer self-test of the serving entry points (test infrastructure;
CPU only): their host code alone, with AddressSanitizer and
UndefinedBehaviorSanitizer, linked with the test's own stand-ins for the HIP runtime.

Outputs go to a build directory given by the caller; nothing is written in-tree.
"""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def build_serving_selftest(out_dir: str) -> str:
    obj, exe = os.path.join(out_dir, "serving_selftest.o"), os.path.join(out_dir, "serving_selftest")
    host_san = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"):
        host_san += ["-Xarch_host", flag]
    subprocess.run([os.path.join(ROCM, "bin", "hipcc"), "-O1", "-g", "-std=c++17", "--offload-arch=gfx950", "--offload-host-only", "-fuse-cuid=none",
                    *host_san, "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "memory_bound_gemv_row_amd", "csrc"),
                    "-c", os.path.join(HERE, "serving_selftest.hip"), "-o", obj], check=True, capture_output=True, text=True)
    # no device code is linked in, so its image is a symbol without contents
    subprocess.run([os.path.join(ROCM, "llvm", "bin", "clang++"), "-fsanitize=address,undefined", obj, "-Wl,--defsym=__hip_fatbin=0", "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe
