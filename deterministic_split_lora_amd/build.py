"""Builds liblora_det.so (the HIP kernels and the C entry points) for gfx950,
and _native.so (compiled argument marshalling for the package, host code).

Run ``python -m deterministic_split_lora_amd.build`` or call ``build()``.  The
library is written next to this file so it travels with the source tree.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblora_det.so")
BINDING = os.path.join(HERE, "_native.so")
SOURCES = ["abi.hip", "shrink.hip", "expand.hip", "fused.hip", "streamed.hip", "sgmv_plan.hip",
           "abi_step.hip", "mx4.hip", "mx4_linear.hip", "block_norm.hip", "sample.hip"]
HEADERS = ["device.h", "kernels.h", "shrink_tile.h", "step_kernels.h", "mx4.h", "mx4_tile.h"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # every fp32 add / multiply in the kernels rounds on its own; fused
    # multiply-adds appear only where the source asks for one (fmaf)
    "-ffp-contract=off",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # only the C ABI (include/lora_det.h) is exported; the kernels' C++
    # launchers stay inside the library
    "-fvisibility=hidden",
    "-Wall",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    p = os.path.join(rocm, "bin", "hipcc")
    return p if os.path.exists(p) else "hipcc"


def _record_revision() -> None:
    """Writes the git revision of the sources next to the library (with
    "-dirty" when tracked files differ from it), so a copy of the tree without
    its history still says what the library was built from.  No git: no file."""
    import subprocess
    root = os.path.dirname(HERE)
    path = os.path.join(HERE, "build_revision.txt")
    try:
        rev = subprocess.run(["git", "-C", root, "rev-parse", "HEAD"], capture_output=True, text=True,
                             timeout=10).stdout.strip()
        dirty = subprocess.run(["git", "-C", root, "status", "--porcelain", "--untracked-files=no"],
                               capture_output=True, text=True, timeout=10).stdout.strip()
    except (OSError, subprocess.SubprocessError):
        return
    if rev:
        with open(path, "w") as f:
            f.write(rev + ("-dirty" if dirty else "") + "\n")


def binding_command(out: str) -> list:
    """The host compiler's line for csrc/binding.cpp, against the installed torch's headers."""
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    include = ["-isystem" + i for i in cpp_extension.include_paths()] + ["-I" + sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
            '-DLORA_TORCH_VERSION="%s"' % torch.__version__, *include,
            os.path.join(CSRC, "binding.cpp"), "-o", out, "-L" + cpp_extension.library_paths()[0],
            "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False) -> str:
    """Compile every source; always recompiles (a cross-compile, no GPU needed).
    Each source is compiled to an object in parallel, then the objects are
    linked into the shared library.  The compiled marshalling needs torch's
    headers besides; if it fails, the library is put in place all the same and
    the failure raised afterwards."""
    from concurrent.futures import ThreadPoolExecutor
    inc = ["-I", os.path.join(os.path.dirname(HERE), "include")]
    tag = "%d" % os.getpid()
    objs = [os.path.join(CSRC, os.path.splitext(s)[0] + ".o.tmp" + tag) for s in SOURCES]
    lib, native = LIB + ".tmp" + tag, BINDING + ".tmp" + tag
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    noise = "'-packed-fp32-ops' is not a recognized feature"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        # hipcc's host pass does not know the packed-fp32 feature and says so;
        # that warning is harmless and filtered here
        return res.returncode, "\n".join(l for l in res.stderr.splitlines() if noise not in l)

    def run_binding():
        try:
            return run(binding_command(native))
        except Exception as e:               # no torch, or one without headers
            return 1, f"{type(e).__name__}: {e}"

    try:
        jobs = [[hipcc(), *compile_flags, *inc, "-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 1)) as ex:
            binding = ex.submit(run_binding)
            results = list(ex.map(run, jobs))
        binding_rc, binding_errs = binding.result()
        errs = "\n".join(e for _, e in results + [(0, binding_errs)] if e.strip())
        if any(rc != 0 for rc, _ in results):
            raise RuntimeError("hipcc failed:\n" + errs)
        if verbose and errs:
            print(errs, file=sys.stderr)
        rc, err = run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", lib])
        if rc != 0:
            raise RuntimeError("hipcc link failed:\n" + err)
        os.replace(lib, LIB)
        _record_revision()
        if binding_rc != 0:
            if os.path.exists(BINDING):      # an earlier one may not fit this library
                os.remove(BINDING)
            raise RuntimeError("the library is built, its compiled marshalling is not:\n" + binding_errs)
        os.replace(native, BINDING)
    finally:
        for o in [*objs, lib, native]:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
