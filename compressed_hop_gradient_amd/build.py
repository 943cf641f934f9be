"""Build the HIP library ``libdq.so`` in-tree for gfx950 (hipcc cross-compiles
without a GPU)."""
import os
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdq.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC",
    # numerics shared with the CPU oracle: no contraction, IEEE division, no fast-math
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-fast-math",
    # packed FP32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # the compile-time check of the level buckets walks every bucket
    "-fconstexpr-steps=100000000",
    "-Wall", "-Wno-unused-command-line-argument",
]
SOURCES = ["dq_kernels.hip", "dq_api.cpp", "dq_dropout.hip", "dq_route.hip", "dq_route_backward.hip",
           "dq_train_api.cpp"]


def build(verbose=False):
    """Compile every HIP source of the package into ``libdq.so`` (always rebuilds);
    the sources compile side by side."""
    noise = "is not a recognized feature for this target"

    def finish(proc):
        _, err = proc.communicate()
        err = "\n".join(l for l in (err or "").splitlines() if noise not in l)
        if proc.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + err)
        if verbose and err.strip():
            print(err)

    def start(args):
        if verbose:
            print(" ".join(args))
        return subprocess.Popen(args, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)

    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory(prefix="dq_build_") as objs:
        out = [os.path.join(objs, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        procs = [start([HIPCC] + FLAGS + ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c",
                                          os.path.join(CSRC, s), "-o", o]) for s, o in zip(SOURCES, out)]
        failed = None
        for p in procs:
            try:
                finish(p)
            except RuntimeError as e:
                failed = failed or e
        if failed:
            raise failed
        finish(start([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared"] + out + ["-o", tmp]))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
