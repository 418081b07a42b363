"""Build libar.so (the HIP all-reduce library) for gfx950 with hipcc.

The translation units compile in parallel; the result lands next to this
file so it travels with the source tree.
"""

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libar.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
SOURCES = ("api.hip", "kernels.hip", "rmsnorm.hip", "noalloc.hip", "ceiling.hip", "ffn.hip", "xent.hip", "rope.hip", "cache.hip", "attention.hip",
           "products.hip", "products_bf16.hip", "products_f32.hip")

# -packed-fp32-ops: keep hipcc from fusing float adds into packed-FP32
# instructions.  No fast-math, no denormal flushing: fp32 adds stay IEEE.
HIPFLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def checks_built_for():
    """What the compiled checks (_marshal.so) depend on, as they are marked."""
    import torch
    return f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"


def build_marshal(out: str = MARSHAL) -> str:
    """Compile the binding's argument checks (host code against torch's headers),
    marked with the torch and Python they are for."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DBUILT_FOR="{checks_built_for()}"', *[f"-I{i}" for i in inc], os.path.join(CSRC, "marshal.cpp"), "-L" + os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-o", out + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{res.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = False, out: str = LIB, defines=()) -> str:
    """Compile every source and link the library (libar.so next to this file
    unless `out` says otherwise); `defines` are extra -D options.  Beside it goes
    the binding's compiled half (_marshal.so), which the binding does without
    where it does not build (no g++, Python headers or torch)."""
    hipcc = _hipcc()
    with tempfile.TemporaryDirectory(prefix="ar_build_") as tmp:
        def compile_one(src):
            obj = os.path.join(tmp, src + ".o")
            cmd = [hipcc, *HIPFLAGS, *[f"-D{d}" for d in defines], "-c", os.path.join(CSRC, src), "-o", obj]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"hipcc failed on {src}:\n{res.stderr}")
            if verbose:
                sys.stderr.write(res.stderr)
            return obj

        with ThreadPoolExecutor(len(SOURCES) + 1) as pool:
            checks = pool.submit(build_marshal) if out == LIB else None
            objs = list(pool.map(compile_one, SOURCES))
        tmp_lib = out + ".tmp"
        cmd = [hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp_lib]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp_lib, out)
    if checks and checks.exception():
        if os.path.exists(MARSHAL):  # of an earlier build
            os.remove(MARSHAL)
        sys.stderr.write(f"the binding's checks are not compiled, and run in Python: {checks.exception()}\n")
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
