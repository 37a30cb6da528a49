"""The library linked with a stand-in for the CUDA runtime (runtime.cpp), so that
its host code runs without a GPU, on as many devices as a test wants."""
import ctypes
import os
import re
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def build(folder):
    """Links it in `folder`; returns its path."""
    from moe_expert_layer_histogram_gb300 import _build
    _build.build()
    objs = [os.path.join(_build.LIBDIR, "obj", s + ".o") for s in _build.SOURCES]
    source = open(os.path.join(HERE, "runtime.cpp")).read()
    used = subprocess.run(["nm", "-u"] + objs, capture_output=True, text=True, check=True).stdout
    # runtime calls that no test makes
    rest = sorted(n for n in set(re.findall(r"\b_*cuda\w+", used)) if n + "(" not in source)
    more = os.path.join(folder, "rest.cpp")
    with open(more, "w") as f:
        f.write("extern \"C\" {\n" + "".join("int %s() { return 999; }\n" % n for n in rest) + "}\n")
    so = os.path.join(folder, "libmoe_fake_cuda.so")
    cuda = os.path.dirname(os.path.dirname(_build._nvcc()))
    # (-Bsymbolic: not the real runtime that torch has loaded)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic",
                    "-I" + os.path.join(cuda, "include"), "-I" + _build.CSRC,
                    os.path.join(HERE, "runtime.cpp"), more] + objs + ["-o", so, "-lpthread"],
                   check=True)
    return so


def load(so, folder):
    """A copy of it, with a state of its own."""
    return ctypes.CDLL(shutil.copy(so, os.path.join(folder, "copy.so")))
