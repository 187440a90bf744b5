"""The library's own objects linked with fake_cudart.c instead of the CUDA
runtime: plans and runs on the CPU, whose launches only leave a line in a log."""
import ctypes
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def load(tmp):
    """The library (its C ABI untyped, and fake_log, fake_clear, fake_queued, fake_kernel), linked under `tmp`."""
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    objects = [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build._sources()]
    fake, lib = os.path.join(str(tmp), "fake_cudart.o"), os.path.join(str(tmp), "libconv_fake.so")
    subprocess.run(["gcc", "-std=gnu11", "-O1", "-fPIC", "-w", "-I", cuda, "-c", os.path.join(HERE, "fake_cudart.c"), "-o", fake], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", lib, fake] + objects, check=True)
    out = ctypes.CDLL(lib)
    out.fake_log.restype = out.fake_kernel.restype = ctypes.c_char_p
    return out
