"""The library's host code over a stand-in CUDA runtime (tests/c/fake_runtime.cpp): what its calls
ask of the runtime, seen without a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from combine_topk_ids_dest_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
ADDRESS = 1 << 40  # of operands, which nothing reads


class Fake:
    """The library (.L, with ep_moe.h's functions) and the records of its calls."""

    def __init__(self, folder):
        if shutil.which("g++") is None:
            pytest.skip("g++ not available")
        objects = [os.path.join(build.BUILD, os.path.basename(s) + ".o") for s in build.sources()]
        build.build(force=not all(os.path.exists(o) for o in objects))
        so = os.path.join(str(folder), "libep_fake.so")
        cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", os.path.join(CUDA, "include"),
               "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(ROOT, "tests", "c", "fake_runtime.cpp"), *objects,
               "-o", so, "-ldl", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        self.L = L = ctypes.CDLL(so)
        declared = _lib.load()
        for name in _lib.MOE_EXPORTS + ("ep_last_error",):
            getattr(L, name).argtypes = getattr(declared, name).argtypes
            getattr(L, name).restype = getattr(declared, name).restype
        L.fake_launch.restype = L.fake_call.restype = ctypes.c_char_p
        L.fake_error_words.restype = ctypes.POINTER(ctypes.c_uint)

    def message(self):
        return self.L.ep_last_error().decode()

    def launches(self):
        """(kernel, device, grid, block, dynamic shared memory) of each launch since the last clear."""
        out, v = [], (ctypes.c_longlong * 8)()
        for i in range(self.L.fake_launches()):
            name = self.L.fake_launch(i, v).decode()
            out.append((name, v[0], tuple(v[1:4]), tuple(v[4:7]), v[7]))
        return out

    def calls(self):
        """The runtime's calls that wait for a device or free memory, since the last clear."""
        return [self.L.fake_call(i).decode() for i in range(self.L.fake_calls())]

    def box(self):
        """Box of the last tensor map."""
        v = (ctypes.c_int * 3)()
        self.L.fake_box(v)
        return tuple(v)

    def router(self, **kw):
        b = dict(num_experts=256, top_k=8, hidden=7168, dtype=_lib.EP_DTYPE_BF16, scoring=0, num_groups=1, top_groups=1,
                 renormalize=1, scale=1.0, weight=ADDRESS, bias=0)
        b.update(kw)
        cfg = _lib.EpRouterConfigC(*[b[f] for f, _ in _lib.EpRouterConfigC._fields_])
        h = ctypes.c_void_p()
        assert self.L.ep_router_create(ctypes.byref(cfg), ctypes.byref(h)) == _lib.EP_OK, self.message()
        return h.value

    def route(self, h, n, hidden=7168):
        """Status and workspace of ep_router_run with n rows."""
        size = ctypes.c_size_t(0)
        assert self.L.ep_router_workspace_size(h, n, ctypes.byref(size)) == _lib.EP_OK
        return self.L.ep_router_run(h, ADDRESS, hidden, n, ADDRESS, ADDRESS, ADDRESS, size.value, None), size.value

    def experts(self, group=0, zeros=0, **kw):
        b = dict(num_experts=8, first_expert=0, top_k=8, hidden=256, intermediate=256, max_tokens=64)
        b.update(kw)
        w = [_lib.EpWeightC(ADDRESS, group, zeros, 0)] * 2
        cfg = _lib.EpExpertsConfigC(*b.values(), *w)
        h = ctypes.c_void_p()
        assert self.L.ep_experts_create(ctypes.byref(cfg), None, 0, ctypes.byref(h)) == _lib.EP_OK, self.message()
        return h.value

    def linear(self, inputs=256, outputs=300, max_tokens=64):
        cfg = _lib.EpLinearConfigC(inputs, outputs, max_tokens, _lib.EpWeightC(ADDRESS, 128, 0, 0))
        h = ctypes.c_void_p()
        assert self.L.ep_linear_create(ctypes.byref(cfg), None, 0, ctypes.byref(h)) == _lib.EP_OK, self.message()
        return h.value

    def run_experts(self, h, n, hidden=256):
        return self.L.ep_experts_run(h, ADDRESS, hidden, ADDRESS, ADDRESS, n, ADDRESS, hidden, None)

    def run_linear(self, h, n, inputs=256, outputs=300):
        return self.L.ep_linear_run(h, _lib.EP_DTYPE_BF16, ADDRESS, inputs, n, ADDRESS, outputs, None)

    def run_layer(self, r, h, n, hidden=256):
        return self.L.ep_layer_run(r, h, ADDRESS, hidden, n, ADDRESS, ADDRESS, ADDRESS, hidden, None)
