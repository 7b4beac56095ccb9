"""csrc/work.cpp over a fake of the CUDA runtime (tests/native/work_shim.cpp), for the CPU
tests of its host logic: handles, failures, order of calls, refusals, choice of kernels."""
import ctypes
import os
import subprocess

import pytest

import server_side_fedavg_gb300 as fa

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "server_side_fedavg_gb300", "csrc")
SO = os.path.join(HERE, "_build", "libwork_shim.so")
CUDA_INC = "/usr/local/cuda/include"

_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.isdir(CUDA_INC):
            pytest.skip("CUDA headers are not installed")
        os.makedirs(os.path.dirname(SO), exist_ok=True)
        srcs = [os.path.join(HERE, "native", "work_shim.cpp"), os.path.join(CSRC, "work.cpp")]
        deps = srcs + [os.path.join(CSRC, f) for f in ("product.cuh", "product_tc.cuh", "distill.cuh", "kernels.cuh")]
        deps.append(os.path.join(ROOT, "include", "fedavg.h"))
        if not os.path.exists(SO) or any(os.path.getmtime(s) > os.path.getmtime(SO) for s in deps):
            # -Bsymbolic: the fake's functions, also where a real runtime is loaded
            subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", CSRC, "-I",
                            os.path.join(ROOT, "include"), "-I", CUDA_INC] + srcs + ["-o", SO], check=True)
        L = ctypes.CDLL(SO)
        vp = ctypes.c_void_p
        L.ws_log.restype = ctypes.c_char_p
        L.ws_fail.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.c_int]
        L.ws_pending.argtypes = [ctypes.c_int]
        L.ws_choice.argtypes = [vp, vp, vp]
        for name in ("ws_sync", "ws_close"):
            getattr(L, name).argtypes = [vp]
        L.fa_work_open.argtypes = [vp, vp]
        L.fa_work_get_stats.argtypes = [vp, vp]
        L.fa_work_last_error.argtypes = [vp]
        L.fa_work_last_error.restype = ctypes.c_char_p
        for name in ("fa_product", "fa_product_backward", "fa_distill_loss", "fa_distill_grad"):
            getattr(L, name).argtypes = [vp, vp, vp]
        _lib = L
    return _lib


class Work:
    """A handle on the fake device.  Addresses are plain numbers: nothing is read."""

    def __init__(self, **opts):
        self.L = lib()
        self.L.ws_reset()
        self.h = ctypes.c_void_p()
        o = fa.fa_work_opts(ctypes.sizeof(fa.fa_work_opts), opts.get("timeout_ms", 0), opts.get("workspace_bytes", 0), 0, 0)
        assert self.L.fa_work_open(ctypes.byref(o), ctypes.byref(self.h)) == fa.FA_OK
        self.opened = self.log()
        self.L.ws_clear_log()

    def log(self):
        return self.L.ws_log().decode().split()

    def fail(self, name, after=0, throwing=False):
        self.L.ws_fail(name.encode(), after, throwing)

    def error(self):
        return self.L.fa_work_last_error(self.h).decode()

    def stats(self):
        st = fa.fa_work_stats()
        assert self.L.fa_work_get_stats(self.h, ctypes.byref(st)) == fa.FA_OK
        return st

    def product(self, m, n, k, a, b, out, din="f32", dout="f32", lda=None, ldb=None, ldo=None, ta=False, tb=True,
                bias=None, residual=None, ldr=0, pre=None, beta=1.0, stream=0):
        args = fa.fa_product_args(
            ctypes.sizeof(fa.fa_product_args), ta | tb << 1, fa.DTYPES[din], fa.DTYPES[dout], 0, 0, m, n, k, a,
            lda or (m if ta else k), b, ldb or (k if tb else n), bias, residual, ldr, out, ldo or n, pre, 1.0, beta)
        return self.L.fa_product(self.h, ctypes.byref(args), stream)

    def backward(self, m, n, k, a, b, dout, d_a, d_b, dtypes=("f32", "f32", "f32"), act="none", pre=None, ldp=0,
                 d_bias=None, ldda=None, lddb=None, ldd=None, stream=0):
        args = fa.fa_product_backward_args(
            ctypes.sizeof(fa.fa_product_backward_args), 2, *(fa.DTYPES[t] for t in dtypes), fa.ACTS[act], m, n, k, a, k, b,
            k, dout, ldd or n, pre, ldp, d_a, ldda or k, d_b, lddb or k, d_bias, 1.0)
        return self.L.fa_product_backward(self.h, ctypes.byref(args), stream)

    def distill_grad(self, rows, vocab, logits, grad, index, value, topk=4, ld=None, ldg=None, loss=None, lse=None,
                     row_weight=None, dtype="f32", stream=0):
        client = fa.fa_distill_client(index, value, topk, 0, 1.0)
        args = fa.fa_distill_args(ctypes.sizeof(fa.fa_distill_args), 1, fa.DTYPES[dtype], 0, rows, vocab, logits, ld or vocab,
                                  ctypes.addressof(client), 1.0, row_weight, loss, lse, grad, ldg or vocab)
        return self.L.fa_distill_grad(self.h, ctypes.byref(args), stream)

    def choice(self):
        cfg, splits, drain = ctypes.c_int(), ctypes.c_uint32(), ctypes.c_int()
        self.L.ws_choice(ctypes.byref(cfg), ctypes.byref(splits), ctypes.byref(drain))
        return cfg.value, splits.value, bool(drain.value)

    def sync(self):
        return self.L.ws_sync(self.h)

    def close(self):
        return self.L.ws_close(self.h)
