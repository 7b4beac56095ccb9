"""csrc/layers.cpp and csrc/orthogonalise.cpp over fakes of the CUDA runtime and of their kernels'
launches (tests/native/work_shim.cpp, step_shim.cpp), for the CPU tests of their host logic."""
import ctypes
import os
import subprocess

import pytest

import server_side_fedavg_gb300 as fa

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "server_side_fedavg_gb300", "csrc")
SO = os.path.join(HERE, "_build", "libstep_shim.so")
CUDA_INC = "/usr/local/cuda/include"

_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.isdir(CUDA_INC):
            pytest.skip("CUDA headers are not installed")
        os.makedirs(os.path.dirname(SO), exist_ok=True)
        srcs = [os.path.join(HERE, "native", f) for f in ("work_shim.cpp", "step_shim.cpp")]
        srcs += [os.path.join(CSRC, f) for f in ("work.cpp", "layers.cpp", "orthogonalise.cpp")]
        deps = srcs + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".hpp"))]
        deps.append(os.path.join(ROOT, "include", "fedavg.h"))
        if not os.path.exists(SO) or any(os.path.getmtime(s) > os.path.getmtime(SO) for s in deps):
            subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", CSRC, "-I",
                            os.path.join(ROOT, "include"), "-I", CUDA_INC] + srcs + ["-o", SO], check=True)
        L = ctypes.CDLL(SO)
        vp = ctypes.c_void_p
        L.ws_log.restype = ctypes.c_char_p
        L.ss_reset.argtypes = [ctypes.c_uint32]
        L.ss_turn.restype = ctypes.c_uint64
        L.fa_work_open.argtypes = [vp, vp]
        L.fa_work_close.argtypes = [vp]
        L.fa_work_last_error.argtypes = [vp]
        L.fa_work_last_error.restype = ctypes.c_char_p
        for name in ("fa_rotary", "fa_group_norm", "fa_group_norm_backward", "fa_orthogonalise"):
            getattr(L, name).argtypes = [vp, vp, vp]
        _lib = L
    return _lib


class Step:
    """A handle on the fake device.  Addresses are plain numbers: nothing is read."""

    def __init__(self, workspace_bytes=1 << 30):
        self.L = lib()
        self.L.ws_reset()
        self.L.ss_reset(0)
        self.h = ctypes.c_void_p()
        o = fa.fa_work_opts(ctypes.sizeof(fa.fa_work_opts), 0, workspace_bytes, 0, 0)
        assert self.L.fa_work_open(ctypes.byref(o), ctypes.byref(self.h)) == fa.FA_OK
        self.L.ws_clear_log()

    def error(self):
        return self.L.fa_work_last_error(self.h).decode()

    def log(self):
        return self.L.ws_log().decode().split()

    def call(self, name, args, stream=0):
        return getattr(self.L, name)(self.h, ctypes.byref(args), stream)

    def close(self):
        return self.L.fa_work_close(self.h)


FAR = [i << 40 for i in range(1, 16)]
_turns = (ctypes.c_uint64 * 256)(*range(1, 257))


def rotary(batch=2, seq=8, dim=64, r=64, qh=4, kh=2, dtype="bf16", flags=0, q=FAR[0], qo=FAR[1], k=FAR[2], ko=FAR[3], position=FAR[4],
           first=0, scale=1.0, turns=True, qs=None, qos=None, ks=None, kos=None, size=None):
    own = lambda h: (seq * h * dim, h * dim, dim)  # noqa: E731
    part = lambda x, o, h, s, t: fa.fa_rotary_part(x, o, h, 0, *(s or own(h)), *(t or own(h)))  # noqa: E731
    return fa.fa_rotary_args(ctypes.sizeof(fa.fa_rotary_args) if size is None else size, flags, fa.DTYPES.get(dtype, dtype), dim, r, 0,
                             batch, seq, ctypes.addressof(_turns) if turns else None, position, first, scale,
                             part(q, qo, qh, qs, qos), part(k, ko, kh, ks, kos))


def norm(n=2, P=100, C=32, G=4, dtype="bf16", param="f32", act=0, flags=0, x=FAR[0], ldx=None, sx=0, y=FAR[1], ldy=None, sy=0,
         gamma=FAR[2], beta=FAR[3], eps=1e-5, mean=FAR[4], rstd=FAR[5]):
    return fa.fa_group_norm_args(ctypes.sizeof(fa.fa_group_norm_args), flags, fa.DTYPES.get(dtype, dtype), fa.DTYPES.get(param, param),
                                 act, 0, n, P, C, G, x, C if ldx is None else ldx, sx, y, C if ldy is None else ldy, sy, gamma, beta,
                                 eps, mean, rstd)


def norm_backward(n=2, P=100, C=32, G=4, dtype="bf16", param="f32", act=0, flags=0, x=FAR[0], dout=FAR[1], gamma=FAR[2], beta=FAR[3],
                  mean=FAR[4], rstd=FAR[5], dx=FAR[6], d_gamma=FAR[7], d_beta=FAR[8], ldx=None, ldd=None, lddx=None):
    return fa.fa_group_norm_backward_args(
        ctypes.sizeof(fa.fa_group_norm_backward_args), flags, fa.DTYPES.get(dtype, dtype), fa.DTYPES.get(param, param), act, 0, n, P, C,
        G, x, ldx or C, 0, dout, ldd or C, 0, gamma, beta, mean, rstd, dx, lddx or C, 0, d_gamma, d_beta)


def ortho(count=2, rows=100, cols=60, din="bf16", dout="bf16", steps=5, flags=0, u=FAR[0], ldu=None, su=0, m=None, ldm=None, sm=0, mo=None,
          ldmo=None, smo=0, res=None, ldr=None, sr=0, out=FAR[4], ldo=None, so=0, mu=0.9, eps=1e-7, alpha=1.0, beta=1.0,
          abc=(3.4445, -4.7750, 2.0315)):
    ld = lambda v: cols if v is None else v  # noqa: E731
    return fa.fa_orthogonalise_args(ctypes.sizeof(fa.fa_orthogonalise_args), flags, fa.DTYPES.get(din, din), fa.DTYPES.get(dout, dout),
                                    steps, 0, count, rows, cols, u, ld(ldu), su, m, ld(ldm), sm, mo, ld(ldmo), smo, res, ld(ldr), sr, out,
                                    ld(ldo), so, mu, eps, alpha, beta, *abc)
