"""C-ABI checks of the routing, combine and clipping entry points that need no
GPU: every argument error is found on the host before any launch, under the
sanitizers too."""
import ctypes
import glob
import os
import subprocess
import sys
import tempfile

import pytest

from mxfp4_precision_numerics_amd import mx

FAKE = 0x1000   # aligned, never dereferenced (validation fails first)
NULL, SHAPE, ALIGN, DTYPE, UNSUPPORTED = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def L():
    return mx.lib()


def caller(fn, **ok):
    def call(**kw):
        assert set(kw) <= set(ok), kw
        return fn(*dict(ok, **kw).values())
    return call


def test_symbols(L):
    names = set(mx.declared_functions())
    assert names >= {"mx_route", "mx_route_bwd", "mx_route_plan", "mx_route_plan_workspace", "mx_combine",
                     "mx_combine_bwd", "mx_grad_workspace", "mx_grad_norm", "mx_grad_clip"}
    for n in names:
        assert hasattr(L, n), n


def test_route_validation(L):
    call = caller(L.mx_route, l=FAKE, lt=mx.MX_F32, t=4, e=32, ld=0, bias=None, score=0, g=1, tg=1, gb=1, k=4, rn=1,
                  scale=1.0, ids=FAKE, w=FAKE, s=None)
    assert call(lt=2) == DTYPE and call(score=2) == UNSUPPORTED
    for bad in (dict(t=-1), dict(t=2 ** 24 + 1), dict(e=0), dict(e=1025), dict(k=0), dict(k=33), dict(e=2), dict(ld=31),
                dict(ld=-1), dict(g=0), dict(g=5), dict(g=4, tg=5), dict(g=4, tg=0), dict(gb=0), dict(gb=3),
                dict(g=8, tg=1, k=5), dict(e=128, g=128), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**bad) == SHAPE, bad
    assert call(l=None) == NULL and call(ids=None) == NULL and call(w=None) == NULL
    assert call(l=FAKE + 2) == ALIGN and call(bias=FAKE + 1) == ALIGN and call(ids=FAKE + 2) == ALIGN
    assert call(w=FAKE + 2) == ALIGN and call(lt=mx.MX_BF16, l=FAKE + 1) == ALIGN
    assert call(t=0, l=None, ids=None, w=None) == 0


def test_route_bwd_validation(L):
    call = caller(L.mx_route_bwd, l=FAKE, lt=mx.MX_F32, t=4, e=32, ld=0, score=0, k=4, rn=1, scale=1.0, ids=FAKE,
                  dw=FAKE, dl=FAKE, dld=0, s=None)
    assert call(lt=7) == DTYPE and call(score=-1) == UNSUPPORTED
    for bad in (dict(t=-1), dict(e=1025), dict(k=33), dict(k=0), dict(ld=8), dict(dld=31), dict(dld=-4)):
        assert call(**bad) == SHAPE, bad
    for name in ("l", "ids", "dw", "dl"):
        assert call(**{name: None}) == NULL and call(**{name: FAKE + 2}) == ALIGN
    assert call(t=0, l=None, ids=None, dw=None, dl=None) == 0


def test_route_plan_validation(L):
    call = caller(L.mx_route_plan, ids=FAKE, t=65536, k=4, e=32, off=FAKE, row=FAKE, slot=FAKE, ws=FAKE, s=None)
    for bad in (dict(t=-1), dict(k=0), dict(e=0), dict(e=1025), dict(t=2 ** 30, k=2)):
        assert call(**bad) == SHAPE, bad
    for name in ("ids", "off", "row", "slot", "ws"):
        assert call(**{name: None}) == NULL and call(**{name: FAKE + 2}) == ALIGN
    assert call(t=0, off=None) == NULL
    ws = L.mx_route_plan_workspace
    assert ws(0, 4, 32) == 0 and ws(4, 4, 32) >= 0 and ws(65536, 4, 32) > 0 and ws(65536, 8, 256) > 0
    for bad in ((-1, 4, 32), (4, 0, 32), (4, 4, 0), (4, 4, 1025), (2 ** 30, 2, 32)):
        assert ws(*bad) == 0


def test_combine_validation(L):
    call = caller(L.mx_combine, y=FAKE, yt=mx.MX_BF16, rows=16, cols=64, yld=0, slot=FAKE, w=FAKE, t=4, k=4, res=None,
                  rld=0, out=FAKE, ot=mx.MX_F32, old=0, s=None)
    assert call(yt=5) == DTYPE and call(ot=-1) == DTYPE
    for bad in (dict(rows=-1), dict(rows=2 ** 31), dict(cols=0), dict(yld=63), dict(t=-1), dict(k=0), dict(rld=1),
                dict(old=63), dict(t=2 ** 30, k=2), dict(t=2 ** 26, k=1), dict(t=2 ** 20, cols=2 ** 15)):
        assert call(**bad) == SHAPE, bad
    for name in ("y", "slot", "out"):
        assert call(**{name: None}) == NULL
    for name in ("y", "slot", "out", "w", "res"):
        assert call(**{name: FAKE + 1}) == ALIGN
    assert call(t=0, y=None, slot=None, out=None) == 0


def test_combine_bwd_validation(L):
    call = caller(L.mx_combine_bwd, do=FAKE, dt=mx.MX_BF16, dld=0, y=FAKE, yt=mx.MX_BF16, rows=16, cols=64, yld=0,
                  slot=FAKE, w=FAKE, t=4, k=4, used=None, dy=FAKE, dyld=0, dw=FAKE, s=None)
    assert call(dt=9) == DTYPE and call(yt=9) == DTYPE
    for bad in (dict(rows=-1), dict(cols=0), dict(yld=63), dict(dld=63), dict(dyld=63), dict(t=-1), dict(k=0),
                dict(t=2 ** 23)):
        assert call(**bad) == SHAPE, bad
    for name in ("do", "y", "slot", "dy"):
        assert call(**{name: None}) == NULL
    for name in ("do", "y", "slot", "dy", "w", "used", "dw"):
        assert call(**{name: FAKE + 1}) == ALIGN
    assert call(t=0, do=None, slot=None) == 0


def test_grad_validation(L):
    def arrays(types, numels, ptrs):
        n = len(types)
        return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int * n)(*types), (ctypes.c_int64 * n)(*numels), n)

    good = arrays([0, 1], [5, 6], [FAKE, FAKE])
    outs = (ctypes.c_void_p * 9)(*[FAKE] * 9)

    def norm(a=good, ws=FAKE, out=FAKE):
        return L.mx_grad_norm(*a, ws, out, None)

    def clip(a=good, o=outs, m=1.0, ws=FAKE, out=FAKE):
        return L.mx_grad_clip(*a, o, m, ws, out, None)

    for call in (norm, clip):
        assert call(a=arrays([0, 2], [5, 6], [FAKE, FAKE])) == DTYPE
        assert call(a=arrays([0, 0], [5, -1], [FAKE, FAKE])) == SHAPE
        assert call(a=arrays([0, 0], [2 ** 40, 1], [FAKE, FAKE])) == SHAPE
        assert call(a=arrays([0, 0], [2 ** 62, 2 ** 62], [FAKE, FAKE])) == SHAPE
        assert call(a=arrays([0], [2 ** 34 + 1], [FAKE])) == SHAPE          # over 64 GB in one tensor
        assert call(a=arrays([1] * 9, [2 ** 34] * 9, [FAKE] * 9)) == SHAPE  # over 2^37 elements
        assert call(a=arrays([0, 0], [5, 6], [FAKE, None])) == NULL
        assert call(a=arrays([0, 1], [5, 6], [FAKE + 2, FAKE])) == ALIGN
        assert call(a=(None, good[1], good[2], 2)) == NULL
        assert call(a=(good[0], good[1], good[2], -1)) == SHAPE
        assert call(ws=None) == NULL and call(out=None) == NULL
        assert call(ws=FAKE + 4) == ALIGN and call(out=FAKE + 2) == ALIGN
    assert clip(m=-1.0) == SHAPE and clip(m=float("nan")) == SHAPE
    assert clip(o=(ctypes.c_void_p * 2)(FAKE, None)) == NULL
    assert clip(o=(ctypes.c_void_p * 2)(FAKE, FAKE + 1)) == ALIGN
    assert L.mx_grad_workspace(0) == 0 and L.mx_grad_workspace(-3) == 0
    assert L.mx_grad_workspace(1000) >= L.mx_grad_workspace(1) > 0


class FakeGrad:
    """What the binding asks of a gradient, on a device of our choice."""

    def __init__(self, device, contiguous=True):
        import torch
        self.dtype, self.device, self.contiguous = torch.float32, device, contiguous

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return 4

    def data_ptr(self):
        return FAKE

    @property
    def is_cuda(self):
        return self.device >= 0


def test_gradients_of_two_devices_are_refused(L):
    mx._torch()
    grads = [FakeGrad(0), FakeGrad(0)]
    assert list(mx._grad_list(grads, "grads")[2]) == [4, 4] and mx._grad_list(grads, "grads")[-1] == 0
    for bad in ([FakeGrad(0), FakeGrad(1)], [FakeGrad(0), FakeGrad(-1)], [FakeGrad(0), FakeGrad(0, contiguous=False)]):
        with pytest.raises(ValueError):
            mx._grad_list(bad, "grads")
        with pytest.raises(ValueError):
            mx.grad_norm(bad)
        with pytest.raises(ValueError):
            mx.grad_clip(grads, 1.0, outs=bad)
    with pytest.raises(ValueError):                        # outs elsewhere than grads
        mx.grad_clip(grads, 1.0, outs=[FakeGrad(1), FakeGrad(1)])
    assert mx._grad_list([], "grads", 0)[-1] is None


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG_RT = (glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so") + [""])[0]


@pytest.mark.skipif(not os.path.exists(CLANG_RT), reason="no clang AddressSanitizer runtime")
def test_host_validation_under_sanitizers():
    """This file's other tests on a library whose host code has the address
    and undefined-behaviour sanitizers on."""
    src = os.path.join(ROOT, "mxfp4_precision_numerics_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        lib = os.path.join(d, "libmx355_asan.so")
        cmd = ["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
               "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Xarch_host", "-fsanitize=address,undefined",
               # C callers may pass any int where the header says an enum
               "-Xarch_host", "-fno-sanitize=enum",
               "-Xarch_host", "-fno-sanitize-recover=all", "-o", lib]
        cmd += [os.path.join(src, n) for n in ("mx_quant.hip", "mx_gemm.hip", "mx_route.hip", "mx_combine.hip",
                                               "mx_grad.hip")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        code = ("import sys; sys.path[:0] = [%r, %r]\n"
                "from mxfp4_precision_numerics_amd import mx\n"
                "mx.LIB_PATH = %r\n"
                "import test_abi_moe as t\n"
                "for n, f in sorted(vars(t).items()):\n"
                "    if n.startswith('test_') and n.endswith('_validation'): f(mx.lib()); print(n)\n"
                "print('library ok')\n") % (ROOT, os.path.join(ROOT, "tests"), lib)
        env = dict(os.environ, LD_PRELOAD=CLANG_RT, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", PYTHONPATH=ROOT)
        r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=600)
        out = r.stdout + r.stderr
        assert r.returncode == 0 and "library ok" in out and "runtime error" not in out, out[-4000:]
