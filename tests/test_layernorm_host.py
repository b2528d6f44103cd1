"""Host-side checks of include/delta_layernorm.h and its binding (no GPU needed): exports, refusals with
their documented codes before any launch, workspace sizes, the environment switches."""
import ctypes
import os

import pytest

import chunkwise_delta_rule_chunked_amd as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "delta_layernorm.h")
A = 1 << 24   # fake, never-dereferenced device addresses, this far apart
EPS = ctypes.c_float(1e-5)
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(D.lib_path()):
        pytest.fail("libdelta.so is not built (run `python -m chunkwise_delta_rule_chunked_amd.build`)")
    from chunkwise_delta_rule_chunked_amd import layernorm
    return layernorm._load()


@pytest.fixture
def no_gpu():
    # a guard against a validation slip that reaches a launch with a fake address
    if torch.cuda.is_available():
        pytest.skip("fake-pointer argument checks run on hosts without a GPU")


def fake(i, off=0):
    return ctypes.c_void_p(A * (i + 1) + off)


def drop(p=0.1, step=None):
    from chunkwise_delta_rule_chunked_amd.layernorm import Dropout
    return ctypes.byref(Dropout(p, 1, 2, step))


def call(fn, names, none, rows, width, dtype, head, kw, tail=()):
    args = [kw[n] if n in kw else None if n in none else fake(i) for i, n in enumerate(names)]
    return getattr(D.load_library(), fn)(rows, width, dtype, *head, *args, *tail, None)


def dropout(rows=4, width=100, dtype=D.F32, d=0, **kw):
    return call("delta_layer_dropout", ["x", "r", "y"], (), rows, width, dtype, [drop() if d == 0 else d], kw)


def fwd(rows=4, width=100, dtype=D.F32, eps=EPS, d=0, **kw):
    return call("delta_layer_layernorm", ["x", "r", "w", "b", "sum", "y"], (), rows, width, dtype, [eps, drop() if d == 0 else d], kw)


def bwd(rows=4, width=100, dtype=D.F32, eps=EPS, d=0, wbytes=1 << 20, **kw):
    names = ["dy", "s", "w", "dsum", "dr", "dx", "dw", "db", "ws"]
    return call("delta_layer_layernorm_bwd", names, (), rows, width, dtype, [eps, drop() if d == 0 else d], kw, (wbytes,))


def test_exports_every_header_function(lib):
    names = D.header_functions(HEADER)
    assert set(names) == {"delta_layer_dropout", "delta_layer_layernorm", "delta_layer_layernorm_bwd_workspace_bytes",
                          "delta_layer_layernorm_bwd"}
    for n in names:
        assert hasattr(lib, n), n


def test_refusals(lib, no_gpu):
    for f in (dropout, fwd, bwd):
        assert f(rows=-1) == -2 and f(rows=1 << 31) == -2 and f(width=0) == -2 and f(width=(1 << 20) + 1) == -2
        assert f(dtype=9) == -3
        for p in (-0.1, 1.1, float("nan"), float("inf")):
            assert f(d=drop(p)) == -2, p
        assert f(d=drop(0.1, A + 4)) == -4
    assert dropout(d=None) == -1 and dropout(x=None) == -1 and dropout(y=None) == -1
    for f in (fwd, bwd):
        assert f(eps=ctypes.c_float(-1.0)) == -2 and f(eps=ctypes.c_float(float("nan"))) == -2
    for n in ("x", "w", "sum", "y"):
        assert fwd(**{n: None}) == -1, n
    assert fwd(sum=None, r=None) == -1                                             # dropped: s is a tensor of its own
    for n in ("dy", "s", "w", "dr", "dx"):
        assert bwd(**{n: None}) == -1, n
    for i, n in enumerate(["x", "r", "w", "b", "sum", "y"]):
        assert fwd(**{n: fake(i, 8 if n in "wb" else 2)}) == -4, n
    for i, n in enumerate(["dy", "s", "w", "dsum", "dr", "dx", "dw", "db", "ws"]):
        assert bwd(**{n: fake(i, 4 if n in ("w", "dw", "db", "ws") else 2)}) == -4, n
    assert dropout(x=fake(0, 2)) == -4 and dropout(r=fake(1, 1), dtype=D.BF16) == -4
    assert fwd(y=fake(0)) == -6 and fwd(y=fake(4)) == -6 and fwd(sum=fake(0, 16)) == -6 and fwd(y=fake(3)) == -6
    assert bwd(dr=fake(0)) == -6 and bwd(dx=fake(4)) == -6 and bwd(db=fake(6)) == -6 and bwd(ws=fake(1)) == -6
    assert dropout(y=fake(0, 16)) == -6 and dropout(y=fake(1, 16)) == -6
    assert dropout(d=drop(0.1, A * 3)) == -6 and fwd(d=drop(0.1, A * 6)) == -6     # the step in what is written


def test_workspace(lib, no_gpu):
    n = ctypes.c_size_t(0)
    f = lib.delta_layer_layernorm_bwd_workspace_bytes
    assert f(0, 100, D.F32, ctypes.byref(n)) == 0 and n.value == 0
    assert f(4, 0, D.F32, ctypes.byref(n)) == -2 and f(4, 8, 7, ctypes.byref(n)) == -3 and f(4, 8, D.F32, None) == -1
    assert f(4, 100, D.F32, ctypes.byref(n)) == 0 and n.value >= 2 * 4 * 100
    assert bwd(wbytes=n.value - 1) == -5 and bwd(ws=None) == -5


def test_fault_injection(lib, no_gpu, monkeypatch):
    """Every call here passes all checks, so with the switch on it ends with DELTA_ERR_HIP."""
    monkeypatch.setenv("DELTA_FAULT", "launch")
    assert dropout() == -7 and dropout(r=None) == -7 and dropout(y=fake(0)) == -7 and dropout(y=fake(1)) == -7
    assert dropout(d=drop(0.1, A * 9)) == -7 and dropout(rows=0) == 0 and dropout(d=drop(1.0)) == -7
    assert fwd() == -7 and fwd(b=None) == -7 and fwd(r=None) == -7 and fwd(d=None) == -7
    assert fwd(sum=fake(0)) == -7 and fwd(sum=fake(1)) == -7                       # over x, over the residual
    assert fwd(r=None, d=None, sum=None) == -7 and fwd(r=None, d=drop(0.0), sum=None) == -7
    assert fwd(r=None, d=None, sum=fake(0)) == -7                                  # not used
    assert bwd() == -7 and bwd(dsum=None) == -7 and bwd(dw=None) == -7 and bwd(db=None) == -7
    assert bwd(d=None, dx=None) == -7 and bwd(dw=None, db=None, ws=None, wbytes=0) == -7
    assert bwd(d=None, dx=fake(4)) == -7                                           # not used
    assert dropout(x=fake(0, 2), y=fake(2, 6), dtype=D.BF16) == -7 and fwd(x=fake(0, 4), sum=fake(4, 12)) == -7   # rows at any element
    assert fwd(rows=0) == 0 and bwd(rows=0) == -7 and bwd(rows=0, dw=None, db=None) == 0


def test_binding_refuses_before_the_library(lib):
    x, w = torch.zeros(4, 16), torch.ones(16)
    for f in (lambda: D.layer_dropout(x, p=0.1, seed=1), lambda: D.layer_layernorm(x, w), lambda: D.layer_layernorm_bwd(x, x, w)):
        with pytest.raises(ValueError):
            f()


def test_host_checks_under_the_sanitizers(tmp_path):
    """This file again in a child process, with layernorm_abi.cpp rebuilt under AddressSanitizer and
    UndefinedBehaviorSanitizer and linked with the kernels' objects as built."""
    base = pytest.importorskip("test_sanitizers")
    if "layernorm_abi_san" in os.environ.get("DELTA_TEST_CHILD", ""):
        pytest.skip("the child itself")
    import glob
    import subprocess
    clang = os.path.join(base.ROCM, "lib", "llvm", "bin", "clang++")
    rt = sorted(glob.glob(os.path.join(base.ROCM, "lib", "llvm", "lib", "clang", "*", "lib", "linux",
                                       "libclang_rt.asan-x86_64.so")))
    pkg = os.path.join(base.ROOT, "chunkwise_delta_rule_chunked_amd")
    objs = [o for o in sorted(glob.glob(os.path.join(pkg, "_build", "*.o"))) if os.path.basename(o) != "layernorm_abi.o"]
    if not os.path.exists(clang) or not rt or len(objs) < 5:
        pytest.skip("needs ROCm's clang, its sanitizer runtime and the library's built objects")
    abi, so = str(tmp_path / "layernorm_abi_san.o"), str(tmp_path / "libdelta_san.so")
    subprocess.run([clang, "-x", "c++", "-std=c++17", "-O1", "-g", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I" + os.path.join(base.ROCM, "include")] + base.SAN +
                   ["-c", os.path.join(pkg, "csrc", "layernorm_abi.cpp"), "-o", abi], check=True)
    subprocess.run([os.path.join(base.ROCM, "bin", "hipcc"), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", so, abi] + objs,
                   check=True, capture_output=True)
    undef = subprocess.run(["nm", "-D", "--undefined-only", so], capture_output=True, text=True).stdout
    assert "__asan_" in undef and "__ubsan_" in undef
    run = base.ABI_RUN.replace("tests/test_abi_host.py", "tests/test_layernorm_host.py")
    out = base._child("import os\nos.environ['DELTA_TEST_CHILD'] = 'layernorm_abi_san'\n" + run % so, rt[-1])
    assert " passed" in out and " failed" not in out
