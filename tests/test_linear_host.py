"""Host-side checks of include/delta_linear.h and its binding (no GPU needed): exports, refusals with
their documented codes before any launch, workspace sizes, the environment switches."""
import ctypes
import os

import pytest

import chunkwise_delta_rule_chunked_amd as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "delta_linear.h")
A = 1 << 28   # fake, never-dereferenced device addresses, this far apart
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(D.lib_path()):
        pytest.fail("libdelta.so is not built (run `python -m chunkwise_delta_rule_chunked_amd.build`)")
    from chunkwise_delta_rule_chunked_amd import linear
    return linear._load()


@pytest.fixture
def no_gpu():
    # a guard against a validation slip that reaches a launch with a fake address
    if torch.cuda.is_available():
        pytest.skip("fake-pointer argument checks run on hosts without a GPU")


def fake(i, off=0):
    return ctypes.c_void_p(A * (i + 1) + off)


def shape(**kw):
    base = dict(B=2, L=100, H=6, dk=64, dv=32, n_h=1, chunk=64, dtype=D.BF16, scale=1.0)
    base.update(kw)
    return D.make_shape(**base)


def size(fn, *args):
    n = ctypes.c_size_t(12345)
    rc = getattr(D.load_library(), fn)(*args, ctypes.byref(n))
    return rc, n.value


FWD = ["q", "k", "v", "g", "S0", "O", "Sf", "w"]
BWD = ["q", "k", "v", "g", "S0", "dO", "dSf", "dq", "dk", "dv", "dg", "dS0", "w"]


def call(fn, names, optional, sh, hk, gate, kw):
    args = [kw[n] if n in kw else None if n in optional else fake(i) for i, n in enumerate(names)]
    return getattr(D.load_library(), fn)(ctypes.byref(sh), hk, gate, *args, kw.get("wbytes", A), None)


def fwd(sh=None, hk=3, gate=1, **kw):
    return call("delta_fwd_lin", FWD, ("S0", "Sf"), sh or shape(), hk, gate, kw)


def bwd(sh=None, hk=3, gate=1, **kw):
    return call("delta_bwd_lin", BWD, ("S0", "dSf", "dS0"), sh or shape(), hk, gate, kw)


def dec(sh=None, hk=3, gate=1, **kw):
    args = [kw[n] if n in kw else fake(i) for i, n in enumerate(["q", "k", "v", "g", "S", "O"])]
    return D.load_library().delta_decode_lin(ctypes.byref(sh or shape(L=1)), hk, gate, *args, None)


def test_exports_every_header_function(lib):
    names = D.header_functions(HEADER)
    assert set(names) == {"delta_fwd_lin_workspace_bytes", "delta_fwd_lin", "delta_bwd_lin_workspace_bytes", "delta_bwd_lin",
                          "delta_decode_lin"}
    for n in names:
        assert hasattr(lib, n), n


def test_fwd_refusals(lib, no_gpu):
    for n in ("q", "k", "v", "g", "O"):
        assert fwd(**{n: None}) == -1, n
    assert fwd(gate=0) == -1                                                       # gates given, none said
    assert fwd(gate=3) == -3 and fwd(gate=-1) == -3
    for kw in (dict(dk=48), dict(dk=256), dict(dv=24), dict(dv=272), dict(dtype=7)):
        assert fwd(shape(**kw)) == -3, kw
    for kw in (dict(n_h=2), dict(L=-1), dict(B=-1), dict(H=1 << 15), dict(L=(1 << 30) + 1)):
        assert fwd(shape(**kw), hk=1) == -2, kw
    assert fwd(hk=0) == -2 and fwd(hk=-3) == -2 and fwd(hk=4) == -2 and fwd(hk=12) == -2
    assert fwd(q=fake(0, 8)) == -4 and fwd(Sf=fake(20, 4)) == -4 and fwd(w=fake(7, 2)) == -4 and fwd(g=fake(3, 2)) == -4
    assert fwd(O=fake(0)) == -6 and fwd(O=fake(2)) == -6 and fwd(Sf=fake(5)) == -6
    assert fwd(S0=fake(20), Sf=fake(20, 256)) == -6                                # part of S0
    long = shape(L=5000)                                                           # in segments: with a workspace
    assert fwd(long, w=None) == -5 and fwd(long, w=fake(0)) == -6
    assert D.load_library().delta_fwd_lin(None, 1, 0, *[None] * 8, 0, None) == -1


def test_bwd_refusals(lib, no_gpu):
    for n in ("q", "k", "v", "g", "dO", "dq", "dk", "dv"):
        assert bwd(**{n: None}) == -1, n
    assert bwd(gate=0, g=None) == -3 and bwd(gate=5) == -3 and bwd(hk=5) == -2     # dg_log without gates
    for i, n in enumerate(BWD):
        assert bwd(**{n: fake(i, 2)}) == -4, n
    assert bwd(g=fake(3, 4), w=None) == -5                                         # gates need 4 bytes only
    assert bwd(dq=fake(1)) == -6 and bwd(dk=fake(7)) == -6 and bwd(dg=fake(3)) == -6 and bwd(dv=fake(5)) == -6
    assert bwd(dSf=fake(20), dS0=fake(20)) == -6 and bwd(S0=fake(20), dS0=fake(20)) == -6


def test_sizes_whose_launches_would_not_fit(lib, no_gpu):
    F, B = "delta_fwd_lin_workspace_bytes", "delta_bwd_lin_workspace_bytes"
    big = dict(L=1, dk=16, dv=16)
    for kw, rc in ((dict(big, B=1 << 20, H=1), 0), (dict(big, B=(1 << 20) + 1, H=1), -2), (dict(big, B=1 << 12, H=1 << 9), -2),
                   (dict(L=1, dk=128, dv=256, B=1 << 18, H=1), 0), (dict(L=1, dk=128, dv=256, B=(1 << 18) + 1, H=1), -2)):
        assert size(F, ctypes.byref(shape(**kw)), 1)[0] == rc and size(B, ctypes.byref(shape(**kw)), 1, 1)[0] == rc, kw
        if rc:
            assert fwd(shape(**kw), hk=1) == rc and bwd(shape(**kw), hk=1) == rc and dec(shape(**kw), hk=1) == rc, kw


def test_decode_refusals(lib, no_gpu):
    for n in ("q", "k", "v", "g", "S", "O"):
        assert dec(**{n: None}) == -1, n
    assert dec(shape(L=2)) == -2 and dec(shape(L=0)) == -2 and dec(hk=4) == -2 and dec(gate=9) == -3
    assert dec(S=fake(4, 8)) == -4 and dec(g=fake(3, 1)) == -4 and dec(O=fake(2)) == -6 and dec(S=fake(0)) == -6


def test_workspace_sizes(lib, no_gpu):
    F, B = "delta_fwd_lin_workspace_bytes", "delta_bwd_lin_workspace_bytes"
    ref = lambda **kw: ctypes.byref(shape(**kw))
    assert size(F, ref(L=0), 3) == (0, 0) and size(B, ref(L=0), 6, 0) == (0, 0)
    assert size(F, ref(L=40), 3) == (0, 0)                                         # one chunk
    assert size(F, ref(dk=8), 3)[0] == -3 and size(F, ref(), 4)[0] == -2 and size(B, ref(), 3, 9)[0] == -3
    assert getattr(lib, F)(ref(), 3, None) == -1 and getattr(lib, B)(ref(), 3, 1, None) == -1
    rc, need = size(F, ref(L=5000), 3)
    assert rc == 0 and need >= 2 * 6 * 64 * 32 * 4 * 2
    assert fwd(shape(L=5000), wbytes=need - 1) == -5
    none, token, head = (size(B, ref(L=5000), 3, g)[1] for g in range(3))
    assert need < none < token < head
    assert size(B, ref(L=5000), 6, 1)[1] < token                                   # shared heads have parts to add up
    assert bwd(shape(L=5000), wbytes=token - 1) == -5
    # the size fits what a call with fewer outputs takes too, and never falls with the length
    sizes = [size(B, ref(L=L, B=1), 3, 1)[1] for L in (1, 64, 65, 1000, 4096)]
    assert sizes == sorted(sizes)


def test_fault_injection(lib, no_gpu, monkeypatch):
    """Every call here passes all checks, so with the switch on it ends with DELTA_ERR_HIP."""
    monkeypatch.setenv("DELTA_FAULT", "launch")
    assert fwd() == -7 and bwd() == -7 and dec() == -7
    assert fwd(gate=2) == -7 and fwd(gate=0, g=None) == -7 and dec(gate=0, g=None) == -7 and dec(gate=2) == -7
    assert fwd(hk=1) == -7 and fwd(hk=6) == -7
    assert fwd(S0=fake(20), Sf=fake(20)) == -7                                     # in place
    assert bwd(gate=0, g=None, dg=None) == -7 and bwd(dg=None) == -7
    none = dict(q=None, k=None, v=None, g=None, O=None)
    assert fwd(shape(L=0), **none, Sf=fake(20)) == -7                              # the state as it was
    assert fwd(shape(L=0), **none) == 0 and fwd(shape(B=0)) == 0
    assert bwd(shape(L=0), dS0=fake(20)) == -7 and bwd(shape(L=0)) == 0
    assert bwd(shape(L=0), gate=2) == -7 and bwd(shape(B=0), gate=2) == -7         # a gradient to clear
    assert dec(shape(L=1, B=0)) == 0


def test_binding_refuses_before_the_library(lib):
    x, s = torch.zeros(1, 4, 1, 16), torch.zeros(1, 1, 16, 16)
    for f in (lambda: D.fwd_lin(x, x, x), lambda: D.bwd_lin(x, x, x, None, None, x), lambda: D.decode_lin(x[:, :1], x[:, :1], x[:, :1], None, s)):
        with pytest.raises(ValueError):
            f()


def test_host_checks_under_the_sanitizers(tmp_path):
    """This file again in a child process, with linear_abi.cpp rebuilt under AddressSanitizer and
    UndefinedBehaviorSanitizer and linked with the kernels' objects as built."""
    base = pytest.importorskip("test_sanitizers")
    if "linear_abi_san" in os.environ.get("DELTA_TEST_CHILD", ""):
        pytest.skip("the child itself")
    import glob
    import subprocess
    clang = os.path.join(base.ROCM, "lib", "llvm", "bin", "clang++")
    rt = sorted(glob.glob(os.path.join(base.ROCM, "lib", "llvm", "lib", "clang", "*", "lib", "linux",
                                       "libclang_rt.asan-x86_64.so")))
    pkg = os.path.join(base.ROOT, "chunkwise_delta_rule_chunked_amd")
    objs = [o for o in sorted(glob.glob(os.path.join(pkg, "_build", "*.o"))) if os.path.basename(o) != "linear_abi.o"]
    if not os.path.exists(clang) or not rt or len(objs) < 5:
        pytest.skip("needs ROCm's clang, its sanitizer runtime and the library's built objects")
    abi, so = str(tmp_path / "linear_abi_san.o"), str(tmp_path / "libdelta_san.so")
    subprocess.run([clang, "-x", "c++", "-std=c++17", "-O1", "-g", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I" + os.path.join(base.ROCM, "include")] + base.SAN +
                   ["-c", os.path.join(pkg, "csrc", "linear_abi.cpp"), "-o", abi], check=True)
    subprocess.run([os.path.join(base.ROCM, "bin", "hipcc"), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", so, abi] + objs,
                   check=True, capture_output=True)
    undef = subprocess.run(["nm", "-D", "--undefined-only", so], capture_output=True, text=True).stdout
    assert "__asan_" in undef and "__ubsan_" in undef
    run = base.ABI_RUN.replace("tests/test_abi_host.py", "tests/test_linear_host.py")
    out = base._child("import os\nos.environ['DELTA_TEST_CHILD'] = 'linear_abi_san'\n" + run % so, rt[-1])
    assert " passed" in out and " failed" not in out
