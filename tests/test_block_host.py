"""Host-side checks of the block operators' C ABI and binding (no GPU needed).

block_api.cpp (argument checks and planning) is built with g++ and stub
launchers (tests/host_shim/block_stubs.cpp) under the address and
undefined-behaviour sanitizers, and driven through ctypes in a child
interpreter: with RETENTION_BLOCK_TEST_LIB set, this file's calls go to that
build, where valid arguments reach a stub; otherwise the refusals alone run,
against the real library. No pointer below is ever dereferenced.
"""

import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import retnet_retention_msr_amd as ret
from retnet_retention_msr_amd import _lib, block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "retnet_retention_msr_amd", "csrc")
HEADER = os.path.join(ROOT, "include", "retention_block.h")
SHIM = os.environ.get("RETENTION_BLOCK_TEST_LIB")
shim_only = pytest.mark.skipif(not SHIM, reason="valid-argument calls only run against the host shim")

INVALID, UNSUPPORTED = _lib.RET_ERR_INVALID_ARG, _lib.RET_ERR_UNSUPPORTED
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not SHIM:
        return _lib.load()
    return _lib.declare_block(ctypes.CDLL(SHIM))


def _v(at, sb=0, sh=0, sn=0):
    return ctypes.byref(_lib.View(at, sb, sh, sn))


def _norm(eps=1e-5, rms=0, weight=None, bias=None):
    return ctypes.byref(_lib.NormStruct(eps, rms, weight, bias))


A = [0x100000000 + i * 1024 * MB for i in range(12)]  # far apart
WS = A[11]


def recurrence(lib, B=2, H=3, N=100, d=64, form=0, dtype=1, x=A[0], g=A[1], h=A[2], s_in=None, s_out=None, cu=None, S=None,
               max_len=None, ws=WS, ws_bytes=1 << 40, strides=None, h_strides=None):
    st = (H * N * d, N * d, d) if strides is None else strides
    return lib.retention_gated_recurrence(_v(x, *st), _v(g, *st), _v(h, *(h_strides or st)), B, H, N, d, form, dtype, s_in, s_out,
                                          cu, B if S is None else S, N if max_len is None else max_len, ws, ws_bytes, None)


def backward(lib, B=2, H=3, N=100, d=64, form=0, dtype=1, x=A[1], dx=A[4], dg=A[5], s_in=None, ds=None, ds_in=None, ws=WS):
    st = (H * N * d, N * d, d)
    return lib.retention_gated_recurrence_backward(_v(A[0], *st), _v(x, *st) if x else None, _v(A[2], *st), _v(A[3], *st),
                                                   _v(dx, *st), _v(dg, *st), B, H, N, d, form, dtype, s_in, ds, ds_in, None,
                                                   B, N, ws, 1 << 40, None)


def step(lib, B=4, H=2, d=64, form=0, dtype=1, x=A[0], g=A[1], h=A[2], states=A[3], n=4, slots=None):
    st = (H * d, d, 0)
    return lib.retention_gated_recurrence_step(_v(x, *st), _v(g, *st), _v(h, *st), B, H, d, form, dtype, states, n, slots, None)


def gnorm(lib, B=2, H=3, N=10, d=64, dtype=1, o=A[0], gate=A[1], y=A[2], norm=None):
    st = (H * N * d, N * d, d)
    return lib.retention_gated_norm(_v(o, *st), _v(gate, *st) if gate else None, _v(y, *st), B, H, N, d, dtype,
                                    norm or _norm(), None)


def gnorm_back(lib, B=2, H=3, N=10, d=64, gate=A[2], do=A[3], dg=A[4], dw=A[5], db=A[6], ws=WS, ws_bytes=1 << 40):
    st = (H * N * d, N * d, d)
    return lib.retention_gated_norm_backward(_v(A[0], *st), _v(A[1], *st), _v(gate, *st) if gate else None, _v(do, *st),
                                             _v(dg, *st) if dg else None, B, H, N, d, 1, _norm(), dw, db, ws, ws_bytes, None)


def rnorm(lib, B=2, N=10, D=64, dtype=1, stream=1, x=A[0], res=A[1], y=A[2], r=A[3], norm=None, scale=None, alpha=1.0):
    st = (N * D, 0, D)
    return lib.retention_residual_norm(_v(x, *st), _v(res, *st), _v(y, *st), _v(r, *st), B, N, D, dtype, stream,
                                       norm or _norm(), scale, alpha, None)


def rnorm_back(lib, B=2, N=10, D=64, dr=A[1], r=A[2], x=A[3], res=None, dx=A[4], dres=A[5], dscale=A[6], dw=A[7], db=A[8], ws=WS,
               ws_bytes=1 << 40, alpha=1.0):
    st = (N * D, 0, D)
    return lib.retention_residual_norm_backward(_v(A[0], *st), _v(dr, *st) if dr else None,
                                                _v(r, *st) if r else None, _v(x, *st) if x else None,
                                                _v(res, *st) if res else None, _v(dx, *st) if dx else None, _v(dres, *st), B, N, D,
                                                1, 1, _norm(), None, alpha, dscale, dw, db, ws, ws_bytes, None)


def test_header_declares_the_binding_symbols(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(retention_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(_lib.BLOCK_EXPORTED)
    assert all(hasattr(lib, n) for n in names)


BAD_SIZES = [dict(B=0), dict(N=-1), dict(d=0), dict(dtype=2)]


@pytest.mark.parametrize("kw", BAD_SIZES + [
    dict(H=0), dict(form=2), dict(form=-1), dict(x=None), dict(g=None), dict(h=None), dict(x=A[0] + 1), dict(h=A[2] + 1),
    dict(S=1), dict(max_len=99), dict(cu=A[5]), dict(cu=A[5], B=1, S=0), dict(cu=A[5] + 2, B=1, S=3),
    dict(cu=A[5], B=1, S=3, max_len=0), dict(h=A[0]), dict(h=A[1] + 128), dict(s_in=A[4] + 2), dict(s_out=A[0]),
    dict(s_in=A[4], s_out=A[4] + 4), dict(strides=(-1, 64, 64)), dict(h_strides=(0, 6400, 64)), dict(h_strides=(19200, 6400, 32)),
    dict(h_strides=(64, 64, 64)),
])
def test_recurrence_refuses(lib, kw):
    assert recurrence(lib, **kw) == INVALID


def test_recurrence_limits(lib):
    assert recurrence(lib, B=1 << 16, H=1 << 10, N=1 << 10) == UNSUPPORTED
    assert recurrence(lib, d=(1 << 20) + 1) == UNSUPPORTED
    assert recurrence(lib, B=1, H=(1 << 31) - 2, N=1, d=1 << 20, cu=A[5], S=1 << 20, strides=(0, 0, 0), h_strides=(0, 1 << 20, 0)) == UNSUPPORTED
    assert recurrence(lib, B=1, cu=A[5], S=(1 << 20) + 1) == UNSUPPORTED
    assert recurrence(lib, strides=(1 << 34, 1 << 32, 1 << 24), h_strides=(19200, 6400, 64)) == UNSUPPORTED
    assert recurrence(lib, strides=(1 << 60, 6400, 64), h_strides=(19200, 6400, 64)) == UNSUPPORTED


def test_recurrence_workspace(lib):
    f = lib.retention_gated_recurrence_workspace_bytes
    for bad in ((0, 1, 9, 9, 0, 1, 1), (1, 0, 9, 9, 0, 1, 1), (1, 1, 0, 0, 0, 1, 1), (1, 1, 9, 9, 0, 0, 1), (1, 1, 9, 9, 0, 1, 2),
                (1, 1, 9, 8, 0, 1, 1), (1, 1, 9, 0, 1, 1, 1)):
        assert f(*bad) == 0
    need = f(1, 3, 60000, 60000, 0, 64, 1)
    assert need > 0 == f(1, 3, 32, 32, 0, 64, 1)
    # A packed row's need goes with its tokens and the number of its sequences, not with their product.
    assert f(64, 3, 60000, 60000, 1, 64, 1) < 2 * need
    if need:
        assert recurrence(lib, B=1, N=60000, ws=None) == INVALID
        assert recurrence(lib, B=1, N=60000, ws_bytes=need - 1) == INVALID
        assert recurrence(lib, B=1, N=60000, ws=WS + 4) == INVALID
        assert recurrence(lib, B=1, N=60000, ws=A[0]) == INVALID


@pytest.mark.parametrize("kw", BAD_SIZES + [
    dict(x=None), dict(dx=A[5]), dict(dx=A[0]), dict(dg=A[3]), dict(ds=A[6], ds_in=A[6] + 8), dict(ds_in=A[4]),
    dict(s_in=A[6], ds_in=A[6]), dict(s_in=A[6] + 1),
])
def test_recurrence_backward_refuses(lib, kw):
    assert backward(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(B=0), dict(H=0), dict(d=-3), dict(dtype=5), dict(form=3), dict(x=None), dict(states=None),
                                dict(n=3), dict(n=0, slots=A[5]), dict(slots=A[5] + 1), dict(h=A[3]), dict(h=A[0]), dict(states=A[0])])
def test_step_refuses(lib, kw):
    assert step(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", BAD_SIZES + [
    dict(o=None), dict(y=None), dict(y=A[0]), dict(y=A[1]), dict(norm=_norm(eps=-1.0)), dict(norm=_norm(eps=float("nan"))),
    dict(norm=_norm(weight=A[3] + 2)), dict(norm=_norm(bias=A[2]))])
def test_gated_norm_refuses(lib, kw):
    assert gnorm(lib, **kw) == INVALID


def test_norm_limits(lib):
    assert gnorm(lib, d=1025) == UNSUPPORTED and gnorm(lib, H=257) == UNSUPPORTED
    assert rnorm(lib, D=16385) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(gate=None), dict(dg=None), dict(do=A[0]), dict(dg=A[3]), dict(dw=A[0]), dict(dw=A[6]),
                                dict(ws=None), dict(ws_bytes=64), dict(ws=A[1]), dict(ws=WS + 2)])
def test_gated_norm_backward_refuses(lib, kw):
    assert gnorm_back(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(N=-1), dict(D=0), dict(dtype=2), dict(dtype=0, stream=1), dict(stream=3), dict(alpha=float("inf")), dict(x=None), dict(res=None), dict(r=None), dict(r=A[2]),
    dict(y=A[1]), dict(scale=A[2]), dict(scale=A[4] + 1)])
def test_residual_norm_refuses(lib, kw):
    assert rnorm(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(x=None), dict(r=None), dict(res=A[9], r=None, x=None, dscale=None), dict(res=A[5]), dict(dres=A[4]), dict(dx=A[2]), dict(dscale=A[0]), dict(ws=None), dict(ws_bytes=8),
                                dict(alpha=float("nan")), dict(db=A[7])])
def test_residual_norm_backward_refuses(lib, kw):
    assert rnorm_back(lib, **kw) == INVALID


@shim_only
def test_valid_calls_reach_the_launchers(lib):
    calls = [
        (recurrence, {}), (recurrence, dict(cu=A[5], B=1, S=7, max_len=50)), (recurrence, dict(s_in=A[4], s_out=A[4])),
        (recurrence, dict(strides=(0, 6400, 64), h_strides=(19200, 6400, 64))),
        (recurrence, dict(N=60000, B=1)), (recurrence, dict(B=1, H=1, N=1, d=1, strides=(0, 0, 0))),
        (backward, {}), (backward, dict(form=1, x=None)), (backward, dict(ds=A[6], ds_in=A[6], s_in=A[7])),
        (step, {}), (step, dict(slots=A[5], n=2)), (gnorm, {}), (gnorm, dict(gate=None)), (gnorm_back, {}),
        (gnorm_back, dict(dw=None, db=None, ws=None)), (gnorm_back, dict(gate=None, dg=None)), (rnorm, {}),
        (rnorm, dict(stream=0)), (rnorm_back, {}), (rnorm_back, dict(dr=None, x=None, dx=None, dscale=None)), (rnorm_back, dict(r=None, res=A[9])),
        (rnorm_back, dict(dscale=None, dw=None, db=None, ws=None)),
    ]
    for fn, kw in calls:
        before = lib.retention_shim_launches()
        assert fn(lib, **kw) == 0, (fn.__name__, kw)
        assert lib.retention_shim_launches() == before + 1


@shim_only
def test_columns_of_one_tensor_may_lie_side_by_side(lib):
    """x, gate and h as thirds of one [B, N, 3 D] tensor; a shift by one element makes them overlap."""
    B, N, D = 2, 10, 64
    st = (N * 3 * D, 0, 3 * D)

    def call(shift):
        v = [_v(A[0] + 2 * (D * i + (shift if i == 2 else 0)), *st) for i in range(3)]
        return lib.retention_gated_recurrence(*v, B, 1, N, D, 0, 1, None, None, None, B, N, WS, 1 << 40, None)

    assert call(0) == 0
    assert call(-1) == INVALID and call(1) == INVALID


def _asan_runtime():
    out = subprocess.run(["g++", "-print-file-name=libasan.so"], capture_output=True, text=True)
    path = out.stdout.strip()
    return path if out.returncode == 0 and os.path.isabs(path) and os.path.exists(path) else None


@pytest.mark.skipif(bool(SHIM) or shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP runtime headers")
def test_checks_pass_under_the_sanitizers(tmp_path):
    asan = _asan_runtime()
    if asan is None:
        pytest.skip("no ASan runtime for g++")
    out = tmp_path / "libblock_host.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fno-omit-frame-pointer",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "block_api.cpp"),
                    os.path.join(ROOT, "tests", "host_shim", "block_stubs.cpp"), "-o", str(out)], check=True)
    env = dict(os.environ, RETENTION_BLOCK_TEST_LIB=str(out), LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=600)
    report = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, report
    assert "ERROR: AddressSanitizer" not in report and "runtime error" not in report, report


# ---------------------------------------------------------------------------
# The binding


@pytest.fixture
def no_library(monkeypatch):
    def refuse():
        raise AssertionError("the C library was reached before the arguments were checked")

    monkeypatch.setattr(_lib, "load", refuse)


def test_host_tensors_and_non_tensors_are_refused(no_library):
    x = torch.zeros(2, 8, 16)
    o = torch.zeros(1, 2, 8, 16)
    norm = ret.Norm()
    for call in (lambda: ret.gated_recurrence(x, x), lambda: ret.gated_recurrence_backward(x, x, x, x),
                 lambda: ret.gated_recurrence_step(x[:, 0], x[:, 0], x[:, 0]), lambda: ret.gated_norm(o),
                 lambda: ret.gated_norm_backward(o, o), lambda: ret.residual_norm(x, x, norm),
                 lambda: ret.residual_norm_backward(x, x, norm)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="must be a tensor"):
        ret.gated_recurrence([1.0], x)


@pytest.mark.parametrize("bad, match", [
    (torch.zeros(2, 8, 16, device="meta"), "must be on cpu"), (torch.zeros(2, 8, 16, dtype=torch.bfloat16), "must be torch.float32"),
    (torch.zeros(2, 8, 17), "must have shape"), (torch.zeros(2, 16, 8).transpose(1, 2), "contiguous last dimension"), (3.0, "must be a tensor"),
])
def test_same_checks_device_dtype_shape_and_layout(bad, match):
    with pytest.raises(ValueError, match=match):
        block._same(bad, "gate", torch.zeros(2, 8, 16))
    with pytest.raises(ValueError, match=match):
        block._Like(torch.zeros(2, 8, 16)).view(bad, "gate")


def _rows_view(t):
    return block._rows_like(t).view(t, "x")


def test_strided_views_are_taken_as_they_are():
    wide = torch.zeros(2, 8, 40)
    v = block._view(wide[..., 3:19])  # [B, N, D]: one head, whose stride is not read
    assert (v.data, v.stride_b, v.stride_n) == (wide.data_ptr() + 12, 320, 40)
    t = torch.zeros(2, 8, 3, 16).transpose(1, 2)  # [B, H, N, d] of a token-major tensor
    v = block._view(t)
    assert (v.stride_b, v.stride_h, v.stride_n) == (8 * 48, 16, 48)
    v = block._view(t[:, :, 0])  # [B, H, d]: one token
    assert (v.stride_b, v.stride_h) == (8 * 48, 16)
    v = block._view(wide[:, 0])  # [B, D]
    assert v.stride_b == 320
    v = _rows_view(torch.zeros(2, 3, 4, 16))
    assert v.stride_n == 16 and block._row_dims((2, 3, 4, 16)) == (1, 24, 16)
    v = _rows_view(wide[0])  # [R, D]
    assert v.stride_n == 40 and block._row_dims(wide[0].shape) == (1, 8, 40)
    assert block._row_dims((16,)) == (1, 1, 16)


def test_unsupported_dtypes_are_type_errors():
    class Device(torch.Tensor):  # a host tensor that says it is on the device: the dtype is looked at before any use
        is_cuda = True

    with pytest.raises(TypeError, match="unsupported dtype"):
        block._activations(torch.zeros(2, 8, 16, dtype=torch.float16).as_subclass(Device), "x", (3, 4))
    assert block._activations(torch.zeros(2, 8, 16).as_subclass(Device), "x", (3, 4)) == _lib.RET_F32
    with pytest.raises(ValueError, match="contiguous last dimension"):
        block._activations(torch.zeros(2, 16, 8).transpose(1, 2).as_subclass(Device), "x", (3, 4))
    with pytest.raises(ValueError, match="3 or 4 dimensions"):
        block._activations(torch.zeros(8, 16).as_subclass(Device), "x", (3, 4))


def test_sequence_arguments(no_library):
    x = torch.zeros(1, 8, 16)
    cu = torch.tensor([0, 3, 8], dtype=torch.int32)
    assert block._sequences(x, cu, None) == ((1, 1, 8, 16), (2, 16), 2, 8)
    assert block._sequences(torch.zeros(1, 4, 8, 16), cu, 5) == ((1, 4, 8, 16), (2, 4, 16), 2, 5)
    assert block._sequences(torch.zeros(3, 8, 16), None, None) == ((3, 1, 8, 16), (3, 16), 3, 8)
    for args, match in (((x, cu.long(), None), "torch.int32"), ((x, cu[:1], None), "two offsets"), ((x, [0, 8], None), "two offsets"),
                        ((x, None, 8), "needs cu_seqlens"), ((x, cu, 0), "positive"), ((x.expand(2, 8, 16), cu, None), "one row"),
                        ((x, cu.to("meta"), None), "must be on")):
        with pytest.raises(ValueError, match=match):
            block._sequences(*args)
    with pytest.raises(ValueError, match="form must be"):
        block._form("tanh")


def test_norm_arguments():
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="Norm or a GroupNorm"):
        block._norm_struct((1e-5,), 8, cpu)
    with pytest.raises(ValueError, match="weight must have shape"):
        block._norm_struct(ret.Norm(1e-5, torch.ones(9)), 8, cpu)
    with pytest.raises(ValueError, match="bias must be torch.float32"):
        block._norm_struct(ret.GroupNorm(1e-5, None, torch.ones(8, dtype=torch.bfloat16)), 8, cpu)
    s = block._norm_struct(ret.Norm(0.5, rms=True), 8, cpu)
    assert (s.eps, s.rms, s.weight, s.bias) == (0.5, 1, None, None)
    assert block._norm_struct(ret.GroupNorm(), 8, cpu).rms == 0


def test_the_epilogue_refuses_the_rms_form():
    with pytest.raises(ValueError, match="root-mean-square"):
        ret._gn_struct(ret.Norm(rms=True), 2, 8, torch.device("cpu"))


def test_rows_of_many_dimensions_are_told_by_their_length():
    """Contiguous is said whatever the stride of a dimension of one element: the rows of such a tensor are D apart."""
    t = torch.zeros(2, 3, 1, 4, 16).transpose(2, 3)  # [2, 3, 4, 1, 16], 64 the stride of the 1
    assert t.is_contiguous() and t.stride(-2) == 64
    assert _rows_view(t).stride_n == 16 and block._row_dims(t.shape) == (1, 24, 16)
    with pytest.raises(ValueError, match="contiguous when"):
        _rows_view(torch.zeros(2, 3, 4, 32)[..., :16])


def test_sizes_beyond_an_int_are_refused(no_library):
    """A broadcast tensor has as many elements as it likes; its sizes reach the C library as ints."""
    long = torch.zeros(1, 1, 8).expand(1, (1 << 32) + 3, 8)
    for call in (lambda: block._sequences(long, None, None), lambda: block._row_dims(long.shape),
                 lambda: block._head_dims(long.unsqueeze(1).shape), lambda: block._step_dims((1, 8), 1 << 32),
                 lambda: block._step_dims(long[0].shape, 5), lambda: block._row_dims((1 << 20, 1 << 10, 1 << 10, 8))):
        with pytest.raises(ValueError, match="too large"):
            call()
    x, cu = torch.zeros(1, 8, 16), torch.tensor([0, 3, 8], dtype=torch.int32)
    assert block._sequences(x, cu, (1 << 32) + 5)[3] == 8  # no sequence is longer than the row


def test_launches_beyond_the_grid_are_refused(lib):
    """A launch holds at most 2^32 threads: 2^26 units of one wave each are too many, one XCD's round less is not."""
    for B, want in ((1 << 26, UNSUPPORTED), ((1 << 26) - 8, 0)):
        if want or SHIM:
            assert recurrence(lib, B=B, H=1, N=1, h=A[11] + (1 << 40), strides=(0, 0, 0), h_strides=(64, 0, 0)) == want


def test_residual_norm_backward_workspace_is_what_its_launch_fills(lib):
    """Three sums of D values for each of 1024 workgroups, 512 for rows beyond 2048 values, 256 beyond 4096."""
    f = lib.retention_residual_norm_backward_workspace_bytes
    assert f(1, 1 << 20, 2048, 1, 1) == 1024 * 3 * 2048 * 4
    assert f(1, 1 << 20, 4096, 1, 1) == 512 * 3 * 4096 * 4
    assert f(1, 1 << 16, 16384, 0, 1) == 256 * 3 * 16384 * 4
    assert f(1, 100, 4096, 1, 1) == 100 * 3 * 4096 * 4 and f(1, 100, 4096, 1, 0) == 0


def test_h_may_be_float32_alone(lib):
    """With the flag h's elements are four bytes, the others two: told by what h's bytes meet and by its alignment."""
    wide = 1 | _lib.H_F32
    n = 2 * 3 * 100 * 64  # values of h
    assert recurrence(lib, dtype=wide, h=A[2] + 2) == INVALID
    assert recurrence(lib, dtype=wide, h=A[1] - 4 * n + 4) == INVALID
    assert recurrence(lib, dtype=_lib.H_F32 | 2) == INVALID and recurrence(lib, dtype=1 | 2 * _lib.H_F32) == INVALID
    assert backward(lib, dtype=wide, dx=A[3] + 4 * n - 2) == INVALID
    assert step(lib, dtype=wide) == INVALID and gnorm(lib, dtype=wide) == INVALID
    f = lib.retention_gated_recurrence_workspace_bytes
    assert f(1, 3, 60000, 60000, 0, 64, wide) == f(1, 3, 60000, 60000, 0, 64, 1) > 0
    if SHIM:
        assert recurrence(lib, dtype=wide) == recurrence(lib, dtype=wide, h=A[1] - 4 * n) == 0
        assert recurrence(lib, dtype=1, h=A[1] - 2 * n) == 0
        assert backward(lib, dtype=wide) == backward(lib, dtype=wide, dx=A[3] + 4 * n) == 0


def test_the_dtype_of_h():
    bf16, f32 = torch.bfloat16, torch.float32
    assert block._h_dtype(None, "out", bf16) is bf16 and block._h_dtype(f32, "out", bf16) is f32
    assert block._h_dtype(torch.zeros(1), "h", bf16) is f32 and block._h_dtype(torch.zeros(1), "h", f32) is f32
    for bad, dtype in ((torch.zeros(1, dtype=bf16), f32), (torch.float64, f32), (torch.float16, bf16)):
        with pytest.raises(ValueError, match="out must be"):
            block._h_dtype(bad, "out", dtype)


@shim_only
def test_heads_of_one_tensor_may_lie_side_by_side(lib):
    """x, gate and h as thirds of one [B, N, 3, H, d] tensor, 3 elements to a row more or none; a shift by one element, or
    heads of all three in turn ([B, N, H, 3, d], where h's d lie between the others'), told by their places."""
    B, H, N, d = 2, 5, 10, 24
    for more in (0, 3):
        pitch = 3 * H * d + more

        def call(shift=0, head_stride=d, third=H * d):
            st = (N * pitch, head_stride, pitch)
            v = [_v(A[0] + 2 * (third * i + (shift if i == 2 else 0)), *st) for i in range(3)]
            return lib.retention_gated_recurrence(*v, B, H, N, d, 0, 1, None, None, None, B, N, WS, 1 << 40, None)

        assert call() == 0
        assert call(shift=-1) == INVALID and call(third=H * d - 8) == INVALID
        assert call(shift=1) == (INVALID if more == 0 else 0)  # into the row's spare elements
        # One head's thirds beside one another: columns of d at a distance of 3 d, if that divides the rows' distance.
        assert call(head_stride=3 * d, third=d) == (0 if more == 0 else INVALID)


def test_the_residual_stream_may_be_updated_in_place(lib):
    """r is the residual itself or lies apart from it; shifted, or with other strides, it is refused, as is y in its place."""
    st = (10 * 64, 0, 64)

    def call(r, strides=st, y=A[2]):
        return lib.retention_residual_norm(_v(A[0], *st), _v(A[1], *st), _v(y, *st), _v(r, *strides), 2, 10, 64, 1, 1, _norm(), None,
                                           1.0, None)

    assert call(A[1] + 2) == call(A[1] + 128) == call(A[1], (64, 0, 128)) == call(A[1], y=A[1]) == call(A[0]) == INVALID
    if SHIM:
        assert call(A[1]) == call(A[3]) == 0


@pytest.mark.parametrize("bad", ["float32", 3, [torch.zeros(1)], torch.int32])
def test_what_is_no_dtype_of_h_is_refused(bad):
    with pytest.raises(ValueError, match="out must be"):
        block._h_dtype(bad, "out", torch.bfloat16)
