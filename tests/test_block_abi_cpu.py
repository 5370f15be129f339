"""CPU checks of the state space blocks' entry points: struct layouts, sizes, refusals before any CUDA call."""
import ctypes as C
import os
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

TYPES = ("conv_shape", "conv_tokens", "conv_grads", "scan_shape", "scan_tokens", "scan_grads", "norm_shape", "gated_rows",
         "residual_rows")


@pytest.fixture(scope="module")
def lib():
    from offline_rl_step_gb300 import _abi, build
    build.build()
    return _abi.load()


def _mirror(name):
    from offline_rl_step_gb300 import _abi
    return getattr(_abi, "".join(x.capitalize() for x in name.split("_")))


def test_struct_layouts(tmp_path):
    from offline_rl_step_gb300 import _abi
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = []
    for n in TYPES:
        lines.append(f'printf("{n} %zu\\n", sizeof(ofrl_{n}));')
        lines += [f'printf("{n}.{f} %zu\\n", offsetof(ofrl_{n}, {f}));' for f, _ in _mirror(n)._fields_]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ofrl.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    seen = 0
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        key, val = line.split()
        n, _, field = key.partition(".")
        assert (getattr(_mirror(n), field).offset if field else C.sizeof(_mirror(n))) == int(val), key
        seen += 1
    assert seen > 60
    # the packed forms the binding passes
    for fmt, n in ((_abi.CONV_TOKENS_FMT, "conv_tokens"), (_abi.CONV_GRADS_FMT, "conv_grads"),
                   (_abi.SCAN_TOKENS_FMT, "scan_tokens"), (_abi.SCAN_GRADS_FMT, "scan_grads"),
                   (_abi.GATED_ROWS_FMT, "gated_rows"), (_abi.RESIDUAL_ROWS_FMT, "residual_rows")):
        assert struct.calcsize(fmt) == C.sizeof(_mirror(n)), n


def test_sizes(lib):
    from offline_rl_step_gb300 import _abi
    ok = _abi.ScanShape(512, 16, 1, 1, 1)
    # a state for every eight tokens
    assert lib.ofrl_scan_saved_bytes(C.byref(ok), 33) == 5 * 512 * 16 * 4
    assert lib.ofrl_scan_saved_bytes(C.byref(ok), 0) == 0
    assert lib.ofrl_scan_saved_bytes(C.byref(_abi.ScanShape(4096, 64, 1, 1, 1)), 2 ** 20) == 2 ** 37      # past 32 bits
    for bad in (-1, 2 ** 31 - 2 ** 17 + 1, 2 ** 31):
        assert lib.ofrl_scan_saved_bytes(C.byref(ok), bad) == -1
        assert lib.ofrl_scan_workspace_bytes(C.byref(ok), bad, 1, 1) == -1
    reading = lib.ofrl_scan_workspace_bytes(C.byref(ok), 65536, 228, 0)
    assert 0 < reading < lib.ofrl_scan_workspace_bytes(C.byref(ok), 65536, 228, 1)
    conv = _abi.ConvShape(1024, 4, 1, 1)
    assert 0 < lib.ofrl_conv_workspace_bytes(C.byref(conv), 65536, 228, 0) < \
        lib.ofrl_conv_workspace_bytes(C.byref(conv), 65536, 228, 1)
    norm = _abi.NormShape(1024, 1, 1, 0)
    assert 0 < lib.ofrl_norm_workspace_bytes(C.byref(norm), 0) < lib.ofrl_norm_workspace_bytes(C.byref(norm), 1)
    assert lib.ofrl_norm_workspace_bytes(C.byref(norm), 2) == -1


def test_workspace_covers_smaller_calls(lib):
    """The workspace of a call of fewer tokens is never larger."""
    from offline_rl_step_gb300 import _abi
    for shape in ((8, 4, 1), (512, 16, 1), (1024, 64, 2), (72, 12, 3), (65536, 8, 1)):
        s, last = C.byref(_abi.ScanShape(shape[0], shape[1], shape[2], 1, 1)), 0
        for t in (0, 1, 15, 16, 63, 64, 65, 1000, 4096, 50000, 10 ** 6, 10 ** 7, 2 ** 31 - 2 ** 17):
            n = lib.ofrl_scan_workspace_bytes(s, t, 1, 1)
            assert n >= last
            last = n


SCAN_BAD = (((0, 16, 1, 0, 1), "EINVAL"), ((64, 0, 1, 0, 1), "EINVAL"), ((64, 16, 3, 0, 1), "EINVAL"),
            ((64, 16, 1, 2, 1), "EINVAL"), ((64, 16, 1, 0, 2), "EINVAL"), ((64, 16, 0, 0, 1), "EINVAL"),
            ((64, 6, 1, 0, 1), "EUNSUPPORTED"), ((64, 68, 1, 0, 1), "EUNSUPPORTED"), ((60, 16, 1, 0, 1), "EUNSUPPORTED"),
            ((64, 16, 16, 0, 1), "EUNSUPPORTED"), ((65544, 16, 1, 0, 1), "EUNSUPPORTED"))
CONV_BAD = (((0, 4, 1, 0), "EINVAL"), ((64, 0, 1, 0), "EINVAL"), ((64, 4, 2, 0), "EINVAL"), ((64, 4, 1, 3), "EINVAL"),
            ((60, 4, 1, 0), "EUNSUPPORTED"), ((64, 1, 1, 0), "EUNSUPPORTED"), ((64, 5, 1, 0), "EUNSUPPORTED"),
            ((65544, 4, 1, 0), "EUNSUPPORTED"))
NORM_BAD = (((0, 1, 0, 0), "EINVAL"), ((64, 0, 0, 0), "EINVAL"), ((64, 3, 0, 0), "EINVAL"), ((64, 1, 2, 0), "EINVAL"),
            ((64, 1, 0, 1), "EINVAL"), ((64, 16, 0, 0), "EUNSUPPORTED"), ((8200, 1, 1, 1), "EUNSUPPORTED"),
            ((65544, 9, 1, 1), "EINVAL"))


def test_shapes_refused(lib):
    from offline_rl_step_gb300 import _abi
    out = C.c_void_p(1)
    for bad, code in SCAN_BAD:
        s = _abi.ScanShape(*bad)
        assert lib.ofrl_scan_create(C.byref(s), 64, 1, 1, C.byref(out)) == getattr(_abi, code), bad
        assert out.value is None
        assert lib.ofrl_scan_saved_bytes(C.byref(s), 64) == -1
        out = C.c_void_p(1)
    for bad, code in CONV_BAD:
        assert lib.ofrl_conv_create(C.byref(_abi.ConvShape(*bad)), 64, 1, 1, C.byref(out)) == getattr(_abi, code), bad
        assert out.value is None
        out = C.c_void_p(1)
    for bad, code in NORM_BAD:
        assert lib.ofrl_norm_create(C.byref(_abi.NormShape(*bad)), 1, C.byref(out)) == getattr(_abi, code), bad
        assert out.value is None
        out = C.c_void_p(1)
    scan, conv, norm = _abi.ScanShape(64, 16, 1, 0, 1), _abi.ConvShape(64, 4, 1, 0), _abi.NormShape(64, 1, 0, 0)
    for create, shape in ((lib.ofrl_scan_create, scan), (lib.ofrl_conv_create, conv)):
        assert create(C.byref(shape), -1, 1, 1, C.byref(out)) == _abi.EINVAL
        assert create(C.byref(shape), 64, -1, 1, C.byref(out)) == _abi.EINVAL
        assert create(C.byref(shape), 64, 1, 2, C.byref(out)) == _abi.EINVAL
        assert create(C.byref(shape), 64, 1, 1, None) == _abi.EINVAL
        assert create(None, 64, 1, 1, C.byref(out)) == _abi.EINVAL
    assert lib.ofrl_norm_create(C.byref(norm), 2, C.byref(out)) == _abi.EINVAL
    assert lib.ofrl_norm_create(C.byref(norm), 1, None) == _abi.EINVAL


def test_null_contexts_refused(lib):
    from offline_rl_step_gb300 import _abi
    assert lib.ofrl_conv_forward(None, None, None, 0, None, None, 0, None, None) == _abi.EINVAL
    assert lib.ofrl_conv_backward(None, None, None, 0, None, None, 0, None, None, None, None) == _abi.EINVAL
    assert lib.ofrl_conv_step(None, None, None, 0, None, None, None, 0, None) == _abi.EINVAL
    assert lib.ofrl_scan_forward(None, None, None, 0, None, None, 0, None, None, None) == _abi.EINVAL
    assert lib.ofrl_scan_backward(None, None, None, 0, None, None, None, 0, None, None, None, None) == _abi.EINVAL
    assert lib.ofrl_scan_step(None, None, None, 0, None, None, None, 0, None) == _abi.EINVAL
    assert lib.ofrl_gated_norm(None, None, None, 0, None) == _abi.EINVAL
    assert lib.ofrl_gated_norm_backward(None, None, None, 0, None, 0, None, 0, None, None) == _abi.EINVAL
    assert lib.ofrl_residual_norm(None, None, None, 0, None, 0, None) == _abi.EINVAL
    assert lib.ofrl_residual_norm_backward(None, None, None, 0, None, 0, None, 0, None, 0, None, None, None) == _abi.EINVAL
    for poll in (lib.ofrl_conv_poll_status, lib.ofrl_scan_poll_status):
        assert poll(None, None, None) == _abi.EINVAL
    for destroy in (lib.ofrl_conv_destroy, lib.ofrl_scan_destroy, lib.ofrl_norm_destroy):
        assert destroy(None) == _abi.OK


def test_binding_refuses_wrong_contexts():
    import offline_rl_step_gb300 as ofrl
    with pytest.raises(TypeError, match="CausalConv"):
        ofrl.conv_forward(None, None, None, None, None)
    with pytest.raises(TypeError, match="SelectiveScan"):
        ofrl.scan_forward(object(), None, None, None, None, None, None, None)
    with pytest.raises(TypeError, match="BlockNorm"):
        ofrl.gated_norm(None, None, None, None, None)
    with pytest.raises(KeyError):
        ofrl.CausalConv(64, activation="gelu")
    closed = ofrl.BlockNorm.__new__(ofrl.BlockNorm)
    closed.handle = None
    with pytest.raises(ValueError, match="closed"):
        ofrl.residual_norm(closed, None, None, None, None, None)


def test_last_kernels_of_a_call_do_not_let_go_early():
    """What follows a call may be a kernel that reads its results before it waits: only kernels that one of the same
    call follows let it start ahead."""
    src = os.path.join(ROOT, "offline_rl_step_gb300", "csrc")
    last = {"conv.cu": ("conv_forward_kernel", "conv_init_grad_kernel", "conv_step_kernel"),
            "block_norm.cu": ("gated_norm_kernel", "residual_norm_kernel", "norm_join_kernel"),
            "scan_fwd.cu": ("scan_forward_kernel",), "scan_bwd.cu": ("scan_grad_join_kernel",),
            "scan_step.cu": ("scan_step_kernel",)}
    for name, kernels in last.items():
        text = open(os.path.join(src, name)).read()
        bodies = text.split("__global__")[1:]
        for k in kernels:
            mine = [b for b in bodies if f" {k}(const __grid_constant__" in b.split("{")[0]]
            assert len(mine) == 1 and "pdl_wait();" in mine[0] and "pdl_trigger" not in mine[0], k
        for b in bodies:      # every kernel waits before it lets go
            assert "pdl_wait();" in b
            if "pdl_trigger" in b:
                assert b.index("pdl_wait();") < b.index("pdl_trigger")
