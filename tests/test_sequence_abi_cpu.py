"""CPU checks of the sequence entry points: struct layouts and host-side answers."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <stddef.h>
#include <stdio.h>
#include "ofrl.h"
#define P(T, F) printf(#T "." #F " %zu\n", offsetof(T, F));
int main(void) {
  printf("ofrl_delta_shape %zu\nofrl_delta_tokens %zu\nofrl_delta_grads %zu\n", sizeof(ofrl_delta_shape),
         sizeof(ofrl_delta_tokens), sizeof(ofrl_delta_grads));
  P(ofrl_delta_shape, dtype) P(ofrl_delta_tokens, beta) P(ofrl_delta_tokens, q_stride) P(ofrl_delta_tokens, tokens)
  P(ofrl_delta_tokens, scale) P(ofrl_delta_grads, dbeta) P(ofrl_delta_grads, beta_stride)
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib():
    from offline_rl_step_gb300 import _abi, build
    build.build()
    return _abi.load()


def test_struct_layouts(tmp_path):
    from offline_rl_step_gb300 import _abi
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(PROBE)
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    mirrors = {"ofrl_delta_shape": _abi.DeltaShape, "ofrl_delta_tokens": _abi.DeltaTokens,
               "ofrl_delta_grads": _abi.DeltaGrads}
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        key, val = line.split()
        cname, _, field = key.partition(".")
        assert (getattr(mirrors[cname], field).offset if field else C.sizeof(mirrors[cname])) == int(val), key


def test_sizes(lib):
    from offline_rl_step_gb300 import _abi
    ok = C.byref(_abi.DeltaShape(2, 4, 64, 64, 1))
    small, large = lib.ofrl_delta_saved_bytes(ok, 64, 1), lib.ofrl_delta_saved_bytes(ok, 6400, 100)
    assert 0 < small < large
    # 64-bit sizes: a long buffer of large heads is past 4 GB
    assert lib.ofrl_delta_saved_bytes(C.byref(_abi.DeltaShape(4, 16, 128, 128, 1)), 2 ** 24, 1) > 2 ** 35
    for shape in ((2, 3, 64, 64, 1), (1, 1, 12, 64, 1), (1, 1, 64, 136, 1), (1, 1, 64, 64, 2), (0, 0, 64, 64, 1)):
        assert lib.ofrl_delta_saved_bytes(C.byref(_abi.DeltaShape(*shape)), 64, 1) == -1
    assert lib.ofrl_delta_saved_bytes(ok, -1, 1) == -1
    assert lib.ofrl_delta_saved_bytes(ok, 2 ** 31, 1) == -1


def test_refusals_before_any_cuda_call(lib):
    from offline_rl_step_gb300 import _abi
    out = C.c_void_p(1)
    for shape, code in (((2, 3, 64, 64, 1), _abi.EINVAL), ((1, 1, 64, 64, 2), _abi.EINVAL),
                        ((1, 1, 130, 64, 1), _abi.EUNSUPPORTED), ((1, 1, 64, 20, 1), _abi.EUNSUPPORTED)):
        assert lib.ofrl_delta_create(C.byref(_abi.DeltaShape(*shape)), 64, 1, 1, C.byref(out)) == code
        assert out.value is None
    ok = C.byref(_abi.DeltaShape(1, 1, 64, 64, 1))
    assert lib.ofrl_delta_create(ok, -1, 1, 1, C.byref(out)) == _abi.EINVAL
    assert lib.ofrl_delta_create(ok, 64, 1, 2, C.byref(out)) == _abi.EINVAL
    assert lib.ofrl_delta_create(ok, 64, 1, 1, None) == _abi.EINVAL
    assert lib.ofrl_delta_forward(None, None, None, 0, None, None, None, None, None) == _abi.EINVAL
    assert lib.ofrl_delta_backward(None, None, None, 0, None, None, None, None, None, None) == _abi.EINVAL
    assert lib.ofrl_delta_step(None, None, None, 0, None, None, None, None) == _abi.EINVAL
    assert lib.ofrl_delta_destroy(None) == _abi.OK
    ptr, size, dt = (C.c_void_p * 1)(256), (C.c_int64 * 1)(4), (C.c_int32 * 1)(0)
    assert lib.ofrl_tensors_create(ptr, size, dt, 0, C.byref(out)) == _abi.EINVAL
    assert lib.ofrl_tensors_create(None, size, dt, 1, C.byref(out)) == _abi.EINVAL
    for p, n, d in ((0, 4, 0), (258, 4, 0), (257, 4, 1), (256, -1, 0), (256, 4, 2)):
        ptr[0], size[0], dt[0] = p, n, d
        assert lib.ofrl_tensors_create(ptr, size, dt, 1, C.byref(out)) == _abi.EINVAL
    assert lib.ofrl_global_norm(None, None, None) == _abi.EINVAL
    assert lib.ofrl_global_norm_clip(None, 1.0, None, None, None) == _abi.EINVAL
    assert lib.ofrl_tensors_destroy(None) == _abi.OK
