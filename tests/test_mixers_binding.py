"""The token mixers' binding and tensors that a kernel cannot read: batches of torch.vmap and tensors
without memory.  Each has to be refused with a Python exception (no GPU needed).

The calls run in a child process, since a binding that lets a C++ exception out of the part that runs
without the interpreter lock ends the process.  A stand-in for the runtime's device queries takes the
calls past the point where a machine without a GPU would refuse them for that.
"""
import os
import shutil
import subprocess
import sys

import pytest

from tests.test_sanitized_host import ROOT

DEVICE_QUERIES = """
extern "C" {
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipSetDevice(int) { return 0; }
int hipGetDeviceCount(int* n) { *n = 1; return 0; }
int hipDeviceGetStreamPriorityRange(int* lo, int* hi) { *lo = 0; *hi = -1; return 0; }
int hipDevicePrimaryCtxGetState(int, unsigned* flags, int* active) { *flags = 0; *active = 1; return 0; }
}
"""

CHILD = """
import sys
import torch
import chunked_gated_delta_13_amd as kda

class Bare(torch.Tensor):   # a float32 (or int32) tensor on the device with no memory behind it
    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")
    @classmethod
    def __torch_dispatch__(cls, f, types, args=(), kwargs=None):
        raise RuntimeError("nothing to run on")

B, T, D, W, H, n, p, win = 2, 5, 8, 4, 2, 64, 64, 7
w, s = Bare(D, W), Bare(B, W - 1, D)
bt, b1 = Bare(B, T, 1, n), Bare(B, 1, n)
qt, q1 = Bare(B, T, H, 64), Bare(B, H, 64)
cache = Bare(B, win, H, 64)
calls = {
    "conv_prefill": ((B, T, D), lambda x: kda.conv_prefill(x, w, y=Bare(B, T, D), state_out=s)),
    "conv_step": ((B, D), lambda x: kda.conv_step(x, w, s, y=Bare(B, D))),
    "ssm_prefill": ((B, T, H, p), lambda x: kda.ssm_prefill(x, Bare(B, T, H), Bare(H), bt, bt, y=qt, S_T=Bare(B, H, n, p))),
    "ssm_step": ((B, H, p), lambda x: kda.ssm_step(x, Bare(B, H), Bare(H), b1, b1, Bare(B, H, n, p), y=q1)),
    "window_prefill": ((B, T, H, 64), lambda x: kda.window_prefill(x, qt, qt, win, o=qt)),
    "window_step": ((B, H, 64), lambda x: kda.window_step(x, q1, q1, cache, cache, Bare(B, dtype=torch.int32), win, o=q1)),
}
shape, call = calls[sys.argv[1]]
ways = {
    "vmap": lambda: torch.vmap(call)(Bare(3, *shape)),
    "vmap of vmap": lambda: torch.vmap(torch.vmap(call))(Bare(3, 2, *shape)),
    "plain": lambda: call(Bare(*shape)),
}
for name, way in ways.items():
    print(name, flush=True)
    try:
        way()
    except ValueError as e:
        assert "no memory" in str(e), e
    else:
        raise AssertionError("not refused")
print("done")
"""


@pytest.mark.parametrize("op", ["conv_prefill", "conv_step", "ssm_prefill", "ssm_step", "window_prefill", "window_step"])
def test_tensors_without_memory_are_refused(tmp_path, op):
    if not shutil.which("g++"):
        pytest.skip("no compiler for the stand-in of the device queries")
    src, lib = tmp_path / "queries.cpp", tmp_path / "queries.so"
    src.write_text(DEVICE_QUERIES)
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, op], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), (r.returncode, r.stdout, r.stderr[-2000:])


def test_the_package_is_imported_without_torch():
    """torch is needed by calls, not by the import (plans of a launcher, the C library's signatures)."""
    child = ("import sys; sys.modules['torch'] = None\n"
             "import chunked_gated_delta_13_amd as kda\n"
             "from chunked_gated_delta_13_amd import _lib\n"
             "assert 'kda_ssm_prefill' in _lib.SIGNATURES and callable(kda.conv_step)\n"
             "print('done')")
    r = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "done\n", r.stderr[-2000:]


def test_sizes_of_workspaces_default_to_bfloat16():
    import torch
    import chunked_gated_delta_13_amd as kda
    for size, args in ((kda.ssm_workspace_bytes, (1, 5000, 2, 1, 64, 64)),
                       (kda.window_step_workspace_bytes, (1, 8, 2, 128, 5000, 4))):
        assert size(*args) == size(*args, dtype=torch.bfloat16) > 0
        with pytest.raises(TypeError, match="bfloat16 or float32"):
            size(*args, dtype=torch.float16)


def test_the_c_library_is_built_without_torch(monkeypatch):
    """The binding is left out where torch is missing; libkda is compiled and linked all the same."""
    from chunked_gated_delta_13_amd import build as kbuild
    linked = []
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(kbuild, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(kbuild, "_link", lambda objs, out: linked.append(out))
    assert kbuild.build() == kbuild.LIB and linked == [kbuild.LIB, kbuild.PEAKS_LIB]


@pytest.mark.parametrize("scale,status", [(2.2e38, 0), (2.4e38, 1), (3.0e38, 1)])
def test_a_scale_whose_base_2_form_is_infinite_is_refused(scale, status):
    """fp32 holds numbers up to 3.40e38; scale log2(e) passes it from 2.36e38 on, and scores of 0 became NaN.
    Without tokens an accepted call is a no-op."""
    from chunked_gated_delta_13_amd import _lib
    lib = _lib.load()
    none = [None] * 8
    assert lib.kda_window_prefill(*none, 1, 0, 2, 1, 64, 5, 0, scale, 128, 64, 64, 0, None, 0, None) == status
    assert lib.kda_window_step(*[None] * 7, 0, 2, 1, 64, 5, 0, scale, 128, 64, 64, 0, None, 0, None) == status
