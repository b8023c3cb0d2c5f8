"""Full-attention and gated delta layers: their binding and tensors that a kernel cannot read (batches of torch.vmap,
tensors without memory), and their host code under AddressSanitizer and UndefinedBehaviorSanitizer.  No GPU needed.
"""
import os
import shutil
import subprocess
import sys

import pytest

from tests.test_mixers_binding import DEVICE_QUERIES
from tests.test_sanitized_host import ROOT, _runtime

CHILD = """
import sys
import torch
import chunked_gated_delta_13_amd as kda

class Bare(torch.Tensor):   # a tensor on the device with no memory behind it
    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")
    @classmethod
    def __torch_dispatch__(cls, f, types, args=(), kwargs=None):
        raise RuntimeError("nothing to run on")

B, T, H, d = 2, 5, 2, 64
i32 = torch.int32
kv, cu, pages, n = Bare(B * T, H, d), Bare(B + 1, dtype=i32), Bare(B, 3, dtype=i32), Bare(B, dtype=i32)
pool = lambda: Bare(6, H, 16 * 34, dtype=torch.uint8)
S = Bare(B, H, d, d)
calls = {
    "attn_prefill": ((B * T, H, d), lambda x: kda.attn_prefill(x, kv, kv, cu, o=kv)),
    "cache_write": ((B * T, H, d), lambda x: kda.cache_write(x, kv, pool(), pool(), pages, cu)),
    "cache_read": ((6, H, 16 * 34), lambda x: kda.cache_read(x, pool(), pages, cu, B * T, d, dtype=torch.float32, k=kv, v=kv)),
    "attn_step": ((B, H, d), lambda x: kda.attn_step(x, pool(), pool(), pages, n, o=Bare(B, H, d))),
    "delta_prefill": ((B, T, H, d), lambda x: kda.delta_prefill(x, Bare(B, T, H, d), Bare(B, T, H, d), Bare(B, T, H), Bare(B, T, H),
                                                                o=Bare(B, T, H, d), S_T=S)),
    "delta_step": ((B, H, d), lambda x: kda.delta_step(x, Bare(B, H, d), Bare(B, H, d), Bare(B, H), Bare(B, H), S, o=Bare(B, H, d))),
}
shape, call = calls[sys.argv[1]]
dtype = torch.uint8 if sys.argv[1] == "cache_read" else torch.float32
ways = {
    "vmap": lambda: torch.vmap(call)(Bare(3, *shape, dtype=dtype)),
    "vmap of vmap": lambda: torch.vmap(torch.vmap(call))(Bare(3, 2, *shape, dtype=dtype)),
    "plain": lambda: call(Bare(*shape, dtype=dtype)),
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


@pytest.mark.parametrize("op", ["attn_prefill", "cache_write", "cache_read", "attn_step", "delta_prefill", "delta_step"])
def test_tensors_without_memory_are_refused(tmp_path, op):
    if not shutil.which("g++"):
        pytest.skip("no compiler for the stand-in of the device queries")
    src, lib = tmp_path / "queries.cpp", tmp_path / "queries.so"
    src.write_text(DEVICE_QUERIES)
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, op], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), (r.returncode, r.stdout, r.stderr[-2000:])


def test_host_code_is_clean_under_sanitizers(tmp_path):
    from chunked_gated_delta_13_amd import build as kbuild
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not asan or not ubsan:
        pytest.skip("gcc sanitizer runtimes not installed")
    if not (os.path.isdir(kbuild.BUILD_DIR) and any(f.endswith(".hip.o") for f in os.listdir(kbuild.BUILD_DIR))):
        pytest.skip("no device objects: the regular build has not run here")
    lib = kbuild.build_sanitized(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=f"{asan} {ubsan}",
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                        f"--kda-library={lib}", "tests/test_layers_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-3000:]
    print(tail)
    assert r.returncode == 0, tail
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, tail
