"""A host allocation that fails inside a call is an error code, not an exception that
leaves the C ABI (which would end the process).  The allocation functions are replaced
in a child process, and fail only during the call."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

ALLOCATOR = r'''
#include <cstdlib>
#include <new>
static thread_local bool failing = false;
extern "C" void set_failing(int f) { failing = f != 0; }
void* operator new(std::size_t n) {
  void* p = failing ? nullptr : std::malloc(n ? n : 1);
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void* operator new(std::size_t n, std::align_val_t a) {
  void* p = failing ? nullptr : std::aligned_alloc((std::size_t)a, (n + (std::size_t)a - 1) & ~((std::size_t)a - 1));
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void* operator new[](std::size_t n) { return operator new(n); }
void* operator new[](std::size_t n, std::align_val_t a) { return operator new(n, a); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
void operator delete(void* p, std::align_val_t) noexcept { std::free(p); }
void operator delete(void* p, std::size_t, std::align_val_t) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t) noexcept { std::free(p); }
void operator delete[](void* p, std::align_val_t) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t, std::align_val_t) noexcept { std::free(p); }
'''

CHILD = r'''
import ctypes, sys
import torch
import roofline_driven_optimisation_gb300 as g
g.load()
set_failing = ctypes.CDLL(sys.argv[1]).set_failing
message = lambda: g.load().gemm_get_last_error().decode()


def cache(pages):
    k = torch.zeros(pages, 2, 16, 64, dtype=torch.int8, device="cuda")
    s = torch.ones(pages, 2, device="cuda")
    return g.KVCache(k, k.clone(), s, s, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))


Q = torch.randn(1, 4, 64, device="cuda").bfloat16()
O = torch.empty_like(Q)
lens = torch.ones(1, dtype=torch.int32, device="cuda")
ws = torch.zeros(g.gemm_kv_attention_workspace(1, 2, 4, 64, 1), dtype=torch.uint8, device="cuda")
A = torch.randn(64, 64, device="cuda").bfloat16()
C = torch.empty_like(A)
calls = [lambda c: g.load().gemm_kv_attention(c.address, 1, 4, Q.data_ptr(), 256, O.data_ptr(), 256, lens.data_ptr(), None, 1,
                                              0.0, ws.data_ptr(), ws.numel(), 0),
         lambda c: g.load().gemm_bf16(64, 64, 64, 1.0, A.data_ptr(), 64, A.data_ptr(), 64, 0.0, C.data_ptr(), 64, 0)]
first, other = cache(3), cache(5)
calls[0](first)                                        # everything that is set up once
torch.cuda.synchronize()
for call in calls:
    set_failing(1)
    rc = call(other)                                   # maps that are not kept yet
    set_failing(0)
    assert rc == g.GEMM_ERR_CUDA and "host memory" in message(), (rc, message())
    assert call(other) == 0, message()
torch.cuda.synchronize()
assert g.device_status()[0] == 0
print("done")
'''


def test_a_failed_allocation_is_an_error_code(cuda_lib, tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    source, lib, child = tmp_path / "failing.cpp", tmp_path / "libfailing.so", tmp_path / "child.py"
    source.write_text(ALLOCATOR)
    child.write_text(CHILD)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(source), "-o", str(lib)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, str(child), str(lib)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
