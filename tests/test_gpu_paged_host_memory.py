"""Host memory that runs out inside a paged call: an error code, nothing launched, nothing
changed, and the same call works afterwards.

A child process runs with a small library in front of the C++ runtime whose operator new fails
while it is armed (around one C call at a time)."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAILING_NEW = r"""
#include <cstdlib>
#include <new>
static thread_local int armed = 0, failed = 0;
extern "C" void fail_new(int on) { armed = on; if (on) failed = 0; }
extern "C" int new_failed() { return failed; }
static void* get(std::size_t n) {
    if (armed) { ++failed; return nullptr; }
    return std::malloc(n ? n : 1);
}
void* operator new(std::size_t n) { void* p = get(n); if (!p) throw std::bad_alloc(); return p; }
void* operator new[](std::size_t n) { void* p = get(n); if (!p) throw std::bad_alloc(); return p; }
void* operator new(std::size_t n, const std::nothrow_t&) noexcept { return get(n); }
void* operator new[](std::size_t n, const std::nothrow_t&) noexcept { return get(n); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t) noexcept { std::free(p); }
"""

CHILD = r"""
import ctypes, sys
import torch
from bit_kivi_kv_gb300 import kivi as K
front = ctypes.CDLL(sys.argv[1])
G, R, H, D = 32, 32, 2, 64
c = K.KiviPagedCache(3, H, H, D, 2, G, R, 8, 16)
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
kp, vp, q, k, v = rnd(H, 96, D), rnd(H, 96, D), rnd(1, H, D), rnd(1, H, D), rnd(1, H, D)
out, st = torch.zeros_like(q), torch.cuda.current_stream().cuda_stream
seq, one = ctypes.c_int(-1), (ctypes.c_int * 1)(0)
assert c.add(kp, vp) == 0 and c.counts(0) == (64, 32)                # a full residual: an append flushes
other = c.add(kp, vp)

def add():
    return K.lib.kivi_paged_add(c.handle, kp.data_ptr(), vp.data_ptr(), 96, st, ctypes.byref(seq))
def append_decode():
    return K.lib.kivi_paged_append_decode(c.handle, one, 1, k.data_ptr(), v.data_ptr(), q.data_ptr(), out.data_ptr(),
                                          0.0, c.workspace.data_ptr(), c.workspace.numel(), st)
def append():
    return K.lib.kivi_paged_append(c.handle, one, 1, k.data_ptr(), v.data_ptr(), st)

for call in (add, append_decode, append):
    if call is append:
        one[0] = other
    torch.cuda.synchronize()
    before = [c.counts(0), c.counts(other), c.pages(0), c.free(), c.buffer.clone(), K.kivi_launch_count()]
    front.fail_new(1)
    status = call()
    front.fail_new(0)
    assert front.new_failed(), call.__name__
    assert status == K.KIVI_ERR_INVALID_ARG and "host memory" in K.kivi_last_error_string(), (call.__name__, status)
    torch.cuda.synchronize()
    after = [c.counts(0), c.counts(other), c.pages(0), c.free(), c.buffer.clone(), K.kivi_launch_count()]
    assert torch.equal(before.pop(4), after.pop(4)) and before == after, (call.__name__, before, after)
    assert call() == K.KIVI_OK, call.__name__
assert c.counts(0) == (96, 1) and c.counts(other) == (96, 1)
torch.cuda.synchronize()
assert out.isfinite().all() and out.abs().max() > 0
print("fine")
"""


def test_paged_calls_survive_a_failing_allocation(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, lib = tmp_path / "failing_new.cpp", tmp_path / "failing_new.so"
    src.write_text(FAILING_NEW)
    r = subprocess.run([gxx, "-O1", "-fPIC", "-shared", str(src), "-o", str(lib)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib)], capture_output=True, text=True, timeout=200, env=env, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), (r.returncode, r.stdout[-500:], r.stderr[-2000:])
