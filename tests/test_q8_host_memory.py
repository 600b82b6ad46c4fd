"""A host without memory for the library's own state: the entry points return a status, and
the next call works.  (The child's operator new fails once, when it is told to.)"""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdlib>
#include <new>
static thread_local bool fail = false;
extern "C" void fail_next_new(int on) { fail = on != 0; }
extern "C" int new_has_failed() { return !fail; }
void *operator new(std::size_t n) {
    if (fail) {
        fail = false;
        throw std::bad_alloc();
    }
    if (void *p = std::malloc(n ? n : 1)) return p;
    throw std::bad_alloc();
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
"""

CHILD = r"""
import ctypes
import torch
import dense_fp32_sgemm_gb300 as sg

own = ctypes.CDLL(None)
x, w = torch.randn(40, 64, device="cuda"), torch.ones(64, device="cuda")
dx, dw = torch.empty_like(x), torch.empty_like(w)
want = sg.rms_norm_backward(x, x, w)
lib = sg.library()
x_at, w_at = x.data_ptr(), w.data_ptr()
# The first call on a stream makes its workspace's state: from C, and through the extension.
stream = torch.cuda.Stream()
torch.cuda.synchronize()


def from_c():
    return lib.sgemm_rms_norm_backward(40, 64, 0, x_at, 64, None, 64, w_at, 0, 1e-6, x_at, 64, None, 64,
                                       dx.data_ptr(), 64, dw.data_ptr(), stream.cuda_stream)


own.fail_next_new(1)
status = from_c()
assert own.new_has_failed() and status == 2, status
assert from_c() == 0
torch.cuda.synchronize()
assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
stream = torch.cuda.Stream()
with torch.cuda.stream(stream):
    own.fail_next_new(1)
    try:
        sg.rms_norm_backward(x, x, w, dx=dx, dweight=dw)
        print("no error")
    except sg.SgemmError as e:
        assert own.new_has_failed()
        print("status", e.status)
    sg.rms_norm_backward(x, x, w, dx=dx, dweight=dw)
torch.cuda.synchronize()
assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
print("done")
"""


@pytest.mark.gpu
def test_entry_points_return_a_status(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not shutil.which("g++"):
        pytest.skip("no compiler")
    sg.build()
    source, lib = tmp_path / "new.cpp", tmp_path / "new.so"
    source.write_text(SOURCE)
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", str(lib), str(source)], check=True)
    preload = " ".join(filter(None, [str(lib), os.environ.get("LD_PRELOAD")]))
    env = dict(os.environ, LD_PRELOAD=preload, PYTHONPATH=ROOT)
    child = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True,
                           timeout=300)
    assert child.returncode == 0, child.stderr[-2000:]
    assert child.stdout.split() == ["status", "2", "done"]
