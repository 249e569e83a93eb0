"""CPU test that a kv_* call without host memory for anything returns a status: an
exception that left a C entry point would end the process."""
import os
import subprocess
import sys

import affine_group_quantized_b200 as agq
from affine_group_quantized_b200 import build

# operator new of every library of the process; refuses while `refuse` is set
NEW = r"""
#include <cstdlib>
#include <new>
extern "C" { int refuse = 0, refused = 0; }
void *operator new(std::size_t n) {
  if (refuse) { ++refused; throw std::bad_alloc(); }
  if (void *p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
"""

CALLS = r"""
import ctypes, sys
new, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
lib.qmv_kv_last_error.restype = ctypes.c_char_p
refuse = ctypes.c_int.in_dll(new, "refuse")
null, zero = ctypes.c_void_p(), ctypes.c_int(0)
calls = [(lib.kv_append, 17), (lib.kv_read, 13), (lib.kv_attention, 16), (lib.kv_evict, 17)]
for f, n in calls:
    refuse.value = 1
    rc = f(*[null] * n)          # no cache at all
    refuse.value = 0
    print(f.__name__, rc, lib.qmv_kv_last_error().decode(), flush=True)
"""


def test_a_refusal_needs_no_memory(tmp_path):
    src, so = tmp_path / "new.cc", tmp_path / "libnew.so"
    src.write_text(NEW)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    build.build()
    r = subprocess.run([sys.executable, "-c", CALLS, str(so), agq.LIB_PATH], capture_output=True,
                       text=True, timeout=300, env=dict(os.environ, LD_PRELOAD=str(so)))
    assert r.returncode == 0, r.stderr[-500:]
    lines = r.stdout.splitlines()
    assert len(lines) == 4
    for line, name in zip(lines, ("kv_append", "kv_read", "kv_attention", "kv_evict")):
        assert line == f"{name} {agq.QMV_ERR_NULL} {name}: the cache or its k or v is NULL"
