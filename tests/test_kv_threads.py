"""CPU test that other Python threads run while a kv_* call is in the library (a
launch waits where the stream's queue is full, and what it waits for may be a
Python callback): the binding's module, built against a stand-in of the library
whose calls take a while."""
import ctypes
import importlib.machinery
import importlib.util
import os
import subprocess
import sysconfig
import threading
import time

import pytest

import affine_group_quantized_b200 as agq
from affine_group_quantized_b200 import build

STAND_IN = r"""
#include <unistd.h>
#include "qmv.h"
static int slow(void) { usleep(300000); return 7; }
int kv_append(const qmv_kv_cache *c, const void *k, const void *v, long long ks, long long vs,
              const int *t, const int *l, const int *s, int b, int n, int w, const int *seen, int *p,
              float *wt, int sw, int *st, void *stream) { return slow(); }
int kv_read(const qmv_kv_cache *c, void *k, void *v, long long ks, long long vs, const int *t,
            const int *l, const int *s, int b, int n, int w, int *st, void *stream) { return slow(); }
int kv_attention(const qmv_kv_cache *c, const void *q, long long qs, const int *t, const int *l,
                 void *o, int b, int h, int w, float sc, float *wt, int sw, void *ws, size_t n, int *st,
                 void *stream) { return slow(); }
int kv_evict(const qmv_kv_cache *c, const int *t, const int *l, const int *s, const float *w,
             const int *p, int *nl, float *nw, int *np, int b, int tw, int sw, int bu, int r, int si,
             int *st, void *stream) { return slow(); }
const char *qmv_kv_last_error(void) { return ""; }
"""
A = 0x10000


class Workspace:
    nbytes = 16
    dtype = None

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return A


@pytest.fixture(scope="module")
def module(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_native")
    (d / "q.c").write_text(STAND_IN)
    lib, ext = d / "libkvstandin.so", d / ("_kv_native" + sysconfig.get_config_var("EXT_SUFFIX"))
    run = lambda *a: subprocess.run([build.CC, "-O1", "-shared", "-fPIC", "-I", build.INCLUDE, *map(str, a)], check=True)  # noqa: E731
    run("-o", lib, d / "q.c")
    run("-I", sysconfig.get_paths()["include"], "-o", ext, os.path.join(build.CSRC, "kv_native.c"),
        "-L", d, "-l:libkvstandin.so", "-Wl,-rpath,$ORIGIN")
    loader = importlib.machinery.ExtensionFileLoader("_kv_native", str(ext))
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_kv_native", loader))
    loader.exec_module(m)
    agq._setup(m, lambda: 0, lambda d: 0)
    return m


@pytest.mark.parametrize("name", ["append", "read", "attention", "evict"])
def test_other_threads_run_meanwhile(module, name):
    c = agq._KVCacheStruct(A, A, A, A, A, A, 8, 2, 16, 128, 4, 64)
    head = (ctypes.addressof(c), None)
    args = {"append": (A, A, A, A, A, 2, 4, 4, None, None, None, 0, None, None, None, 0),
            "read": (A, A, A, A, A, 2, 4, 4, None, None, None, 0),
            "attention": (A, A, A, A, 2, 4, 4, 0.1, Workspace(), None, 0, None, None, 0),
            "evict": (A, A, A, A, A, A, A, A, 2, 4, 64, 32, 0, 0, None, 0)}[name]
    seen, stop = [], threading.Event()

    def other():
        while not stop.is_set():
            seen.append(time.monotonic())
            time.sleep(0.005)

    t = threading.Thread(target=other)
    t.start()
    try:
        time.sleep(0.05)
        begin = time.monotonic()
        assert getattr(module, name)(*head, *args) == 7
        end = time.monotonic()
    finally:
        stop.set()
        t.join()
    assert end - begin >= 0.29
    # (5 ms apart; a few are enough on a busy machine)
    assert sum(begin + 0.02 < s < end - 0.02 for s in seen) >= 5
