"""The shared memory a kernel is allowed (allow_smem of csrc/qmv_kv.h), asked for
by two threads at once: compiled on the CPU against a stand-in for the runtime
call, which lets the threads meet in the order that matters; and first calls of several
threads on a GPU."""
import os
import subprocess
import sys

import pytest

from affine_group_quantized_b200 import build

CUDA = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "include")

SOURCE = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "qmv_kv.h"

static std::atomic<int> limit{0}, calls{0};       // of the kernel, as the runtime holds it
static std::atomic<bool> small_inside{false}, large_done{false};
constexpr int kSmall = 60000, kLarge = 90000;

// The smaller request is held inside the call until the larger one has been
// served, or for half a second where it cannot be meanwhile.
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute what, int value) {
  if (what != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  ++calls;
  if (value == kSmall) {
    small_inside = true;
    for (int i = 0; i < 500 && !large_done; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  }
  limit = value;
  return cudaSuccess;
}
inline cudaError_t cudaFuncSetAttribute(void (*f)(int), cudaFuncAttribute what, int value) {
  return cudaFuncSetAttribute(reinterpret_cast<const void *>(f), what, value);
}
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }

static void kernel(int) {}

int main() {
  static qmvc::Granted granted;
  qmvc::Device dev;
  dev.id = 1;
  std::thread a([&] { qmvc::allow_smem(kernel, granted, dev, kSmall); });
  while (!small_inside) std::this_thread::yield();
  std::thread b([&] {
    qmvc::allow_smem(kernel, granted, dev, kLarge);
    large_done = true;
  });
  a.join();
  b.join();
  if (limit < kLarge) return printf("the limit was lowered to %d\n", limit.load()), 1;
  // what has been allowed is not asked for again, less neither
  const int before = calls;
  qmvc::allow_smem(kernel, granted, dev, kLarge);
  qmvc::allow_smem(kernel, granted, dev, kSmall / 2);
  if (calls != before || limit < kLarge) return printf("%d calls, limit %d\n", calls - before, limit.load()), 1;
  // more is, and another device asks for itself
  qmvc::allow_smem(kernel, granted, dev, kLarge + 1);
  dev.id = 0;
  qmvc::allow_smem(kernel, granted, dev, kLarge + 1);
  if (calls != before + 2) return printf("%d calls, 2 are due\n", calls - before), 1;
  puts("ok");
}
"""


def test_a_smaller_request_never_lowers_the_limit(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.INCLUDE, "-I", build.CSRC,
                    "-I", CUDA, "-o", str(exe), str(src)], check=True)
    for _ in range(3):
        r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


CALLS = r"""
import threading, torch
import affine_group_quantized_b200 as agq

H, D, page, gs = 1, 64, 16, 32
go = threading.Barrier(4)
failed = []


def calls(batches):
    try:
        torch.cuda.set_device(0)
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            sets = []
            for batch in batches:
                pages = batch
                bufs = [torch.zeros((pages, H, page, w), dtype=t, device="cuda") for w, t in
                        ((D // 8, torch.int32),) * 2 + ((D // gs, torch.bfloat16),) * 4]
                cache = agq.KVCache(*bufs, pages, H, page, D, 4, gs)
                table = torch.arange(batch, dtype=torch.int32, device="cuda").view(batch, 1)
                lens = torch.full((batch,), 5, dtype=torch.int32, device="cuda")
                q = torch.zeros((batch, H, D), dtype=torch.bfloat16, device="cuda")
                out = torch.ones_like(q)
                ws = torch.empty(agq.kv_attention_workspace(cache, batch, H, 1), dtype=torch.uint8,
                                 device="cuda")
                sets.append((cache, q, table, lens, out, batch, H, 1, 0.1, ws))
            stream.synchronize()
            go.wait()
            for s in sets:
                agq.kv_attention(*s)
            stream.synchronize()
            assert all((s[4] == 0).all() for s in sets)
    except Exception as e:
        failed.append(e)
        go.abort()


threads = [threading.Thread(target=calls, args=([64 * i, 4096 - 900 * i, 33 + i, 4000],)) for i in range(1, 5)]
for t in threads: t.start()
for t in threads: t.join()
assert not failed, failed
print("ok")
"""


@pytest.mark.gpu
def test_first_calls_of_four_threads():
    # a process of its own, so that the calls are its first ones
    root = os.path.dirname(os.path.dirname(build.LIB))
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
