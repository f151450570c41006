"""Attributes that the launchers raise before a launch, per device and from
several threads: the header itself against a fake of the setter, and, on a GPU,
two host threads that alternate small and large shapes."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_quantized_wql_gb300", "csrc")

FAKE = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "launch_limits.h"

static std::atomic<size_t> limit[80];          // the fake devices' attribute
static std::atomic<int> calls{0};

int set_on(int device, size_t value) {
  ++calls;
  std::this_thread::sleep_for(std::chrono::microseconds(value % 7 * 20));
  limit[device] = value;
  return 0;
}

int main() {
  static wql::LargestPerDevice largest;
  // device 1 is set although device 0 has had the value
  for (int d : {0, 1, 63, 64, 70}) {
    if (largest.raise(d, 1000, [d](size_t v) { return set_on(d, v); }) != 0) return 1;
    if (limit[d] < 1000) return 2;
  }
  const int before = calls;
  for (int i = 0; i < 10; ++i) largest.raise(0, 900 + i, [](size_t v) { return set_on(0, v); });
  if (calls != before) return 3;               // no call for what is there
  // an error is passed on and not remembered
  if (largest.raise(0, 5000, [](size_t) { return 7; }) != 7) return 4;
  if (largest.raise(0, 5000, [](size_t v) { return set_on(0, v); }) != 0 || limit[0] != 5000) return 5;
  // threads with different sizes: after its own raise() a thread finds room
  std::atomic<int> short_of{0};
  for (int round = 0; round < 20; ++round) {
    wql::LargestPerDevice* fresh = new wql::LargestPerDevice;
    limit[2] = 0;
    std::vector<std::thread> threads;
    for (int t = 0; t < 4; ++t)
      threads.emplace_back([&, t] {
        for (size_t v = 100 + t * 31; v < 1000; v += 97) {
          fresh->raise(2, v, [](size_t w) { return set_on(2, w); });
          if (limit[2] < v) ++short_of;
        }
      });
    for (auto& t : threads) t.join();
    delete fresh;
  }
  if (short_of) return 6;
  wql::LastPerDevice last;
  int got = -1;
  for (int d : {0, 1, 99})
    for (int v : {0, 40, 40, 7}) {
      got = -1;
      last.want(d, v, [&](int w) { got = w; return 0; });
      if (got != v && !(v == 40 && got == -1)) return 8;
    }
  return 0;
}
"""


def test_values_are_kept_per_device_and_never_lowered(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(FAKE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)], timeout=120).returncode == 0


def test_no_launcher_keeps_a_limit_of_its_own():
    for name in os.listdir(CSRC):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                code = f.read()
            raises = code.count("cudaFuncAttributeMaxDynamicSharedMemorySize")
            assert raises == (1 if name == "wql_common.cuh" else 0), name


THREADS = r"""
import ctypes, threading
import torch
import weight_only_quantized_wql_gb300 as wql

lib = wql.load()
dev = torch.device("cuda:0")
wql._binding()
k = 1024
w = wql.wql_mx_quantize(torch.randn(700, k, device=dev))
shapes, want = (1, 300), {}
for m in shapes:
    x = wql.wql_mx_quantize(torch.randn(m, k, device=dev), wql.MX_FP8)
    l = torch.randn(4 if m == 1 else 1, 2000 if m == 1 else 30000, device=dev)
    want[m] = (x, l, torch.full((l.shape[0],), 0.5, device=dev))
torch.cuda.synchronize()
bad = []

def work(order):
    s = torch.cuda.Stream(dev)
    for m in order:
        x, l, u = want[m]
        out = torch.empty(m, 700, dtype=torch.bfloat16, device=dev)
        ids = torch.empty(l.shape[0], dtype=torch.int32, device=dev)
        sx, sw = (wql._WqlMx(a.fmt, 0, a.rows, a.k, a.codes.data_ptr(), a.scales.data_ptr())
                  for a in (x, w))
        torch.cuda.current_stream(dev).synchronize()
        st = lib.wql_mx_logits(ctypes.byref(sx), ctypes.byref(sw), None, wql.BF16, out.data_ptr(),
                               None, 0, s.cuda_stream)
        st2 = lib.wql_sample(l.data_ptr(), wql.F32, l.shape[0], l.shape[1], u.data_ptr(), None, None,
                             None, None, ids.data_ptr(), None, s.cuda_stream)
        s.synchronize()
        if st or st2 or (ids < 0).any():
            bad.append((m, st, st2))

order = [shapes[i % 2] for i in range(60)]
threads = [threading.Thread(target=work, args=(o,)) for o in (order, order[::-1])]
for t in threads: t.start()
for t in threads: t.join()
assert not bad, bad[:4]
"""


@pytest.mark.gpu
def test_two_threads_alternate_small_and_large_shapes():
    """In a process of its own: nothing has raised the limits before."""
    r = subprocess.run([sys.executable, "-c", THREADS], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
