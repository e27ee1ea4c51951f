"""No C++ exception leaves the library when the host's memory runs out: a program whose operator new fails at its
n-th call, for every n that a call reaches, gets a status back each time (an exception would end it)."""
import shutil
import subprocess

import pytest

from muon_newton_schulz_amd import build

PROGRAM = r"""
#include "muon_ns.h"
#include <dlfcn.h>
#include <cstdio>
#include <cstdlib>
#include <new>
#include <vector>

static long left = -1;      // calls of operator new until one fails; -1: none does
void* operator new(size_t n) {
  if (left >= 0 && left-- == 0) throw std::bad_alloc();
  void* p = std::malloc(n ? n : 1);
  if (!p) std::abort();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

template <typename F>
static void exhaust(const char* name, F call, int at_last) {
  for (long n = 0; n < 1000; ++n) {
    left = n;
    const int st = (int)call();
    const bool failed = left == -1;
    left = -1;
    if (failed ? st != MNS_ERR_PARAM : st != at_last) {
      std::printf("%s: allocation %ld, status %d\n", name, n, st);
      std::exit(3);
    }
    if (!failed) {
      std::printf("%s: %ld allocations\n", name, n);
      return;
    }
  }
  std::exit(4);
}

int main(int, char** argv) {
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (!lib) { std::printf("%s\n", dlerror()); return 2; }
  auto clip = (decltype(&clip_grad_norm))dlsym(lib, "clip_grad_norm");
  auto norm = (decltype(&grad_norm))dlsym(lib, "grad_norm");
  auto step = (decltype(&muon_step))dlsym(lib, "muon_step");
  auto size = (decltype(&mns_step_workspace_size))dlsym(lib, "mns_step_workspace_size");
  std::vector<mns_tensor> t;
  std::vector<mns_matrix> m;
  for (int i = 0; i < 40; ++i) {
    char* p = (char*)(uintptr_t)(0x100000 + 0x10000 * i);
    t.push_back(mns_tensor{p, p, 8, MNS_F32});
    m.push_back(mns_matrix{p, (float*)(p + 0x1000), p + 0x2000, nullptr, 8 + i % 7, 16});
  }
  const float abc[3] = {3.4445f, -4.775f, 2.0315f};
  mns_hparams hp = {};
  hp.mu = 0.9f; hp.lr = 0.1f; hp.T = 1; hp.abc = abc; hp.row_fraction = 1.0; hp.dtype = MNS_BF16;
  float* out = (float*)(uintptr_t)0x10000;
  size_t bytes;
  exhaust("grad_norm", [&] { return norm(t.data(), 40, out, nullptr, 0, nullptr); }, MNS_ERR_WORKSPACE);
  exhaust("clip_grad_norm", [&] { return clip(t.data(), 40, 1.f, 0.f, out, nullptr, 0, nullptr); },
          MNS_ERR_WORKSPACE);
  exhaust("mns_step_workspace_size", [&] { return size(m.data(), 40, &hp, &bytes); }, MNS_OK);
  exhaust("muon_step", [&] { return step(m.data(), 40, &hp, nullptr, 0, nullptr); }, MNS_ERR_WORKSPACE);
  std::puts("done");
  return 0;
}
"""


def test_statuses_when_memory_runs_out(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "exhaust.cpp", tmp_path / "exhaust"
    src.write_text(PROGRAM)
    # (the library takes operator new from the program: -rdynamic)
    subprocess.run([cxx, "-std=c++17", "-O1", "-rdynamic", "-I", build.INCLUDE, str(src), "-o", str(exe), "-ldl"],
                   check=True)
    run = subprocess.run([str(exe), build.LIB_PATH], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and run.stdout.endswith("done\n"), (run.returncode, run.stdout, run.stderr)
    assert "clip_grad_norm: 0" not in run.stdout and "muon_step: 0" not in run.stdout      # it did interpose
