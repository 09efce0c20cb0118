"""The tensor-map encoder's address as threads ask for it at the same time, and after a failure (CPU only: the
runtime's lookup is replaced by a slow one)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

static std::atomic<int> asked{0};
static std::atomic<bool> works{true};
static cudaError_t slow_lookup(const char*, void** f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  ++asked;
  std::this_thread::sleep_for(std::chrono::milliseconds(100));
  *f = (void*)&asked;
  *q = cudaDriverEntryPointSuccess;
  return works ? cudaSuccess : cudaErrorUnknown;
}
#define cudaGetDriverEntryPointByVersion slow_lookup
#include "tma.cuh"

int main() {
  works = false;
  const bool none = ctr::encode_fn() == nullptr;
  works = true;
  std::atomic<int> missing{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&] { if (!ctr::encode_fn()) ++missing; });
  for (auto& t : threads) t.join();
  const int before = asked;
  const bool found = ctr::encode_fn() != nullptr;
  std::printf("%d %d %d %d\n", (int)none, (int)missing, (int)found, asked - before);
}
"""


def test_every_thread_gets_the_address(tmp_path):
    from sparse_embeddings_feature_gb300 import build as B
    src, exe = tmp_path / "ask.cu", tmp_path / "ask"
    src.write_text(PROGRAM)
    r = subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.CSRC, "-I", B.INCLUDE,
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split()
    assert out == ["1", "0", "1", "0"]     # a failure gives none; then no thread misses it; it is kept
