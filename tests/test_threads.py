"""Several host threads on one handle (no GPU): every thread makes refused
calls, which touch the handle and nothing else, and has to find the text of its
own refusal."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>
#include "gmm_handle.hpp"
#include "gmm_moe.h"

int main() {
  gmm_handle h;  // (what gmm_create makes, without its device memory)
  std::atomic<int> wrong{0}, ready{0};
  const gmm_tensor vec{nullptr, GMM_F32, 1, {4, 0, 0, 0}}, mat{nullptr, GMM_F32, 2, {4, 4, 0, 0}};
  auto run = [&](int which) {
    ++ready;
    while (ready < 6) std::this_thread::yield();
    for (int i = 0; i < 20000; ++i) {
      const char* want = "";
      gmm_status st = GMM_OK;
      switch (which) {
        case 0: want = "lhs, rhs, group_sizes and out are required";
          st = gmm_run(&h, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, nullptr); break;
        case 1: want = "expected 2-tensors for lhs and rhs";
          st = gmm_tgmm_run(&h, &vec, &vec, &vec, nullptr, &vec, nullptr); break;
        case 2: want = "x, slot_row and out are required";
          st = gmm_dispatch_run(&h, nullptr, nullptr, nullptr, nullptr); break;
        case 3: want = "expert_ids must be int32 or int64";
          st = gmm_sort_tokens_run(&h, &mat, &vec, &mat, nullptr, 0, nullptr); break;
        case 4: want = "x must be a bf16 2-tensor";
          st = gmm_quant_fp8_run(&h, &vec, &vec, &vec, nullptr); break;
        default: want = "existing_out is required (gmm_run writes zeros instead)";
          st = gmm_run_existing_out(&h, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr,
                                    nullptr, nullptr);
      }
      if (st != GMM_E_INVALID || std::strcmp(gmm_last_error(&h), want)) ++wrong;
    }
  };
  std::vector<std::thread> threads;
  for (int i = 0; i < 6; ++i) threads.emplace_back(run, i);
  for (auto& t : threads) t.join();
  if (std::strcmp(gmm_last_error(&h), "")) ++wrong;  // this thread made no call
  std::printf("wrong %d\n", wrong.load());
  return wrong ? 1 : 0;
}
"""


def test_threads_find_their_own_errors(tmp_path):
    from moe_grouped_matrix_amd import _binding, build
    if not CXX or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("no C++ compiler or HIP headers")
    if not os.path.exists(_binding.LIB_PATH):
        build.build()
    (tmp_path / "t.cpp").write_text(PROGRAM)
    exe, pkg = tmp_path / "t", os.path.dirname(_binding.LIB_PATH)
    subprocess.run([CXX, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(pkg, "csrc"), str(tmp_path / "t.cpp"),
                    _binding.LIB_PATH, "-L" + os.path.join(ROCM, "lib"), "-lamdhip64", "-pthread",
                    "-Wl,-rpath," + pkg, "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout == "wrong 0\n", (run.returncode, run.stdout, run.stderr[-500:])
