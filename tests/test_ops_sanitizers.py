"""The host paths of the ragged products, the int8 products and the block norms under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): moe_ops_api.hip built with host-side
sanitizers, linked with the library's other objects and a driver that calls every size query over
valid and overflowing shapes and every entry point with arguments that must be refused before any
HIP call. Any sanitizer report aborts the program, which fails the test."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routing_expert_grouped_amd", "csrc")
BUILD = os.path.join(ROOT, "routing_expert_grouped_amd", "_build")
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
           UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")

DRIVER = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <vector>
#include "moe.h"
static int bad = 0;
static void refused(int line, int st, int want) {
  if (st != want) { std::printf("line %d returned %d, want %d\n", line, st, want); ++bad; }
}
int main() {
  const int M = 2147483647, E = MOE_EINVAL, U = MOE_EUNSUPPORTED;
  const std::vector<moe_gemm_shape> shapes = {
      {64, 100, 60, 4}, {0, 1, 1, 1}, {65536, 6144, 4096, 256}, {-1, 1, 1, 1}, {1, 0, 1, 1},
      {M, M, M, M}, {1 << 30, 1 << 20, 1 << 20, 1024}, {1 << 30, 64, 64, 1},
      {-M, -M, -M, -M}, {1, 131071, 16, 1}, {1, 1 << 20, 1 << 20, 1}};
  unsigned long long acc = 0;
  for (const moe_gemm_shape& s : shapes) {
    acc += moe_int8_weight_bytes(&s) + moe_grouped_gemm_wgrad_workspace_bytes(&s);
    acc += moe_int8_pitch(s.K) + moe_norm_backward_workspace_bytes(s.R, s.K);
  }
  for (int32_t T : {-M, -1, 0, 1, 4096, 1 << 30, M})
    for (int32_t h : {-M, 0, 1, 16384, 16385, M}) acc += moe_norm_backward_workspace_bytes(T, h);
  acc += moe_int8_pitch(-M) + moe_int8_pitch(M);
  refused(__LINE__, moe_int8_weight_bytes(nullptr) != 0, 0);
  refused(__LINE__, moe_grouped_gemm_wgrad_workspace_bytes(nullptr) != 0, 0);
  const moe_gemm_shape s = shapes[0], huge = shapes[5], one = {64, 100, 60, 1};
  int8_t* q = reinterpret_cast<int8_t*>(uintptr_t(0x1000));
  void* p = q;
  float* f = reinterpret_cast<float*>(p);
  int32_t* i = reinterpret_cast<int32_t*>(p);
  void* mis = reinterpret_cast<void*>(uintptr_t(0x1004));
  const int B = MOE_ELT_BF16;
  for (auto fn : {moe_grouped_gemm, moe_grouped_gemm_dgrad}) {
    refused(__LINE__, fn(&s, B, nullptr, 200, nullptr, 1, 64, p, i, p, 200, B, nullptr), E);
    refused(__LINE__, fn(&s, B, p, -M, nullptr, 1, 64, p, i, p, 200, B, nullptr), E);
    refused(__LINE__, fn(&s, B, p, 200, nullptr, 1, 64, mis, i, p, 200, B, nullptr), E);
    refused(__LINE__, fn(&s, 77, p, 200, nullptr, 1, 64, p, i, p, 200, B, nullptr), E);
    refused(__LINE__, fn(&huge, B, p, 200, nullptr, 1, 64, p, i, p, 200, B, nullptr), U);
    refused(__LINE__, fn(nullptr, B, p, 200, nullptr, 1, 64, p, i, p, 200, B, nullptr), E);
  }
  refused(__LINE__, moe_grouped_gemm_wgrad(&s, B, p, 100, i, 0, 64, p, 60, i, p, MOE_ELT_F32, p,
                                           nullptr), E);
  refused(__LINE__, moe_grouped_gemm_wgrad(&shapes[6], B, p, 1 << 20, nullptr, 1, 1 << 30, p,
                                           1 << 20, i, p, MOE_ELT_F32, p, nullptr), U);
  refused(__LINE__, moe_quantize_int8(4, M, B, p, M, 0, q, f, nullptr), U);
  refused(__LINE__, moe_quantize_int8(4, 16384, B, p, 16384, 1, q, f, nullptr), E);
  refused(__LINE__, moe_int8_pack_weights(&huge, q, p, nullptr), U);
  refused(__LINE__, moe_int8_prepare_weights(&s, nullptr, p, f, nullptr), E);
  refused(__LINE__, moe_gemm_int8(&s, q, f, p, f, nullptr, p, 60, B, nullptr), E);
  refused(__LINE__, moe_gemm_int8(&one, q, f, p, f, nullptr, p, 59, B, nullptr), E);
  refused(__LINE__, moe_grouped_gemm_int8(&s, q, f, i, 1, -5, i, p, f, nullptr, p, 60, B,
                                          nullptr), E);
  refused(__LINE__, moe_pre_norm(4, 100, B, p, p, NAN, p, nullptr, nullptr, nullptr, nullptr), E);
  refused(__LINE__, moe_pre_norm(M, M, B, p, p, 1e-6f, p, nullptr, nullptr, nullptr, nullptr), U);
  refused(__LINE__, moe_post_norm(4, 100, B, p, nullptr, p, p, f, 1.0f, 1e-6f, p, f, nullptr,
                                  nullptr, nullptr, nullptr, nullptr, nullptr), E);
  refused(__LINE__, moe_pre_norm_backward(4, 100, B, p, p, f, p, mis, p, f, p, nullptr), E);
  refused(__LINE__, moe_post_norm_backward(4, 100, B, nullptr, p, f, p, p, f, 1.0f, nullptr,
                                           nullptr, nullptr, nullptr, p, p, f, f, f, nullptr, p,
                                           nullptr), E);
  std::printf("%s %llu\n", bad ? "FAILED" : "OK", acc);
  return bad != 0;
}
"""


def _run(cmd, **kw):
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=600, **kw)
    assert res.returncode == 0, (" ".join(cmd[:3]), res.stdout[-2000:], res.stderr[-3000:])
    return res


def test_ops_host_paths_under_asan_ubsan():
    hipcc = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    others = sorted(os.path.join(BUILD, f) for f in os.listdir(BUILD)
                    if f.endswith(".o") and f != "moe_ops_api.o") if os.path.isdir(BUILD) else []
    if not others:
        pytest.fail("no library objects: build with `python -m routing_expert_grouped_amd.build`")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    with tempfile.TemporaryDirectory() as d:
        api, drv_src = os.path.join(d, "moe_ops_api.o"), os.path.join(d, "drv.cpp")
        drv, exe = os.path.join(d, "drv.o"), os.path.join(d, "drv")
        with open(drv_src, "w") as f:
            f.write(DRIVER)
        _run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *san,
              "-c", os.path.join(CSRC, "moe_ops_api.hip"), "-o", api])
        _run([hipcc, "--cuda-host-only", "-O1", "-g", "-std=c++17", *san,
              "-I", os.path.join(ROOT, "include"), "-c", drv_src, "-o", drv])
        _run([hipcc, "--offload-arch=gfx950", *san[:4], api, drv, *others, "-o", exe])
        out = _run([exe], env=ENV)
    assert out.stdout.startswith("OK"), out.stdout
    assert "runtime error" not in out.stderr
