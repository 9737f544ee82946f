"""Host code of routing from logits and of the 4-bit expert calls under
AddressSanitizer and UndefinedBehaviorSanitizer: a C program built with both
drives every entry point of the sanitized library with valid and invalid
arguments and the largest sizes.  No GPU is needed: every call returns from its
host-side checks, does nothing (no tokens), or finds no device."""
import os
import subprocess

import pytest

from test_sanitized_abi import CLANG, LIBDIR, ROOT

C_SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "beam_moe.h"

static int fails = 0;
#define EXPECT(cond) do { if (!(cond)) { printf("FAIL line %d: %s\n", __LINE__, #cond); ++fails; } } while (0)

int main(void) {
  /* never dereferenced */
  void* p[8];
  void* odd = (void*)(uintptr_t)0x100001;
  moe_select_config_t c, d;
  moe_config_t m, b;
  size_t n, big = (size_t)1 << 45;
  int i, e;
  int64_t ts[] = {0, 1, 15, 16, 17, 2048, 2049, 1000000, ((int64_t)1 << 26) - 1};
  for (i = 0; i < 8; ++i) p[i] = (void*)((uintptr_t)(i + 1) << 50);
  memset(&c, 0, sizeof c);
  c.num_experts = 256; c.num_groups = 8; c.topk_groups = 4; c.group_best = 2; c.topk = 8;
  c.score = MOE_SCORE_SOFTMAX; c.renormalize = 1; c.logits_dtype = MOE_DTYPE_FP32;
  memset(&m, 0, sizeof m);
  m.hidden = 5120; m.intermediate = 2560; m.num_experts = 256; m.num_groups = 1;
  m.topk_groups = 1; m.topk = 8; m.renormalize = 1; m.routed_scaling = 1.0f;
  m.weight_layout = MOE_LAYOUT_FP4_PACKED;

  for (i = 0; i < (int)(sizeof ts / sizeof ts[0]); ++i) {
    for (e = 1; e <= 1024; e = e * 2 + 1) {
      c.num_tokens = ts[i]; c.num_experts = e; c.topk = 1;
      EXPECT(moe_balance_workspace_bytes(&c, &n) == MOE_OK);
      EXPECT((n > 0) == (ts[i] > 0) && n <= 128 * (8 * (size_t)e + 4) + 256);
      if (n) EXPECT(moe_balance_loss(&c, p[0], p[1], 1.0f, p[2], p[3], p[4], n - 1, NULL) == MOE_ERR_WORKSPACE);
    }
  }
  c.num_experts = 256; c.topk = 8;
  c.num_tokens = INT64_MAX;
  EXPECT(moe_select(&c, p[0], NULL, p[1], p[2], NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_select_backward(&c, p[0], p[1], p[2], NULL, NULL, p[3], NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_balance_workspace_bytes(&c, &n) == MOE_ERR_UNSUPPORTED);
  c.num_tokens = INT64_MIN;
  EXPECT(moe_select(&c, p[0], NULL, p[1], p[2], NULL) == MOE_ERR_INVALID_ARG);
  c.num_tokens = 0;
  EXPECT(moe_select(&c, p[0], NULL, p[1], p[2], NULL) == MOE_OK);
  EXPECT(moe_select(NULL, p[0], NULL, p[1], p[2], NULL) == MOE_ERR_INVALID_ARG);
  d = c; d.num_groups = 0; EXPECT(moe_select(&d, p[0], NULL, p[1], p[2], NULL) == MOE_ERR_INVALID_ARG);
  d = c; d.topk_groups = INT32_MAX; d.num_groups = INT32_MAX; EXPECT(moe_select(&d, p[0], NULL, p[1], p[2], NULL) == MOE_ERR_INVALID_ARG);
  d = c; d.num_experts = INT32_MAX; d.num_groups = INT32_MAX; d.topk_groups = INT32_MAX; d.topk = INT32_MAX;
  EXPECT(moe_select(&d, p[0], NULL, p[1], p[2], NULL) == MOE_ERR_UNSUPPORTED);
  d = c; d.num_experts = INT32_MIN; EXPECT(moe_balance_workspace_bytes(&d, &n) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_balance_loss(&c, p[0], p[1], NAN, p[2], p[3], NULL, 0, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_balance_loss(&c, p[0], p[1], 1.0f, p[2], p[3], NULL, 0, NULL) == MOE_OK);
  EXPECT(moe_select_backward(&c, p[0], p[1], NULL, p[2], p[4], p[3], NULL) == MOE_OK);
  EXPECT(moe_select_backward(&c, p[0], p[1], p[2], NULL, p[4], p[3], NULL) == MOE_ERR_INVALID_ARG);
  c.num_tokens = ((int64_t)1 << 26) - 1; c.num_experts = 1024;
  EXPECT(moe_select(&c, p[0], NULL, p[0], p[2], NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_select_backward(&c, p[0], p[1], p[2], NULL, NULL, (char*)p[0] + ((size_t)1 << 37), NULL) == MOE_ERR_INVALID_ARG);
  c.num_tokens = 0; c.num_experts = 256;
  EXPECT(moe_route_select(&m, &c, p[0], p[1], NULL, p[2], p[3], NULL, NULL, 0, NULL) == MOE_OK);
  EXPECT(moe_route_select(NULL, &c, p[0], p[1], NULL, p[2], p[3], NULL, NULL, 0, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_route_select(&m, NULL, p[0], p[1], NULL, p[2], p[3], NULL, NULL, 0, NULL) == MOE_ERR_INVALID_ARG);
  c.num_tokens = 9;
  EXPECT(moe_route_select(&m, &c, p[0], p[1], NULL, p[2], p[3], NULL, p[4], big, NULL) == MOE_ERR_INVALID_ARG);

  /* 4-bit weights */
  for (i = 0; i < (int)(sizeof ts / sizeof ts[0]); ++i) {
    m.num_tokens = ts[i];
    EXPECT(moe_workspace_bytes(&m, MOE_ENTRY_EXPERT_FFN, &n) == MOE_OK);
    if (ts[i]) {
      EXPECT(n > 0);
      EXPECT(moe_expert_ffn_fp4(&m, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], odd, n - 1, NULL) == MOE_ERR_WORKSPACE);
    }
    EXPECT(moe_workspace_bytes(&m, MOE_ENTRY_LAYER, &n) == MOE_OK);
    EXPECT(moe_workspace_bytes(&m, MOE_ENTRY_EXPERT_STAGE, &n) == MOE_OK);
  }
  m.num_tokens = 0;
  EXPECT(moe_expert_ffn_fp4(&m, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[0], big, NULL) == MOE_OK);
  EXPECT(moe_expert_gate_up_fp4(&m, p[0], p[1], p[2], p[3], odd, p[5], p[6], big, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_expert_down_fp4(&m, p[0], p[1], p[2], NULL, p[4], p[5], big, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_layer_forward_fp4(&m, p[0], p[1], NULL, p[2], p[3], p[4], p[5], p[6], NULL, NULL, p[7], big, NULL) == MOE_OK);
  b = m; b.weight_layout = MOE_LAYOUT_PACKED;
  EXPECT(moe_layer_forward_fp4(&b, p[0], p[1], NULL, p[2], p[3], p[4], p[5], p[6], NULL, NULL, p[7], big, NULL) == MOE_ERR_INVALID_ARG);
  b = m; b.hidden = 1 << 30; b.intermediate = 1 << 30;
  EXPECT(moe_expert_down_fp4(&b, p[0], p[1], p[2], p[3], p[4], p[5], big, NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_quantize_fp4(&b, p[0], NULL, p[1], p[2], NULL, NULL, NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_quantize_fp4(NULL, p[0], NULL, p[1], p[2], NULL, NULL, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_quantize_fp4(&m, p[0], NULL, p[1], NULL, NULL, NULL, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_quantize_fp4(&m, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == MOE_OK);
  EXPECT(moe_quantize_fp4(&m, p[0], NULL, (uint8_t*)p[0] + 4096, p[2], NULL, NULL, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_pack_fp4(&m, NULL, NULL, p[0], p[1], NULL, NULL, p[2], p[1], NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_pack_fp4(&m, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == MOE_OK);
  printf("%s (%d failures)\n", fails ? "checks failed" : "checks passed", fails);
  return fails != 0;
}
"""


def test_validation_under_asan_and_ubsan(tmp_path):
    from grouped_top_routing_amd import build as b
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang not available")
    if not os.path.exists(b.LIB_SANITIZED):
        pytest.fail(f"{b.LIB_SANITIZED} is missing: build it with "
                    "`python -m grouped_top_routing_amd.build`")
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text(C_SOURCE)
    r = subprocess.run([CLANG, "-std=c99", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                        "-fno-omit-frame-pointer", "-shared-libasan", str(src), "-lm",
                        "-I", os.path.join(ROOT, "include"), "-L", LIBDIR, "-lbeam_moe_sanitized",
                        "-Wl,-rpath," + LIBDIR, "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env["LD_LIBRARY_PATH"] = b.clang_rt_dir() + ":" + env.get("LD_LIBRARY_PATH", "")
    # leak checking stays off: the HIP runtime keeps allocations for the life
    # of the process; every memory error and undefined behaviour aborts
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "checks passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr
