"""The training calls' host code under AddressSanitizer and
UndefinedBehaviorSanitizer: a C program built with both drives every entry
point of the sanitized library with valid and invalid arguments, workspace
sizes up to the largest batch and long tensor lists.  No GPU is needed: every
call returns from its host-side checks, does nothing (no tokens, no elements),
or finds no device."""
import os
import subprocess

import pytest

from test_sanitized_abi import CLANG, LIBDIR, ROOT

C_SOURCE = r"""
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "beam_moe.h"

static int fails = 0;
#define EXPECT(cond) do { if (!(cond)) { printf("FAIL line %d: %s\n", __LINE__, #cond); ++fails; } } while (0)

int main(void) {
  void* p = (void*)(uintptr_t)0x100000;   /* never dereferenced */
  void* odd = (void*)(uintptr_t)0x100002;
  moe_config_t c;
  moe_adamw_t o;
  moe_adamw_tensor_t* t;
  size_t n;
  int i;
  int64_t ts[] = {0, 1, 128, 129, 4096, 1000000, (((int64_t)1 << 31) - 1) / 8};
  memset(&c, 0, sizeof c);
  c.hidden = 5120; c.intermediate = 128; c.num_experts = 256; c.num_groups = 1;
  c.topk_groups = 1; c.topk = 8; c.renormalize = 1; c.routed_scaling = 1.0f;
  for (i = 0; i < (int)(sizeof ts / sizeof ts[0]); ++i) {
    c.num_tokens = ts[i];
    EXPECT(moe_workspace_bytes(&c, MOE_ENTRY_ROUTE_BACKWARD, &n) == MOE_OK);
    EXPECT((n > 0) == (ts[i] > 128));
    /* enough tokens to need a launch: the missing workspace is found first */
    if (n) EXPECT(moe_route_backward(&c, p, p, p, p, p, p, p, NULL, 0, p, p, NULL, 0, NULL) ==
                  (ts[i] > 100000000 ? MOE_ERR_UNSUPPORTED : MOE_ERR_WORKSPACE));
  }
  c.num_tokens = INT64_MAX;
  EXPECT(moe_dispatch(&c, 0, p, p, NULL, p, NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_combine_rows(&c, 1, p, p, p, p, NULL) == MOE_ERR_UNSUPPORTED);
  c.num_tokens = INT64_MIN;
  EXPECT(moe_dispatch(&c, 0, p, p, NULL, p, NULL) == MOE_ERR_INVALID_ARG);
  c.num_tokens = 0;
  EXPECT(moe_dispatch(&c, 0, p, p, NULL, p, NULL) == MOE_OK);
  EXPECT(moe_dispatch(NULL, 0, p, p, NULL, p, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_dispatch(&c, 0, odd, p, NULL, p, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_dispatch_backward(&c, 1, p, p, p, p, p, p, NULL) == MOE_OK);
  EXPECT(moe_dispatch_backward(&c, 1, p, p, NULL, p, p, p, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_combine_backward(&c, 0, p, p, p, p, p, p, NULL) == MOE_OK);
  EXPECT(moe_combine_backward(&c, 0, p, NULL, p, p, p, p, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_route_logits(&c, p, p, NULL, 1, p, p, p, p, (size_t)1 << 40, NULL) == MOE_OK);
  EXPECT(moe_route_backward(&c, p, p, p, p, p, p, p, p, 0, p, NULL, p, 0, NULL) == MOE_ERR_INVALID_ARG);

  memset(&o, 0, sizeof o);
  o.lr = 1e-3; o.beta1 = 0.9; o.beta2 = 0.999; o.eps = 1e-8; o.grad_scale = 1.0; o.step = 1;
  t = calloc(100, sizeof *t);  /* exactly as many as are passed */
  for (i = 0; i < 100; ++i) {
    t[i].param = t[i].m = t[i].v = p; t[i].grad = p;
    t[i].param_dtype = t[i].grad_dtype = MOE_DTYPE_FP32; t[i].state_bits = 32;
  }
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_OK);  /* no elements */
  t[99].state_bits = 8;
  t[99].n = 5;
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_ERR_INVALID_ARG);  /* no scales */
  t[99].m_scale = t[99].v_scale = odd;
  t[99].n = (int64_t)1 << 34;
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_ERR_UNSUPPORTED);
  t[99].n = INT64_MAX;
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_ERR_UNSUPPORTED);
  t[99].n = -1;
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_ERR_INVALID_ARG);
  t[99].n = 0;
  o.step = INT64_MAX;
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_OK);
  o.step = 0;
  EXPECT(moe_adamw_step(&o, t, 100, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_adamw_step(NULL, t, 100, NULL) == MOE_ERR_INVALID_ARG);
  free(t);
  printf("%s\n", fails ? "failed" : "sanitized training calls passed");
  return fails != 0;
}
"""


def test_training_calls_under_asan_and_ubsan(tmp_path):
    from grouped_top_routing_amd import build as b
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang not available")
    src, exe = tmp_path / "train.c", tmp_path / "train"
    src.write_text(C_SOURCE)
    r = subprocess.run([CLANG, "-std=c99", "-g", "-Wall", "-fsanitize=address,undefined",
                        "-fno-omit-frame-pointer", "-shared-libasan", str(src),
                        "-I", os.path.join(ROOT, "include"), "-L", LIBDIR, "-lbeam_moe_sanitized",
                        "-Wl,-rpath," + LIBDIR, "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env["LD_LIBRARY_PATH"] = b.clang_rt_dir() + ":" + env.get("LD_LIBRARY_PATH", "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr
