"""CPU tests of the scratch that attention and token scores ask for on devices of other sizes:
the host side is built on its own, on a device of a given CU count whose launches
do nothing."""
import os
import shutil
import subprocess

import pytest

from weight_only_int4_unpack_amd import attn, build, scoring
from weight_only_int4_unpack_amd import w4a16 as W

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

MAIN = r"""
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <hip/hip_runtime.h>
#include "serve_internal.h"
static int g_cus;
extern "C" const char* hipGetErrorString(hipError_t) { return ""; }
namespace w4a16 {
w4a16_status report(w4a16_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vfprintf(stderr, fmt, ap);
  va_end(ap);
  return st;
}
w4a16_status current_device(int* cus) {
  if (g_cus == 0) return W4A16_ERR_DEVICE;
  *cus = g_cus;
  return W4A16_OK;
}
hipError_t launch_rope_table(const RopeTableParams&, hipStream_t) { return hipSuccess; }
hipError_t launch_rope_kv(const RopeKvParams&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_read(const KvReadParams&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_token_logprobs(const ScoreParams&, int, hipStream_t) { return hipSuccess; }
#define KERNEL(name) hipError_t name(const AttnParams&, AttnKind, hipStream_t) { return hipSuccess; }
KERNEL(attn_f16_same) KERNEL(attn_f16_e4m3) KERNEL(attn_f16_int8)
KERNEL(attn_bf16_same) KERNEL(attn_bf16_e4m3) KERNEL(attn_bf16_int8)
}  // namespace w4a16
// cus, bytes: one new token of one sequence, 32 / 8 heads of 128, in e4m3; then 64 x 151667 scores, top 20
int main(int argc, char** argv) {
  g_cus = atoi(argv[1]);
  const int64_t bytes[2] = {atoll(argv[2]), atoll(argv[3])};
  alignas(16) static char one[64];
  void* p = one;
  w4a16_tree_attention_t a{};
  a.cache = {p, p, (float*)p, (float*)p, 4, 64, 8, 128, W4A16_KV_E4M3};
  a.q = p; a.out = p; a.lse = (float*)p;
  a.block_table = a.kv_lens = a.q_starts = (const int32_t*)p;
  a.tokens = 1; a.q_token = 4096; a.q_head = 128; a.table_stride = 64;
  a.sequences = 1; a.table_pages = 64; a.max_q = 1; a.q_heads = 32; a.dtype = W4A16_BF16; a.scale = 0.1f;
  w4a16_token_logprobs_t s{};
  s.logits = p; s.ids = (const int64_t*)p; s.logprobs = s.entropy = s.top_logprobs = (float*)p;
  s.top_ids = (int64_t*)p; s.tokens = 64; s.row_stride = s.vocab = 151667; s.top_k = 20; s.dtype = W4A16_BF16;
  printf("%d %d\n", (int)w4a16_tree_attention(&a, p, bytes[0], nullptr),
         (int)w4a16_token_logprobs(&s, p, bytes[1], nullptr));
  return 0;
}
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    at = tmp_path_factory.mktemp("host")
    (at / "main.cpp").write_text(MAIN)
    exe = str(at / "main")
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{build.CSRC}",
                    str(at / "main.cpp"), os.path.join(build.CSRC, "serve_host.cpp"), "-o", exe],
                   check=True, env=env)

    def run(cus, *nbytes):
        out = subprocess.run([exe, str(cus), *map(str, nbytes)], check=True, capture_output=True, text=True,
                             env=env).stdout
        return [int(x) for x in out.split()]
    return run


def sizes(cus):
    return (attn.tree_attention_workspace_bytes(1, 1, 32, 8, 128, cus), scoring.workspace_bytes(64, 151667, 20, cus))


@pytest.mark.parametrize("cus", [32, 64, 128, 256, 304])
def test_the_devices_own_size_is_enough(cus, calls):
    assert calls(cus, *sizes(cus)) == [W.OK, W.OK]


@pytest.mark.parametrize("cus", [64, 128, 256, 304])
def test_less_is_refused(cus, calls):
    a, s = sizes(cus)
    assert a > W.WORKSPACE_COUNTER_BYTES and s > W.WORKSPACE_COUNTER_BYTES
    assert calls(cus, a - 1, s - 1) == [W.ERR_WORKSPACE, W.ERR_WORKSPACE]


def test_without_a_device_the_scratch_of_a_whole_one_is_checked_first(calls):
    a, s = sizes(256)
    assert calls(0, a - 1, s - 1) == [W.ERR_WORKSPACE, W.ERR_WORKSPACE]
    assert calls(0, a, s) == [W.ERR_DEVICE, W.ERR_DEVICE]
