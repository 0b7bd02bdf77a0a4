"""What the serving operators promise that shows without a GPU: in their sources, their host code and their arguments."""

import re
import subprocess
from pathlib import Path

from conftest import ROOT

PACKAGE = ROOT / "dsa_sparse_attention_fp8_gb300"


def test_the_norm_reads_by_ordinary_loads():
    """The kernel may write its sum over x or the residual: no read of it by way of the read-only path."""
    text = (PACKAGE / "csrc" / "norm.cuh").read_text()
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", text)


def test_a_prompt_of_a_million_tokens_is_within_the_share():
    """The cost that the attention kernel gives a prompt of 2^20 tokens, 128 heads over 8 key heads, on 152 SMs, and
    that of four such prompts, are within a CTA's share; a share, and a unit before or after it, are within 32 bits."""
    text = (PACKAGE / "csrc" / "paged_attention.cuh").read_text()
    most = 1 << int(re.search(r"kAttnMaxShare = 1 << (\d+)", text).group(1))
    tokens, group, kv_heads, sms = 1 << 20, 16, 8, 152
    unit = 2 * (128 // group)                       # tokens of two query tiles
    cost = sum(2 * (1 + -(-end // 128)) for end in range(unit, tokens + 1, unit)) * kv_heads
    assert 4 * cost // sms <= most
    longest = 2 * (1 + (1 << 31) // 128)            # a unit over all the positions there are
    assert most + 2 * longest < 1 << 31


def test_attributes_are_set_for_each_device(tmp_path):
    """Host code under a runtime of its own: once a device, again where it failed."""
    source = tmp_path / "per_device.cpp"
    source.write_text(r'''
#include "host.h"
static int current = 0;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = current; return current < 0 ? cudaErrorInvalidDevice : cudaSuccess; }
static dsa_host::PerDevice done;
int main() {
  int calls = 0;
  auto call = [&](int dev, cudaError_t answer) { current = dev; return done.once([&] { ++calls; return answer; }); };
  if (call(0, cudaSuccess) != cudaSuccess || call(0, cudaSuccess) != cudaSuccess || calls != 1) return 1;
  if (call(1, cudaErrorInvalidValue) != cudaErrorInvalidValue || calls != 2) return 2;
  if (call(1, cudaSuccess) != cudaSuccess || call(1, cudaSuccess) != cudaSuccess || calls != 3) return 3;
  if (call(0, cudaSuccess) != cudaSuccess || calls != 3) return 4;
  if (call(200, cudaSuccess) != cudaSuccess || call(200, cudaSuccess) != cudaSuccess || calls != 5) return 5;
  if (call(-1, cudaSuccess) == cudaSuccess || calls != 5) return 6;
  return 0;
}
''')
    from dsa_sparse_attention_fp8_gb300 import _build
    toolkit = Path(_build._nvcc()).resolve().parents[1] / "include"
    program = tmp_path / "per_device"
    subprocess.run(["g++", "-std=c++17", "-I", str(PACKAGE / "csrc"), "-I", str(toolkit), str(source), "-o", str(program)],
                   check=True)
    assert subprocess.run([str(program)]).returncode == 0
    for name in ("serving.cu", "dsa_indexer.cu"):
        text = (PACKAGE / "csrc" / name).read_text()
        assert not re.search(r"call_once\(once, \[\] \{\s*attr_err", text)
