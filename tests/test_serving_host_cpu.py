"""What the serving operators promise that shows without a GPU: in their sources, their host code and their arguments."""

import re
import subprocess
from pathlib import Path

import pytest
import torch

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


class On(torch.Tensor):
    """A host tensor that says it lies on cuda:1."""

    def get_device(self):
        return 1

    is_cuda = True


def test_tensors_of_another_device_are_refused(monkeypatch):
    """A call launches on the current device: with tensors of another one it is refused before it reaches the library."""
    from dsa_sparse_attention_fp8_gb300 import binding as B
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "load", lambda: pytest.fail("the call went on"))

    def t(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(On)
    bf = torch.bfloat16
    rows, cache = t(2, 4, 64, dtype=bf), t(1, 64, 4, 64, dtype=bf)
    calls = [lambda: B.build_block_tables(t(1), t(1), t(1), t(1, 1), t(2), t(2), t(2, dtype=torch.int64), t(1)),
             lambda: B.kv_write(rows, rows, t(2, dtype=torch.int64), cache, cache),
             lambda: B.paged_attention(rows, cache, cache, t(2), t(1), t(1, 1), 1.0, t(8, dtype=torch.uint8)),
             lambda: B.add_rms_norm(rows[0], None, t(64, dtype=bf), 1e-6, out=rows[0]),
             lambda: B.quantize_fp8_blocks(t(2, 128, dtype=torch.float32))]
    for call in calls:
        with pytest.raises(ValueError, match="cuda:1.*cuda:0 is the current device"):
            call()


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace

    from dsa_sparse_attention_fp8_gb300 import binding as B
    assert B._stream_of(SimpleNamespace(cuda_stream=7, device_index=1), 1) == 7
    with pytest.raises(ValueError, match="stream is one of cuda:0"):
        B._stream_of(SimpleNamespace(cuda_stream=7, device_index=0), 1)


def test_strides_of_zero_are_refused(lib):
    """Rows that would be written over one another, and what a tensor map does not read."""
    import ctypes

    from test_serving_cpu import FAKE, P, attention, cache, write
    e4m3 = dict(type=3, k_scale=0x1000, v_scale=0x1000)
    for name in ("k_page_stride", "k_token_stride", "k_head_stride", "v_page_stride", "v_token_stride", "v_head_stride"):
        for kind in ({}, e4m3):
            c = cache(**kind, **{name: 0})
            assert write(lib, c) == -1 and b"stride of 0" in lib.dsa_last_error(), name
            assert attention(lib, c, ws_bytes=0) == -1 and b"stride of 0" in lib.dsa_last_error(), name
    for name in ("k_scale_page_stride", "k_scale_head_stride", "v_scale_page_stride", "v_scale_head_stride"):
        c = cache(**e4m3, **{name: 0})
        assert write(lib, c) == -1 and b"written" in lib.dsa_last_error(), name
        assert attention(lib, c, ws_bytes=0) == -3              # one scale for all heads or pages may be read
    c = cache()

    def call(q=(8192, 128), out=(8192, 128), T=4, Hq=64, c=c):
        return lib.dsa_paged_attention(FAKE, *q, 0, T, Hq, ctypes.byref(c), FAKE, FAKE, 1, FAKE, 4, 0.1, 0, 0, FAKE, *out,
                                       None, P(0x1000), 0, None, None)
    assert call() == -3                                         # (no workspace: everything before it is as it should be)
    for bad in (dict(q=(0, 128)), dict(q=(8192, 0)), dict(out=(0, 128)), dict(out=(8192, 0))):
        assert call(**bad) == -1 and b"stride of 0" in lib.dsa_last_error()
    one = cache(num_kv_heads=1, k_head_stride=0, v_head_stride=0)
    assert call(q=(0, 0), out=(0, 0), T=1, Hq=1, c=one) == -3


def test_queries_as_two_e4m3_terms_are_as_near_as_stated():
    """Over an E4M3 cache a row, times a power of two that brings its maximum to [128, 256), is a sum of two E4M3 terms:
    exactly down to 2^-9 of the maximum, and below that as near as the header and the kernel say."""
    stated = [int(re.search(r"by 2\^-(\d+) of (?:it|that)[\s*/]*at[\s*/]*most", path.read_text()).group(1))
              for path in (ROOT / "include" / "dsa_indexer.h", PACKAGE / "csrc" / "paged_attention.cuh")]
    x = torch.arange(0x3000, 0x4380).to(torch.int16).view(torch.bfloat16).float()      # BF16 numbers from 2^-31 to 256
    first = x.to(torch.float8_e4m3fn).float()
    off = (first + (x - first).to(torch.float8_e4m3fn).float() - x).abs()
    assert x.max() < 256
    worst = 0.0
    for top in (128.0, 255.0):                          # the row's maximum
        row = x <= top
        assert (off[row & (x >= top * 2.0 ** -9)] == 0).all()
        worst = max(worst, (off[row].max() / top).item())
    assert all(worst <= 2.0 ** -n for n in stated), (worst, stated)
    assert worst > 2.0 ** -18


def test_fp16_queries_over_an_e4m3_cache_are_refused_with_the_reason(lib):
    from test_serving_cpu import attention, cache, write
    c = cache(type=3, k_scale=0x1000, v_scale=0x1000)
    assert attention(lib, c, type=1) == -2 and b"significant bits" in lib.dsa_last_error()
    assert attention(lib, c, type=0, ws_bytes=0) == -3 and write(lib, c, type=1, T=0) == 0
    x = torch.arange(0x5800, 0x5C00).to(torch.int16).view(torch.float16).float()      # the FP16 numbers from 128 to 256
    first = x.to(torch.float8_e4m3fn).float()
    off = (first + (x - first).to(torch.float8_e4m3fn).float() - x).abs() / x
    assert off.max() > 2.0 ** -10                                                      # their rounding is 2^-11


def test_the_library_is_rebuilt_when_any_of_its_sources_changes():
    from dsa_sparse_attention_fp8_gb300 import _build
    included = set()
    for path in (PACKAGE / "csrc").iterdir():
        included |= set(re.findall(r'#include "([^"]+)"', path.read_text()))
    known = {path.name for path in _build._sources()}
    assert included <= known and "host.h" in known


def test_the_scoring_kernels_counters_are_of_its_present_sources():
    """Additions for other kernels go where they leave the committed counters, and the bench's traffic figure, valid."""
    import bench
    assert bench.profiled_traffic("long_context_decode") and bench.profiled_traffic("batched_decode")
    included = re.findall(r'#include "(\w+\.cuh)"', "".join((PACKAGE / "csrc" / n).read_text() for n in bench.KERNEL_SOURCES))
    assert set(included) <= set(bench.KERNEL_SOURCES)
