"""What the serving operators promise that shows without a GPU: in their sources, their host code and their arguments."""

import re

from conftest import ROOT

PACKAGE = ROOT / "dsa_sparse_attention_fp8_gb300"


def test_the_norm_reads_by_ordinary_loads():
    """The kernel may write its sum over x or the residual: no read of it by way of the read-only path."""
    text = (PACKAGE / "csrc" / "norm.cuh").read_text()
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", text)
