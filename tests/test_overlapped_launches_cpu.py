"""Kernels that are launched while the stream's previous kernel still runs, by their
source: what a test on a GPU would show only by chance."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dsa_sparse_attention_quant_gb300",
                    "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["attn_rows.cu", "attn_prompt.cu", "pages.cu"])
def test_nothing_is_read_as_read_only(name):
    # every load of these kernels stands behind the wait for a kernel that may have
    # written what it reads, and that was running when this one began
    text = source(name)
    assert "launch_pdl(" in text and "pdl_wait();" in text
    for word in ("__ldg", "__restrict__", "ld.global.nc"):
        assert word not in text, word
