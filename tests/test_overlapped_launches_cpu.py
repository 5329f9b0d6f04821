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


def bodies():
    """Name and body of every kernel of the library."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        text = source(name)
        for m in re.finditer(r"__global__ void (?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(", text):
            i = text.index("{", m.end())
            end, depth = i + 1, 1
            while depth:
                depth += (text[end] == "{") - (text[end] == "}")
                end += 1
            yield m.group(1), text[i + 1:end - 1]


def test_kernels_launched_early_wait_whatever_they_have_to_do():
    # a kernel that ends without having waited lets the next one begin, and write,
    # while the one before it still reads. The score kernel's two forms wait in
    # branches that are decided when it is compiled.
    launched = set()
    for name in os.listdir(CSRC):
        launched |= set(re.findall(r"launch_pdl\((\w+)", source(name) if name.endswith(".cu") else ""))
    seen = {}
    for name, body in bodies():
        depth = 0
        for word in re.findall(r"[{}]|pdl_wait\(\);", body):
            depth += (word == "{") - (word == "}")
            if word.startswith("pdl_wait") and depth == 0:
                seen[name] = True
        seen.setdefault(name, False)
    assert {"prologue_kernel", "topk_kernel", "resolve_kernel", "kv_write_kernel", "attn_join_kernel"} <= launched
    for name in (launched & set(seen)) | {"attn_rows_kernel", "attn_prompt_kernel"}:
        assert seen[name] or name == "logits_kernel", name


def test_no_input_is_declared_read_only():
    text = "".join(source(name) for name in os.listdir(CSRC) if name.endswith(".cu"))
    launched = set(re.findall(r"launch_pdl\((\w+)", text)) | {"attn_rows_kernel", "attn_prompt_kernel"}
    found = set()
    for m in re.finditer(r"__global__ void (?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(([^)]*)\)", text):
        if m.group(1) in launched:
            found.add(m.group(1))
            assert not re.search(r"const \w+\s*\*\s*__restrict__", m.group(2)), m.group(1)
    assert {"topk_kernel", "prologue_kernel", "attn_rows_kernel", "fork_move_kernel"} <= found
