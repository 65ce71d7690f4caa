"""A kernel that may be launched while the kernel before it on the stream still runs
(programmatic dependent launches) waits for that one (griddepcontrol.wait) before it touches
global memory. Read from the sources, whichever files there are; kernels launched with <<< >>>
alone carry no such attribute."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rank_bottleneck_online_gb300", "csrc")


def source(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def sources():
    return [p for p in sorted(glob.glob(os.path.join(CSRC, "*")))
            if p.endswith((".cu", ".cuh", ".h", ".inc"))]


def matching(text, at, opening, closing):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == opening) - (text[i] == closing)
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced")


def kernels():
    """(file, name, parameter's name, body) of every __global__ definition."""
    out = []
    for path in sources():
        text = source(path)
        for m in re.finditer(r"__global__\s+void\s*", text):
            at = m.end()
            if text.startswith("__launch_bounds__", at):
                at = matching(text, text.index("(", at), "(", ")")
            name = re.match(r"\s*(\w+)\s*\(", text[at:])
            assert name, (path, text[at:at + 80])
            params = at + name.end() - 1
            end = matching(text, params, "(", ")")
            rest = text[end:].lstrip()
            if rest.startswith(";"):
                continue                               # a declaration
            body = text.index("{", end)
            out.append((os.path.basename(path), name.group(1), text[params + 1:end - 1],
                        text[body + 1:matching(text, body, "{", "}") - 1]))
    return out


def test_every_kernel_is_found():
    found = kernels()
    assert len(found) == sum(source(p).count("__global__") for p in sources())
    assert {"rope_kernel", "dropout_kernel", "quant_rows_kernel", "quant_tile_kernel",
            "fp8_gemm_kernel", "gemm_kernel", "add_kernel"} <= {k[1] for k in found}


@pytest.mark.parametrize("file,name,params,body", kernels(), ids=lambda v: v if re.fullmatch(r"[\w.]+", v) else "")
def test_waits_before_it_touches_global_memory(file, name, params, body):
    text = "".join(source(p) for p in sources())
    uses = re.findall(rf"\b{name}\b\s*(?:<[\w, ]*>)?\s*(<<<)?", text)
    if uses.count("<<<") and uses.count("<<<") == len(uses) - 1:
        return                                         # its definition and plain launches
    first = body.strip().split(";")[0].strip()
    if first == "pdl_enter()":
        return
    # a kernel with a prologue: nothing of its parameters but tensor maps' addresses (their
    # prefetch) and sizes before the wait, and the next kernel is let go after it
    wait = body.index("griddep_wait();")
    assert body.index("griddep_launch_dependents();") > wait
    pointers = set(re.findall(r"\bp\.(\w+)", body[:wait])) & pointer_fields()
    assert not pointers, f"{name} in {file} uses {pointers} before it waits"
    for access in ("tma_load", "tma_store", "ld_global", "st_global", "atomic", "__ldg", "store_chunk"):
        assert access not in body[:wait], f"{name} in {file}: {access} before it waits"


def pointer_fields():
    """Names of the pointer members of the kernels' parameter structs."""
    out = set()
    for path in sources():
        text = source(path)
        for m in re.finditer(r"struct\s+\w*Params\s*\{", text):
            body = text[m.end():matching(text, m.end() - 1, "{", "}") - 1]
            for line in body.split(";"):
                out |= set(re.findall(r"\*\s*(\w+)", line))
    return out


def test_pointer_fields_are_found():
    assert {"row_scale", "out", "err", "x", "res", "q", "sft"} <= pointer_fields()
