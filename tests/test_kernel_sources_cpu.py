"""Rules that every kernel's source keeps, checked by reading the source: a
kernel that breaks one may still compute the right values on most runs."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_dsq_b200", "csrc")


def matching(text, start, pair="{}"):
    """Index just past the bracket that closes the one at start."""
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise ValueError("unbalanced")


def without_blocks(text, head):
    """text without the bodies of the statements that `head` matches up to their condition's bracket."""
    while m := re.search(head, text):
        end = matching(text, m.end() - 1, "()")
        while text[end] in " \n":
            end += 1
        end = matching(text, end) if text[end] == "{" else text.index(";", end) + 1
        text = text[:m.start()] + text[end:]
    return text


def source(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def kernels():
    """(file, name, body) of every kernel."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = source(path)
        for m in re.finditer(r"__global__\s+void\s+", text):
            at = m.end()
            if text.startswith("__launch_bounds__", at):
                at = matching(text, text.index("(", at), "()")
            name = re.compile(r"\s*(\w+)\(").match(text, at)
            args_end = matching(text, name.end() - 1, "()")
            start = text.index("{", args_end)
            yield os.path.basename(path), name[1], text[start:matching(text, start)]


KERNELS = list(kernels())


def test_the_reader_finds_the_kernels():
    names = {n for _, n, _ in KERNELS}
    assert {"gemv_rows_kernel", "gemv_fused_kernel", "gemv_kernel", "gemv_tokens_kernel", "gemv_tokens_mma_kernel", "prefill_kernel",
            "x_to_f16_kernel", "act_q8_kernel", "norm_block_kernel", "sort_place_kernel", "combine_kernel"} <= names


@pytest.mark.parametrize("name,body", [(n, b) for _, n, b in KERNELS if "mbar_init" in b], ids=lambda v: v if len(v) < 40 else "")
def test_barriers_exist_before_any_lane_waits(name, body):
    """One lane initialises a shared-memory barrier.  Whatever the template's
    switches, a warp's, block's or cluster's barrier follows before a wait, an
    arrival or a copy on it, unless the initialising thread itself makes it."""
    body = without_blocks(body, r"if constexpr \(")
    body = without_blocks(body, r"auto \w+ = \[&\]\(")   # called later
    body = body[body.rindex("mbar_init"):]
    wait = re.search(r"mbar_wait_for|mbar_try_wait|wait_or_abort|convert_role|fused_epilogue", body)
    assert wait, name
    assert re.search(r"__syncwarp\(\)|__syncthreads\(\)|cluster_sync\(\)", body[:wait.start()]), name


def test_read_only_loads_only_where_no_kernel_before_may_still_write():
    """A kernel that waits for the one before (pdl_wait) runs while that one
    writes: what it reads through the read-only path may be stale, since such a
    load is defined only for data that nobody writes during the kernel's run and
    may be moved above the wait.  Kernels without the wait start after it."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = source(path)
        for m in reversed(list(re.finditer(r"__global__\s+void\s+", text))):
            start = text.index("{", matching(text, text.index("(", re.compile(r"(?:__launch_bounds__\([^)]*\))?\s*\w+").match(text, m.end()).end()), "()"))
            end = matching(text, start)
            if "pdl_wait" not in text[start:end]:
                text = text[:m.start()] + text[end:]
        left = re.findall(r"[^\n]*(?:__ldg|__restrict__|ld\.global\.nc)[^\n]*", text)
        assert not left, (os.path.basename(path), left)
