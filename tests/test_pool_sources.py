"""Launches and waits of the paged attention: what the sources have to hold, since a missing acquire,
or a copy left in flight by a wait that gave up, shows in no result."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "h2o_heavy_hitter_gb300" / "csrc"


def kernels(name):
    """{kernel: body} of a source file."""
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    found = {}
    for m in re.finditer(r"__global__", text):
        kernel = re.search(r"(\w+)\s*\((?:const|PoolView)", text[m.end():]).group(1)
        at = text.index("{", text.index(kernel, m.end()))
        depth, end = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        found[kernel] = text[at:end]
    return found


@pytest.mark.parametrize("source", ["pool_attend.cu", "pool_prefix.cu", "pool_pages.cu"])
def test_every_kernel_waits_or_acquires_before_it_reads(source):
    """The first thing that a kernel does with memory is behind a wait of its own, or behind an acquire
    of what the kernel before it released."""
    found = kernels(source)
    assert found
    for kernel, body in found.items():
        if kernel == "pool_finish_kernel":  # below
            continue
        first = min((body.index(x) for x in ("grid_dependency_wait()", "grid_acquire()") if x in body), default=-1)
        assert first >= 0, kernel
        # (shared barriers and the addresses of kernel parameters aside)
        for read in ("checked_length(", "build_list(", "produce_tma<", "finish_block<", "list_entry(", "v.meta[",
                     "v.table[", "plan[", "seqs["):
            assert read not in body or body.index(read) > first, (kernel, read)


def test_kernels_whose_followers_read_before_they_wait_release_first():
    found = kernels("pool_attend.cu") | kernels("pool_prefix.cu")
    for kernel in ("pool_prefix_kernel", "pool_rows_kernel", "pool_prefix_score_kernel", "pool_finish_kernel"):
        assert "grid_release_dependents()" in found[kernel], kernel
    for kernel in ("pool_rows_kernel", "pool_prefix_score_kernel"):
        assert "grid_acquire()" in found[kernel], kernel


def test_the_joining_kernel_reads_what_others_wrote_from_l2():
    """It may begin without a wait: every load of finish_block goes past L1."""
    text = re.sub(r"//[^\n]*", "", (CSRC / "pool_attend.cu").read_text())
    body = text[text.index("void finish_block("):text.index("pool_finish_kernel(")]
    for array in ("p.w.cum", "p.w.seq", "v.meta"):
        assert len(re.findall(re.escape(array), body)) == len(re.findall(r"load<L2>\(" + re.escape(array), body)), array
    loads = [m for m in re.findall(r"= (\S*)reinterpret_cast<const float[24]\*>", body)]
    assert loads and all(x == "load<L2>(" for x in loads)
    assert "= *" not in body
    tiles = (CSRC / "pool_tiles.cuh").read_text()
    for name, form in (("checked_length(", "__ldcg("), ("float2 record_ml(", "load<L2>("), (" load(", "__ldcg(")):
        at = tiles.index(name)
        assert form in tiles[at:tiles.index("}", at)], name
    assert "row_lse<32, L2>" in body and "record_ml(" not in body and "finish_block<D, beside>" in text


def test_roles_wait_for_their_copies_and_products_before_they_leave():
    """A wait that gives up anywhere in a CTA leaves no copy into its shared memory and no product
    into its Tensor Memory in flight: nobody returns early, and every role that issues drains."""
    tiles = (CSRC / "pool_tiles.cuh").read_text()
    for name in ("produce_tma(", "produce_codes("):
        body = tiles[tiles.index("__device__ void " + name):]
        body = body[:body.index("\n}\n")]
        assert "return" not in body and body.rstrip().endswith("drain_copies(bars.full, n, v.err);"), name
    for source, names in (("pool_attend.cu", ["pool_rows_kernel"]),
                          ("pool_prefix.cu", ["pool_prefix_kernel", "pool_prefix_score_kernel"])):
        for name in names:
            body = kernels(source)[name]
            assert body.index("tma_load_4d(") < body.index("drain_copies(bars->q_full,"), name
            assert body.rindex("umma_ss(") < body.index("drain_products(&bars->drained,") < body.index("tmem_dealloc("), name
            assert "mbar_init(&bars->drained, 1)" in body, name
