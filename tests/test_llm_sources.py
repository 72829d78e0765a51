"""What the kernels' sources may not contain. The library also serves the loops with one rank per device, whose
operands can lie in another GPU's memory, and TMA loads with cluster multicast are fit for a GPU's own memory only."""

import glob
import os
import re

BULK_COPY = "cp.async.bulk"

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "collective_fusedallreduce_gb300", "csrc")


def statements():
    """Every asm statement of the sources, its string literals joined."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.h"))):
        with open(path) as f:
            for m in re.finditer(r"asm(?: volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", f.read()):
                yield os.path.basename(path), "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))


def test_statements_are_found():
    text = [s for _, s in statements()]
    assert any(f"{BULK_COPY}.tensor.3d.shared::cluster" in s for s in text)
    assert any("tcgen05.commit" in s for s in text)


def test_no_bulk_copy_is_multicast():
    for name, s in statements():
        if BULK_COPY in s:
            assert "multicast" not in s, (name, s)


def kernels():
    """(file, name, text) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            parts = f.read().split("__global__")[1:]
        for part in parts:
            body = part[:part.index("\n}\n")]
            yield os.path.basename(path), re.search(r"k_\w+", body).group(0), body


def test_no_cta_leaves_before_its_stages_are_handed_back():
    """A commit arrives on a barrier some time after it was issued: the producer waits for the last ones, or they may
    reach shared memory that the CTA has given up (of its own, or of the other CTA of a pair)."""
    seen = 0
    for name, kernel, body in kernels():
        if "umma_commit" not in body:
            continue
        seen += 1
        assert "await_hand_back(empty_bar(0)" in body or re.search(r"wait\(a?empty(_bar)?\(s\), .*, never\)", body), kernel
    assert seen >= 5


def test_releases_to_another_cta_have_its_scope():
    for name, s in statements():
        assert not ("mbarrier.arrive.release.cta" in s and "shared::cluster" in s), (name, s)
