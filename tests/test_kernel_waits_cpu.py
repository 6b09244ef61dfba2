"""What the kernels' sources have to say before they reach beyond their own CTA, read here because no run shows it missing."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_weight_only_w4a16_gb300", "csrc")


def _code(path):
    """A source without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _kernels():
    """(file, kernel, its text up to the next one)"""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        for text in _code(path).split("__global__")[1:]:
            yield os.path.basename(path), re.search(r"(\w+_kernel)\s*\(", text).group(1), text


REACHES = r"\b(?:st_cluster|ld_cluster|map_rank)\("
KERNELS = [pytest.param(text, id=f"{file}-{name}") for file, name, text in _kernels() if re.search(REACHES, text)]


def test_the_kernels_are_found():
    assert len(list(_kernels())) > 20 and len(KERNELS) >= 4


@pytest.mark.parametrize("text", KERNELS)
def test_every_cta_of_a_cluster_has_begun_before_another_reaches_into_it(text):
    """Another CTA's shared memory may be read, written or signalled once that CTA runs: a barrier of the cluster comes
    before, in the order of the text."""
    barrier = re.search(r"\bcluster_(?:wait|sync_all)\(\)", text)
    assert barrier and barrier.start() < re.search(REACHES, text).start()


@pytest.mark.parametrize("file,rings", [("norm.cu", 1), ("int8.cu", 2), ("grouped.cu", 2)])
def test_a_producer_waits_for_its_copies_however_it_ends(file, rings):
    """A consumer whose wait has run out leaves copies in flight that a producer at its end no longer knows of: no copy
    may land in the shared memory of a CTA that has left, so the wait for them hangs on no verdict of the producer's."""
    code = _code(os.path.join(CSRC, file))
    ends = [m.start() for m in re.finditer(r"\bdrain_copies\(", code)]
    assert len(ends) == rings
    for at in ends:
        assert "ok" not in re.search(r"[;}][^;}]*$", code[:at]).group(0)
