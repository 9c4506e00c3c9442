"""A warp of a softmax group whose wait runs out must not leave the others at a named barrier,
which has no limit of its own: it goes on and meets every barrier (CPU only: the sources)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_301_gb300", "csrc")


def code(text):
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["pa_multi.cuh", "pa_latent_prefill.cu"])
def test_no_softmax_warp_leaves_its_barriers(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert text.count("softmax and output rows --") == 1
    part = text[text.index("softmax and output rows --"):]
    part = code(part[:part.index("tmem_dealloc(")])
    assert "barrier" in part or "any_of" in part
    assert not re.search(r"\b(break|return)\s*;", part)
    for loop in re.findall(r"\b(?:for|while) \(.*", part):
        assert not re.search(r"\bok\b", loop), loop
    # nor is a barrier or a vote behind what one warp knows alone
    for line in part.splitlines():
        if re.search(r"\b(sync\(\)|named_barrier|any_of)", line):
            assert not re.search(r"\bok\b", line), line
