"""A wait that gives up after a second has to begin behind the wait for earlier work on the stream: in kernels that start before that work has
finished (programmatic dependents), its time would count.  Shown on the source, as no call here has a predecessor of that length."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_q1_q8_gb300", "csrc")
LIMITED = re.compile(r"\b(?:wait_or_abort(?:_sleep)?|mbar_wait)\(")


def roles(text, kernel):
    """The kernel's body, cut where its comments name a role of the block's warps."""
    body = text[text.index(f"{kernel}("):]
    body = body[:body.index("\n}\n")]
    return re.split(r"// -{10,} ", body)[1:]


@pytest.mark.parametrize("file,kernel", [("linear_tiles.cu", "linear_tiles_kernel")])
def test_limits_begin_behind_the_dependency(file, kernel):
    found = [r for r in roles(open(os.path.join(CSRC, file)).read(), kernel) if LIMITED.search(r)]
    names = [r.split("\n")[0].split(":")[0] for r in found]
    assert names == ["sums", "MMAs", "copies of the activations", "weights", "teardown"], names
    for r in found[:-1]:                                                   # what the teardown waits for was issued behind the other roles' waits
        at = r.find("griddepcontrol.wait")
        assert 0 <= at < LIMITED.search(r).start(), r.split("\n")[0]
