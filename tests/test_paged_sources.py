"""Rules of the paged kernels' sources that no call on a healthy GPU shows broken."""
import os
import re

import pytest

from top_cache_gb300 import build

FILES = sorted(f for f in os.listdir(build.CSRC) if f.startswith("kvo_paged"))


def _kernels():
    for f in FILES:
        with open(os.path.join(build.CSRC, f)) as src:
            for text in re.split(r"(?=__global__ void )", src.read())[1:]:
                yield f, re.search(r"(\w+_kernel)\(", text).group(1), text


DEPENDENT = [(f, name, text) for f, name, text in _kernels() if "grid_wait();" in text]


def test_dependent_kernels_are_found():
    assert {name for _, name, _ in DEPENDENT} >= {"attend_paged_kernel", "attend_paged_f8_kernel", "join_paged_kernel"}


@pytest.mark.parametrize("file,name,text", DEPENDENT, ids=[name for _, name, _ in DEPENDENT])
def test_nothing_is_reported_while_the_launch_before_may_still_write(file, name, text):
    # the kernel before it in the stream writes the status and the list's head too, and may come last
    early = text[:text.index("grid_wait();")]
    assert not re.search(r"\*a\.status\s*=|a\.head\[\w+\]\s*=(?!=)", early), "%s: %s" % (file, name)


def test_a_join_that_may_meet_more_parts_than_it_holds_does_not_compile():
    with open(os.path.join(build.CSRC, "kvo_paged_attend.cu")) as f:
        assert re.search(r"static_assert\(kMaxWorkers <= kJoinParts,", f.read())
