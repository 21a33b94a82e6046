"""How a kernel that gives up ends. A wait that runs out sets the block's abort
flag and the other roles stop; what the block still has in flight has to land
before it ends, so the waits for that are mbar_drain's, which the flag does not
end. Giving up takes a lost signal, which no test can make without harm, so the
sources are read."""
import os
import re

import pytest

from fine_grained_fp8_sigmoid_b200.build import HERE


def _source(name):
    with open(os.path.join(HERE, "csrc", name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_drain_has_a_limit_and_no_abort_flag():
    body = re.search(r"bool mbar_drain\((.*?)\n}", _source("common.cuh"), re.S).group(1)
    assert "abort" not in body and "limit_ns" in body and "set_device_error(MOE_ERR_TIMEOUT)" in body


@pytest.mark.parametrize("name,loops", [("few.cu", 2), ("norm.cu", 1)])
def test_rings_are_drained(name, loops):
    """The last laps of the copies' rings."""
    found = re.findall(r"for \(int j = max\(0, \w+ - [\w.]+\); j < \w+; \+\+j\)\s*([^;]*);", _source(name))
    assert len(found) == loops and all("mbar_drain(" in f and "abort" not in f for f in found)


def test_few_tokens_drains_its_mmas_and_the_tokens_codes():
    s = _source("few.cu")
    end = s[s.index("umma_commit(&sm->drained)"):s.index("tmem_dealloc(")]
    assert end.index("mbar_drain(&sm->drained, 0)") < end.index("mbar_drain(&sm->x_ready, 0)") < end.index("__syncthreads()")
