"""Every file under csrc/ is built into the library or included by one that is."""
import os
import re

from block_diffusion_lm_gb300 import build


def test_no_source_is_left_over():
    files = sorted(f for f in os.listdir(build.CSRC)
                   if os.path.isfile(os.path.join(build.CSRC, f)))
    included = set()
    for f in files:
        with open(os.path.join(build.CSRC, f)) as h:
            included.update(re.findall(r'#include "([^"]+)"', h.read()))
    assert [f for f in files if f not in build.SOURCES and f not in included] == []
    assert sorted(set(build.SOURCES) - set(files)) == []
