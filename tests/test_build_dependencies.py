"""What an edit has to rebuild."""
import os
import re

from rotary_position_embedding_rope_gb300 import _build


def test_every_included_file_is_a_dependency_of_the_library():
    deps = {os.path.realpath(d) for d in _build._deps()}
    for source in sorted(deps):
        for name in re.findall(r'^#include "([^"]+)"', open(source).read(), re.M):
            at = [p for p in (os.path.join(d, name) for d in (_build.CSRC, _build.INCLUDE)) if os.path.exists(p)]
            assert at and os.path.realpath(at[0]) in deps, "%s of %s" % (name, os.path.basename(source))
