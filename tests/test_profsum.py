"""The sources that the committed traffic profile is stamped with."""

import json
import os
import re

from ternary_weight_int8_tb_amd import profsum


def included(path, seen):
    """`path` and the headers of its own folder that it includes, directly or not."""
    seen.add(path)
    for name in re.findall(r'^#include "([^"]+)"', open(path).read(), re.M):
        header = os.path.join(os.path.dirname(path), name)
        if os.path.exists(header) and header not in seen:
            included(header, seen)
    return seen


def test_the_stamp_covers_every_source_of_the_profiled_kernels():
    csrc = os.path.join(profsum.ROOT, "ternary_weight_int8_tb_amd", "csrc")
    sources = included(os.path.join(csrc, "tb.hip"), set())
    assert sorted(os.path.join(profsum.ROOT, f) for f in profsum.SOURCES) == sorted(sources)


def test_the_committed_profile_names_the_sources():
    with open(os.path.join(profsum.ROOT, "profiles", "ffn64_stream_traffic.json")) as fh:
        assert json.load(fh)["source_files"] == profsum.SOURCES
