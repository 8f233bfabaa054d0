"""The library is rebuilt when any file that it is compiled from is newer."""
import os
import re

from block_causal_streaming_b200 import build as wf_build


def _included(path, seen):
    """Files that `path` includes by name, and theirs."""
    if path in seen:
        return
    seen.add(path)
    with open(path) as f:
        names = re.findall(r'^#include "([^"]+)"', f.read(), re.M)
    for n in names:
        for folder in (os.path.dirname(path), os.path.join(wf_build.ROOT, "include")):
            at = os.path.normpath(os.path.join(folder, n))
            if os.path.exists(at):
                _included(at, seen)


def test_every_included_file_is_watched():
    seen = set()
    for s in wf_build.SOURCES:
        _included(s, seen)
    watched = {os.path.normpath(f) for f in wf_build.DEPENDS}
    assert len(seen) > 10 and seen <= watched, sorted(seen - watched)
