"""What a build watches (no GPU needed)."""
import os
import re

from mixture_experts_layer_rmsnorm_gb300 import _build


def test_every_included_file_is_watched():
    """A file that a source includes by name makes the library stale when it is newer."""
    watched = {os.path.realpath(p) for p in _build.sources() + _build.headers()}
    for src in sorted(watched):
        with open(src) as f:
            for name in re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M):
                places = [os.path.join(d, name) for d in (os.path.dirname(src), _build.CSRC, _build.INCLUDE)]
                found = [os.path.realpath(p) for p in places if os.path.exists(p)]
                assert found and found[0] in watched, f"{os.path.basename(src)} includes {name}"
