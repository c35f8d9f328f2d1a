"""The guard on the accumulator ring of the key-weights kernel, on CPU: a ring in which a copy
could overwrite accumulators that are still to be read does not compile."""
import os
import subprocess

import pytest

from load_balanced_split_gb300 import build as hbuild

RING = "kAccs = kSmall ? 8 : 16;"


def _front_end(tmp_path, ring):
    text = open(os.path.join(hbuild.CSRC, "key_weights.cu"), encoding="utf-8").read()
    assert text.count(RING) == 1
    src = tmp_path / "key_weights.cu"
    src.write_text(text.replace(RING, "kAccs = %s;" % ring))
    cmd = [hbuild.nvcc()] + hbuild.ARCH + hbuild.FLAGS + ["--fatbin", "-Xcicc", "-O0", str(src),
                                                          "-o", str(tmp_path / "out.fatbin")]
    return subprocess.run(cmd, capture_output=True, text=True)


@pytest.mark.parametrize("ring", ["kStages + kBufs", "(kStages + kBufs + 1) & ~1",
                                  "kStages + kBufs + kGroups - 1"])
def test_a_ring_without_slack_is_refused(tmp_path, ring):
    r = _front_end(tmp_path, ring)
    assert r.returncode != 0 and "accumulator ring" in r.stderr
