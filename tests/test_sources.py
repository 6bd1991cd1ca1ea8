"""What the sources must not hold (no GPU needed)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def instructions():
    """(file, text) of each piece of inline assembly, its string literals joined."""
    for path in glob.glob(os.path.join(ROOT, "attention_forward_gb300", "csrc", "*")):
        with open(path) as f:
            text = re.sub(r'"\s*\n\s*"', "", f.read())
        for literal in re.findall(r'"((?:[^"\\]|\\.)*)"', text):
            for line in literal.replace("\\t", " ").split("\\n"):
                yield os.path.basename(path), line


def test_no_load_is_multicast_to_a_cluster():
    """Every rank of a run on several GPUs loads this library, and a call may be given
    another GPU's memory, from which no multicast load may read: each CTA loads its own
    tiles."""
    loads = [(f, i) for f, i in instructions() if "cp.async.bulk" in i]
    assert len(loads) > 5
    assert not [x for x in loads if "multicast" in x[1]]
