"""What the compiler reports of the tree attention's kernel."""
import os
import re
import subprocess

from sparse_attention_td_gb300 import build as libbuild


def test_tree_attention_has_no_local_memory(tmp_path):
    """A kernel whose first launch has the driver find local memory is one unknown more in a
    kernel that is launched early; nothing in this one needs any."""
    cmd = [libbuild.nvcc(), "-c", os.path.join(libbuild.CSRC, "td_tree.cu"), "-o", str(tmp_path / "t.o")]
    r = subprocess.run(cmd + libbuild._flags(True), capture_output=True, text=True, check=True)
    lines = r.stderr.splitlines()
    seen = 0
    for line, after in zip(lines, lines[1:]):
        if "Function properties" in line and re.search(r"tree_(attention|join)_kernel", line):
            assert "0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads" in after
            seen += 1
    assert seen == 2
