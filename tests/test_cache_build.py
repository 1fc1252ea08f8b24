"""What the compiler reports of the kernels on small caches."""
import os
import subprocess

import pytest

from sparse_attention_td_gb300 import build as libbuild


@pytest.mark.parametrize("source,kernels", [("td_cache_attn.cu", 5), ("td_cache_rows.cu", 8), ("td_prompt.cu", 3)])
def test_kernels_have_no_local_memory(source, kernels, tmp_path):
    """All of them are launched early, as the tree attention's: none has, nor any function that it calls."""
    cmd = [libbuild.nvcc(), "-c", os.path.join(libbuild.CSRC, source), "-o", str(tmp_path / "t.o")]
    r = subprocess.run(cmd + libbuild._flags(True), capture_output=True, text=True, check=True)
    lines = r.stderr.splitlines()
    assert sum("Compiling entry function" in line for line in lines) == kernels
    seen = 0
    for line, after in zip(lines, lines[1:]):
        if "Function properties" in line:
            assert "0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads" in after, line
            seen += 1
    assert seen >= kernels
