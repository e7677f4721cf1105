"""The host side of the orthogonalised updates: workspace sizes and the optimiser that chunks a tensor's
matrices (CPU: no kernel runs)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = [(64, 96), (128, 3000), (128, 3100), (300, 520), (7168, 100), (100, 7168), (2112, 1088), (512, 2048), (1, 32768),
          (32768, 32768)]


def test_workspace_of_no_matrices():
    # (in a process of its own: the division by the number of matrices ended it)
    code = ("from expert_routed_ffn_router_gb300 import binding as B\n"
            f"for s in {SHAPES!r}: assert 0 < B.moe_orthogonalize_workspace_bytes(0, *s) <= 4096, s\n")
    assert subprocess.run([sys.executable, "-c", code], timeout=300, cwd=ROOT).returncode == 0
