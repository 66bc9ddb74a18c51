"""The draft-serving calls on the host: refusals, and what the binding needs."""
import os
import subprocess
import sys

import numpy as np
import pytest

import discrete_diffusion_block_gb300 as dgp
from test_draft_ops_host import AT, LP, L, call  # noqa: F401  (L: a fixture)

MOST = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("factor", [MOST, MOST / 1.44])
def test_factors_whose_product_with_log2_e_overflows_are_refused(L, factor):  # noqa: F811
    # the kernels work in units of log2: factor log2(e) would be infinite, and
    # infinity times the distance 0 of a row's maximum NaN
    assert call(L.dg_op_tree_attention, AT, scale=factor) == dgp.DG_EINVAL
    assert call(L.dg_op_token_logprobs, LP, inv_tau=factor) == dgp.DG_EINVAL


def test_the_largest_factor_is_accepted(L):  # noqa: F811
    # (calls without rows: the checks alone)
    most = float(np.float32(2.3e38))
    assert np.isfinite(np.float32(most * 1.4426950408889634))
    assert call(L.dg_op_tree_attention, AT, scale=most, n_tok=0) == dgp.DG_OK
    assert call(L.dg_op_token_logprobs, LP, inv_tau=most, rows=0) == dgp.DG_OK


def test_the_package_is_imported_and_built_without_torch():
    code = """
import sys
sys.modules["torch"] = None                  # as if it were not installed
import discrete_diffusion_block_gb300 as dgp
from discrete_diffusion_block_gb300 import build
build.build()
assert dgp.load().dg_last_error() is not None
assert dgp.load().dg_op_tree_attention_workspace_bytes(5, 2, 16, 8, 128) > 0
print("works")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600)
    assert p.returncode == 0 and "works" in p.stdout, p.stderr[-2000:]
