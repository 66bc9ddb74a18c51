"""The draft-serving calls on the host: refusals, and what the binding needs."""
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
