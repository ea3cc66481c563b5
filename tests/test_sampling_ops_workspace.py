"""Sizes of the workspaces of the sampling operators, without a GPU."""
from decoder_only_transformer_fwd_b200 import nc


def test_prefix_attention_workspace_may_start_at_any_16_byte_boundary():
    """Piece rows are stored 32 bytes at a time, so the areas start at a multiple of 32 within the workspace, and its
    size has room for that.  These sizes leave no slack between the areas: one slot per unit and CTA (32 + 296), each
    of 64 rows of 128 fp32 values and a log-sum-exp, then 8 bytes per unit."""
    full = (32 + 296) * 64 * (128 + 1) * 4 + 32 * 8
    assert full % 256 == 0
    assert nc.nc_prefix_attention_workspace_bytes(32, 32, 1, 64, 1, 100, 0) >= full + 16
