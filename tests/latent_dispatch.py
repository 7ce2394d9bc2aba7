"""Which kernel a call of spec_latent_attention takes, told by its workspace."""

import torch


def item_rows(c, heads, most):
    """Rows of an item: 16 to 64 (slots are the products' rows) or 128 (a row a thread; two items a row tile above 256 dimensions).
    The workspace holds flags, cut items and two shares for each of 152 parts."""
    import speculative_decoding_verification_29_gb300 as sv

    need = sv.latent_workspace_bytes(torch.empty(1, c.bs, c.C + c.R, dtype=c.dt), c.C, heads, most)
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    for rows in (16, 32, 48, 64, 128):
        dims = c.C // 2 if rows == 128 and c.C > 256 else c.C
        if need == up(152 * 4) + up(304 * 16) + up(304 * rows * 8) + up(304 * rows * dims * 4):
            return rows
    raise AssertionError(need)
