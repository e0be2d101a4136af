"""Sizes at the paged calls' limits (none of the calls reaches a device)."""

from test_paged_oracle import UNSUPPORTED, calls, lib  # noqa: F401


def test_tokens_of_a_call(lib):  # noqa: F811
    """More tokens than tiles of queries can be counted in 32 bits."""
    for T in ((1 << 30) + 1, (1 << 31) - 1):
        for dtype in (0, 1):
            assert calls(lib, T=T, H=1, dtype=dtype, o_dtype=dtype, max_new=T)["attend"]() == UNSUPPORTED
