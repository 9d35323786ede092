"""Sizes that the attention over the 8-bit cache refuses, without a GPU."""
import pytest

from test_heads_host import INVALID, P, UNSUPPORTED, attend, lib, seqs  # noqa: F401


def test_more_tiles_than_a_block_counts(lib):  # noqa: F811
    """A block's share of the call's tiles is an int: 300 * (2^31 - 1) of them are refused, and what comes close is not."""
    prompt = dict(cu=P, tokens=1 << 20, table_width=1 << 16, table_stride=1 << 16)
    assert attend(lib, s=seqs(heads=64, **prompt), group=16) == UNSUPPORTED
    assert attend(lib, s=seqs(heads=32, **prompt), group=16, q=None) == INVALID      # (the next check)
    assert attend(lib, s=seqs(heads=1024, cu=P, tokens=1 << 16, batch=1 << 16), select=P, kept=1 << 20, group=1) == UNSUPPORTED
    assert attend(lib, s=seqs(heads=64, cu=P, tokens=1 << 16, batch=1 << 16), select=P, kept=1 << 20, group=1, q=None) == INVALID
    # many sequences under a wide table are no more than their tokens
    assert attend(lib, s=seqs(heads=32, **{**prompt, "batch": 1 << 20}), group=4, q=None) == UNSUPPORTED
    assert attend(lib, s=seqs(heads=32, **{**prompt, "batch": 1 << 10}), group=4, q=None) == INVALID


def test_more_query_heads_than_are_counted(lib):  # noqa: F811
    assert attend(lib, s=seqs(heads=32769, batch=1, tokens=1), group=65535) == UNSUPPORTED
    assert attend(lib, s=seqs(heads=32768, batch=1, tokens=1), group=65535, q=None) == INVALID
