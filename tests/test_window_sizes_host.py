"""The size queries of the windowed decode and the chunk attention refuse what does not fit a C int in
any argument, instead of answering for the size that it wraps to."""

import pytest

import paged_kv_cache_422_b200 as nvpa

DECODE = dict(batch=4, num_q_heads=16, num_kv_heads=8, head_dim=128, max_context_len=4096, block_size=256, window=512,
              num_sinks=4, num_splits=2)
CHUNK = dict(DECODE, total_q=100, max_seqlen_q=40)


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_422_b200.build import build
    build()


@pytest.mark.parametrize("query,sizes", [(nvpa.paged_decode_window_workspace_size, DECODE),
                                         (nvpa.chunk_attention_workspace_size, CHUNK)])
def test_sizes_that_do_not_fit(query, sizes):
    assert query(**sizes) > 0
    for name, value in sizes.items():
        for wide in (value + (1 << 32), 1 << 31, -(1 << 31) - 1, 1 << 70):
            with pytest.raises(ValueError, match="32 bits"):
                query(**dict(sizes, **{name: wide}))
    for name in ("batch", "num_q_heads", "num_kv_heads", "max_context_len", "window", "num_sinks", "num_splits"):
        assert query(**dict(sizes, **{name: -1})) == 0
