"""Sizes and numbers behind the prompt and 4-bit cache calls that need no GPU."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from quantised_gemv_norm_gb300 import build, dq

    build.build()
    return dq.load()


def test_decode_scratch_goes_by_the_query_heads(lib):
    size = lib.dq_attention_decode_kv4_workspace_bytes
    one = size(5, 3, 3, 100000)
    assert one > 0
    for group in range(2, 9):
        assert size(5, 3 * group, 3, 100000) == group * one


@pytest.mark.parametrize("n_seq,n_q,n_kv,max_keys", [
    (2**31 - 1, 2**31 - 1, 2**31 - 1, 2**30), (2**31 - 1, 8, 1, 4096), (4, 9, 1, 4096), (4, 10, 4, 4096), (1, 8, 8, 2**30 + 1),
    (1, 1 << 17, 1 << 17, 4096),
])
def test_decode_scratch_is_zero_for_counts_that_the_call_refuses(lib, n_seq, n_q, n_kv, max_keys):
    assert lib.dq_attention_decode_kv4_workspace_bytes(n_seq, n_q, n_kv, max_keys) == 0
