"""The speculative decode step's limits on counts, at their borders, without a GPU: a call that is within them is refused
for the next thing that is wrong with it (a workspace too small, an address that is not aligned), before any CUDA call."""
import ctypes

import pytest

P = ctypes.c_void_p
SHAPE, ALIGN, UNSUPPORTED = -2, -3, -4
A, ODD = P(4096), P(4104)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from quantised_gemv_norm_gb300 import build, dq

    build.build()
    return dq.load()


# tiles of work: row tiles x key tiles x sequences x KV heads, 2^30 or more are refused
@pytest.mark.parametrize("kw,status", [
    # 43 heads a KV head: two tokens in 128 rows, four in an item, 64 of them in 16 items (not the 11 of their rows)
    (dict(n_q=43, n_seq=8, max_new=64, max_pages=1 << 24), UNSUPPORTED),
    (dict(n_q=43, n_seq=7, max_new=64, max_pages=1 << 24), SHAPE),
    (dict(n_q=33, n_seq=12, max_new=64, max_pages=1 << 24), UNSUPPORTED),  # three in 128 rows: 11 items
    (dict(n_q=33, n_seq=11, max_new=64, max_pages=1 << 24), SHAPE),
    (dict(n_q=4, n_seq=64, max_new=4, max_pages=1 << 24), UNSUPPORTED),  # up to 16 rows: tiles of 64 keys, one item
    (dict(n_q=4, n_seq=63, max_new=4, max_pages=1 << 24), SHAPE),
    (dict(n_q=8, n_seq=128, max_new=16, max_pages=1 << 24), UNSUPPORTED),  # one tile of 128 rows and keys
    (dict(n_q=8, n_seq=127, max_new=16, max_pages=1 << 24), SHAPE),
])
def test_attention_tiles(lib, kw, status):
    from quantised_gemv_norm_gb300 import dq

    d = dict(q=4096, out=4096, q_row_stride=1 << 13, q_head_stride=128, out_row_stride=1 << 13, out_head_stride=128, pool=4096,
             pages=4096, n_past=4096, cu_new=4096, seen=None, type=1, n_seq=1, total_new=64, max_new=1, n_q=1, n_kv=1,
             head_dim=128, n_pages=10, page_size=64, max_pages=5, workspace=4096, workspace_bytes=16)
    d.update(kw)
    assert lib.dq_attention_tree(ctypes.byref(dq._Tree(**d)), None) == status


@pytest.mark.parametrize("layers,n_seq,n_kv,status", [
    (1 << 16, 1 << 12, 8, UNSUPPORTED), (1 << 16, (1 << 12) - 1, 8, ALIGN), (1, 1 << 27, 16, UNSUPPORTED),
    (1, (1 << 27) - 1, 16, ALIGN), (1, 1 << 29, 1, ALIGN), (1, (1 << 29) + 1, 1, UNSUPPORTED), ((1 << 16) + 1, 1, 1, UNSUPPORTED),
    (1 << 16, 1, 1, ALIGN),
])
def test_kept_rows(lib, layers, n_seq, n_kv, status):
    """2^31 (sequence, layer, head) triples, 2^16 layers, 2^29 sequences."""
    assert lib.dq_kv16_keep(ODD, 1, A, A, A, A, layers, 4 * 64 * n_kv * 512, n_seq, 8, n_kv, 128, 4, 64, 2, None) == status


@pytest.mark.parametrize("n_q,n_kv,rows,status", [
    (2, 1, (1 << 31) - 1, UNSUPPORTED), (2, 1, (1 << 31) - 256, ALIGN), (2, 1, (1 << 31) - 255, UNSUPPORTED),
    (32, 8, 178956949, ALIGN), (32, 8, 178956950, UNSUPPORTED),  # 12 fours of heads a row: 2^31 - 256 = 12 x 178956949.3
])
def test_appended_rows(lib, n_q, n_kv, rows, status):
    """2^31 - 256 fours of heads."""
    heads = n_q + 2 * n_kv
    assert lib.dq_kv16_append(ODD, 0, heads * 128, A, A, None, None, A, 1e-6, rows, n_q, n_kv, 128, 64, 1, A, A, 4, 64,
                              None) == status
