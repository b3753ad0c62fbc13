"""Refusals of the prompt, packed-row and 4-bit cache entry points, and the layout the header
defines, without a GPU: every check returns before any CUDA call."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
NULL, SHAPE, ALIGN, UNSUPPORTED = -1, -2, -3, -4
A = P(4096)  # an aligned address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from quantised_gemv_norm_gb300 import build, dq

    build.build()
    return dq.load()


def changed(base, **kw):
    d = dict(base)
    d.update(kw)
    return list(d.values())


ROPE = dict(qkv=A, stride=48 * 128, pos=A, qn=A, kn=A, rope=A, eps=1e-6, rows=3, n_q=32, n_kv=8, hd=128, ctx=64, type=1,
            q=A, k=A, v=A, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(qkv=None), NULL), (dict(pos=None), NULL), (dict(rope=None), NULL), (dict(q=None), NULL), (dict(v=None), NULL),
    (dict(qn=None), NULL), (dict(kn=None), NULL),  # one norm alone
    (dict(rows=0), SHAPE), (dict(n_q=0), SHAPE), (dict(n_kv=-1), SHAPE), (dict(ctx=0), SHAPE), (dict(type=3), SHAPE),
    (dict(type=-1), SHAPE), (dict(stride=48 * 128 - 4), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(hd=64), UNSUPPORTED), (dict(stride=48 * 128 + 2), ALIGN), (dict(qkv=P(4100)), ALIGN), (dict(k=P(4104)), ALIGN),
    (dict(qn=P(4104)), ALIGN),
])
def test_qkv_rope_refuses(lib, kw, status):
    assert lib.dq_qkv_rope(*changed(ROPE, **kw)) == status


def prompt(**kw):
    from quantised_gemv_norm_gb300 import dq

    d = dict(q=4096, k=4096, v=4096, out=4096, q_row_stride=6144, q_head_stride=128, k_row_stride=6144, k_head_stride=128,
             v_row_stride=6144, v_head_stride=128, out_row_stride=4096, out_head_stride=128, cu_q=4096, cu_k=None, type=1,
             n_seq=2, total_q=10, total_k=10, n_q=32, n_kv=8, head_dim=128, workspace=None, workspace_bytes=0)
    d.update(kw)
    return dq._Prompt(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL), (dict(cu_q=None), NULL),
    (dict(n_seq=0), SHAPE), (dict(total_q=0), SHAPE), (dict(total_k=0), SHAPE), (dict(n_q=30), SHAPE), (dict(n_kv=0), SHAPE),
    (dict(type=0), SHAPE), (dict(type=7), SHAPE), (dict(q_row_stride=64), SHAPE), (dict(k_head_stride=0), SHAPE),
    (dict(v_row_stride=0), SHAPE), (dict(out_head_stride=-128), SHAPE), (dict(head_dim=64), UNSUPPORTED),
    (dict(n_q=129, n_kv=1), UNSUPPORTED), (dict(total_q=(1 << 30) + 1), UNSUPPORTED), (dict(k_row_stride=6148), ALIGN),
    (dict(q=4104), ALIGN), (dict(out=4097), ALIGN),
])
def test_attention_prompt_refuses(lib, kw, status):
    assert lib.dq_attention_prompt(ctypes.byref(prompt(**kw)), None) == status


def test_attention_prompt_refuses_no_description(lib):
    assert lib.dq_attention_prompt(None, None) == NULL


APPEND = dict(k=A, v=A, type=1, kr=1024, kh=128, vr=1024, vh=128, slots=A, pool=A, rows=5, n_kv=8, hd=128, pages=4, page=64,
              stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(pool=None), NULL),
    (dict(rows=0), SHAPE), (dict(n_kv=0), SHAPE), (dict(pages=0), SHAPE), (dict(page=0), SHAPE), (dict(page=24), SHAPE),
    (dict(type=9), SHAPE), (dict(kr=0), SHAPE), (dict(vh=64), SHAPE), (dict(hd=64), UNSUPPORTED),
    (dict(pages=1 << 20, page=2048), UNSUPPORTED), (dict(k=P(4104)), ALIGN), (dict(pool=P(4098)), ALIGN),
    (dict(vr=1028), ALIGN),
])
def test_kv4_append_refuses(lib, kw, status):
    assert lib.dq_kv4_append(*changed(APPEND, **kw)) == status


READ = dict(pool=A, slots=A, type=1, k=A, v=A, rows=5, n_kv=8, hd=128, pages=4, page=64, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(pool=None), NULL), (dict(slots=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(rows=0), SHAPE),
    (dict(page=8), SHAPE), (dict(type=3), SHAPE), (dict(hd=256), UNSUPPORTED), (dict(v=P(4104)), ALIGN),
])
def test_kv4_read_refuses(lib, kw, status):
    assert lib.dq_kv4_read(*changed(READ, **kw)) == status


DECODE = dict(q=A, type=0, pool=A, table=A, n=A, out=A, n_seq=1, n_q=32, n_kv=8, hd=128, pages=4, page=64, max_pages=4,
              max_keys=200, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(pool=None), NULL), (dict(table=None), NULL), (dict(n=None), NULL), (dict(out=None), NULL),
    (dict(n_seq=0), SHAPE), (dict(n_q=30), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_keys=0), SHAPE),
    (dict(max_keys=257), SHAPE), (dict(max_keys=(1 << 30) + 1, max_pages=1 << 25), UNSUPPORTED), (dict(page=40), SHAPE), (dict(type=4), SHAPE), (dict(n_q=72), UNSUPPORTED),
    (dict(hd=64), UNSUPPORTED), (dict(q=P(4100)), ALIGN), (dict(out=P(4104)), ALIGN), (dict(pool=P(4104)), ALIGN),
])
def test_attention_decode_kv4_refuses(lib, kw, status):
    assert lib.dq_attention_decode_kv4(*changed(DECODE, **kw)) == status


def test_binding_refuses_shapes_and_types():
    from quantised_gemv_norm_gb300 import dq

    q, k = torch.zeros(4, 8, 128, dtype=torch.float16), torch.zeros(4, 2, 128, dtype=torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        dq.attention_prompt(q, k, k.bfloat16(), cu)
    with pytest.raises(ValueError):
        dq.attention_prompt(q, k, k[:3], cu)
    with pytest.raises(ValueError):
        dq.attention_prompt(q, k, k, cu.long())
    with pytest.raises(ValueError):
        dq.attention_prompt(q[..., :64], k, k, cu)
    with pytest.raises(ValueError):
        dq.attention_prompt(q, k, k, cu, cu_k=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        dq.kv4_pool(2, 2, 24, device="cpu")
    pool = dq.kv4_pool(2, 2, 32, device="cpu")
    assert tuple(pool.shape) == (2, 2, 2, 2560)
    slots = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dq.kv4_append(k.double(), k.double(), slots, pool)
    with pytest.raises(ValueError):
        dq.kv4_append(k, k, slots[:3], pool)
    with pytest.raises(ValueError):
        dq.kv4_append(k, k, slots, pool[:, :1])
    with pytest.raises(ValueError):
        dq.kv4_read(pool.float(), slots)
    with pytest.raises(ValueError):
        dq.attention_decode_kv4(q, pool, torch.zeros(4, 1, dtype=torch.int64), slots)
    with pytest.raises(ValueError):
        dq.qkv_rope(torch.zeros(4, 128), slots, torch.zeros(8, 64, 2), 2, 1)


def test_prompt_struct_matches_the_header(tmp_path):
    from quantised_gemv_norm_gb300 import dq

    fields = [n for n, _ in dq._Prompt._fields_]
    consts = {"DQ_TYPE_F32": dq.TYPE_F32, "DQ_TYPE_F16": dq.TYPE_F16, "DQ_TYPE_BF16": dq.TYPE_BF16,
              "DQ_KV4_BLOCK_ROWS": dq.KV4_BLOCK_ROWS, "DQ_KV4_BLOCK_BYTES": dq.KV4_BLOCK_BYTES}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "dq.h"', "int main(void) {",
           '  printf("size %zu\\n", sizeof(dq_prompt));']
    src += ['  printf("%s %%zu\\n", offsetof(dq_prompt, %s));' % (f, f) for f in fields]
    src += ['  printf("%s %%d\\n", (int)(%s));' % (c, c) for c in consts]
    src += ["  return 0;", "}"]
    c = tmp_path / "layout.c"
    c.write_text("\n".join(src) + "\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                           text=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(dq._Prompt)
    for f in fields:
        assert int(got[f]) == getattr(dq._Prompt, f).offset, f
    for n, v in consts.items():
        assert int(got[n]) == v
