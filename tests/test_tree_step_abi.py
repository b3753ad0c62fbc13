"""Refusals of the speculative decode step's entry points, and the layouts the header defines, without a GPU: every check
returns before any CUDA call."""
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
    assert set(kw) <= set(base)
    d = dict(base)
    d.update(kw)
    return list(d.values())


APPEND = dict(qkv=A, in_type=0, stride=48 * 128, pos=A, slots=A, qn=A, kn=A, rope=A, eps=1e-6, rows=3, n_q=32, n_kv=8, hd=128,
              ctx=64, type=1, q=A, pool=A, pages=4, page=64, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(qkv=None), NULL), (dict(pos=None), NULL), (dict(slots=None), NULL), (dict(rope=None), NULL), (dict(q=None), NULL),
    (dict(pool=None), NULL), (dict(qn=None), NULL), (dict(kn=None), NULL),
    (dict(rows=0), SHAPE), (dict(n_q=0), SHAPE), (dict(n_kv=-1), SHAPE), (dict(ctx=0), SHAPE), (dict(in_type=3), SHAPE),
    (dict(type=0), SHAPE), (dict(type=5), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(stride=47 * 128), SHAPE), (dict(page=24), SHAPE), (dict(page=0), SHAPE), (dict(pages=0), SHAPE),
    (dict(hd=64), UNSUPPORTED), (dict(pages=1 << 20, page=2048), UNSUPPORTED), (dict(pages=1 << 21, page=64), UNSUPPORTED),
    (dict(n_q=(1 << 16) + 1, stride=1 << 24), UNSUPPORTED), (dict(stride=48 * 128 + 2), ALIGN),
    (dict(in_type=1, stride=48 * 128 + 4), ALIGN), (dict(qkv=P(4104)), ALIGN), (dict(q=P(4104)), ALIGN),
    (dict(pool=P(4098)), ALIGN), (dict(kn=P(4100)), ALIGN), (dict(slots=P(4098)), ALIGN),
])
def test_append_refuses(lib, kw, status):
    assert lib.dq_kv16_append(*changed(APPEND, **kw)) == status


def tree(**kw):
    from quantised_gemv_norm_gb300 import dq

    d = dict(q=4096, out=4096, q_row_stride=4096, q_head_stride=128, out_row_stride=4096, out_head_stride=128, pool=4096,
             pages=4096, n_past=4096, cu_new=4096, seen=None, type=1, n_seq=2, total_new=6, max_new=4, n_q=32, n_kv=8,
             head_dim=128, n_pages=10, page_size=64, max_pages=5, workspace=4096, workspace_bytes=1 << 40)
    assert set(kw) <= set(d)
    d.update(kw)
    return dq._Tree(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(pool=None), NULL), (dict(pages=None), NULL), (dict(n_past=None), NULL),
    (dict(workspace=None), NULL), (dict(n_seq=0), SHAPE), (dict(total_new=0), SHAPE), (dict(max_new=0), SHAPE),
    (dict(n_q=30), SHAPE), (dict(n_kv=0), SHAPE), (dict(type=0), SHAPE), (dict(type=3), SHAPE), (dict(page_size=40), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(q_row_stride=64), SHAPE), (dict(out_head_stride=0), SHAPE),
    (dict(cu_new=None), SHAPE), (dict(workspace_bytes=8), SHAPE), (dict(head_dim=64), UNSUPPORTED),
    (dict(max_new=65), UNSUPPORTED), (dict(n_q=65 * 8), UNSUPPORTED), (dict(total_new=(1 << 30) + 1), UNSUPPORTED),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(n_seq=1 << 21), UNSUPPORTED), (dict(n_pages=1 << 21), UNSUPPORTED),
    (dict(q_row_stride=1 << 38), UNSUPPORTED), (dict(q_row_stride=4100), ALIGN), (dict(q=4104), ALIGN), (dict(out=4097), ALIGN),
    (dict(pool=4104), ALIGN), (dict(workspace=4104), ALIGN), (dict(seen=4100), ALIGN), (dict(n_past=4098), ALIGN),
])
def test_attention_refuses(lib, kw, status):
    assert lib.dq_attention_tree(ctypes.byref(tree(**kw)), None) == status


def test_no_description(lib):
    assert lib.dq_attention_tree(None, None) == NULL
    assert lib.dq_verify_draft(None, None) == NULL


def verify(**kw):
    from quantised_gemv_norm_gb300 import dq

    d = dict(logits=4096, logits_stride=1000, draft_probs=None, draft_stride=0, noise=4096, noise_stride=1000, tokens=4096,
             parents=None, uniform=4096, temperature=None, cu_new=None, path=4096, n_path=4096, next=4096, type=0, n_seq=2,
             total_new=6, max_new=3, vocab=1000, workspace=4096, workspace_bytes=1 << 40)
    assert set(kw) <= set(d)
    d.update(kw)
    return dq._Verify(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), NULL), (dict(noise=None), NULL), (dict(tokens=None), NULL), (dict(uniform=None), NULL),
    (dict(path=None), NULL), (dict(n_path=None), NULL), (dict(next=None), NULL), (dict(workspace=None), NULL),
    (dict(n_seq=0), SHAPE), (dict(total_new=0), SHAPE), (dict(total_new=5), SHAPE), (dict(max_new=0), SHAPE),
    (dict(vocab=0), SHAPE), (dict(type=3), SHAPE), (dict(logits_stride=999), SHAPE), (dict(noise_stride=0), SHAPE),
    (dict(draft_probs=4096, draft_stride=10), SHAPE), (dict(workspace_bytes=64), SHAPE),
    (dict(max_new=65, cu_new=4096), UNSUPPORTED), (dict(draft_probs=4096, draft_stride=1000, parents=4096), UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1, logits_stride=1 << 25, noise_stride=1 << 25), UNSUPPORTED),
    (dict(total_new=(1 << 24) + 1, cu_new=4096), UNSUPPORTED),
    (dict(total_new=1 << 24, cu_new=4096, vocab=1 << 24, logits_stride=1 << 24, noise_stride=1 << 24), UNSUPPORTED),
    (dict(logits=4098), ALIGN), (dict(logits=4097, type=1), ALIGN), (dict(noise=4098), ALIGN), (dict(next=4097), ALIGN),
    (dict(workspace=4104), ALIGN), (dict(cu_new=4098), ALIGN),
])
def test_verify_refuses(lib, kw, status):
    assert lib.dq_verify_draft(ctypes.byref(verify(**kw)), None) == status


KEEP = dict(pool=A, type=1, pages=A, n_past=A, path=A, n_path=A, layers=3, stride=4 * 64 * 8 * 512, n_seq=2, max_new=8, n_kv=8,
            hd=128, n_pages=4, page=64, max_pages=2, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(pool=None), NULL), (dict(pages=None), NULL), (dict(n_past=None), NULL), (dict(path=None), NULL),
    (dict(n_path=None), NULL), (dict(layers=0), SHAPE), (dict(n_seq=0), SHAPE), (dict(max_new=0), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(type=0), SHAPE), (dict(page=8), SHAPE), (dict(stride=4 * 64 * 8 * 512 - 16), SHAPE),
    (dict(max_new=65), UNSUPPORTED), (dict(hd=96), UNSUPPORTED), (dict(n_seq=1 << 27), UNSUPPORTED),
    (dict(layers=(1 << 16) + 1), UNSUPPORTED), (dict(pool=P(4104)), ALIGN), (dict(stride=4 * 64 * 8 * 512 + 8), ALIGN),
    (dict(path=P(4098)), ALIGN),
])
def test_keep_refuses(lib, kw, status):
    assert lib.dq_kv16_keep(*changed(KEEP, **kw)) == status


def test_workspace_sizes(lib):
    assert lib.dq_attention_tree_workspace_bytes(0, 1, 32, 8) == 0
    assert lib.dq_attention_tree_workspace_bytes(1, 65, 32, 8) == 0
    assert lib.dq_attention_tree_workspace_bytes(1, 4, 30, 8) == 0
    assert lib.dq_attention_tree_workspace_bytes(1, 4, 32, 8) > 0
    assert lib.dq_verify_draft_workspace_bytes(0, 100) == 0
    assert lib.dq_verify_draft_workspace_bytes(3, 0) == 0
    n = lib.dq_verify_draft_workspace_bytes(3, 8193)
    assert n >= 3 * 16 and n % 48 == 0
    assert lib.dq_verify_draft_workspace_bytes(6, 8193) <= 2 * n


def test_binding_refuses_shapes_and_types():
    from quantised_gemv_norm_gb300 import dq

    with pytest.raises(ValueError):
        dq.kv16_pool(2, 2, 24, device="cpu")
    with pytest.raises(ValueError):
        dq.kv16_pool(2, 2, 16, dtype=torch.float32, device="cpu")
    pool = dq.kv16_pool(2, 2, 32, device="cpu")
    assert tuple(pool.shape) == (2, 2, 2, 32, 128)
    assert tuple(dq.kv16_pool(2, 2, 32, n_layers=3, device="cpu").shape) == (3, 2, 2, 2, 32, 128)
    n = torch.zeros(4, dtype=torch.int32)
    pages = torch.zeros(4, 1, dtype=torch.int32)
    q = torch.zeros(4, 8, 128, dtype=torch.float16)
    for bad in (dict(q=q.bfloat16()), dict(q=q[..., :64]), dict(pool=pool[:, :1]), dict(pool=pool.float()),
                dict(pages=pages.long()), dict(pages=pages[0]), dict(n_past=n[:3]), dict(seen=n), dict(cu_new=n),
                dict(q=torch.cat([q, q[:1]])), dict(max_new=2)):
        a = dict(q=q, pool=pool, pages=pages, n_past=n)
        a.update(bad)
        with pytest.raises(ValueError):
            dq.attention_tree(**a)
    rope = torch.zeros(8, 64, 2)
    for bad in (dict(qkv=torch.zeros(4, 128)), dict(positions=n.long()), dict(slots=n[:2]), dict(rope=rope[..., :1]),
                dict(q_norm=torch.zeros(128)), dict(qkv=torch.zeros(4, 12 * 128).double()), dict(pool=pool.float())):
        a = dict(qkv=torch.zeros(4, 12 * 128), positions=n, slots=n, rope=rope, pool=pool, n_q=8)
        a.update(bad)
        with pytest.raises(ValueError):
            dq.kv16_append(**a)
    for bad in (dict(logits=torch.zeros(4)), dict(logits=torch.zeros(4, 10).double()), dict(tokens=n.long()),
                dict(uniform=torch.zeros(3)), dict(noise=torch.zeros(2, 9)), dict(noise=torch.zeros(3, 10)),
                dict(parents=n[:3]), dict(draft_probs=torch.zeros(4, 9)), dict(temperature=torch.zeros(4)),
                dict(cu_new=n), dict(max_new=3), dict(logits=torch.zeros(10, 4).T)):
        a = dict(logits=torch.zeros(4, 10), tokens=n, uniform=torch.zeros(4), noise=torch.zeros(2, 10))
        a.update(bad)
        with pytest.raises(ValueError):
            dq.verify_draft(**a)
    for bad in (dict(pool=pool[0]), dict(path=n), dict(pages=pages[:3]), dict(n_path=n.long()), dict(n_past=n[:2])):
        a = dict(pool=pool, pages=pages, n_past=n, path=torch.zeros(4, 3, dtype=torch.int32), n_path=n)
        a.update(bad)
        with pytest.raises(ValueError):
            dq.kv16_keep(**a)


@pytest.mark.parametrize("name", ["_Tree", "_Verify"])
def test_packed_descriptions_are_the_structures(name):
    from quantised_gemv_norm_gb300 import dq

    cls, pack = getattr(dq, name), {"_Tree": dq._pack_tree, "_Verify": dq._pack_verify}[name]
    values = [1000 + 7 * i for i in range(len(cls._fields_))]
    made = cls.from_buffer_copy(pack(*values).ljust(ctypes.sizeof(cls), b"\0"))
    assert [getattr(made, f) for f, _ in cls._fields_] == values


def test_structs_match_the_header(tmp_path):
    from quantised_gemv_norm_gb300 import dq

    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "dq.h"', "int main(void) {"]
    for name, cls in (("dq_tree", dq._Tree), ("dq_verify", dq._Verify)):
        src.append('  printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        src += ['  printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f) for f, _ in cls._fields_]
    src += ["  return 0;", "}"]
    c = tmp_path / "layout.c"
    c.write_text("\n".join(src) + "\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                       text=True).stdout.splitlines())
    for name, cls in (("dq_tree", dq._Tree), ("dq_verify", dq._Verify)):
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got["%s.%s" % (name, f)]) == getattr(cls, f).offset, f
