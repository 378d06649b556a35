"""Argument checks of draft trees and page sharing on the host, and the tests'
own plain forms (CPU only)."""
import numpy as np
import pytest

import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

FAKE = 1 << 20  # aligned, never dereferenced on a failed check
BAD = B.PA_ERR_INVALID_ARG


def shape(**kw):
    d = dict(B=2, H_q=4, H_kv=2, L=5, D=128, num_pages=16, page_size=16, max_pages_per_seq=3,
             dtype=B.PA_BF16)
    d.update(kw)
    return B.make_shape(**d)


def pool(**kw):
    d = dict(key_codes=FAKE, key_scales=FAKE, value_codes=FAKE, value_scales=FAKE)
    d.update(kw)
    return tuple(d.values())


def test_mask_refusals():
    def call(b=2, L=5, parents=FAKE, mask=FAKE, depths=FAKE, ws=FAKE, n=256):
        return B.pa_tree_mask(b, L, parents, mask, depths, ws, n, 0)
    assert call(b=0) == BAD and call(L=0) == BAD and call(L=-1) == BAD
    assert call(parents=None) == BAD and call(mask=FAKE + 2) == BAD and call(depths=None) == BAD
    assert call(L=B.TREE_MAX + 1) == B.PA_ERR_UNSUPPORTED
    assert call(ws=None) == B.PA_ERR_WORKSPACE and call(n=255) == B.PA_ERR_WORKSPACE


@pytest.mark.parametrize("q4", [False, True])
def test_attention_refusals(q4):
    def call(sh=None, q=FAKE, p=pool(), bt=FAKE, ctx=FAKE, mask=FAKE, scale=0.1, out=FAKE, ws=FAKE):
        sh = sh or shape()
        if q4:
            return B.pa_paged_attention_tree_q4(sh, q, p, bt, ctx, mask, scale, out, ws, 1 << 30, 0)
        return B.pa_paged_attention_tree(sh, q, p[0], p[2], bt, ctx, mask, scale, out, ws, 1 << 30,
                                         0)
    assert call(q=None) == BAD and call(bt=None) == BAD and call(ctx=FAKE + 2) == BAD
    assert call(mask=None) == BAD and call(mask=FAKE + 2) == BAD and call(out=FAKE + 8) == BAD
    assert call(p=pool(key_codes=FAKE + 8)) == BAD and call(p=pool(value_codes=None)) == BAD
    assert call(scale=float("inf")) == BAD and call(scale=-1.0) == BAD
    assert call(sh=shape(H_q=5)) == BAD
    assert call(sh=shape(D=64)) == B.PA_ERR_UNSUPPORTED
    assert call(sh=shape(L=B.TREE_MAX + 1)) == B.PA_ERR_UNSUPPORTED
    assert call(ws=None) == B.PA_ERR_WORKSPACE and call(ws=FAKE + 16) == B.PA_ERR_WORKSPACE
    assert B.pa_tree_workspace_bytes(shape(L=B.TREE_MAX + 1)) == 0
    assert B.pa_tree_workspace_bytes(shape(L=0)) == 0


@pytest.mark.parametrize("q4", [False, True])
def test_compaction_refusals(q4):
    def call(sh=None, p=pool(), bt=FAKE, ctx=FAKE, path=FAKE, n=4, lens=FAKE, out=FAKE + 64,
             ws=FAKE, wn=256):
        args = (bt, ctx, path, n, lens, out, ws, wn, 0)
        if q4:
            return B.pa_compact_kv_q4(sh or shape(), p, *args)
        return B.pa_compact_kv(sh or shape(), p[0], p[2], *args)
    assert call(p=pool(key_codes=None)) == BAD and call(path=None) == BAD and call(n=0) == BAD
    assert call(lens=FAKE + 1) == BAD and call(out=None) == BAD
    assert call(out=FAKE) == BAD  # the lengths themselves
    assert call(sh=shape(B=0)) == BAD
    assert call(ws=None) == B.PA_ERR_WORKSPACE and call(wn=8) == B.PA_ERR_WORKSPACE


def test_page_refusals():
    n = B.pa_pages_workspace_bytes(shape())
    assert n >= 256 and B.pa_pages_workspace_bytes(shape(num_pages=0)) == 0

    def fork(bt=FAKE, refs=FAKE, s=FAKE, t=FAKE, lens=None, k=3, ws=FAKE, wn=256):
        return B.pa_fork_pages(shape(), bt, FAKE, refs, s, t, lens, k, ws, wn, 0)
    assert fork(bt=None) == BAD and fork(refs=None) == BAD and fork(s=None) == BAD
    assert fork(t=FAKE + 2) == BAD and fork(k=-1) == BAD and fork(lens=FAKE + 1) == BAD
    assert fork(ws=None) == B.PA_ERR_WORKSPACE and fork(wn=255) == B.PA_ERR_WORKSPACE
    assert fork(k=0) == B.PA_OK  # nothing to do

    def resize(bt=FAKE, ctx=FAKE, new=FAKE + 64, copies=FAKE, ws=FAKE, wn=n):
        return B.pa_resize_pages(shape(), bt, ctx, FAKE, new, copies, ws, wn, 0)
    assert resize(bt=None) == BAD and resize(new=None) == BAD and resize(copies=None) == BAD
    assert resize(new=FAKE) == BAD  # the lengths themselves
    assert resize(ws=None) == B.PA_ERR_WORKSPACE and resize(ws=FAKE + 64) == B.PA_ERR_WORKSPACE
    assert resize(wn=n - 1) == B.PA_ERR_WORKSPACE

    def copy(p=pool(), c=FAKE, k=2, ws=FAKE):
        return (B.pa_copy_pages(shape(), p[0], p[2], c, k, ws, 256, 0),
                B.pa_copy_pages_q4(shape(), p, c, k, ws, 256, 0))
    assert copy(p=pool(value_codes=FAKE + 8)) == (BAD, BAD)
    assert copy(c=None) == (BAD, BAD) and copy(k=-1) == (BAD, BAD)
    assert copy(ws=None) == (B.PA_ERR_WORKSPACE,) * 2
    assert copy(k=0) == (B.PA_OK,) * 2


def test_python_refusals():
    import torch
    i = torch.int32

    def z(*s, dtype=i):
        return torch.zeros(s, dtype=dtype)
    with pytest.raises(ValueError):
        B.tree_mask(z(2, 3))  # not on a GPU
    with pytest.raises(ValueError):
        B.tree_mask(z(2, 3, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.paged_attention_tree(z(1, 4, 2, 128, dtype=torch.bfloat16),
                               *[z(4, 2, 16, 128, dtype=torch.bfloat16)] * 2, z(1, 2), z(1),
                               z(1, 2, 1), 16)
    for sources in (z(2), z(2, dtype=torch.int64)):
        with pytest.raises(ValueError):
            B.fork_pages(z(4, 2), z(4), z(9), sources, z(2), 16)
    with pytest.raises(ValueError):
        B.resize_pages(z(4, 2), z(3), z(9), z(4), 16)  # lengths of other rows
    with pytest.raises(ValueError):
        B._copy_pages("", None, (), (4, 2, 16), 0, torch.device("cpu"), z(4, 2), z(256))


def test_the_tests_own_trees():
    parents = np.array([[-1, 0, 0, 2, -2, 4, -1]], np.int32)
    see = tr.visible(parents)[0]
    assert [np.flatnonzero(r).tolist() for r in see] == [[0], [0, 1], [0, 2], [0, 2, 3], [], [], [6]]
    assert tr.words(see[None])[0, :, 0].tolist() == [1, 3, 5, 13, 0, 0, 64]


def test_the_tests_own_pages():
    p = tr.Pages(3, 4, 6, 4)
    p.resize([6, 0, 0])
    p.fork([0], [1])
    assert p.table[1].tolist() == [0, 1, -1, -1] and p.refs.tolist() == [2, 2, 0, 0, 0, 0]
    copies, short = p.resize([-1, 9, 0])
    assert copies[1].tolist() == [1, 2, 2] and not short and p.table[1].tolist() == [0, 2, 3, -1]
    copies, short = p.resize([0, 16, 12])
    # row 0 gives up page 1 alone: row 1 takes it, row 2 finds two of three
    assert short and p.ctx.tolist() == [0, 16, 0] and p.table[1].tolist() == [0, 2, 3, 1]
    assert p.consistent()
