"""Argument checks of the cache operators on the host (CPU only)."""
import ctypes

import numpy as np
import pytest

import cache_ref as ref
from paged_kv_cache_03_gb300 import binding as B

FAKE = 1 << 20  # aligned, never dereferenced on a failed check


def shape(**kw):
    d = dict(B=2, H_q=4, H_kv=2, L=5, D=128, num_pages=16, page_size=16, max_pages_per_seq=3,
             dtype=B.PA_BF16)
    d.update(kw)
    return B.make_shape(**d)


def pool(**kw):
    d = dict(key_codes=FAKE, key_scales=FAKE, value_codes=FAKE, value_scales=FAKE)
    d.update(kw)
    return tuple(d.values())


def attend(sh=None, q=FAKE, p=pool(), bt=FAKE, ctx=FAKE, scale=0.1, w=None, w_out=None, w_S=0,
           out=FAKE, ws=FAKE):
    return B.pa_paged_attention_q4(sh or shape(), q, p, bt, ctx, scale, 1, w, w_out, w_S, out, ws,
                                   1 << 30, 0)


def test_q4_attention_refusals():
    bad = B.PA_ERR_INVALID_ARG
    assert attend(q=None) == bad and attend(bt=None) == bad and attend(ctx=None) == bad
    assert attend(out=FAKE + 8) == bad and attend(p=None) == bad
    assert attend(p=pool(key_codes=FAKE + 8)) == bad
    assert attend(p=pool(value_codes=None)) == bad
    assert attend(p=pool(key_scales=FAKE + 8)) == bad
    assert attend(scale=float("nan")) == bad and attend(scale=-1.0) == bad
    assert attend(sh=shape(H_q=5)) == bad
    assert attend(sh=shape(D=64)) == B.PA_ERR_UNSUPPORTED
    assert attend(w=FAKE) == bad                                 # nowhere to write
    assert attend(w_out=FAKE, w_S=47) == bad                     # shorter than the table
    assert attend(w_out=FAKE + 2, w_S=48) == bad
    assert attend(ws=None) == B.PA_ERR_WORKSPACE
    assert attend(ws=FAKE + 16) == B.PA_ERR_WORKSPACE
    assert B.pa_q4_workspace_bytes(shape(L=0)) == 0


def test_weights_refusals():
    def call(sh=None, w_out=FAKE, w_S=48):
        return B.pa_paged_attention_weights(sh or shape(), FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, 1,
                                            None, w_out, w_S, FAKE, None, 0, 0)
    assert call(w_out=None) == B.PA_ERR_INVALID_ARG
    assert call(w_S=47) == B.PA_ERR_INVALID_ARG
    assert call(sh=shape(dtype=B.PA_F32)) == B.PA_ERR_UNSUPPORTED
    assert call() == B.PA_ERR_WORKSPACE
    assert B.pa_weights_workspace_bytes(shape(dtype=B.PA_F32)) == 0


def test_append_and_gather_refusals():
    def append(k=FAKE, p=pool(), ws=FAKE, n=256):
        return B.pa_append_kv_q4(shape(), k, FAKE, p, FAKE, FAKE, ws, n, 0)
    assert append(k=None) == B.PA_ERR_INVALID_ARG
    assert append(k=FAKE + 8) == B.PA_ERR_INVALID_ARG
    assert append(p=pool(value_scales=None)) == B.PA_ERR_INVALID_ARG
    assert append(ws=None) == B.PA_ERR_WORKSPACE and append(n=255) == B.PA_ERR_WORKSPACE

    def gather(n=4, k=FAKE):
        return B.pa_gather_kv_q4(shape(), pool(), FAKE, FAKE, n, 0, k, FAKE, None, 0, 0)
    assert gather(n=0) == B.PA_ERR_INVALID_ARG and gather(k=FAKE + 4) == B.PA_ERR_INVALID_ARG
    assert gather() == B.PA_ERR_WORKSPACE


@pytest.mark.parametrize("q4", [False, True])
def test_evict_refusals(q4):
    def call(w_S=48, keep=20, recent=5, dst=FAKE + 64, dst_n=2, ctx_out=FAKE + 64,
             w_out=FAKE + 64, w_out_S=20, kept=FAKE, ws=FAKE):
        args = (FAKE, FAKE, FAKE, w_S, keep, recent, dst, dst_n, ctx_out, w_out, w_out_S, kept, ws,
                256, 0)
        if q4:
            return B.pa_evict_kv_q4(shape(), pool(), *args)
        return B.pa_evict_kv(shape(), FAKE, FAKE, *args)
    bad = B.PA_ERR_INVALID_ARG
    assert call(w_S=47) == bad and call(keep=0) == bad and call(recent=-1) == bad
    assert call(recent=21) == bad
    assert call(dst=FAKE) == bad and call(ctx_out=FAKE) == bad and call(w_out=FAKE) == bad
    assert call(dst_n=1) == bad and call(w_out_S=19) == bad
    assert call(kept=None) == bad
    assert call(ws=None) == B.PA_ERR_WORKSPACE


def test_python_refusals():
    import torch
    z = torch.zeros
    u8 = torch.uint8
    with pytest.raises(ValueError):  # not on a GPU
        B.Q4Pool(z(4, 2, 16, 64, dtype=u8), z(4, 2, 16, 8, dtype=u8), z(4, 2, 16, 64, dtype=u8),
                 z(4, 2, 16, 8, dtype=u8))
    with pytest.raises(ValueError):
        B.Q4Pool(z(4, 2, 16, 32, dtype=u8), z(4, 2, 16, 8, dtype=u8), z(4, 2, 16, 64, dtype=u8),
                 z(4, 2, 16, 8, dtype=u8))
    with pytest.raises(ValueError):
        B.paged_attention_weights(z(1, 4, 1, 128), z(4, 2, 16, 128), z(4, 2, 16, 128),
                                  z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32), 16,
                                  key_weights_out=z(1, 2, 32))
    with pytest.raises(ValueError):
        B._pages_dims(z(4, 2, 16, 128), z(4, 2, 16, 128, dtype=torch.bfloat16))


def test_the_tests_own_quantiser():
    """The 64-bit form against hand-made rows."""
    x = np.zeros((1, 128))
    x[0, :8] = [6, -6, 5, 2.5, -0.25, 0.75, 3.5, 0.26]  # scale 1: ties to even codes
    x[0, 16:18] = [2690, -1e9]                          # past the range
    x[0, 32] = 2.0 ** -12                               # below the smallest scale's codes
    codes, scales = ref.quantise(x)
    assert scales[0, 0] == 0x38 and scales[0, 1] == 0x7e and scales[0, 2] == 1
    v = ref.dequantise(codes, scales)[0]
    assert v[:8].tolist() == [6, -6, 4, 2, 0, 1, 4, 0.5]
    assert v[16:18].tolist() == [2688, -2688] and v[32] == 0
    assert ctypes.sizeof(B.pa_q4_pool) == 32


def test_the_tests_own_eviction():
    w = np.array([[[3, 1, 3, 2, 3, 9, 0, 0]]], np.float32)
    assert ref.evict(w, [6], 3, 1)[0].tolist() == [[[0, 2, 5]]]
    assert ref.evict(w, [6], 3, 3)[0].tolist() == [[[3, 4, 5]]]
    assert ref.evict(w, [2], 3, 1)[0].tolist() == [[[0, 1, -1]]]
