"""Operands of the cache operators that share memory where they must not (CPU only): refused on the host before anything
is enqueued.  The addresses are never read."""
import ctypes

import pytest
import torch

import latent_kv_attention_b200 as lka
from latent_kv_attention_b200 import build, cache_ops

P = ctypes.c_void_p
INVALID, WORKSPACE = 1, 3
Q, K, V, QO, KC, VC, LENS, FREQ, TABLE, SCALE, WS = (P((i + 1) << 24) for i in range(11))
ST = (ctypes.c_int64 * 9)(*([64] * 9))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lka.library()


def at(p, off):
    return P(p.value + off)


def gqa(lib, q_out=QO, kc=KC, vc=VC, ws=WS):
    """Caches of 3 x 2 x 32 rows of 64 bf16 values: 24,576 bytes; queries of 3 x 4 x 1 rows: 1536 bytes."""
    return lib.gqa_rope_append(Q, K, V, ST, LENS, None, FREQ, q_out, kc, vc, 3, 4, 2, 1, 64, 64, 32, 0, 1.0, 0, ws, 256, None)


def paged(lib, q_out=QO, kc=KC, vc=VC, ws=WS):
    """Pools of 5 x 2 x 16 rows of 64 bf16 values: 20,480 bytes."""
    return lib.gqa_rope_append_paged(Q, K, V, ST, TABLE, LENS, None, FREQ, q_out, kc, vc, 3, 4, 2, 1, 64, 64, 16, 2, 5, 0, 1.0,
                                     0, ws, 256, None)


def fp8(lib, q_out=QO, kc=KC, vc=VC, ws=WS):
    """Caches of 12,288 bytes."""
    return lib.gqa_rope_append_fp8kv(Q, K, V, ST, SCALE, SCALE, LENS, None, FREQ, q_out, kc, vc, 3, 4, 2, 1, 64, 64, 32, 0, 1.0,
                                     ws, 256, None)


def latent(lib, q_out=QO, cache=KC, ws=WS):
    """A cache of 3 x 32 rows of 512 + 64 bf16 values: 110,592 bytes."""
    return lib.latent_rope_append(Q, K, V, ST, LENS, None, FREQ, q_out, cache, 3, 8, 1, 512, 64, 32, 0, 1.0, 0, ws, 256, None)


@pytest.mark.parametrize("call,size", [(gqa, 24576), (paged, 20480), (fp8, 12288)])
def test_append_refuses_overlapping_caches_and_queries(lib, call, size):
    assert call(lib, vc=at(KC, size - 16)) == INVALID
    assert call(lib, kc=at(VC, size - 16)) == INVALID
    assert call(lib, q_out=KC) == INVALID
    assert call(lib, q_out=at(VC, size - 16)) == INVALID
    assert call(lib, q_out=at(KC, -1536 + 16)) == INVALID
    # next to each other is apart: what is missing then is the workspace
    assert call(lib, vc=at(KC, size), q_out=at(KC, -1536), ws=None) == WORKSPACE


def test_latent_append_refuses_queries_in_the_cache(lib):
    assert latent(lib, q_out=at(KC, 110592 - 16)) == INVALID
    assert latent(lib, q_out=at(KC, 1024)) == INVALID  # in its values
    assert latent(lib, q_out=at(KC, 110592), ws=None) == WORKSPACE


def test_paged_evict_refuses_overlapping_pools(lib):
    """Pools of 5 x 2 x 16 rows of 64 bf16 values: 20,480 bytes."""
    def call(vp, ws=WS):
        return lib.gqa_evict_paged(KC, vp, P(20 << 24), TABLE, LENS, P(21 << 24), P(22 << 24), 1, 2, 64, 16, 2, 5, 8, 0, 0, 0, ws,
                                   256, None)
    assert call(KC) == INVALID
    assert call(at(KC, 20480 - 16)) == INVALID
    assert call(at(KC, -20480 + 16)) == INVALID
    assert call(at(KC, 20480), ws=None) == WORKSPACE


# ------------------------------------------------------------------ the binding
@pytest.mark.parametrize("strides,ok", [((384, 128, 32, 1), True), ((384, 32, 96, 1), True), ((0, 128, 32, 1), False),
                                        ((384, 128, 16, 1), False), ((384, 16, 32, 1), False), ((64, 128, 32, 1), False)])
def test_in_place_needs_rows_of_their_own(strides, ok):
    """A tensor [2, 3, 4, 32] of these strides, rotated in place: rows that are met twice would be turned twice."""
    x = torch.empty(2048).as_strided((2, 3, 4, 32), strides)
    assert ok == (len({int(i) for i in torch.arange(2048).as_strided(x.shape, strides).flatten()}) == x.numel())
    if ok:
        cache_ops._separate(x, strides, x, strides, "x", itself=True)
    else:
        with pytest.raises(ValueError):
            cache_ops._separate(x, strides, x, strides, "x", itself=True)
