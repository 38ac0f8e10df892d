"""The calls on drafted trees and the sinks' setting refuse bad arguments on the host, before any CUDA call: pointers
here are never followed."""
import ctypes

import pytest

from paged_kv_decode_09_gb300 import api, build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
SCORES = api._Scores(0.1, 0.0, None, None)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


@pytest.fixture(scope="module")
def pools(lib):
    out = {}
    for kv in (api.F16, api.Q8_0, api.BF16, api.F32):
        h = ctypes.c_void_p()
        sc = FAKE if kv == api.Q8_0 else None
        assert lib.kv_pool_create(ctypes.byref(h), 3, 64, 8, 128, kv, FAKE, FAKE, sc, sc, None) == 0
        out[kv] = h
    yield out
    for h in out.values():
        lib.kv_pool_destroy(h)


def refused(lib, fn, args, changes, status):
    args = dict(args, **changes)
    assert getattr(lib, fn)(*args.values()) == status, changes
    assert lib.pkv_last_error_message()


def tree(pools, kv=api.F16, sc=SCORES):
    return dict(pool=pools[kv], layer=0, q=FAKE, qs=4096, t=api.F16, parents=FAKE, cu=FAKE, tokens=5, bt=FAKE, stride=4,
                lens=FAKE, rows=2, n_q=32, sc=ctypes.byref(sc), out=ctypes.c_void_p(1 << 22), lse=None, ws=FAKE,
                ws_bytes=1 << 40, chunks=8, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(pool=None), INVALID), (dict(layer=7), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(parents=None), INVALID), (dict(parents=ODD), INVALID), (dict(out=None), INVALID), (dict(out=FAKE), INVALID),
    (dict(t=api.BF16), UNSUPPORTED), (dict(t=api.F32), UNSUPPORTED), (dict(n_q=24), UNSUPPORTED), (dict(qs=4088), INVALID),
    (dict(cu=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID), (dict(stride=0), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=2049), UNSUPPORTED), (dict(tokens=-1), INVALID),
    (dict(tokens=(1 << 22) + 1), UNSUPPORTED), (dict(sc=None), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=0), WORKSPACE), (dict(chunks=-1), INVALID), (dict(chunks=4097), UNSUPPORTED),
    (dict(sc=ctypes.pointer(api._Scores(0.1, 0.0, FAKE, None))), UNSUPPORTED),
    (dict(sc=ctypes.pointer(api._Scores(0.1, 0.0, None, FAKE))), UNSUPPORTED),
    (dict(sc=ctypes.pointer(api._Scores(float("nan"), 0.0, None, None))), INVALID),
    (dict(sc=ctypes.pointer(api._Scores(0.1, -1.0, None, None))), INVALID),
])
def test_tree_attention(lib, pools, changes, status):
    refused(lib, "paged_tree_attention", tree(pools), changes, status)


def test_f32_pools_have_no_tree_attention(lib, pools):
    for t in (api.F16, api.BF16, api.F32):
        refused(lib, "paged_tree_attention", tree(pools, api.F32), dict(t=t), UNSUPPORTED)


def commit(pools, kv=api.F16):
    other = lambda n: ctypes.c_void_p((1 << 20) + 4096 * n)  # noqa: E731
    return dict(pool=pools[kv], first=0, layers=3, parents=FAKE, leaves=other(1), cu=FAKE, tokens=5, bt=FAKE, stride=4,
                lens=other(2), rows=2, path=None, path_stride=1, new=other(3), stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(pool=None), INVALID), (dict(first=-1), INVALID), (dict(first=3), INVALID), (dict(layers=4), INVALID),
    (dict(layers=-1), INVALID), (dict(first=1), INVALID), (dict(first=2, layers=2 ** 31 - 1), INVALID),
    (dict(parents=None), INVALID), (dict(parents=ODD), INVALID), (dict(leaves=None), INVALID), (dict(leaves=ODD), INVALID),
    (dict(cu=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID), (dict(stride=0), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=2049), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(new=None), INVALID),
    (dict(new=ODD), INVALID), (dict(path=FAKE, path_stride=0), INVALID), (dict(path=ODD), INVALID),
    (dict(new=ctypes.c_void_p((1 << 20) + 8192)), INVALID), (dict(new=ctypes.c_void_p((1 << 20) + 4096)), INVALID),
    (dict(new=FAKE), INVALID), (dict(path=ctypes.c_void_p((1 << 20) + 8192)), INVALID), (dict(path=FAKE), INVALID),
    (dict(path=ctypes.c_void_p((1 << 20) + 4096 * 3)), INVALID),
])
def test_commit(lib, pools, changes, status):
    refused(lib, "kv_tree_commit", commit(pools), changes, status)


def test_nothing_to_do_is_fine(lib, pools):
    for changes in (dict(rows=0), dict(tokens=0)):
        assert lib.paged_tree_attention(*dict(tree(pools), **changes, q=None, ws=None, parents=None).values()) == 0
    assert lib.kv_tree_commit(*dict(commit(pools), rows=0, parents=None, leaves=None).values()) == 0


def test_sinks_setting(lib, pools):
    p, n = pools[api.F16], ctypes.c_int(-1)
    assert lib.kv_pool_get_sinks(p, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.kv_pool_set_sinks(p, 1, 4) == 0
    assert lib.kv_pool_get_sinks(p, 1, ctypes.byref(n)) == 0 and n.value == 4
    assert lib.kv_pool_get_sinks(p, 0, ctypes.byref(n)) == 0 and n.value == 0
    for layer, sinks in ((1, -1), (3, 1), (-1, 1), (1, (1 << 30) + 1)):
        assert lib.kv_pool_set_sinks(p, layer, sinks) == INVALID
    assert lib.kv_pool_set_sinks(None, 0, 1) == INVALID and lib.kv_pool_get_sinks(None, 0, ctypes.byref(n)) == INVALID
    assert lib.kv_pool_get_sinks(p, 0, None) == INVALID
    assert lib.kv_pool_set_sinks(p, 1, 0) == 0


def test_calls_that_do_not_serve_sinks(lib, pools):
    """The two-launch form, several queries a row and attention weights refuse a layer with sinks and a window; one
    without a window has none."""
    p = pools[api.F16]
    assert lib.kv_pool_set_sinks(p, 2, 4) == 0 and lib.kv_pool_set_window(p, 2, 100) == 0
    step = [p, 2, FAKE, FAKE, 4, FAKE, 2, 32, 0.1, FAKE, FAKE, 1 << 40, 8, None]
    assert lib.paged_decode_split(*step) == UNSUPPORTED and b"sinks" in lib.pkv_last_error_message()
    several = [p, 2, FAKE, FAKE, 4, FAKE, 2, 4, 32, 0.1, FAKE, FAKE, 1 << 40, 8, None]
    assert lib.paged_decode_attention_mq(*several) == UNSUPPORTED and b"sinks" in lib.pkv_last_error_message()
    assert lib.pkv_decode_step_mq(*several[:3], FAKE, FAKE, *several[3:]) == UNSUPPORTED
    mass = [p, 2, FAKE, 4096, api.F16, FAKE, FAKE, 5, FAKE, 4, FAKE, 2, 32, ctypes.byref(SCORES), 0, None, FAKE, 64, FAKE,
            1 << 40, 8, None]
    assert lib.paged_attention_mass(*mass) == UNSUPPORTED and b"sinks" in lib.pkv_last_error_message()
    assert lib.kv_pool_set_window(p, 2, 0) == 0 and lib.kv_pool_set_sinks(p, 2, 0) == 0
