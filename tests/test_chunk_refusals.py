"""The long-prompt calls refuse bad arguments on the host, before any CUDA call: pointers here are never followed."""
import ctypes

import pytest

from paged_kv_decode_09_gb300 import api, build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


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
        assert lib.kv_pool_create(ctypes.byref(h), 2, 64, 8, 128, kv, FAKE, FAKE, sc, sc, None) == 0
        out[kv] = h
    yield out
    for h in out.values():
        lib.kv_pool_destroy(h)


def refused(lib, fn, args, changes, status):
    """The call with `changes` to its arguments is refused with `status`, and says why."""
    args = dict(args, **changes)
    assert getattr(lib, fn)(*args.values()) == status, changes
    assert lib.pkv_last_error_message()


def rope(pools, kv=api.F16):
    return dict(pool=pools[kv], layer=0, q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, t_in=api.F16, q_out=ODD,
                t_out=api.F16, pos=FAKE, axes=2, sec=(ctypes.c_int * 2)(30, 34), inv=FAKE, rot=128, inter=0, cu=FAKE,
                tokens=5, bt=FAKE, stride=4, lens=FAKE, rows=2, n_q=32, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(pool=None), INVALID), (dict(layer=2), INVALID), (dict(layer=-1), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=ODD), INVALID), (dict(), INVALID),  # q_out unaligned
    (dict(q_out=None), INVALID), (dict(q_out=FAKE, t_out=api.BF16), INVALID),  # in place, another type
    (dict(q_out=FAKE, qs=8192), INVALID),  # in place, another stride
    (dict(qs=4095), INVALID), (dict(ks=1023), INVALID), (dict(vs=1028), INVALID), (dict(qs=1 << 31), INVALID),
    (dict(t_in=api.Q8_0), UNSUPPORTED), (dict(t_out=api.Q8_0), UNSUPPORTED), (dict(t_in=9), UNSUPPORTED),
    (dict(rot=120), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
    (dict(axes=0), UNSUPPORTED), (dict(axes=5), UNSUPPORTED), (dict(sec=None), INVALID),
    (dict(sec=(ctypes.c_int * 2)(30, 33)), INVALID), (dict(sec=(ctypes.c_int * 2)(0, 64)), INVALID),
    (dict(inv=None), INVALID), (dict(pos=None), INVALID), (dict(cu=None), INVALID), (dict(bt=None), INVALID),
    (dict(lens=ODD), INVALID), (dict(stride=0), INVALID), (dict(rows=-1), INVALID), (dict(rows=2049), UNSUPPORTED),
    (dict(tokens=-1), INVALID), (dict(tokens=(1 << 22) + 1), UNSUPPORTED), (dict(n_q=-1), INVALID),
])
def test_rope_append(lib, pools, changes, status):
    refused(lib, "kv_rope_append", rope(pools), changes, status)


SCORES = api._Scores(0.1, 0.0, None, None)


def attention(pools, kv=api.F16, sc=SCORES):
    return dict(pool=pools[kv], layer=0, q=FAKE, qs=4096, t=api.F16, cu=FAKE, tokens=5, bt=FAKE, stride=4, lens=FAKE,
                rows=2, n_q=32, sc=ctypes.byref(sc), out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, chunks=8,
                stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(pool=None), INVALID), (dict(layer=7), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(lse=ctypes.c_void_p((1 << 20) + 1)), INVALID),
    (dict(t=api.BF16), UNSUPPORTED), (dict(t=api.F32), UNSUPPORTED), (dict(n_q=0), INVALID), (dict(n_q=12), INVALID),
    (dict(n_q=24), UNSUPPORTED), (dict(n_q=64, qs=8192), UNSUPPORTED), (dict(qs=4088), INVALID),
    (dict(qs=4100), INVALID), (dict(cu=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(stride=0), INVALID), (dict(stride=1 << 27), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=2049), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(sc=None), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=0), WORKSPACE), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), INVALID), (dict(chunks=-1), INVALID),
    (dict(chunks=4097), UNSUPPORTED),
])
def test_chunk_attention(lib, pools, changes, status):
    refused(lib, "paged_chunk_attention", attention(pools), changes, status)


@pytest.mark.parametrize("sc", [api._Scores(float("nan"), 0, None, None), api._Scores(float("inf"), 0, None, None),
                                api._Scores(0.1, -1, None, None), api._Scores(0.1, float("nan"), None, None),
                                api._Scores(0.1, float("inf"), None, None), api._Scores(0.1, 0, ODD, None),
                                api._Scores(0.1, 0, None, ctypes.c_void_p((1 << 20) + 1))])
def test_scores(lib, pools, sc):
    refused(lib, "paged_chunk_attention", attention(pools, sc=sc), {}, INVALID)
    refused(lib, "paged_attention_mass", mass(pools, sc=sc), {}, INVALID)


def test_pools_take_their_own_type(lib, pools):
    refused(lib, "paged_chunk_attention", attention(pools, api.BF16), {}, UNSUPPORTED)
    refused(lib, "paged_chunk_attention", attention(pools, api.Q8_0), dict(t=api.BF16), UNSUPPORTED)
    for t in (api.F16, api.BF16, api.F32):
        refused(lib, "paged_chunk_attention", attention(pools, api.F32), dict(t=t), UNSUPPORTED)
        refused(lib, "paged_attention_mass", mass(pools, api.F32), dict(t=t), UNSUPPORTED)


def test_nothing_to_do_is_fine(lib, pools):
    for changes in (dict(rows=0), dict(tokens=0)):
        assert lib.paged_chunk_attention(*dict(attention(pools), **changes, q=None, ws=None).values()) == 0
        assert lib.kv_rope_append(*dict(rope(pools), **changes, q=None).values()) == 0
    assert lib.paged_attention_mass(*dict(mass(pools), rows=0, q=None).values()) == 0
    assert lib.kv_evict(*dict(evict(pools), rows=0, mass=None).values()) == 0


def test_workspace_bytes(lib, pools):
    f = lib.paged_chunk_workspace_bytes
    assert f(pools[api.F16], 32, 8) > 0
    assert f(None, 32, 8) == 0 and f(pools[api.F16], 30, 8) == 0 and f(pools[api.F16], 24, 8) == 0
    assert f(pools[api.F16], 32, 0) == 0 and f(pools[api.F16], 32, 4097) == 0
    g = lib.paged_attention_mass_workspace_bytes
    assert g(8) > 0 and g(0) == 0 and g(4097) == 0


def mass(pools, kv=api.F16, sc=SCORES):
    return dict(pool=pools[kv], layer=0, q=FAKE, qs=4096, t=api.F16, lse=FAKE, cu=FAKE, tokens=5, bt=FAKE, stride=4,
                lens=FAKE, rows=2, n_q=32, sc=ctypes.byref(sc), last=0, mass_in=None, mass_out=FAKE, mass_stride=64,
                ws=FAKE, ws_bytes=1 << 40, chunks=8, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(pool=None), INVALID), (dict(layer=7), INVALID), (dict(q=None), INVALID), (dict(lse=None), INVALID),
    (dict(t=api.BF16), UNSUPPORTED), (dict(n_q=24), UNSUPPORTED), (dict(qs=4100), INVALID),
    (dict(mass_out=None), INVALID), (dict(mass_in=ctypes.c_void_p((1 << 20) + 1)), INVALID),
    (dict(mass_stride=0), INVALID), (dict(last=-1), INVALID), (dict(sc=None), INVALID), (dict(cu=None), INVALID),
    (dict(rows=2049), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), INVALID), (dict(chunks=-1), INVALID), (dict(chunks=4097), UNSUPPORTED),
])
def test_mass(lib, pools, changes, status):
    refused(lib, "paged_attention_mass", mass(pools), changes, status)


def evict(pools, kv=api.F16):
    other = lambda n: ctypes.c_void_p((1 << 20) + 4096 * n)  # noqa: E731
    return dict(pool=pools[kv], layer=0, mass=FAKE, mass_stride=64, bt=other(1), stride=4, lens=other(2), rows=2,
                keep=other(3), first=1, recent=1, dst=other(4), dst_stride=2, idx=other(5), keep_stride=32,
                dst_mass=None, new_lens=other(6), stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(pool=None), INVALID), (dict(layer=7), INVALID), (dict(mass=None), INVALID), (dict(bt=None), INVALID),
    (dict(lens=None), INVALID), (dict(keep=None), INVALID), (dict(dst=None), INVALID), (dict(idx=None), INVALID),
    (dict(new_lens=None), INVALID), (dict(mass_stride=0), INVALID), (dict(stride=0), INVALID),
    (dict(dst_stride=0), INVALID), (dict(keep_stride=0), INVALID), (dict(first=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=2049), UNSUPPORTED),
    (dict(dst_mass=FAKE), INVALID),  # the weights themselves
    (dict(new_lens=ctypes.c_void_p((1 << 20) + 8192)), INVALID),  # seq_lens
    (dict(mass=ctypes.c_void_p((1 << 20) + 1)), INVALID),
])
def test_evict(lib, pools, changes, status):
    refused(lib, "kv_evict", evict(pools), changes, status)


@pytest.mark.parametrize("scale,softcap", [(0.1, 1e-31), (0.1, 2e30), (1e38, 1e-3)])
def test_caps_whose_scores_leave_fp32(lib, pools, scale, softcap):
    changes = dict(sc=ctypes.pointer(api._Scores(scale, softcap, None, None)))
    refused(lib, "paged_chunk_attention", attention(pools), changes, INVALID)


def test_out_is_not_q(lib, pools):
    refused(lib, "paged_chunk_attention", attention(pools), dict(out=FAKE), INVALID)
    assert b"out" in lib.pkv_last_error_message()
