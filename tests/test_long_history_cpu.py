"""Refusals of the long-history operators that need no GPU: host argument errors of the C ABI and
the checks of the Python wrappers."""

import ctypes
import os

import pytest
import torch

from candidate_isolated_jagged_b200 import jca


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(jca.LIB_PATH):
        from candidate_isolated_jagged_b200 import build
        build.build()
    return jca.lib()


P, ST, WS = 0x10000, 0x20000, 0x40000   # never dereferenced: every call fails its host checks


def _caller(fn, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults), set(kw) - set(defaults)
        return fn(*{**defaults, **kw}.values())
    return call


def test_rope_axes_host_errors(L):
    sec = (ctypes.c_int32 * 4)(4, 2, 2, 0)
    for fn in (L.jca_rope_axes_fwd, L.jca_rope_axes_bwd):
        call = _caller(fn, q=P, k=P, qo=P, ko=P, pos=P, sec=sec, n_axes=3, per_axis=0, T=5, H=4, Hkv=2,
                       d=16, qs=64, ks=32, qos=64, kos=32, base=10000.0, dtype=0, idx_bits=64,
                       stream=None)
        assert call(idx_bits=16) == -5
        assert call(d=24) == -3
        assert call(dtype=3) == -10
        assert call(T=-1) == -2
        assert call(H=0) == -2
        assert call(Hkv=0) == -2
        assert call(n_axes=0) == -2
        assert call(n_axes=5) == -2
        assert call(base=1.0) == -2
        assert call(base=float("nan")) == -2
        assert call(sec=(ctypes.c_int32 * 3)(4, 4, 4)) == -2      # more pairs than the head has
        assert call(sec=(ctypes.c_int32 * 3)(4, -1, 4)) == -2
        assert call(sec=(ctypes.c_int32 * 3)(2**31 - 1, 2**31 - 1, 2)) == -2
        assert call(sec=None) == -1
        assert call(qs=48) == -2
        assert call(kos=16) == -2
        assert call(q=None) == -1
        assert call(ko=None) == -1
        assert call(pos=None) == -1
        assert call(q=P + 8) == -4
        assert call(qs=66) == -4
        assert call(T=0, q=None, qo=None, pos=None) == 0


def _window(L, which):
    ptrs = dict(q=P, k=P, v=P, out=P)
    if which == "fwd":
        ptrs.update(lse=P)
    else:
        ptrs.update(dout=P, lse=P, dq=P, dk=P, dv=P)
    fn = L.jagged_window_attn_fwd if which == "fwd" else L.jagged_window_attn_bwd
    return _caller(fn, **ptrs, off=P, valid=None, B=3, T=20, H=4, Hkv=2, d=16, window=8, n_sinks=2,
                   qs=64, ks=32, vs=32, scale=0.0, idx_bits=64, ws=WS, ws_bytes=1 << 22, status=ST,
                   stream=None)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_window_host_errors(L, which):
    call = _window(L, which)
    assert call(idx_bits=8) == -5
    assert call(d=48) == -3
    assert call(B=-1) == -2
    assert call(B=0) == -2            # rows without users
    assert call(T=-1) == -2
    assert call(T=1 << 31) == -2
    assert call(H=3) == -2            # not a multiple of Hkv
    assert call(Hkv=0) == -2
    assert call(window=0) == -2
    assert call(window=-5) == -2
    assert call(n_sinks=-1) == -2
    assert call(n_sinks=129) == -2
    assert call(qs=32) == -2
    assert call(ks=36) == -4
    assert call(off=None) == -1
    assert call(status=None) == -1
    assert call(ws=None) == -1
    assert call(v=None) == -1
    assert call(out=P + 2) == -4
    assert call(ws=WS + 16) == -4
    assert call(ws_bytes=8) == -6
    if which == "bwd":
        assert call(lse=None) == -1
        assert call(dk=None) == -1
        assert call(dout=P + 8) == -4


def test_window_workspace_bytes(L):
    for f in (L.jca_window_workspace_bytes, L.jca_window_bwd_workspace_bytes):
        assert f(3, 20, 4, 2, 16, 2) > 0
        assert f(0, 0, 4, 2, 16, 2) > 0
        assert f(3, 20, 4, 3, 16, 2) == 0
        assert f(3, 20, 4, 2, 20, 2) == 0
        assert f(3, 20, 4, 2, 16, 129) == 0
        assert f(-1, 20, 4, 2, 16, 2) == 0


def test_decode_host_errors(L):
    call = _caller(L.jagged_window_decode_fwd, q=P, kn=P, vn=P, kc=P, vc=P, out=P, off=P, len=P, B=3,
                   R=50, H=4, Hkv=2, d=16, window=8, n_sinks=2, qs=64, ks=32, vs=32, scale=0.0,
                   idx_bits=64, status=ST, stream=None)
    assert call(idx_bits=8) == -5
    assert call(d=20) == -3
    assert call(B=-1) == -2
    assert call(R=-1) == -2
    assert call(H=5) == -2
    assert call(window=0) == -2
    assert call(n_sinks=-1) == -2
    assert call(vs=24) == -2
    assert call(qs=68) == -4
    for name in ("q", "kn", "vn", "kc", "vc", "out", "off", "len", "status"):
        assert call(**{name: None}) == -1, name
    assert call(kc=P + 4) == -4
    assert call(B=0) == 0


def test_tree_host_errors(L):
    call = _caller(L.cand_tree_attn_fwd, q=P, k=P, v=P, off=P, parent=P, hk=P, hv=P, hoff=P, hlen=None,
                   out=P, B=3, N=9, R=50, H=4, Hkv=2, d=16, max_cand=8, qs=64, ks=32, vs=32, scale=0.0,
                   idx_bits=64, status=ST, stream=None)
    assert call(idx_bits=8) == -5
    assert call(d=20) == -3
    assert call(B=0) == -2
    assert call(N=-1) == -2
    assert call(H=5) == -2
    assert call(max_cand=0) == -2
    assert call(max_cand=1025) == -2
    assert call(ks=24) == -2
    for name in ("q", "k", "v", "off", "parent", "hk", "hv", "hoff", "out", "status"):
        assert call(**{name: None}) == -1, name
    assert call(out=P + 4) == -4
    assert call(B=0, N=0) == 0


def test_wrappers_refuse_cpu_tensors_and_shapes(L):
    q = torch.zeros(4, 2, 16, dtype=torch.bfloat16)
    off = torch.tensor([0, 4])
    with pytest.raises(ValueError, match="CUDA"):
        jca.jagged_window_attn_fwd(q, q, q, q, off, 2)
    with pytest.raises(ValueError, match="CUDA"):
        jca.jca_rope_axes_fwd(q, None, q, None, off[:, None], [8])
    with pytest.raises(ValueError, match="three"):
        jca.jagged_window_decode_fwd(q[0], q, q, q, q, q, off, off, 2)
    dev = q.device
    with pytest.raises(TypeError, match="k must"):
        jca._rows("k", q.float(), 4, 2, 16, torch.bfloat16, dev)
    with pytest.raises(ValueError, match="k must"):
        jca._rows("k", q, 4, 2, 8, torch.bfloat16, dev)
    with pytest.raises(ValueError, match="packed"):
        jca._rows("k", q.transpose(0, 1).contiguous().transpose(0, 1), 4, 2, 16, torch.bfloat16, dev)
    with pytest.raises(ValueError, match="contiguous"):
        jca._packed("out", torch.zeros(4, 6, 16, dtype=torch.bfloat16)[:, :2], 4, 2, 16, torch.bfloat16,
                    dev)
    assert jca._rows("q", torch.zeros(4, 6, 16, dtype=torch.bfloat16)[:, :2], 4, 2, 16, torch.bfloat16,
                     dev) == 96
    with pytest.raises(ValueError, match="elements"):
        jca._vector("valid", torch.zeros(3, dtype=torch.uint8), 4, torch.uint8, dev)


def test_status_names(L):
    assert "parent" in jca.status_string(8) and "type" in jca.status_string(-10)


def test_rope_axes_in_place_needs_one_stride(L):
    sec = (ctypes.c_int32 * 1)(4)
    for fn in (L.jca_rope_axes_fwd, L.jca_rope_axes_bwd):
        call = _caller(fn, q=P, k=P, qo=P, ko=P, pos=P, sec=sec, n_axes=1, per_axis=0, T=5, H=4, Hkv=2,
                       d=16, qs=64, ks=32, qos=64, kos=32, base=10000.0, dtype=0, idx_bits=64,
                       stream=None)
        assert call(qs=128) == -2
        assert call(kos=64) == -2


def test_wrappers_refuse_scratch_of_another_kind(L):
    dev = torch.device("cpu")
    with pytest.raises(TypeError, match="status"):
        jca._status_on(torch.zeros(1), dev, None)
    with pytest.raises(ValueError, match="status"):
        jca._status_on(torch.zeros(2, dtype=torch.int32), dev, None)
    status = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        jca._window_scratch(torch.zeros(8, 2, dtype=torch.uint8)[:, 0], status, lambda: 0, dev, None)
    assert jca._status_on(status, dev, None) is status


def test_integers_past_the_c_types_stay_large(L):
    assert jca._clip(1 << 70, 64) == 2**63 - 1 and jca._clip((1 << 32) + 1, 32) == 2**31 - 1
    assert jca._clip(-(1 << 40), 32) == -2**31 and jca._clip(128, 32) == 128


def test_section_counts_past_32_bits_are_refused(L):
    """ctypes alone would drop the upper bits and rotate by other sections."""
    for given, kept in (((2**32 + 4, 3), (2**31 - 1, 3)), ((-(2**32) + 4,), (-2**31,)),
                        ((1 << 70, 1), (2**31 - 1, 1)), ((3, 2, 2), (3, 2, 2))):
        assert tuple(jca._sections(given)) == kept
    call = _caller(L.jca_rope_axes_fwd, q=P, k=None, qo=P, ko=None, pos=P, sec=None, n_axes=2, per_axis=0,
                   T=5, H=4, Hkv=0, d=16, qs=64, ks=0, qos=64, kos=0, base=10000.0, dtype=0, idx_bits=64,
                   stream=None)
    assert call(sec=jca._sections((2**32 + 4, 3))) == -2
    assert call(sec=jca._sections((4, -(2**32) + 3))) == -2
    assert tuple(jca._sections([8])) == (8,)
    for bad in (2.5, 8.0, "8", None):   # 8.0 too, although it equals an accepted number
        with pytest.raises(TypeError):
            jca._sections((bad,))


def test_workspace_sizes_of_numbers_past_the_c_types(L):
    """0, as for other sizes that the calls refuse, and not the size of what the lower bits hold."""
    for f in (jca.jca_window_workspace_bytes, jca.jca_window_bwd_workspace_bytes):
        assert f(3, 20, 4, 2, 16, 2) > 0
        wide = 1 << 32
        for args in ((3 + (1 << 64), 20, 4, 2, 16, 2), (3, 20 + (1 << 64), 4, 2, 16, 2), (3, 20, 4 + wide, 2, 16, 2),
                     (3, 20, 4, 2 + wide, 16, 2), (3, 20, 4, 2, 16 + wide, 2), (3, 20, 4, 2, 16, 2 + wide),
                     (3, 20, 4, 2, 16, 2 - wide)):
            assert f(*args) == 0, args


def test_gradient_workspace_is_for_users_longer_than_the_window(L):
    """Partial sums of first tokens are kept only for users that can be longer than the window."""
    f = jca.jca_window_bwd_workspace_bytes
    rows, heads = 10000 * 50, (8, 8, 128)
    stats = f(10000, rows, *heads, 0)                      # without first tokens
    part = 8 * 8 * 64 * 128                                # bytes of one user's, or one chunk's, sums
    assert f(10000, rows, *heads, 64) == L.jca_window_bwd_workspace_bytes(10000, rows, *heads, 64)
    assert f(10000, rows, *heads, 64) >= stats + 2 * 10000 * part
    for window, users in ((49, 10000), (99, 5000), (1023, 488), (rows // 2, 1), (rows - 1, 1)):
        extra = f(10000, rows, *heads, 64, window) - stats
        slots = 2 * users + rows // 256 + 1
        assert slots * part <= extra <= slots * (part + 32) + 1024, window
    for window in (rows, rows + 1, 1 << 62, 1 << 70):
        assert f(10000, rows, *heads, 64, window) == stats
    for window in (0, -1, -(1 << 70)):
        assert f(10000, rows, *heads, 64, window) == 0
    sizes = [f(700, 40000, 4, 2, 64, 8, w) for w in range(1, 40100, 37)]
    assert sizes == sorted(sizes, reverse=True)


@pytest.mark.parametrize("window", [1, 7, 40])
def test_gradient_call_refuses_less_than_the_size_for_its_window(L, window):
    call = _window(L, "bwd")
    n = jca.jca_window_bwd_workspace_bytes(3, 20, 4, 2, 16, 2, window)
    assert call(window=window, ws_bytes=n - 1) == -6
