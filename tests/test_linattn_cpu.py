"""include/gdn_linattn.h on the host: exported symbols, struct layouts, and refusals (every call
here fails validation or launches nothing, so no GPU is needed).  The 64-bit definitions that the
GPU tests compare with are checked against independent forms."""
import ctypes
import os
import re
import time

import numpy as np
import pytest
import torch

from gated_delta_rule_64_b200 import gdn
from oracle import linattn as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE
A = 1 << 40  # fake, 256-byte aligned "device" addresses; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_64_b200 import build
    build.build()
    return gdn.load_library()


def _p(i, off=0):
    return None if i is None else ctypes.c_void_p(A + i * (1 << 36) + off)


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "gdn_linattn.h")).read()
    names = set(re.findall(r"\b(gdn_[a-z_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(gdn.EXPORTED_LINATTN)
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layouts():
    assert ctypes.sizeof(gdn.GdnQkRopeDesc) == 56 and gdn.GdnQkRopeDesc.q_stride.offset == 32
    assert ctypes.sizeof(gdn.GdnBeamDesc) == 32 and gdn.GdnBeamDesc.row_stride.offset == 24


# ---------------------------------------------------------------------------
# gdn_linattn_chunk_fwd, gdn_linattn_decode_step
# ---------------------------------------------------------------------------

def _desc(B=2, T=130, H=3, dk=128, dv=128, dtype=gdn.GDN_BF16, gate=gdn.GDN_GATE_HEAD, scale=1.0, hk=0):
    return gdn.GdnDesc(B, T, H, dk, dv, dtype, gate, scale, hk)


def _fwd(lib, d, *, q=0, k=1, v=2, g=3, h0=None, cu=None, n=0, snap=0, out=5, fin=None, snaps=None, ws=7,
         ws_bytes=1 << 34, off=None):
    off = off or {}
    p = lambda i, name: _p(i, off.get(name, 0))  # noqa: E731
    return lib.gdn_linattn_chunk_fwd(ctypes.byref(d), p(q, "q"), p(k, "k"), p(v, "v"), p(g, "g"), p(h0, "h0"),
                                     p(cu, "cu"), n, snap, p(out, "out"), p(fin, "fin"), p(snaps, "snaps"),
                                     p(ws, "ws"), ws_bytes, None)


@pytest.mark.parametrize("field,value,status", [
    ("dk", 96, UNS), ("dv", 32, UNS), ("H", 0, INV), ("T", -1, INV), ("B", -1, INV), ("dtype", 7, INV),
    ("gate", gdn.GDN_GATE_CHANNEL, UNS), ("gate", 3, INV), ("gate", -1, INV), ("hk", 2, INV), ("hk", 6, INV),
    ("scale", float("inf"), INV), ("T", 1 << 31, UNS)])
def test_chunk_bad_descriptor(lib, field, value, status):
    d = _desc()
    setattr(d, field, value)
    assert _fwd(lib, d) == status and lib.gdn_last_error().decode()


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "out"])
def test_chunk_null_pointer(lib, name):
    assert _fwd(lib, _desc(), **{name: None}) == INV


@pytest.mark.parametrize("name,off", [("q", 8), ("k", 8), ("v", 8), ("out", 8), ("g", 2), ("h0", 8), ("fin", 8)])
def test_chunk_misaligned(lib, name, off):
    kw = {"h0": {"h0": 10}, "fin": {"fin": 10}}.get(name, {})
    assert _fwd(lib, _desc(), off={name: off}, **kw) == INV and "aligned" in lib.gdn_last_error().decode()


def test_chunk_refusals(lib):
    d = _desc()
    assert _fwd(lib, d, snap=32) == INV and _fwd(lib, d, snap=-64) == INV
    assert _fwd(lib, d, snap=64) == INV  # no buffer
    assert _fwd(lib, d, cu=8, n=2) == INV  # packed needs B == 1
    one = _desc(B=1)
    assert _fwd(lib, one, cu=8, n=-1) == INV
    assert _fwd(lib, one, cu=8, n=2, snap=64, snaps=9) == UNS
    assert _fwd(lib, one, cu=8, n=2, off={"cu": 2}) == INV
    assert _fwd(lib, d, ws=None) == WS and _fwd(lib, d, ws_bytes=64) == WS
    assert _fwd(lib, d, off={"ws": 64}) == WS


@pytest.mark.parametrize("kw", [dict(out=0), dict(out=2), dict(out=3), dict(h0=10, out=10), dict(fin=10, out=10),
                                dict(fin=2), dict(fin=10, snaps=10, snap=64), dict(ws=0), dict(ws=5),
                                dict(fin=7), dict(h0=7)])
def test_chunk_overlaps(lib, kw):
    assert _fwd(lib, _desc(), **kw) == INV and "overlap" in lib.gdn_last_error().decode()


def test_chunk_final_state_partly_over_initial(lib):
    assert _fwd(lib, _desc(), h0=10, fin=10, off={"fin": 64}) == INV


def test_chunk_no_sequences_is_a_no_op(lib):
    assert _fwd(lib, _desc(B=0), ws=None) == gdn.GDN_OK
    assert _fwd(lib, _desc(B=1, T=0), cu=8, n=0, ws=None) == gdn.GDN_OK


def test_chunk_no_sequences_takes_no_planning(lib):
    """Without sequences there are no segments to weigh up, however many tokens each would have (2^26 chunks
    here, each of which would count as a split to look at)."""
    n = ctypes.c_size_t()
    d = _desc(B=0, T=1 << 32)
    start = time.perf_counter()
    assert lib.gdn_linattn_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)) == gdn.GDN_OK
    assert _fwd(lib, d, ws=None) == gdn.GDN_OK
    assert time.perf_counter() - start < 0.05


def test_no_barrier_over_part_of_a_block():
    """The roles of the tensor-core kernels leave their loops where a wait gives up, each on its own.  A
    barrier that counts some of the block's warps would hold those that reach it for good (the barrier
    of the whole block at the kernels' ends is reached by all), so the kernels have none."""
    text = open(os.path.join(ROOT, "gated_delta_rule_64_b200", "csrc", "linattn_tc.cu")).read()
    code = re.sub(r"//[^\n]*", "", text)
    assert "mbar_wait(" in code and not re.search(r"named_bar|bar\.sync|barrier\.|bar\.arrive", code)


def test_workspace_size(lib):
    n = ctypes.c_size_t()
    size = lambda d, N: (lib.gdn_linattn_workspace_size(ctypes.byref(d), N, ctypes.byref(n)), n.value)[1]  # noqa: E731
    assert size(_desc(), 2) == 256  # short sequences are not split
    state = 128 * 128 * 4
    long = size(_desc(B=1, T=262144, H=16), 1)
    assert long >= 2 * 16 * state  # at least two segments
    # many short packed sequences: room for the longest packing, not for a state per sequence
    assert size(_desc(B=1, T=65536, H=2), 4096) < 4096 * 2 * state
    assert lib.gdn_linattn_workspace_size(ctypes.byref(_desc()), 2, None) == INV
    assert lib.gdn_linattn_workspace_size(ctypes.byref(_desc()), -1, ctypes.byref(n)) == INV
    assert lib.gdn_linattn_workspace_size(None, 2, ctypes.byref(n)) == INV


def test_decode_refusals(lib):
    def call(d, off=(), null=None, out=5, state=4):
        p = [_p(i, 8 if i in off else 0) for i in (0, 1, 2, 3)] + [_p(state), _p(out)]
        if null is not None:
            p[null] = None
        return lib.gdn_linattn_decode_step(ctypes.byref(d), *p, None)
    d = _desc(T=1)
    assert call(_desc(T=2)) == INV
    assert call(_desc(T=1, gate=gdn.GDN_GATE_CHANNEL)) == UNS
    assert call(_desc(T=1, dk=96)) == UNS
    for i in range(6):
        assert call(d, null=i) == INV
    for i in (0, 1, 2):
        assert call(d, off=(i,)) == INV
    assert call(d, out=4) == INV and call(d, out=0) == INV and call(d, state=1) == INV
    assert call(_desc(B=0, T=1)) == gdn.GDN_OK


# ---------------------------------------------------------------------------
# gdn_qk_norm_rope
# ---------------------------------------------------------------------------

def _rope(lib, *, rows=10, hq=4, hk=2, dim=128, rot=128, inter=0, dtype=gdn.GDN_BF16, qs=None, ks=None, eps=1e-6,
          off=0.0, ptr=None, shift=None):
    d = gdn.GdnQkRopeDesc(rows, hq, hk, dim, rot, inter, dtype, hq * dim if qs is None else qs,
                          hk * dim if ks is None else ks, eps, off)
    at = dict(q=0, k=1, pos=2, freq=3, qw=4, kw=5, qo=6, ko=7)
    at.update(ptr or {})
    p = [_p(at[n], (shift or {}).get(n, 0)) for n in ("q", "k", "pos", "freq", "qw", "kw", "qo", "ko")]
    return lib.gdn_qk_norm_rope(ctypes.byref(d), *p, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(hq=0), INV), (dict(hk=-1), INV), (dict(dim=96), UNS), (dict(rot=144), UNS),
    (dict(rot=24), UNS), (dict(rot=-16), UNS), (dict(inter=2), INV), (dict(dtype=5), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(off=float("inf")), INV), (dict(qs=256), INV), (dict(qs=516), INV),
    (dict(ks=260), INV), (dict(rows=1 << 31), UNS),
    (dict(ptr={"q": None}), INV), (dict(ptr={"k": None}), INV), (dict(ptr={"qo": None}), INV),
    (dict(ptr={"ko": None}), INV), (dict(ptr={"pos": None}), INV), (dict(ptr={"freq": None}), INV),
    (dict(shift={"q": 8}), INV), (dict(shift={"ko": 4}), INV), (dict(shift={"pos": 2}), INV),
    (dict(shift={"qw": 2}), INV),
    (dict(ptr={"ko": 6}), INV), (dict(ptr={"qo": 1}), INV), (dict(ptr={"ko": 0}), INV),
    (dict(ptr={"qo": 0}, qs=1024), INV), (dict(ptr={"qo": 0}, shift={"qo": 16}), INV), (dict(ptr={"qo": 2}), INV)])
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status and lib.gdn_last_error().decode()


def test_rope_no_tokens_is_a_no_op(lib):
    assert _rope(lib, rows=0) == gdn.GDN_OK


def test_rope_wrapper_layouts():
    x = torch.zeros(2, 5, 1024)
    assert gdn._token_rows("q", x[..., :512].unflatten(-1, (4, 128))) == 1024
    assert gdn._token_rows("q", x[:, :1, :512].unflatten(-1, (4, 128))) == 5 * 1024
    assert gdn._token_rows("q", x[:1, :1, :512].unflatten(-1, (4, 128))) == 512
    with pytest.raises(ValueError):
        gdn._token_rows("q", x[:, :3, :512].unflatten(-1, (4, 128)))  # uneven over (B, T)
    with pytest.raises(ValueError):
        gdn._token_rows("q", x.unflatten(-1, (8, 128))[:, :, ::2])
    with pytest.raises(ValueError):
        gdn._token_rows("q", x[..., :512].unflatten(-1, (128, 4)).transpose(-1, -2))


# ---------------------------------------------------------------------------
# gdn_beam_select, gdn_state_reorder
# ---------------------------------------------------------------------------

def _beam(lib, *, B=2, W=4, V=1000, K=8, dtype=gdn.GDN_F32, stride=None, ptr=None, shift=None, ws_bytes=1 << 30):
    d = gdn.GdnBeamDesc(B, W, V, K, dtype, V if stride is None else stride)
    at = dict(x=0, s=1, os=2, op=3, ot=4, ws=5)
    at.update(ptr or {})
    p = {n: _p(at[n], (shift or {}).get(n, 0)) for n in at}
    return lib.gdn_beam_select(ctypes.byref(d), p["x"], p["s"], p["os"], p["op"], p["ot"], p["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(W=0), INV), (dict(W=65), INV), (dict(V=0), INV), (dict(K=0), INV), (dict(K=65), INV),
    (dict(V=1, W=4, K=5), INV), (dict(dtype=9), INV), (dict(stride=999), INV), (dict(W=64, V=1 << 25), UNS),
    (dict(ptr={"x": None}), INV), (dict(ptr={"os": None}), INV), (dict(ptr={"op": None}), INV),
    (dict(ptr={"ot": None}), INV), (dict(shift={"x": 2}), INV), (dict(shift={"s": 2}), INV),
    (dict(shift={"ot": 2}), INV), (dict(ptr={"ws": None}), WS), (dict(shift={"ws": 64}), WS),
    (dict(ws_bytes=16), WS), (dict(ptr={"op": 2}), INV), (dict(ptr={"ot": 0}), INV), (dict(ptr={"ws": 0}), INV),
    (dict(ptr={"os": 1}), INV)])
def test_beam_refusals(lib, kw, status):
    assert _beam(lib, **kw) == status and lib.gdn_last_error().decode()


def test_beam_no_requests_is_a_no_op(lib):
    assert _beam(lib, B=0, ptr={"ws": None}) == gdn.GDN_OK
    n = ctypes.c_size_t()
    d = gdn.GdnBeamDesc(1, 4, 1000, 8, gdn.GDN_F32, 1000)
    assert lib.gdn_beam_workspace_size(ctypes.byref(d), ctypes.byref(n)) == gdn.GDN_OK and n.value > 0
    assert lib.gdn_beam_workspace_size(ctypes.byref(d), None) == INV
    assert lib.gdn_beam_workspace_size(None, ctypes.byref(n)) == INV


@pytest.mark.parametrize("V", [(1 << 31) - 1, (1 << 31) - 2000, (1 << 31) - 16384, (1 << 31) - 16385])
@pytest.mark.parametrize("dtype", [gdn.GDN_F32, gdn.GDN_BF16])
def test_beam_workspace_of_the_largest_vocabulary(lib, V, dtype):
    """A key of 8 bytes for each of K = 8 continuations of a slice, and 8 bytes of sums: slices are 2,048
    logits or more."""
    n = ctypes.c_size_t()
    d = gdn.GdnBeamDesc(1, 1, V, 8, dtype, V)
    assert lib.gdn_beam_workspace_size(ctypes.byref(d), ctypes.byref(n)) == gdn.GDN_OK
    assert 64 <= n.value <= (V // 2048 + 1) * 72 + 512


def test_reorder_refusals(lib):
    def call(B=2, W=4, row=64, state=0, parent=1, so=0, po=0):
        return lib.gdn_state_reorder(_p(state, so), _p(parent, po), B, W, row, None)
    assert call(B=-1) == INV and call(W=0) == INV and call(W=65) == INV and call(row=24) == INV
    assert call(state=None) == INV and call(parent=None) == INV and call(so=8) == INV and call(po=2) == INV
    assert call(parent=0, po=256) == INV
    assert call(B=1 << 40) == UNS
    assert call(B=0) == gdn.GDN_OK and call(row=0) == gdn.GDN_OK


# ---------------------------------------------------------------------------
# The definitions
# ---------------------------------------------------------------------------

def test_recurrence_equals_the_masked_product():
    rng = np.random.default_rng(0)
    B, T, H, hk, dk, dv = 2, 9, 4, 2, 5, 3
    q, k, v = rng.normal(size=(B, T, hk, dk)), rng.normal(size=(B, T, hk, dk)), rng.normal(size=(B, T, H, dv))
    g, h0 = -rng.random((B, T, H)), rng.normal(size=(B, H, dv, dk))
    out, fin, snaps = L.linear_attention(q, k, v, g, h0, scale=0.5, snapshot_stride=3)
    G = g.cumsum(1)
    for h in range(H):
        w = np.exp(G[:, :, None, h] - G[:, None, :, h]) * np.tril(np.ones((T, T)))
        s = np.einsum("bid,bjd->bij", q[:, :, h // 2], k[:, :, h // 2]) * w
        inter = np.exp(G[:, :, h])[..., None] * np.einsum("bid,bed->bie", q[:, :, h // 2], h0[:, h])
        assert np.allclose(out[:, :, h], 0.5 * (s @ v[:, :, h] + inter))
        last = np.exp(G[:, -1:, h] - G[:, :, h])
        want = np.exp(G[:, -1, h])[:, None, None] * h0[:, h] + np.einsum("bj,bje,bjd->bed", last, v[:, :, h], k[:, :, h // 2])
        assert np.allclose(fin[:, h], want)
    assert np.allclose(snaps[:, 2], fin)


def test_packed_definition_equals_separate_sequences():
    rng = np.random.default_rng(1)
    q, k, v = (rng.normal(size=(1, 8, 2, 4)) for _ in range(3))
    g = -rng.random((1, 8, 2))
    out, fin, _ = L.linear_attention(q, k, v, g, cu_seqlens=[0, 3, 3, 7])
    for n, (a, b) in enumerate([(0, 3), (3, 3), (3, 7)]):
        o, f, _ = L.linear_attention(q[:, a:b], k[:, a:b], v[:, a:b], g[:, a:b])
        assert np.allclose(out[:, a:b], o) and np.allclose(fin[n], f[0])
    assert np.isnan(out[:, 7]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_adds_angles(interleaved):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(1, 1, 1, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    at = lambda p: L.norm_rope(x, np.array([[p]]), f, eps=0.0, interleaved=interleaved)  # noqa: E731
    assert np.allclose(np.linalg.norm(at(7)), np.sqrt(64))
    assert np.allclose((at(5) * at(9)).sum(), (at(0) * at(4)).sum())  # depends on the distance alone
    assert np.allclose(at(3)[..., 32:], at(0)[..., 32:])


def test_beam_definition():
    x = np.log(np.array([[[0.5, 0.25, 0.25], [0.9, 0.05, 0.05]]]))
    s, p, t = L.beam_select(x, np.log([[0.5, 0.25]]), 4)
    assert np.allclose(np.exp(s), [[0.25, 0.225, 0.125, 0.125]])
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 0, 1, 2]]
    s, p, t = L.beam_select(x, np.array([[-np.inf, np.nan]]), 4)  # dead beams: index order
    assert np.isneginf(s).all() and p.tolist() == [[0, 0, 0, 1]] and t.tolist() == [[0, 1, 2, 0]]
