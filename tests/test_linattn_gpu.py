"""GPU parity of the operators of include/gdn_linattn.h against their 64-bit definitions.

Tolerances (relative L2 over a tensor), from the arithmetic:
  fp32 results.  Sums of n <= 2^9 products in flight at a time: 2^-24 sqrt(n) = 1.3e-6 with random
    signs; the decays' exponentials, 2^-22, on arguments good to 2^-24 * 32 (terms whose argument
    is larger are below 2^-32 of the sum): 1.6e-6.  Together below 5e-6.
  bf16 outputs.  The output's own rounding is at most 2^-8 relative.  On the tensor cores the scores
    and the state are rounded once each before the second product, 2^-8 of each part: 3 * 2^-8.
  norm and rotation, fp32: mean square 2^-24 * 8 at most, rsqrt 2^-22, angle 2^-22 of a turn in the
    sine and cosine (1.5e-6 of the head's length at worst): 3e-6.
"""
import ctypes

import numpy as np
import pytest
import torch

from gated_delta_rule_64_b200 import gdn
from oracle import linattn as L
from tests.gpu_util import rel_l2

pytestmark = pytest.mark.gpu

TOL_F32 = 5e-6
TOL_BF16 = 3 * 2.0 ** -8


def _inputs(B, T, H, hk, dk, dv, dtype, gate="token", h0=True, seed=0, lengths=None, decay=1.0):
    rng = np.random.default_rng(seed)
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    cu = None
    if lengths is not None:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
        B, T = 1, int(cu[-1])
    N = len(lengths) if lengths is not None else B
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(t(B, T, hk, dk)).to(td), unit(t(B, T, hk, dk)).to(td), t(B, T, H, dv).to(td)
    if gate == "token":
        g = -decay * torch.nn.functional.softplus(t(B, T, H) - 2)
    else:
        g = -decay * torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    return dict(q=q, k=k, v=v, g=g, h0=0.3 * t(N, H, dv, dk) if h0 else None, cu=cu)


def _run(x, **kw):
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    ws = torch.empty(gdn.gdn_linattn_workspace_size(*x["v"].shape[:3], x["q"].shape[3], x["v"].shape[3],
                                                    _n(x), dtype=x["q"].dtype,
                                                    hk=x["q"].shape[2]), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # what the workspace holds before the call does not matter
    got = gdn.gdn_linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], workspace=ws, **kw)
    torch.cuda.synchronize()
    assert gdn.gdn_chunk_status(ws) == (gdn.GDN_OK, gdn.GDN_DEV_OK)
    return got


def _n(x):
    return x["cu"].numel() - 1 if x["cu"] is not None else x["q"].shape[0]


def _check(x, scale=1.0, snapshot_stride=0):
    out, fin, snaps = _run(x, scale=scale, snapshot_stride=snapshot_stride)
    o, f, s = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"], x["cu"], scale=scale,
                                 snapshot_stride=snapshot_stride)
    tol = TOL_F32 if x["q"].dtype == torch.float32 else TOL_BF16
    assert rel_l2(out, o) <= tol, ("out", rel_l2(out, o))
    assert rel_l2(fin, f) <= TOL_F32, ("state", rel_l2(fin, f))
    if snapshot_stride:
        assert rel_l2(snaps, s) <= TOL_F32, ("snapshots", rel_l2(snaps, s))


SIZES = [(1, 1, 1, 1), (2, 31, 3, 1), (1, 64, 2, 2), (3, 65, 4, 2), (1, 130, 2, 1), (2, 257, 6, 3)]


@pytest.mark.parametrize("B,T,H,hk", SIZES)
@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("f32", 128, 64), ("f32", 64, 128), ("f32", 128, 128),
                                         ("bf16", 64, 128), ("bf16", 128, 128)])
@pytest.mark.parametrize("gate", ["token", "const"])
def test_chunk(B, T, H, hk, dtype, dk, dv, gate):
    _check(_inputs(B, T, H, hk, dk, dv, dtype, gate, h0=T % 2 == 1, seed=T), scale=0.7)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("gate,decay", [("token", 1.0), ("token", 0.01), ("const", 1.0), ("const", 0.0)])
def test_chunk_long_split_with_snapshots(dtype, d, gate, decay):
    """Long enough for segments (the workspace shows it), states kept every 192 tokens; with weak decays
    the whole sequence reaches its end, with decay 0 nothing fades."""
    x = _inputs(1, 4000, 2, 1, d, d, dtype, gate, seed=7, decay=decay)
    assert gdn.gdn_linattn_workspace_size(1, 4000, 2, d, d, 1, dtype=x["q"].dtype, hk=1) > 2 * 2 * d * d * 4
    _check(x, snapshot_stride=192)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("gate,decay", [("token", 1.0), ("token", 0.002), ("const", 0.0)])
def test_chunk_very_many_segments(dtype, d, gate, decay):
    """One head over 40,000 tokens: so many segments that their start states are chained by a kernel of
    their own; a weak decay carries every segment's state into all that follow."""
    _check(_inputs(1, 40_000, 1, 1, d, d, dtype, gate, seed=16, decay=decay))


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("gate,decay", [("token", 1.0), ("token", 0.01)])
@pytest.mark.parametrize("lengths", [[5], [70, 1, 0, 300, 64, 129], [0, 0, 33], [2500, 3, 1100, 0, 64, 1024, 2049]])
def test_chunk_packed(dtype, d, gate, decay, lengths):
    _check(_inputs(1, 0, 4, 2, d, d, dtype, gate, h0=True, seed=len(lengths), lengths=lengths, decay=decay))


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_chunk_packed_many_sequences(dtype, d):
    """More sequences than a block has threads, empty ones among them, and one of several segments."""
    lengths = [(7 * n) % 5 for n in range(700)] + [3000] + [0, 2] * 30
    _check(_inputs(1, 0, 1, 1, d, d, dtype, h0=True, seed=17, lengths=lengths, decay=0.05))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunk_strong_decays_and_resets(dtype):
    """Gates that erase the state (-1e4, -300) beside gates of zero: nothing overflows, nothing leaks."""
    x = _inputs(1, 300, 2, 2, 128, 128, dtype, seed=3)
    x["g"][:, 50] = -1e4
    x["g"][:, 64] = -300.0
    x["g"][:, 200:230] = -40.0
    x["g"][:, 231:260] = 0.0
    _check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("log2_decay", [-40.0, -61.0, -95.0, -99.0, -101.0, -119.0, -121.0])
def test_chunk_large_values_under_strong_decays(dtype, log2_decay):
    """Queries, keys and values that no norm holds down, while a chunk's decay takes a good part of the
    exponent's range: factors of one side alone (2^99) would carry the products past it.  Sums of q k v
    are 2^26 2^14 2^6 here."""
    x = _inputs(1, 200, 2, 1, 128, 128, dtype, seed=19)
    x["q"], x["k"], x["v"] = x["q"] * 3000, x["k"] * 3000, x["v"] * 10000
    x["g"][:] = log2_decay * float(np.log(2.0)) / 64
    _check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("log2_decay", [-40.0, -100.0, -119.0, -121.0])
def test_chunk_small_values_under_strong_decays(dtype, log2_decay):
    """The other end: contributions |q . k| |v| near 2^-53.  On the tensor cores a factor of 2^-60 meets them, and
    2^-126 is the least normal value, so that what is lost there (below 2^-64) is rarer than one in 2^10
    of them, each 2^-11 of the others."""
    x = _inputs(1, 200, 2, 1, 128, 128, dtype, seed=23)
    x["v"], x["h0"] = x["v"] * 2.0 ** -50, x["h0"] * 2.0 ** -50
    x["g"][:] = log2_decay * float(np.log(2.0)) / 64
    _check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("erase", [torch.finfo(torch.float32).min, float("-inf"), -106.0])
@pytest.mark.parametrize("T", [200, 3000])
def test_chunk_gates_of_the_lowest_value(dtype, erase, T):
    """Gates that erase the state do not take the decays beside them along (sums of such gates are not
    finite); a fixed gate of that value leaves each token with itself."""
    x = _inputs(1, T, 2, 1, 128, 128, dtype, seed=18, decay=0.1)
    for t in (0, 5, 70, 71, 130, 191, 199):
        x["g"][:, t] = erase
    if T > 200:
        x["g"][:, 1000:1003] = erase
    _check(x)
    x["g"] = torch.tensor([erase, -0.01])
    _check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunk_rows_outside_sequences_and_their_neighbours(dtype):
    """Rows behind the last sequence stay as they were, and what lies there (NaN, infinities) reaches
    no result; neither does a NaN in another sequence."""
    lengths = [70, 10, 100]
    x = _inputs(1, 0, 2, 2, 128, 128, dtype, seed=4, lengths=lengths)
    pad = 37
    for n in ("q", "k", "v", "g"):
        bad = torch.full((1, pad) + tuple(x[n].shape[2:]), float("nan"), dtype=x[n].dtype)
        bad[:, ::2] = float("inf")
        x[n] = torch.cat([x[n], bad], 1)
    x["v"][:, 70:80] = float("nan")  # the middle sequence
    x["k"][:, 70:80] = float("inf")
    out = torch.full(x["v"].shape, 3.0, dtype=x["v"].dtype, device="cuda")
    _, fin, _ = _run(x, out=out)
    assert torch.equal(out[:, 180:], torch.full_like(out[:, 180:], 3.0))
    part = lambda a, b: L.linear_attention(*(x[n][:, a:b] for n in "qkvg"), None if x["h0"] is None else  # noqa: E731
                                           x["h0"][[0 if a == 0 else 2]])
    tol = TOL_F32 if dtype == "f32" else TOL_BF16
    for n, (a, b) in ((0, (0, 70)), (2, (80, 180))):
        o, f, _ = part(a, b)
        assert rel_l2(out[:, a:b], o) <= tol and rel_l2(fin[n:n + 1], f) <= TOL_F32


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_chunk_final_state_in_place_and_continued(dtype, d):
    """Two calls that hand the state on, in place, equal one call over all tokens."""
    x = _inputs(2, 500, 2, 2, d, d, dtype, seed=5)
    o, f, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"])
    state = x["h0"].cuda()
    outs = []
    for a, b in ((0, 170), (170, 500)):
        p = [x[n][:, a:b].contiguous().cuda() for n in "qkvg"]
        outs.append(gdn.gdn_linattn_chunk_fwd(*p, state, final_state=state)[0])
    torch.cuda.synchronize()
    assert rel_l2(torch.cat(outs, 1), o) <= (TOL_F32 if dtype == "f32" else TOL_BF16)
    assert rel_l2(state, f) <= TOL_F32


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("decay", [0.02, 0.0])
def test_chunk_long_in_place_split(dtype, d, decay):
    """The final state replaces the initial one, which every segment's start depends on."""
    x = _inputs(1, 6000, 3, 1, d, d, dtype, seed=15, decay=decay)
    _, f, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"])
    state = x["h0"].cuda()
    gdn.gdn_linattn_chunk_fwd(*(x[n].cuda() for n in "qkvg"), state, final_state=state)
    assert rel_l2(state, f) <= TOL_F32


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("h0,final,combined", [(False, "none", False), (True, "none", False), (False, "new", False),
                                               (True, "new", False), (True, "initial", True)])
def test_chunk_split_start_states(dtype, d, h0, final, combined):
    """A split sequence's blocks add up their start states themselves, with or without an initial and a final
    state; the combine kernel runs where the final state replaces the initial one."""
    x = _inputs(1, 6000, 2, 1, d, d, dtype, seed=22, h0=h0, decay=0.02)
    p = [x[n].cuda() for n in "qkvg"] + [x["h0"].cuda() if h0 else None]
    gdn.profile_read()
    gdn.profile_enable(True)
    out, fin, _ = gdn.gdn_linattn_chunk_fwd(*p, final_state={"none": None, "new": True, "initial": p[4]}[final])
    gdn.profile_enable(False)
    names = gdn.profile_read()
    assert any("state" in n for n in names), names  # split
    assert ("gdn_linattn_combine" in names) == combined, names
    o, f, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"])
    assert rel_l2(out, o) <= (TOL_F32 if dtype == "f32" else TOL_BF16)
    assert fin is None or rel_l2(fin, f) <= TOL_F32


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_empty_prompt_copies_the_state(d):
    h0 = torch.randn(2, 3, d, d, device="cuda")
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out, fin, _ = gdn.gdn_linattn_chunk_fwd(e(2, 0, 3, d), e(2, 0, 3, d), e(2, 0, 3, d),
                                            torch.empty(2, 0, 3, device="cuda"), h0)
    assert out.shape == (2, 0, 3, d) and torch.equal(fin, h0)
    _, fin, _ = gdn.gdn_linattn_chunk_fwd(e(2, 0, 3, d), e(2, 0, 3, d), e(2, 0, 3, d),
                                          torch.zeros(3, device="cuda"))
    assert not fin.any()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("gate", [gdn.GDN_GATE_HEAD, gdn.GDN_GATE_CONST])
@pytest.mark.parametrize("packed", [False, True])
def test_chunk_without_tokens_needs_no_inputs(dtype, d, gate, packed):
    """The C entry point takes a call without tokens whose q, k, v, gates and output are NULL: the final states
    are the initial ones."""
    lib = gdn.load_library()
    h0, fin = torch.randn(2, 3, d, d, device="cuda"), torch.full((2, 3, d, d), 5.0, device="cuda")
    ws = torch.full((4096,), 255, dtype=torch.uint8, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    desc = gdn.GdnDesc(1 if packed else 2, 0, 3, d, d, gdn.GDN_F32 if dtype == "f32" else gdn.GDN_BF16, gate, 1.0, 0)
    st = lib.gdn_linattn_chunk_fwd(ctypes.byref(desc), None, None, None, None, h0.data_ptr(),
                                   cu.data_ptr() if packed else None, 2, 0, None, fin.data_ptr(), None,
                                   ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == gdn.GDN_OK, lib.gdn_last_error().decode()
    assert gdn.gdn_chunk_status(ws) == (gdn.GDN_OK, gdn.GDN_DEV_OK) and torch.equal(fin, h0)


@pytest.mark.parametrize("cu", [[0, 90, 40, 200], [-5, 300, 7, 1000], [200, 0, 0, 0], [7, 60, 61, 100]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunk_wrong_offsets_stay_inside(cu, dtype):
    """Offsets that are not non-decreasing from 0 give some result without touching anything else;
    sequences with sound offsets of their own (the last case starts behind row 0) keep theirs."""
    x = _inputs(1, 200, 2, 2, 128, 128, dtype, seed=6, h0=False)
    x["cu"] = torch.tensor(cu, dtype=torch.int32)
    guard = torch.full((3, 200, 2, 128), 5.0, dtype=x["v"].dtype, device="cuda")
    _run(x, out=guard[1:2])
    assert (guard[0] == 5).all() and (guard[2] == 5).all()
    if cu[0] == 7:
        o, _, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], None, cu)
        assert rel_l2(guard[1:2, 7:100], o[:, 7:100]) <= (TOL_F32 if dtype == "f32" else TOL_BF16)
        assert (guard[1, :7] == 5).all() and (guard[1, 100:] == 5).all()


def test_chunk_captured_and_replayed_with_new_inputs():
    """Two captured calls that share a workspace, replayed after their inputs changed."""
    xs = [_inputs(1, 5000, 2, 2, 128, 128, "bf16", seed=s, decay=0.05) for s in (8, 9, 10)]
    bufs = [{n: t.cuda() for n, t in x.items() if t is not None} for x in xs[:2]]
    ws = torch.empty(gdn.gdn_linattn_workspace_size(1, 5000, 2, 128, 128, 1), dtype=torch.uint8, device="cuda")
    run = lambda d: gdn.gdn_linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], workspace=ws)  # noqa: E731
    for d in bufs:
        run(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [run(d) for d in bufs]
    for n in "qkvg":
        bufs[1][n].copy_(xs[2][n])
    bufs[1]["h0"].copy_(xs[2]["h0"])
    graph.replay()
    torch.cuda.synchronize()
    for x, (out, fin, _) in ((xs[0], outs[0]), (xs[2], outs[1])):
        o, f, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"])
        assert rel_l2(out, o) <= TOL_BF16 and rel_l2(fin, f) <= TOL_F32


def test_chunk_two_streams_at_once_and_repeatable():
    """Two calls in flight on two streams (a workspace each) give what each gives alone, bit for bit."""
    xs = [{n: None if t is None else t.cuda() for n, t in
           _inputs(2, 3000, 4, 2, 128, 128, "bf16", seed=s).items()} for s in (11, 12)]
    run = lambda x, **kw: gdn.gdn_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], **kw)  # noqa: E731
    alone = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    both = [[run(x, stream=s) for x, s in zip(xs, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for got in both:
        for (o, f, _), (o1, f1, _) in zip(got, alone):
            assert torch.equal(o, o1) and torch.equal(f, f1)


def test_calls_on_a_given_stream_keep_their_tensors():
    """Inputs freed right after a call on another stream are not overwritten before it has run: memory that
    the current stream asks for next is not theirs."""
    side = torch.cuda.Stream()
    x = _inputs(1, 20_000, 4, 4, 128, 128, "bf16", seed=19)
    o, f, _ = gdn.gdn_linattn_chunk_fwd(*(x[n].cuda() for n in "qkvg"), x["h0"].cuda())
    torch.cuda.synchronize()
    for _ in range(3):
        args = [x[n].cuda() for n in "qkvg"] + [x["h0"].cuda()]
        torch.cuda.synchronize()
        got = gdn.gdn_linattn_chunk_fwd(*args, stream=side)
        sizes = [a.shape for a in args]
        del args
        junk = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in sizes]
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], f)
        del junk, got


# ---------------------------------------------------------------------------
# gdn_linattn_decode_step
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("gate", ["token", "const"])
def test_decode_steps(dtype, dk, dv, gate):
    x = _inputs(3, 5, 4, 2, dk, dv, dtype, gate, seed=dk + dv)
    state = x["h0"].cuda()
    outs = []
    for t in range(5):
        g = x["g"] if gate == "const" else x["g"][:, t:t + 1]
        p = [y.contiguous().cuda() for y in (x["q"][:, t:t + 1], x["k"][:, t:t + 1], x["v"][:, t:t + 1], g)]
        outs.append(gdn.gdn_linattn_decode_step(*p, state, scale=0.5))
    torch.cuda.synchronize()
    o, f, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"], scale=0.5)
    assert rel_l2(torch.cat(outs, 1), o) <= (TOL_F32 if dtype == "f32" else 2.0 ** -8)
    assert rel_l2(state, f) <= TOL_F32


def test_decode_with_erasing_and_full_gates():
    x = _inputs(2, 1, 3, 3, 128, 128, "f32", seed=21)
    x["g"][0] = -1e6
    x["g"][1] = 0.0
    state = x["h0"].cuda()
    out = gdn.gdn_linattn_decode_step(*(x[n][:, 0].contiguous().cuda() for n in "qkvg"), state)
    o, f, _ = L.linear_attention(x["q"], x["k"], x["v"], x["g"], x["h0"])
    assert rel_l2(out, o) <= TOL_F32 and rel_l2(state, f) <= TOL_F32


# ---------------------------------------------------------------------------
# gdn_qk_norm_rope
# ---------------------------------------------------------------------------

TOL_ROPE = 3e-6


def _rope_inputs(B, T, hq, hk, d, rot, dtype, seed=0, extra=0, far=0):
    rng = np.random.default_rng(seed)
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.from_numpy(rng.standard_normal((B, T, (hq + hk) * d + extra), dtype=np.float32)).to(td)
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)) for _ in range(2)]
    pos = torch.from_numpy(rng.integers(-far - 1, far + 100, size=(B, T), dtype=np.int64).astype(np.int32))
    f = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32))
    return x, w, pos, f


def _rope_check(x, w, pos, f, hq, hk, d, inter, offset=0.0, eps=1e-6, weights=True):
    xd = x.cuda()
    q, k = xd[..., :hq * d].unflatten(-1, (hq, d)), xd[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    ws = [t.cuda() for t in w] if weights else [None, None]
    got = gdn.gdn_qk_norm_rope(q, k, pos.cuda(), f.cuda() if len(f) else None, *ws, eps=eps, weight_offset=offset,
                               interleaved=inter)
    torch.cuda.synchronize()
    tol = TOL_ROPE if x.dtype == torch.float32 else 2.0 ** -8
    for y, src, wt in zip(got, (q, k), w):
        want = L.norm_rope(src, pos, f, wt if weights else None, eps=eps, weight_offset=offset, interleaved=inter)
        assert y.is_contiguous() and rel_l2(y, want) <= tol, rel_l2(y, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("share", [0, 0.25, 0.5, 1])
@pytest.mark.parametrize("inter", [False, True])
def test_rope(dtype, d, share, inter):
    for B, T, hq, hk in ((1, 1, 1, 1), (2, 7, 5, 2), (3, 1, 8, 8), (1, 401, 3, 1)):
        x, w, pos, f = _rope_inputs(B, T, hq, hk, d, int(share * d), dtype, seed=T, extra=64 * (T % 2))
        _rope_check(x, w, pos, f, hq, hk, d, inter)


@pytest.mark.parametrize("rot", [16, 48, 112])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_other_widths_offset_and_no_weights(rot, dtype):
    x, w, pos, f = _rope_inputs(2, 9, 4, 2, 128, rot, dtype, seed=rot)
    _rope_check(x, w, pos, f, 4, 2, 128, False, offset=1.0, eps=1e-5)
    _rope_check(x, w, pos, f, 4, 2, 128, True, weights=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_at_far_positions(dtype):
    x, w, pos, f = _rope_inputs(2, 50, 2, 2, 128, 128, dtype, seed=1, far=2 ** 31 - 200)
    _rope_check(x, w, pos, f, 2, 2, 128, False)


def test_rope_many_tokens_and_many_heads():
    x, w, pos, f = _rope_inputs(1, 20000, 2, 1, 64, 64, "bf16", seed=2)
    _rope_check(x, w, pos, f, 2, 1, 64, False)
    x, w, pos, f = _rope_inputs(1, 3, 300, 100, 64, 64, "bf16", seed=3)
    _rope_check(x, w, pos, f, 300, 100, 64, False)


def test_rope_zero_and_tiny_heads():
    """A head of zeros stays zero (eps keeps the norm finite); so does one of denormals, nearly."""
    x, w, pos, f = _rope_inputs(1, 4, 2, 2, 128, 128, "f32", seed=4)
    x[:, 0] = 0
    x[:, 1] *= 1e-30
    _rope_check(x, w, pos, f, 2, 2, 128, False)


def test_rope_in_place():
    x, w, pos, f = _rope_inputs(2, 33, 4, 4, 128, 64, "bf16", seed=5)
    q, k = (t.contiguous().cuda() for t in x.unflatten(-1, (8, 128)).split(4, 2))
    want = gdn.gdn_qk_norm_rope(q, k, pos.cuda(), f.cuda(), w[0].cuda(), w[1].cuda())
    got = gdn.gdn_qk_norm_rope(q, k, pos.cuda(), f.cuda(), w[0].cuda(), w[1].cuda(), q_out=q, k_out=k)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].data_ptr() == q.data_ptr()


# ---------------------------------------------------------------------------
# gdn_beam_select, gdn_state_reorder
# ---------------------------------------------------------------------------

def _beam_check(logits, scores, K):
    s, p, t = gdn.gdn_beam_select(logits.cuda(), None if scores is None else scores.cuda(), K)
    torch.cuda.synchronize()
    ws, wp, wt = L.beam_select(logits, scores, K)
    assert np.array_equal(p.cpu().numpy(), wp) and np.array_equal(t.cpu().numpy(), wt)
    got, fine = s.cpu().double().numpy(), np.isfinite(ws)
    assert np.array_equal(np.isneginf(got), ~fine)
    # a score of magnitude up to 2^5 is rounded to 2^-20 at most; the normaliser's fp32 exponentials: 2^-22
    assert np.all(np.abs(got[fine] - ws[fine]) <= 2e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,W,V,K", [(1, 1, 1, 1), (2, 3, 5, 4), (1, 4, 2, 8), (3, 4, 1000, 8), (2, 2, 8191, 64),
                                     (2, 5, 8193, 5), (1, 8, 50001, 16), (1, 64, 777, 64), (2, 1, 70000, 1)])
def test_beam_select(dtype, B, W, V, K):
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.normal(0, 2, size=(B, W, V)).astype(np.float32)).to(dtype)
    s = torch.from_numpy(-5 * rng.random((B, W), dtype=np.float32))
    _beam_check(x, s, K)
    _beam_check(x, None, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beam_ties_masks_and_dead_beams(dtype):
    x = torch.zeros(9, 4, 9000, dtype=dtype)                      # request 0: all equal
    s = torch.zeros(9, 4)
    x[1] = float("-inf")                                          # nothing allowed
    x[2] = float("-inf")
    x[2, 1, 8999] = 1.0                                           # one continuation, then index order
    x[3, :, 100:] = float("-inf")                                 # a mask that leaves 100 tokens
    x[3, :, :100] = torch.linspace(-3, 3, 100)
    x[4, 2, 17] = float("nan")                                    # that beam is dead
    x[5, 0, 17] = float("inf")                                    # that one too
    s[6, 0], s[6, 1] = float("-inf"), float("nan")                # two beams that had ended
    x[7] = torch.finfo(dtype).min                                 # masks of the type's lowest value
    x[7, 3, 4000:4004] = 2.0
    x[8] = -0.0
    x[8, :, 8200] = 0.0                                           # equal to its neighbours
    for K in (1, 8, 33):
        _beam_check(x, s, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [20, 1000, 9000])
def test_beam_scores_past_the_fp32_range_in_between(dtype, V):
    """A beam whose score less its normaliser passes the range (its continuations' scores do not), beside
    an ordinary one, with masked places that have to fill the last ranks."""
    x = torch.full((3, 2, V), torch.finfo(dtype).min, dtype=dtype)
    x[1:, 1] = torch.linspace(-2, 2, V).to(dtype)
    x[2, :, 5:] = float("-inf")
    s = torch.tensor([[3e38, 2e38], [3e38, -1.0], [3e38, -1.0]])
    for K in (1, 8, 33):
        _beam_check(x, s, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", [(40, 9001), (80, 16500)])
def test_beam_many_requests(dtype, B, V):
    """Enough beams for the larger slices; among them runs of equal values, masks, sorted logits, dead beams."""
    rng = np.random.default_rng(B)
    x = torch.from_numpy(rng.normal(0, 2, size=(B, 8, V)).astype(np.float32))
    x[1] = 0.0
    x[2] = float("-inf")
    x[2, 3, V - 1] = 1.0
    x[3] = torch.arange(V) / V
    x[4] = -torch.arange(V) / V
    x[5, :, 64:] = torch.finfo(dtype).min
    x[6, 2, 17], x[6, 3, 18] = float("nan"), float("inf")
    x[7] = torch.round(x[7])
    s = torch.from_numpy(-5 * rng.random((B, 8), dtype=np.float32))
    for K in (1, 16, 64):
        _beam_check(x.to(dtype), s, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [(1 << 31) - 1, (1 << 31) - 9000])
def test_beam_largest_vocabulary(dtype, V):
    """W V = 2^31 - 1, the most that one request may have: indices of the last slice pass the vocabulary's end
    and 2^31.  All logits but three are 0, so the normaliser is log(V - 3 + the three's exponentials); it is
    good to 2^-17, and the scores near -21 to half an fp32 step, 2^-20."""
    x = torch.zeros(1, 1, V, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    peaks = {V - 1: 3.0, (1 << 30) + 5: 2.5, 7: 2.0}
    for i, y in peaks.items():
        x[0, 0, i] = y
    score, parent, token = gdn.gdn_beam_select(x, None, 8)
    assert token[0].tolist() == [V - 1, (1 << 30) + 5, 7, 0, 1, 2, 3, 4] and not parent.any()
    lse = np.log(V - 3 + sum(np.exp(y) for y in peaks.values()))
    want = np.array([3.0, 2.5, 2.0] + [0.0] * 5) - lse
    assert np.abs(score[0].cpu().double().numpy() - want).max() <= 2.0 ** -17 + 2.0 ** -20
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(1, 300), (1, 40_009), (40, 128_009)])
def test_beam_log_sums(dtype, B, V):
    """The stated bound of a beam's log-sum, at logits where many small exponentials add up.  For a logit d
    below the slice's largest: its fp32 exponential is off by 2^-22 and by 2.25 d 2^-24 for the argument's two
    roundings and the constant's, up to three times 2^-22 over the rescalings (whose d add up); 40 additions of
    2^-24; d is log(16,384) = 9.7 on average at most.  Together (12 + 22 + 40) 2^-24 < 2^-17.  The score's own
    rounding is 2^-24 of it."""
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.zeros(B, 4, V)
    x[:, 1, 1:] = -9.6875
    x[:, 2] = -torch.linspace(0, 20, V)
    x[:, 3] = torch.randn(V, generator=torch.Generator().manual_seed(V)) * 4
    x = x.to(td)
    score, parent, token = (t.cpu() for t in gdn.gdn_beam_select(x.cuda(), None, 4))
    lse = torch.logsumexp(x[0].double(), -1)
    want = x[0].double() - lse[:, None]
    for b in (0, B - 1):
        at = want[parent[b].long(), token[b].long()]
        assert ((score[b].double() - at).abs() <= 2.0 ** -17 + 2.0 ** -24 * at.abs()).all()
    each = gdn.gdn_beam_select(x[:1].transpose(0, 1).contiguous().cuda(), None, 1)  # every beam on its own
    assert ((each[0][:, 0].cpu().double() - (x[0].double().max(-1)[0] - lse)).abs() <= 2.0 ** -17 + 2.0 ** -20).all()


def test_beam_first_step_and_strided_vocabulary():
    """All beams alike (the first step after a prompt): equal scores over beams, the first beam's come first;
    logits cut from rows of a padded vocabulary whose padding holds large values."""
    rng = np.random.default_rng(5)
    row = torch.from_numpy(rng.normal(0, 2, size=10001).astype(np.float32))
    full = torch.full((2, 4, 10048), 50.0)
    full[..., :10001] = row
    for dtype in (torch.float32, torch.bfloat16):
        wide = full.to(dtype).cuda()
        s, p, t = gdn.gdn_beam_select(wide[..., :10001], torch.zeros(2, 4, device="cuda"), 9)
        ws, wp, wt = L.beam_select(wide[..., :10001].cpu(), None, 9)
        assert np.array_equal(p.cpu().numpy(), wp) and np.array_equal(t.cpu().numpy(), wt)
    odd = torch.zeros(1, 2, 1003, device="cuda")[..., 1:1000]  # rows that start between 16-byte boundaries
    odd += torch.from_numpy(rng.normal(size=(1, 2, 999)).astype(np.float32)).cuda()
    s, p, t = gdn.gdn_beam_select(odd, None, 7)
    ws, wp, wt = L.beam_select(odd.cpu(), None, 7)
    assert np.array_equal(p.cpu().numpy(), wp) and np.array_equal(t.cpu().numpy(), wt)


def test_beam_sorted_and_equal_runs():
    """Rising and falling logits put the best values of a slice into few threads' hands; runs of equal
    values cross slices."""
    n = 20000
    up = torch.arange(n, dtype=torch.float32) / n
    x = torch.stack([up, up.flip(0), torch.round(up * 3), torch.round(up.flip(0) * 3)])[None]
    _beam_check(x, torch.tensor([[0.0, -0.1, -0.2, -0.3]]), 64)


@pytest.mark.parametrize("W", [1, 2, 3, 4, 7, 8, 13, 16, 20, 33, 64])
@pytest.mark.parametrize("shape", [(4,), (3, 64), (2, 64, 64)])
def test_state_reorder(W, shape):
    rng = np.random.default_rng(W)
    B = 3
    state = torch.from_numpy(rng.standard_normal((B * W,) + shape).astype(np.float32))
    parent = torch.from_numpy(rng.integers(0, W, size=(B, W)).astype(np.int32))
    parent[0] = torch.arange(W)          # nothing moves
    parent[1] = torch.arange(W).flip(0)  # every row swaps with another
    want = L.state_reorder(state.numpy(), parent.numpy())
    got = gdn.gdn_state_reorder(state.cuda(), parent.cuda())
    assert np.array_equal(got.cpu().numpy(), want)


def test_state_reorder_keeps_rows_with_parents_out_of_range_and_other_types():
    state = torch.arange(2 * 3 * 16, dtype=torch.bfloat16).reshape(6, 16)
    parent = torch.tensor([[-1, 3, 2 ** 31 - 1], [-2 ** 31, 0, 0]], dtype=torch.int32)
    got = gdn.gdn_state_reorder(state.cuda(), parent.cuda()).cpu()
    assert torch.equal(got, state[[0, 1, 2, 3, 3, 3]])


# ---------------------------------------------------------------------------
# Together, as they are used
# ---------------------------------------------------------------------------

def test_prompt_then_beam_search():
    """A layer's projections through norm and rotation, the prompt's linear attention, then three beam
    steps: each step's tokens through the single-token form, its continuations selected, the states moved
    to the beams that go on.  Every beam's outputs equal those of one pass over its own tokens."""
    rng = np.random.default_rng(33)
    H, hk, d, W, T, V, steps = 4, 2, 128, 3, 150, 500, 3
    C = 2 * hk * d + H * d
    proj = torch.from_numpy(rng.standard_normal((V, C), dtype=np.float32)).to(torch.bfloat16).cuda()  # of each token
    head = torch.from_numpy(rng.standard_normal((H * d, V), dtype=np.float32) * 0.2).cuda()
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda() for _ in range(2)]
    f = torch.from_numpy((10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)).cuda()
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1) / H).cuda()

    def layer_inputs(tokens, first):
        x = proj[tokens.long()]
        pos = (first + torch.arange(tokens.shape[1], device="cuda", dtype=torch.int32)).expand(tokens.shape).contiguous()
        q, k = gdn.gdn_qk_norm_rope(x[..., :hk * d].unflatten(-1, (hk, d)),
                                    x[..., hk * d:2 * hk * d].unflatten(-1, (hk, d)), pos, f, *w)
        return q, k, x[..., 2 * hk * d:].unflatten(-1, (H, d)).contiguous()

    prompt = torch.from_numpy(rng.integers(0, V, size=(1, T))).cuda()
    q, k, v = layer_inputs(prompt, 0)
    out, state, _ = gdn.gdn_linattn_chunk_fwd(q, k, v, g, scale=d ** -0.5)
    state = state.expand(W, H, d, d).contiguous()
    scores, parent, token = gdn.gdn_beam_select((out[:, -1].reshape(1, 1, -1).float() @ head), None, W)
    beams = torch.cat([prompt.expand(W, T), token.reshape(W, 1)], 1)
    for n in range(steps):
        q, k, v = layer_inputs(beams[:, -1:], T + n)
        out = gdn.gdn_linattn_decode_step(q, k, v, g, state, scale=d ** -0.5)
        ref_q, ref_k, ref_v = layer_inputs(beams, 0)
        o, s, _ = L.linear_attention(ref_q, ref_k, ref_v, g, scale=d ** -0.5)
        assert rel_l2(out[:, 0], o[:, -1]) <= 2.0 ** -8 and rel_l2(state, s) <= TOL_F32
        logits = (out.reshape(1, W, -1).float() @ head)
        want = L.beam_select(logits, scores, W)
        scores, parent, token = gdn.gdn_beam_select(logits, scores, W)
        assert np.array_equal(parent.cpu().numpy(), want[1]) and np.array_equal(token.cpu().numpy(), want[2])
        gdn.gdn_state_reorder(state, parent)
        beams = torch.cat([beams[parent[0].long()], token.reshape(W, 1)], 1)
