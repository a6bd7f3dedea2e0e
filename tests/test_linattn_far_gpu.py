"""The operators of include/gdn_linattn.h where offsets pass 2^31 elements or 2^32 bytes, segments are cut into
many parts, and in calls that combine options: against 64-bit forms on the GPU.

Tolerances: those of test_linattn_gpu.py (relative L2), except for states that very many tokens add up to, TOL_LONG:
the tensor cores add 256 tokens in one accumulator, 48 products, each cut off by 2^-24 of it on average while it
grows to its size (2/3 on average): 1.9e-6; the chunks of a segment that follow one another, 2,110, 2^-24
sqrt(2110) = 2.7e-6; the products' own 1.3e-6 and the decays' 1.6e-6: together below 1e-5."""
import numpy as np
import pytest
import torch

from gated_delta_rule_64_b200 import gdn
from oracle import linattn as L
from tests.gpu_util import rel_l2

pytestmark = pytest.mark.gpu

TOL_F32 = 5e-6
TOL_BF16 = 3 * 2.0 ** -8
TOL_LONG = 1e-5


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _chunked(q, k, v, g, S, C=64):
    """(T,h,d) in 64 bits, one head per column: outputs and the final state."""
    out = torch.empty_like(v)
    for t in range(0, v.shape[0], C):
        Q, K, V, G = (x[t:t + C].transpose(0, 1) for x in (q, k, v, g))
        G = G.cumsum(1)
        P = (Q @ K.mT) * torch.exp((G[:, :, None] - G[:, None, :]).tril()).tril()
        out[t:t + C] = (P @ V + torch.exp(G)[..., None] * (Q @ S.mT)).transpose(0, 1)
        S = torch.exp(G[:, -1])[:, None, None] * S + (V * torch.exp(G[:, -1:] - G)[..., None]).mT @ K
    return out, S


def _err(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("gate", ["token", "const"])
@pytest.mark.parametrize("in_place", [False, True])
def test_chunk_segments_of_many_parts(gate, in_place):
    """Two sequences of 270,000 tokens and 37 heads: two segments each, of 135,040 tokens, which are more than
    the eight parts of 16,384 tokens whose states are fetched together.  The last head reaches element
    2.5e9 of v and out."""
    B, T, H, d = 2, 270_000, 37, 128
    assert gdn.gdn_linattn_workspace_size(B, T, H, d, d, B, hk=1) >= 2 * B * 9 * H * d * d * 4
    gen = _gen(1)
    r = lambda *s, dtype=torch.bfloat16: torch.randn(s, device="cuda", generator=gen, dtype=dtype)  # noqa: E731
    q, k = (_unit(r(B, T, 1, d, dtype=torch.float32)).bfloat16() for _ in range(2))
    v, h0 = r(B, T, H, d), r(B, H, d, d, dtype=torch.float32)
    if gate == "token":  # sums of -4 or so over the sequence in the heads looked at
        g = -3e-5 * torch.rand(B, T, H, device="cuda", generator=gen)
    else:
        g = -torch.exp2(-torch.arange(H, device="cuda") / 2.0)
    first = h0.double()
    ws = torch.empty(gdn.gdn_linattn_workspace_size(B, T, H, d, d, B, hk=1), dtype=torch.uint8, device="cuda")
    out, fin, _ = gdn.gdn_linattn_chunk_fwd(q, k, v, g, h0, final_state=h0 if in_place else True, workspace=ws)
    assert gdn.gdn_chunk_status(ws) == (gdn.GDN_OK, gdn.GDN_DEV_OK)
    for b in range(B):
        heads = [0, H - 1]
        x = q[b].double().expand(T, 2, d), k[b].double().expand(T, 2, d), v[b, :, heads].double()
        o, f = _chunked(*x, (g[b, :, heads] if gate == "token" else g[heads].expand(T, 2)).double(), first[b, heads])
        for i, h in enumerate(heads):
            assert _err(out[b, :, h], o[:, i]) <= TOL_BF16, (b, h)
            assert _err(fin[b, h], f[i]) <= TOL_LONG, (b, h, _err(fin[b, h], f[i]))


@pytest.mark.parametrize("gate", ["token", "const"])
def test_chunk_cuda_cores_equal_gates_over_a_long_segment(gate):
    """270,000 fp32 tokens of 74 heads in two segments of 4,220 chunks; the state kept 64 tokens into the second
    one is the first one's sum.  A sum of n = 135,040 products in a row, each rounded to 2^-23 / sqrt(12) of the
    sum so far (rms), which grows like its root: 2^-23 sqrt(n / 24) = 8.9e-6, and 1.6e-6 for the decays: 1.1e-5.
    The gate is one whose multiples round the same way in 32 bits, thousands of times."""
    T, H, d, at = 270_000, 74, 64, 135_104
    gen = _gen(9)
    q, k = (_unit(torch.randn(1, T, 1, d, device="cuda", generator=gen)) for _ in range(2))
    v = torch.randn(1, T, H, d, device="cuda", generator=gen)
    x = -1.5274936e-05
    g = torch.full((H,) if gate == "const" else (1, T, H), x, device="cuda")
    _, _, snaps = gdn.gdn_linattn_chunk_fwd(q, k, v, g, snapshot_stride=at)
    for h in (0, H - 1):
        w = torch.exp(float(np.float32(x)) * torch.arange(at - 1, -1, -1, device="cuda", dtype=torch.float64))
        want = (v[0, :at, h].double() * w[:, None]).T @ k[0, :at, 0].double()
        assert _err(snaps[0, 0, h], want) <= 1.1e-5, _err(snaps[0, 0, h], want)


def test_chunk_states_of_a_long_memory():
    """262,144 tokens that hardly fade (sums of -0.13): every segment's state is a sum over all that came before,
    none of which a biased rounding may shorten."""
    T, H, d = 262_144, 16, 128
    gen = _gen(7)
    q, k = (_unit(torch.randn(1, T, 1, d, device="cuda", generator=gen)).bfloat16() for _ in range(2))
    v = torch.randn(1, T, H, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    g = -1e-6 * torch.rand(1, T, H, device="cuda", generator=gen)
    out, fin, _ = gdn.gdn_linattn_chunk_fwd(q, k, v, g)
    heads = [0, 7, 15]
    n = len(heads)
    o, f = _chunked(q[0].double().expand(T, n, d), k[0].double().expand(T, n, d), v[0, :, heads].double(),
                    g[0, :, heads].double(), torch.zeros(n, d, d, dtype=torch.float64, device="cuda"))
    for i, h in enumerate(heads):
        assert _err(out[0, :, h], o[:, i]) <= TOL_BF16
        assert _err(fin[0, h], f[i]) <= TOL_LONG, (h, _err(fin[0, h], f[i]))


@pytest.mark.parametrize("gate", [-1.5e-5, -1.1e-4, -1.9e-3])
def test_chunk_equal_gates_over_many_chunks(gate):
    """Gates per token that are all alike, 2,110 chunks to a segment: every chunk's decay has the same rounding,
    which must not be taken 2,110 times.  The decays' share of the tolerance, 1.6e-6, is that of one."""
    B, T, H, d = 2, 270_000, 37, 128
    gen = _gen(8)
    q, k = (_unit(torch.randn(B, T, 1, d, device="cuda", generator=gen)).bfloat16() for _ in range(2))
    v, h0 = (torch.randn(s, device="cuda", generator=gen, dtype=t) for s, t in
             (((B, T, H, d), torch.bfloat16), ((B, H, d, d), torch.float32)))
    g = torch.full((B, T, H), gate, device="cuda")
    out, fin, _ = gdn.gdn_linattn_chunk_fwd(q, k, v, g, h0)
    for b, h in ((0, 0), (1, H - 1)):
        o, f = _chunked(*(x[b].double() for x in (q, k)), v[b, :, h:h + 1].double(), g[b, :, h:h + 1].double(),
                        h0[b, h:h + 1].double())
        assert _err(out[b, :, h], o[:, 0]) <= TOL_BF16
        assert _err(fin[b, h], f[0]) <= TOL_LONG, _err(fin[b, h], f[0])


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("bf16", 128, 64)])
def test_chunk_cuda_cores_past_2_to_31_elements(dtype, dk, dv):
    """1,040,000 tokens of 33 heads, 64 wide.  A token's decay is 0.25 or more, so what lies 1,000 tokens back
    (2^-360) is gone."""
    T, H, n = 1_040_000, 33, 2000
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = _gen(2)
    q, k = (_unit(torch.randn(1, T, 1, dk, device="cuda", generator=gen)).to(td) for _ in range(2))
    v = torch.randn(1, T, H, dv, device="cuda", generator=gen, dtype=td)
    g = -0.25 - torch.rand(1, T, H, device="cuda", generator=gen)
    out, fin, _ = gdn.gdn_linattn_chunk_fwd(q, k, v, g)
    zero = torch.zeros(H, dv, dk, dtype=torch.float64, device="cuda")
    o, f = _chunked(q[0, -n:].double().expand(n, H, dk), k[0, -n:].double().expand(n, H, dk), v[0, -n:].double(),
                    g[0, -n:].double(), zero)
    assert _err(fin[0], f) <= TOL_F32
    assert _err(out[0, -1000:], o[-1000:]) <= (TOL_F32 if dtype == "f32" else 2.0 ** -8)
    o, _ = _chunked(q[0, :n].double().expand(n, H, dk), k[0, :n].double().expand(n, H, dk), v[0, :n].double(),
                    g[0, :n].double(), zero)
    assert _err(out[0, :n], o) <= (TOL_F32 if dtype == "f32" else 2.0 ** -8)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_chunk_snapshots_and_final_state_in_place_of_a_split(dtype, d):
    """The start states are chained by a kernel of their own here, and the states at every 320 tokens are kept."""
    rng = np.random.default_rng(3)
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    q, k, v = _unit(t(2, 6000, 1, d)).to(td), _unit(t(2, 6000, 1, d)).to(td), t(2, 6000, 2, d).to(td)
    g, h0 = -0.02 * t(2, 6000, 2).abs(), t(2, 2, d, d)
    o, f, s = L.linear_attention(q, k, v, g, h0, snapshot_stride=320)
    state = h0.cuda()
    out, _, snaps = gdn.gdn_linattn_chunk_fwd(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state, final_state=state,
                                              snapshot_stride=320)
    assert rel_l2(state, f) <= TOL_F32 and rel_l2(snaps, s) <= TOL_F32
    assert rel_l2(out, o) <= (TOL_F32 if dtype == "f32" else TOL_BF16)


def test_decode_states_past_2_to_31_elements():
    B, H, d = 4100, 32, 128
    gen = _gen(4)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    q, k, v, g = r(B, 1, H, d), r(B, 1, H, d), r(B, 1, H, d), -r(B, 1, H).abs()
    state = r(B, H, d, d)
    at = [0, B - 1]
    s0 = state[at].double()
    out = gdn.gdn_linattn_decode_step(q, k, v, g, state)
    x = [y[at, 0].double() for y in (q, k, v, g)]
    want = torch.exp(x[3])[..., None, None] * s0 + x[2][..., :, None] * x[1][..., None, :]
    assert _err(state[at], want) <= TOL_F32
    assert _err(out[at, 0], (want @ x[0][..., None])[..., 0]) <= TOL_F32


def test_rope_past_2_to_31_elements_in_place():
    T, hq, d = 66_000, 128, 256
    gen = _gen(5)
    q = torch.randn(1, T, hq, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    f = (10000.0 ** (-torch.arange(128) / 128.0)).cuda()
    at = [0, 1, T // 2, T - 1]
    want = L.norm_rope(q[:, at], pos[:, at], f)
    got, _ = gdn.gdn_qk_norm_rope(q, q[:, :, :0], pos, f, q_out=q)
    assert got.data_ptr() == q.data_ptr() and rel_l2(got[:, at], want) <= 2.0 ** -8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rope_queries_only(dtype, interleaved, d):
    """No key heads: an empty k, and nothing of it is touched."""
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    for B, T, hq in ((1, 1, 1), (2, 33, 7), (300, 1, 16)):
        gen = _gen(T)
        q = torch.randn(B, T, hq, d, device="cuda", generator=gen).to(td)
        pos = torch.randint(0, 5000, (B, T), device="cuda", generator=gen, dtype=torch.int32)
        f = (10000.0 ** (-torch.arange(d // 4) / (d // 4))).float().cuda()
        w = torch.randn(d, device="cuda", generator=gen)
        y, none = gdn.gdn_qk_norm_rope(q, q[:, :, :0], pos, f, w, interleaved=interleaved)
        assert none.shape == (B, T, 0, d)
        want = L.norm_rope(q, pos, f, w, interleaved=interleaved)
        assert rel_l2(y, want) <= (3e-6 if dtype == "f32" else 2.0 ** -8)


def test_reorder_past_2_to_32_bytes():
    """Twelve rows of 400 MB; one parent twice, one beam that nobody goes on with."""
    state = torch.randint(0, 1 << 30, (12, 100_000_000), device="cuda", dtype=torch.int32, generator=_gen(6))
    parent = torch.tensor([[1, 0, 3, 3], [0, 1, 2, 3], [3, 3, 0, 1]], dtype=torch.int32, device="cuda")
    want = state[(parent.long() + 4 * torch.arange(3, device="cuda")[:, None]).flatten()]
    assert torch.equal(gdn.gdn_state_reorder(state, parent), want)


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()
