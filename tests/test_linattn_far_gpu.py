"""The operators of include/gdn_linattn.h where offsets pass 2^31 elements or 2^32 bytes, segments are cut into
many parts, and in calls that combine options: against 64-bit forms on the GPU.

Tolerances: those of test_linattn_gpu.py (relative L2), except for states that very many tokens add up to, TOL_LONG:
the tensor cores add 256 tokens in one accumulator, 48 products, each cut off by 2^-24 of it on average while it
grows to its size (2/3 on average): 1.9e-6; the chunks of a segment that follow one another, 2,110, 2^-24
sqrt(2110) = 2.7e-6; the products' own 1.3e-6 and the decays' 1.6e-6: together below 1e-5."""
import pytest
import torch

from gated_delta_rule_64_b200 import gdn

pytestmark = pytest.mark.gpu

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


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()
