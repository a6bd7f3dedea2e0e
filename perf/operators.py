"""What is measured of the decayed linear attention and of the operators around it.

Five operators, each in a plain form of elementary torch operations (``own`` false) and as the
calls that a user makes of the library (``own`` true):

  chunk    gdn_linattn_chunk_fwd    prompts: S_t = a_t S_{t-1} + v_t k_t^T, o_t = S_t (scale q_t)
  decode   gdn_linattn_decode_step  one token of every live sequence, the state in place
  rope     gdn_qk_norm_rope         norm of every query and key head, then the position rotation
  beam     gdn_beam_select          the best continuations over beams and vocabulary
  reorder  gdn_state_reorder        recurrent states moved to the beams that go on with them
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64  # tokens of a chunk in the plain form


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------

def _chunk(B, T, H, hk, dk, dv, dtype, gate, stride=0, lens="", h0=True):
    return {"op": "chunk", "B": B, "T": T, "H": H, "hk": hk, "dk": dk, "dv": dv, "dtype": dtype, "gate": gate,
            "stride": stride, "lens": lens, "h0": h0}


def _decode(B, H, hk, dk, dv, dtype, gate):
    return {"op": "decode", "B": B, "H": H, "hk": hk, "dk": dk, "dv": dv, "dtype": dtype, "gate": gate}


def _rope(B, T, hq, hk, d, rot, dtype, interleaved, vcols, far):
    return {"op": "rope", "B": B, "T": T, "hq": hq, "hk": hk, "d": d, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "vcols": vcols, "far": far}


def _beam(B, W, V, K, dtype, pad):
    return {"op": "beam", "B": B, "W": W, "V": V, "K": K, "dtype": dtype, "pad": pad}


def _reorder(B, W, H, dk, dv):
    return {"op": "reorder", "B": B, "W": W, "H": H, "dk": dk, "dv": dv}


def listed():
    return [
        # a short fp32 prompt, where the launches count
        dict(_chunk(1, 256, 2, 2, 64, 64, "f32", "token"), name="chunk tiny f32"),
        # an ordinary batch of prompts
        dict(_chunk(4, 4096, 16, 16, 128, 128, "bf16", "token"), name="chunk prefill"),
        # one very long document, a fixed decay for each head, states kept every 8192 tokens
        dict(_chunk(1, 262144, 16, 16, 128, 128, "bf16", "const", stride=8192, h0=False), name="chunk long const"),
        # packed prompts of ragged lengths, query/key heads shared by pairs of value heads
        dict(_chunk(1, 0, 32, 16, 128, 128, "bf16", "token",
                    lens="5111,16023,801,9990,1,13333,0,7717"), name="chunk packed ragged"),
        # one live sequence: the smallest step
        dict(_decode(1, 16, 16, 128, 128, "bf16", "const"), name="decode one"),
        # a full batch of live sequences
        dict(_decode(256, 32, 32, 128, 128, "bf16", "token"), name="decode batch"),
        # the prompts of "chunk prefill": q and k as slices of the layer's mixed projection
        dict(_rope(4, 4096, 16, 16, 128, 128, "bf16", False, 2048, False), name="rope prefill"),
        # a decode step at far positions, fewer key heads, half of each head rotated
        dict(_rope(256, 1, 32, 8, 128, 64, "bf16", False, 1024, True), name="rope decode"),
        # one request, a small vocabulary
        dict(_beam(1, 4, 32000, 8, "f32", 0), name="beam one"),
        # a batch of requests, a large vocabulary padded to a multiple of 64
        dict(_beam(32, 8, 128009, 16, "bf16", 55), name="beam batch"),
        # one request's states of one layer
        dict(_reorder(1, 4, 16, 64, 64), name="reorder one"),
        # a batch's states of one layer
        dict(_reorder(32, 8, 32, 128, 128), name="reorder batch"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    H = rng.choice([h for h in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32) if h <= most])
    return H, rng.choice([h for h in range(1, H + 1) if H % h == 0])


def draw(rng):
    op = rng.choice(["chunk", "chunk", "decode", "rope", "beam", "reorder"])
    if op == "chunk":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if dtype == "bf16" and rng.random() < 0.7:
            dk = dv = 128
        else:
            dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        H, hk = _heads(rng, 32)
        # token-heads in all, at most an eighth of the longest listed case (a hundredth in fp32)
        most = (40_000 if dtype == "f32" else 500_000) // H
        gate = rng.choice(["token", "token", "const"])
        if rng.random() < 0.4:
            n, total = rng.randint(1, 12), _log_int(rng, 16, most)
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
            return _chunk(1, 0, H, hk, dk, dv, dtype, gate, lens=",".join(map(str, lens)), h0=rng.random() < 0.5)
        B = _log_int(rng, 1, 8)
        T = _log_int(rng, 1, max(1, most // B))
        stride = rng.choice([0, 0, 64 * rng.randint(1, 40)])
        return _chunk(B, T, H, hk, dk, dv, dtype, gate, stride=stride, h0=rng.random() < 0.5)
    if op == "decode":
        H, hk = _heads(rng, 32)
        return _decode(_log_int(rng, 1, 256), H, hk, rng.choice([64, 128]), rng.choice([64, 128]),
                       rng.choice(["bf16", "bf16", "f32"]), rng.choice(["token", "const"]))
    if op == "rope":
        hq = rng.choice([1, 2, 3, 4, 8, 16, 24, 32])
        hk = rng.choice([h for h in range(1, hq + 1) if hq % h == 0])
        d = rng.choice([64, 128, 256])
        rot = rng.choice([d, d, d // 2, d // 4])
        rows = _log_int(rng, 1, max(1, 16384 * 32 * 128 // ((hq + hk) * d)))
        B = rng.choice([b for b in (1, 2, 3, 5, 8) if b <= rows])
        return _rope(B, rows // B, hq, hk, d, rot, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.4,
                     rng.choice([0, hk * d]), rng.random() < 0.3)
    if op == "beam":
        W = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        V = _log_int(rng, 500, 200_000)
        B = _log_int(rng, 1, max(1, min(64, 32 * 8 * 128_000 // (W * V))))
        return _beam(B, W, V, rng.choice([W, 2 * W]), rng.choice(["f32", "bf16"]), rng.choice([0, 0, (-V) % 64]))
    W = rng.choice([2, 3, 4, 5, 8, 12, 16])
    H = rng.choice([1, 2, 4, 8, 16, 32])
    return _reorder(_log_int(rng, 1, max(1, 256 // W)), W, H, rng.choice([64, 128]), rng.choice([64, 128]))


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------

def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-30)


def _lengths(case):
    return [int(n) for n in case["lens"].split(",")] if case["lens"] else []


def _slopes(H, device):
    """log of a fixed decay for each head: -2^(-8 (h + 1) / H), from -0.7 to -1/256 for many heads."""
    h = torch.arange(1, H + 1, device=device, dtype=torch.float32)
    return -torch.exp2(-8.0 * h / H)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1_000_003 + 17)
    normal = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    op, s = case["op"], {"case": dict(case)}
    if op in ("chunk", "decode"):
        td, H, hk, dk, dv = DTYPES[case["dtype"]], case["H"], case["hk"], case["dk"], case["dv"]
        lens = _lengths(case) if op == "chunk" else []
        B, T = (1, sum(lens)) if lens else (case["B"], case["T"] if op == "chunk" else 1)
        N = len(lens) or B
        s["q"], s["k"] = _unit(normal(B, T, hk, dk)).to(td), _unit(normal(B, T, hk, dk)).to(td)
        s["v"] = normal(B, T, H, dv).to(td)
        if case["gate"] == "const":
            # drawn a little around the usual slopes, so that another seed gives other decays
            s["g"] = _slopes(H, dev) * torch.exp(0.1 * normal(H))
        else:
            s["g"] = -torch.nn.functional.softplus(normal(B, T, H) - 2.0)
        s["scale"] = dk ** -0.5
        if op == "decode":
            s["state"] = 0.02 * normal(N, H, dv, dk)
            return s
        s["h0"] = 0.02 * normal(N, H, dv, dk) if case["h0"] else None
        s["cu"] = None
        if lens:
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu"], s["lens"] = torch.tensor(cu, dtype=torch.int32, device=dev), lens
    elif op == "rope":
        B, T, hq, hk, d = case["B"], case["T"], case["hq"], case["hk"], case["d"]
        x = normal(B, T, (hq + hk) * d + case["vcols"]).to(DTYPES[case["dtype"]])  # [q heads | k heads | the rest]
        s["q"] = x[..., :hq * d].unflatten(-1, (hq, d))
        s["k"] = x[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
        s["qw"], s["kw"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
        start = torch.randint(0, 260_000 if case["far"] else 1, (B, 1), generator=gen, device=dev)
        s["pos"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        s["inv_freq"] = 10_000.0 ** (-torch.arange(0, case["rot"], 2, device=dev).float() / case["rot"])
    elif op == "beam":
        B, W, V = case["B"], case["W"], case["V"]
        full = (2.0 * normal(B, W, V + case["pad"])).to(DTYPES[case["dtype"]])
        banned = torch.rand(full.shape, generator=gen, device=dev) < 0.01  # tokens that a constraint rules out
        s["logits"] = full.masked_fill_(banned, float("-inf"))[..., :V]
        s["scores"] = -5.0 * torch.rand((B, W), generator=gen, device=dev)
    else:
        B, W = case["B"], case["W"]
        s["state"] = normal(B * W, case["H"], case["dv"], case["dk"])
        s["parent"] = torch.randint(0, W, (B, W), generator=gen, device=dev, dtype=torch.int32)
    return s


# --------------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------------

def _prefix(tot, U, S0):
    """States before item 0 .. n and after the last: S_{c+1} = exp(tot_c) S_c + U_c over axis 2.
    tot (N, H, n) in 64 bits, U (N, H, n, E), S0 (N, H, E); returns (N, H, n + 1, E)."""
    N, H, n, E = U.shape
    if n <= CHUNK:
        D = torch.cat([tot.new_zeros(N, H, 1), tot.cumsum(-1)], -1)
        reach = torch.arange(n + 1, device=U.device)[:, None] > torch.arange(n, device=U.device)[None, :]
        M = torch.exp((D[..., :, None] - D[..., None, 1:]).masked_fill(~reach, float("-inf"))).float()
        return M @ U + torch.exp(D).float()[..., None] * S0[:, :, None]
    pad = -n % CHUNK
    tot = torch.nn.functional.pad(tot, (0, pad))
    U = torch.nn.functional.pad(U, (0, 0, 0, pad))
    blocks = (n + pad) // CHUNK
    tot, U = tot.reshape(N, H, blocks, CHUNK), U.reshape(N, H * blocks, CHUNK, E)
    local = _prefix(tot.reshape(N, H * blocks, CHUNK), U, U.new_zeros(N, H * blocks, E))
    local = local.reshape(N, H, blocks, CHUNK + 1, E)
    starts = _prefix(tot.sum(-1), local[..., -1, :], S0)
    D = tot.cumsum(-1)
    inside = local[..., 1:, :] + torch.exp(D).float()[..., None] * starts[:, :, :blocks, None, :]
    return torch.cat([S0[:, :, None], inside.reshape(N, H, blocks * CHUNK, E)[:, :, :n]], 2)


def _linattn(q, k, v, g, S0, scale, stride):
    """q, k (N, T, H, dk), v (N, T, H, dv), g (N, T, H), all fp32; S0 (N, H, dv, dk)."""
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    pad = -T % CHUNK
    nc = (T + pad) // CHUNK
    rows = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).reshape(N, nc, CHUNK, H, -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v, g = rows(q), rows(k), rows(v), rows(g[..., None])[..., 0]
    G = g.double().cumsum(-1)
    tot = G[..., -1]
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    P = scale * (q @ k.transpose(-1, -2))
    P = P * torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~causal, float("-inf"))).float()
    U = (v * torch.exp(tot[..., None] - G).float()[..., None]).transpose(-1, -2) @ k
    S = _prefix(tot, U.reshape(N, H, nc, dv * dk), S0.reshape(N, H, dv * dk)).reshape(N, H, nc + 1, dv, dk)
    o = P @ v + (scale * torch.exp(G).float())[..., None] * (q @ S[:, :, :nc].transpose(-1, -2))
    o = o.permute(0, 2, 3, 1, 4).reshape(N, nc * CHUNK, H, dv)[:, :T]
    snaps = None
    if stride:
        snaps = S[:, :, stride // CHUNK::stride // CHUNK][:, :, :T // stride].transpose(1, 2)
    return o, S[:, :, nc], snaps


def _plain_chunk(s):
    c = s["case"]
    td, H = s["q"].dtype, c["H"]
    rep = H // c["hk"]
    q, k = (x.float().repeat_interleave(rep, 2) for x in (s["q"], s["k"]))
    v = s["v"].float()
    g = s["g"].expand(v.shape[:3]) if s["g"].dim() == 1 else s["g"]
    if s["cu"] is None:
        S0 = s["h0"] if s["h0"] is not None else v.new_zeros(v.shape[0], H, c["dv"], c["dk"])
        o, fin, snaps = _linattn(q, k, v, g, S0, s["scale"], c["stride"])
        return (o.to(td), fin) + (() if snaps is None else (snaps,))
    lens, cu = s["lens"], s["cu"].long()
    N, longest, total = len(lens), max(max(lens), 1), v.shape[1]
    S0 = s["h0"] if s["h0"] is not None else v.new_zeros(N, H, c["dv"], c["dk"])
    t = torch.arange(longest, device=v.device)
    inside = t[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + t[None, :]).clamp_max(total - 1)
    take = lambda x: x[0][at] * inside.reshape(N, longest, *([1] * (x.dim() - 2)))  # noqa: E731
    o, fin, _ = _linattn(take(q), take(k), take(v), take(g), S0, s["scale"], 0)
    seq = torch.repeat_interleave(torch.arange(N, device=v.device), cu[1:] - cu[:-1], output_size=total)
    row = torch.arange(total, device=v.device)
    return o[seq, row - cu[seq]][None].to(td), fin


def _plain_decode(s):
    c = s["case"]
    rep = c["H"] // c["hk"]
    q, k = (x[:, 0].float().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
    g = s["g"] if s["g"].dim() == 1 else s["g"][:, 0]
    S = s["state"]
    S.mul_(torch.exp(g)[..., None, None])
    S.add_(s["v"][:, 0].float()[..., :, None] * k[..., None, :])
    o = (S @ (s["scale"] * q)[..., None])[..., 0]
    return o.to(s["q"].dtype)[:, None], S


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    angle = s["pos"].double()[..., None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        a, b = a * cos - b * sin, b * cos + a * sin
        head = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        out.append(torch.cat([head, y[..., rot:]], -1).to(x.dtype))
    return tuple(out)


def _plain_beam(s):
    c = s["case"]
    B, W, V, K = c["B"], c["W"], c["V"], c["K"]
    x = s["logits"].double()
    m = x.max(-1, keepdim=True).values
    score = s["scores"].double()[..., None] + (x - (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))))
    score = torch.where(torch.isnan(score), float("-inf"), score).reshape(B, W * V)
    # the K best, the lowest index first among equals: everything above the K-th value, then its equals in order
    kth = torch.topk(score, K, -1).values[:, -1:]
    rank = (score > kth).long() + (score >= kth).long()
    index = torch.arange(W * V, device=x.device)
    best = torch.topk(rank * (W * V) - index, K, -1).indices.sort(-1).values
    value, order = torch.gather(score, -1, best).sort(dim=-1, descending=True, stable=True)
    best = torch.gather(best, -1, order)
    return value.float(), (best // V).int(), (best % V).int()


def _plain_reorder(s):
    c = s["case"]
    B, W = c["B"], c["W"]
    at = torch.arange(B, device=s["parent"].device)[:, None] * W + s["parent"]
    s["state"] = s["state"][at.reshape(-1)]
    return s["state"]


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"chunk": _plain_chunk, "decode": _plain_decode, "rope": _plain_rope, "beam": _plain_beam,
                "reorder": _plain_reorder}[op](s)
    from gated_delta_rule_64_b200 import gdn
    c = s["case"]
    if op == "chunk":
        out, fin, snaps = gdn.gdn_linattn_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"],
                                                    scale=s["scale"], snapshot_stride=c["stride"])
        return (out, fin) + (() if snaps is None else (snaps,))
    if op == "decode":
        return gdn.gdn_linattn_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"]), s["state"]
    if op == "rope":
        return gdn.gdn_qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["qw"], s["kw"], eps=1e-6,
                                    interleaved=c["interleaved"])
    if op == "beam":
        return gdn.gdn_beam_select(s["logits"], s["scores"], c["K"])
    return gdn.gdn_state_reorder(s["state"], s["parent"])


def work(case):
    c, op = case, case["op"]
    el = {"f32": 4, "bf16": 2}.get(case.get("dtype"), 4)
    if op in ("chunk", "decode"):
        H, hk, dk, dv = c["H"], c["hk"], c["dk"], c["dv"]
        lens = _lengths(c) if op == "chunk" else []
        rows = sum(lens) if lens else c["B"] * (c["T"] if op == "chunk" else 1)
        N = len(lens) or c["B"]
        state = 4 * N * H * dv * dk
        states = 2 * state if op == "decode" or c["h0"] else state
        if op == "chunk" and c["stride"]:
            states += state * (c["T"] // c["stride"])
        gate = 4 * H * (rows if c["gate"] == "token" else 1)
        return {"bytes": rows * el * (2 * hk * dk + 2 * H * dv) + gate + states, "flops": 4 * rows * H * dk * dv}
    if op == "rope":
        n = c["B"] * c["T"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * n * el + 4 * c["B"] * c["T"] + 8 * c["d"] + 2 * c["rot"], "flops": 7 * n}
    if op == "beam":
        n = c["B"] * c["W"] * c["V"]
        return {"bytes": n * el + 4 * c["B"] * c["W"] + 12 * c["B"] * c["K"], "flops": 4 * n}
    # with parents drawn alike, W - 1 of W beams change, and a beam is some other's parent with 1 - (1 - 1/W)^(W-1)
    W, row = c["W"], 4 * c["H"] * c["dv"] * c["dk"]
    moved = c["B"] * row * (W * (1 - (1 - 1 / W) ** (W - 1)) + W - 1)
    return {"bytes": moved + 4 * c["B"] * W, "flops": 0}


# --------------------------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------------------------

def _recurrence(q, k, v, a, S, every):
    """Token by token: q, k (T, U, dk), v (T, U, dv), a (T, U), S (U, dv, dk) in 64 bits."""
    T = q.shape[0]
    out, kept = v.new_empty(T, v.shape[1], v.shape[2], 1), []
    a, q, k, v = a[..., None, None], q[..., :, None], k[..., None, :], v[..., :, None]
    for t in range(T):
        S.mul_(a[t])
        S.baddbmm_(v[t], k[t])
        torch.bmm(S, q[t], out=out[t])
        if every and (t + 1) % every == 0:
            kept.append(S.clone())
    return out[..., 0], kept


def _exact_chunk(case, s):
    H, rep = case["H"], case["H"] // case["hk"]
    dk, dv = case["dk"], case["dv"]
    q, k = (x.double().repeat_interleave(rep, 2) for x in (s["q"], s["k"]))
    q, v = q * s["scale"], s["v"].double()
    B, T = v.shape[:2]
    a = torch.exp(s["g"].double())
    a = a.expand(B, T, H)
    lens = _lengths(case) or [T] * B
    N, longest = len(lens), max(lens)
    # every sequence beside the others, the short ones followed by tokens that change nothing
    wide = lambda x, fill: torch.full((longest, N) + x.shape[1:], fill, dtype=x.dtype, device=x.device)  # noqa: E731
    flat = [x.reshape(B * T, *x.shape[2:]) for x in (q, k, v, a)]
    beside, at = [wide(x, 1.0 if i == 3 else 0.0) for i, x in enumerate(flat)], 0
    for n, length in enumerate(lens):
        for x, y in zip(flat, beside):
            y[:length, n] = x[at:at + length]
        at += length
    S = torch.zeros(N * H, dv, dk, dtype=torch.float64, device=v.device)
    if s["h0"] is not None:
        S += s["h0"].double().reshape(N * H, dv, dk)
    qs, ks, vs, al = (x.reshape(longest, N * H, *x.shape[3:]) for x in beside)
    o, kept = _recurrence(qs, ks, vs, al, S, case["stride"])
    o = o.reshape(longest, N, H, dv)
    out = torch.cat([o[:length, n] for n, length in enumerate(lens)]).reshape(B, T, H, dv)
    got = (out, S.reshape(N, H, dv, dk))
    if case["stride"]:
        shape = (N, H, dv, dk)
        got += (torch.stack([x.reshape(shape) for x in kept], 1) if kept else S.new_zeros(N, 0, H, dv, dk),)
    return got


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "chunk":
        return _exact_chunk(case, s)
    if op == "decode":
        rep = case["H"] // case["hk"]
        q, k = (x[:, 0].double().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
        a = torch.exp(s["g"].double()) if s["g"].dim() == 1 else torch.exp(s["g"][:, 0].double())
        S = torch.einsum("bhi,bhj->bhij", s["v"][:, 0].double(), k) + s["state"].double() * a[..., None, None]
        return torch.einsum("bhij,bhj->bhi", S, q * s["scale"])[:, None], S
    if op == "rope":
        rot, got = case["rot"], []
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[..., None] * s["inv_freq"].double())[..., None, :]
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.double()
            y = w.double() * y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["d"] + 1e-6)
            z, tail = y[..., :rot], y[..., rot:]
            pairs = z.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else z.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            got.append(torch.cat([z.flatten(-2), tail], -1))
        return tuple(got)
    if op == "beam":
        value = s["scores"].double()[..., None] + torch.log_softmax(s["logits"].double(), -1)
        value, at = value.flatten(1).sort(dim=-1, descending=True, stable=True)
        value, at = value[:, :case["K"]], at[:, :case["K"]]
        return value, torch.div(at, case["V"], rounding_mode="floor").int(), torch.remainder(at, case["V"]).int()
    B, W = case["B"], case["W"]
    old = s["state"].double().reshape(B, W, -1)
    return torch.stack([old[b, s["parent"][b].long()] for b in range(B)]).reshape(s["state"].shape)
