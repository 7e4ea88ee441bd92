"""What is measured of the latent attention operators, and in what form.

Four operators that serve a layer whose keys and values come from one shared
latent vector a token.  Each case names one of them and its sizes; `run`
computes it with elementary torch operations in fp32 (own = False) or by the
library's entry points (own = True), on the same inputs.

  append    the latent part of the joint down-projection's output, normalised
            (y = w * c / sqrt(mean c^2 + eps)) or as it is, and its rope part,
            rotated by the token's position, go into a paged cache; the rope
            part of the queries' heads is rotated in the same call.
  gather    cached tokens of every sequence as packed bf16 rows, which the
            up-projection expands.
  absorbed  attention in the latent space: all heads read the same keys
            (latent and rope part) and the same values (the latent):
            x[j] = scale * (ql . c[j] + qr . r[j]), out = sum_j softmax(x)[j] c[j];
            also the natural log of the sum of exponentials.
  expanded  attention of packed prompts over keys and values of every head
            (the up-projection's output) and the shared rope part.

L = 512 has rope parts of 64 and heads of 128 + 128, L = 256 half of each.
Cache: latents [blocks, block, L] in bf16, or in e4m3 with one power-of-two
fp32 scale for each token and 128 values [blocks, block, L / 128]; rope parts
[blocks, block, L / 8] in bf16.  A token's rotation takes pairs of neighbours
(2i, 2i + 1), or channels i and i + P/2, and a table of cosines and sines.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-4
EPS = 1e-6
# columns of the joint projection before the latent: the query's latent, as in a 2112-wide projection for L = 512
BEFORE = {512: 1536, 256: 768}


def listed():
    return [
        # one decode step of a batch: what the joint projection gives, and 8 heads of a shard
        {"name": "append_tokens_64", "op": "append", "L": 512, "cache": "bf16", "block": 64, "b": 64, "h": 8, "new": 1,
         "ctx": 1500, "ragged": True, "norm": True, "pairs": True},
        # prompts of different lengths behind a cached prefix, into 8 bits
        {"name": "append_prompts_4", "op": "append", "L": 512, "cache": "e4m3", "block": 64, "b": 4, "h": 32, "new": 4096,
         "ctx": 300, "ragged": True, "norm": False, "pairs": True},
        # the cached prefixes of a few short sequences, odd sizes
        {"name": "gather_short_7", "op": "gather", "L": 256, "cache": "bf16", "block": 16, "b": 7, "kv": 777, "ragged": True},
        # long prefixes out of 8 bits, for the next prompt chunk
        {"name": "gather_long_4", "op": "gather", "L": 512, "cache": "e4m3", "block": 64, "b": 4, "kv": 32768, "ragged": True},
        # one short sequence, one token: latency
        {"name": "absorbed_token_777", "op": "absorbed", "L": 256, "cache": "bf16", "block": 16, "b": 1, "h": 8, "new": 1,
         "kv": 777, "ragged": False},
        # a decode step of a ragged batch, heads split over GPUs
        {"name": "absorbed_shard_64x8192", "op": "absorbed", "L": 512, "cache": "bf16", "block": 64, "b": 64, "h": 16,
         "new": 1, "kv": 8192, "ragged": True},
        # a decode step with all heads on one GPU, 8-bit cache
        {"name": "absorbed_all_heads_32x4096", "op": "absorbed", "L": 512, "cache": "e4m3", "block": 64, "b": 32, "h": 128,
         "new": 1, "kv": 4096, "ragged": True},
        # a few long sequences
        {"name": "absorbed_long_4x65536", "op": "absorbed", "L": 512, "cache": "bf16", "block": 128, "b": 4, "h": 128,
         "new": 1, "kv": 65536, "ragged": False},
        # three drafted tokens of each sequence at once
        {"name": "absorbed_drafts_16x2048", "op": "absorbed", "L": 512, "cache": "e4m3", "block": 32, "b": 16, "h": 20,
         "new": 3, "kv": 2048, "ragged": True},
        # short prompts, odd sizes
        {"name": "expanded_short_9x150", "op": "expanded", "L": 256, "b": 9, "h": 5, "new": 150, "kv": 150, "ragged": True},
        # prompt chunks behind gathered prefixes
        {"name": "expanded_chunks_4x2048", "op": "expanded", "L": 512, "b": 4, "h": 32, "new": 2048, "kv": 4096,
         "ragged": True},
        # one long prompt
        {"name": "expanded_long_8192", "op": "expanded", "L": 512, "b": 1, "h": 32, "new": 8192, "kv": 8192,
         "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _held(case):
    """Scores, and cached values of the padded batch, that the plain form of a case holds."""
    if case["op"] in ("append", "gather"):
        return 0, 0
    return case["b"] * case["h"] * case["new"] * case["kv"], case["b"] * case["kv"] * case["L"] * case.get("h", 1)


def _within(case):
    """Costs no more than the operator's largest listed case."""
    cost = [tuple(work(c).values()) + _held(c) for c in listed() if c["op"] == case["op"]]
    return all(x <= max(top) for x, top in zip(tuple(work(case).values()) + _held(case), zip(*cost)))


def draw(rng):
    op = rng.choice(("append", "append", "gather", "absorbed", "absorbed", "absorbed", "expanded", "expanded"))
    while True:
        case = {"op": op, "L": rng.choice((256, 512, 512)), "b": _log(rng, 1, 128), "ragged": rng.random() < 0.7}
        if op != "expanded":
            case.update(cache=rng.choice(("bf16", "e4m3")), block=rng.choice((16, 32, 64, 128)))
        if op != "gather":
            case["h"] = _log(rng, 1, 128)
        if op == "append":
            case["new"] = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
            case["ctx"] = rng.choice((0, _log(rng, 1, 4096)))
            # codes next to a border would hang on the norm's last bit
            case.update(norm=case["cache"] == "bf16" and rng.random() < 0.7, pairs=rng.random() < 0.6)
        elif op == "gather":
            case["kv"] = _log(rng, 1, 65536)
        elif op == "absorbed":
            case["new"] = 1 if rng.random() < 0.6 else _log(rng, 2, 512)
            case["kv"] = case["new"] + _log(rng, 1, 65536) - 1
        else:
            case["new"] = _log(rng, 1, 8192)
            case["kv"] = case["new"] + rng.choice((0, _log(rng, 1, 8192)))
        if _within(case):
            return case


# ---- sizes that follow from a case alone

def _spread(most, i, b, ragged, least=1):
    """Length of sequence i of b: between a quarter of `most` and `most`."""
    if not ragged or b == 1:
        return most
    return max(least, most - (3 * most // 4) * ((i * 5 + 2) % b) // b)


def _lens(case):
    """(new tokens, tokens in all) of every sequence."""
    b, ragged = case["b"], case["ragged"]
    if case["op"] == "gather":
        kv = [_spread(case["kv"], i, b, ragged) for i in range(b)]
        return kv, kv
    new = [_spread(case["new"], i, b, ragged) for i in range(b)]
    if case["op"] == "append":
        return new, [n + (_spread(case["ctx"], b - 1 - i, b, ragged) if case["ctx"] else 0) for i, n in enumerate(new)]
    return new, [max(n, _spread(case["kv"], b - 1 - i, b, ragged)) for i, n in enumerate(new)]


def _row_bytes(case):
    L = case["L"]
    return L // 4 + (2 * L if case["cache"] == "bf16" else L + L // 32)


def work(case):
    new, kv = _lens(case)
    L, op = case["L"], case["op"]
    P, tokens = L // 8, sum(new)
    if op == "append":
        # the new rows in and out, the table's row, every head's rope part in and out
        return {"bytes": tokens * (2 * (L + P) + _row_bytes(case) + 4 * P + 4 * P * case["h"]),
                "flops": tokens * (4 * L + 3 * P * (1 + case["h"]))}
    if op == "gather":
        return {"bytes": tokens * (_row_bytes(case) + 2 * (L + P)), "flops": tokens * L}
    h = case["h"]
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, kv))
    if op == "absorbed":
        return {"bytes": sum(kv) * _row_bytes(case) + tokens * h * (2 * (L + P) + 2 * L + 4), "flops": 2 * h * (2 * L + P) * pairs}
    d = L // 4
    return {"bytes": sum(kv) * (4 * d * h + 2 * P) + tokens * h * (2 * (d + P) + 2 * d + 4), "flops": 2 * h * (2 * d + P) * pairs}


# ---- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _latents(shape, gen):
    """bf16 latents of unit size, some channels heavier."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * (1 + 2 * (torch.arange(shape[-1], device="cuda") % 64 == 9))).bfloat16()


def _rope_part(shape, gen):
    """bf16 rope parts: unit size, an offset in slow channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x + 2.0 * (torch.arange(shape[-1], device="cuda") >= shape[-1] - 4)).bfloat16()


def _pages(lens, block, gen, spare=3):
    """(block table [b, most], blocks in the pool): blocks handed out in no order."""
    need = [-(-t // block) for t in lens]
    most, total = max(max(need), 1), sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").int()
    need = torch.tensor(need, device="cuda")
    slot = torch.arange(most, device="cuda")
    at = (need.cumsum(0) - need).unsqueeze(1) + slot
    return torch.where(slot < need.unsqueeze(1), order[at.clamp(max=total - 1)], -1).int().contiguous(), total


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (fp32, amax floored)."""
    f, e = torch.frexp(amax.clamp(min=AMAX_FLOOR))
    return torch.ldexp(torch.ones_like(f), e - torch.where(f <= 0.875, 9, 8))


def _to_e4m3(x):
    """fp32 [..., L] -> (codes, scales [..., L / 128])."""
    g = x.unflatten(-1, (-1, 128))
    s = _pow2_scale(g.abs().amax(-1))
    return (g / s.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).flatten(-2), s


def _angles(positions, P):
    """cos | sin [positions, P] in fp32, from angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(P // 2, dtype=torch.float64, device="cuda") * 2 / P)
    a = torch.arange(positions, dtype=torch.float64, device="cuda").unsqueeze(1) * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _running(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = _generator(seed)
    op, L, state = case["op"], case["L"], dict(case)
    P, d = L // 8, L // 4
    new, kv = _lens(case)
    tokens = sum(new)
    state.update(cu=_running(new), most=max(new), scale=(d + P) ** -0.5)
    if op == "expanded":
        h, keys = case["h"], sum(kv)
        state.update(cu_kv=_running(kv), q=_latents((tokens, h, d + P), gen), kv_up=_latents((keys, h, 2 * d), gen),
                     k_rope=_rope_part((keys, P), gen),
                     out=torch.empty(tokens, h, d, dtype=torch.bfloat16, device="cuda"),
                     lse=torch.empty(tokens, h, device="cuda"))
        return state
    table, blocks = _pages(kv, case["block"], gen)
    state.update(table=table, kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                 ctx=torch.tensor([t - n for n, t in zip(new, kv)], dtype=torch.int32, device="cuda"))
    # what the pool holds before the call
    shape = (blocks, case["block"])
    latent = torch.empty(*shape, L, dtype=torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn, device="cuda")
    scales = None if case["cache"] == "bf16" else torch.empty(*shape, L // 128, device="cuda")
    step = max(1, (1 << 26) // (case["block"] * L))
    for at in range(0, blocks, step):
        part = slice(at, min(at + step, blocks))
        x = _latents((part.stop - at, case["block"], L), gen)
        if scales is None:
            latent[part] = x
        else:
            latent[part], scales[part] = _to_e4m3(x.float())
    state["cache_of"] = (latent, _rope_part((*shape, P), gen), scales)
    if op == "append":
        # slices of one joint projection's output and of the query projection's, as a model has them
        joint = torch.cat((_latents((tokens, BEFORE[L]), gen), _latents((tokens, L), gen), _rope_part((tokens, P), gen)), 1)
        q = _latents((tokens, case["h"], d + P), gen)
        state.update(latent=joint[:, BEFORE[L]:BEFORE[L] + L], rope=joint[:, BEFORE[L] + L:], q_rope=q[..., d:],
                     q_out=torch.zeros(tokens, case["h"], P, dtype=torch.bfloat16, device="cuda"),
                     angles=_angles(max(kv), P),
                     w=(1 + 0.1 * torch.randn(L, generator=gen, device="cuda")).bfloat16() if case["norm"] else None)
    elif op == "gather":
        state.update(rows=torch.empty(tokens, L, dtype=torch.bfloat16, device="cuda"),
                     rope_rows=torch.empty(tokens, P, dtype=torch.bfloat16, device="cuda"))
    else:
        state.update(q=_latents((tokens, case["h"], L), gen), q_rope=_rope_part((tokens, case["h"], P), gen),
                     out=torch.empty(tokens, case["h"], L, dtype=torch.bfloat16, device="cuda"),
                     lse=torch.empty(tokens, case["h"], device="cuda"))
    return state


# ---- the plain form

def _values(cache):
    """fp32 latents of (latent, rope, scales), any leading shape."""
    latent, _, scales = cache
    x = latent.float()
    return x if scales is None else (x.unflatten(-1, (-1, 128)) * scales.unsqueeze(-1)).flatten(-2)


def _places(s):
    """(sequence, position) of every packed row."""
    t = torch.arange(int(s["rows_in_all"]), device="cuda")
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, t - cu[seq]


def _rotate(x, angles, pairs):
    """fp32 x [..., P] by angles [..., P] = cos | sin."""
    c, n = angles.chunk(2, -1)
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * n, a * n + b * c), -1)


def _plain_append(s):
    latent, rope, scales = s["cache_of"]
    seq, i = _places({"rows_in_all": s["latent"].shape[0], "cu": s["cu"]})
    pos = s["ctx"].long()[seq] + i
    page, slot = s["table"].long()[seq, pos // s["block"]], pos % s["block"]
    y = s["latent"].float()
    if s["w"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["w"].float()
    if scales is None:
        latent[page, slot] = y.bfloat16()
    else:
        # by bytes: not every form of indexed assignment takes 8-bit floats
        codes, scales[page, slot] = _to_e4m3(y)
        latent.view(torch.uint8)[page, slot] = codes.view(torch.uint8)
    angles = s["angles"][pos]
    rope[page, slot] = _rotate(s["rope"].float(), angles, s["pairs"]).bfloat16()
    s["q_out"].copy_(_rotate(s["q_rope"].float(), angles.unsqueeze(1), s["pairs"]))
    return {"latent": latent, "rope": rope, "scales": scales, "q": s["q_out"]}


def _plain_gather(s):
    latent, rope, scales = s["cache_of"]
    seq, pos = _places({"rows_in_all": s["rows"].shape[0], "cu": s["cu"]})
    page, slot = s["table"].long()[seq, pos // s["block"]], pos % s["block"]
    picked = (latent.view(torch.uint8 if scales is not None else latent.dtype)[page, slot].view(latent.dtype), None,
              None if scales is None else scales[page, slot])
    return {"rows": _values(picked).bfloat16(), "rope_rows": rope[page, slot]}


def _softmax(x):
    """(unnormalised weights, their sum, the log of it) of masked scores x, rows without any key included."""
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    return p, total, (top + torch.log(total)).squeeze(-1)


def _padded(x, cu, most):
    """Packed rows [T, ...] as [b, most, ...]; rows past a sequence's end are some row."""
    at = cu[:-1, None].long() + torch.arange(most, device="cuda")
    return x[at.clamp(max=x.shape[0] - 1)]


def _packed_rows(x, s):
    """[b, h, most, ...] back to packed rows [T, h, ...]."""
    seq, i = _places({"rows_in_all": s["q"].shape[0], "cu": s["cu"]})
    return x[seq, :, i]


def _plain_absorbed(s):
    b, h, L, most = s["b"], s["h"], s["L"], s["most"]
    table = s["table"].long().clamp(min=0)
    latent, rope, scales = s["cache_of"]
    raw = latent.view(torch.uint8) if scales is not None else latent
    c = _values((raw[table].view(latent.dtype), None, None if scales is None else scales[table])).reshape(b, -1, L)
    k = torch.cat((c, rope[table].float().reshape(b, -1, L // 8)), -1)
    q = torch.cat((s["q"], s["q_rope"]), -1).float()
    q = _padded(q, s["cu"], most).transpose(1, 2).reshape(b, h * most, -1)
    x = torch.matmul(q, k.transpose(1, 2).contiguous()).view(b, h, most, -1) * s["scale"]
    at = s["ctx"].long()[:, None] + torch.arange(most, device="cuda")
    sees = torch.arange(x.shape[-1], device="cuda") <= at[..., None]
    x = torch.where(sees[:, None], x, -math.inf)
    p, total, lse = _softmax(x)
    out = torch.matmul(p.view(b, h * most, -1), c).view(b, h, most, L) / total
    return {"out": _packed_rows(torch.where(total > 0, out, 0), s).bfloat16(), "lse": _packed_rows(lse, s)}


def _plain_expanded(s):
    b, h, d, most = s["b"], s["h"], s["L"] // 4, s["most"]
    n_kv = s["cu_kv"].long()[1:] - s["cu_kv"].long()[:-1]
    n_q = s["cu"].long()[1:] - s["cu"].long()[:-1]
    longest = max(_lens(s)[1])
    up = _padded(s["kv_up"].float(), s["cu_kv"], longest).transpose(1, 2)                  # [b, h, keys, 2 d]
    r = _padded(s["k_rope"].float(), s["cu_kv"], longest)[:, None].expand(b, h, longest, -1)
    k, v = torch.cat((up[..., :d], r), -1), up[..., d:].contiguous()
    q = _padded(s["q"].float(), s["cu"], most).transpose(1, 2).contiguous()
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    at = (n_kv - n_q)[:, None] + torch.arange(most, device="cuda")
    sees = torch.arange(longest, device="cuda") <= at[..., None]
    x = torch.where(sees[:, None], x, -math.inf)
    p, total, lse = _softmax(x)
    out = torch.matmul(p, v) / total
    return {"out": _packed_rows(torch.where(total > 0, out, 0), s).bfloat16(), "lse": _packed_rows(lse, s)}


def run(state):
    op = state["op"]
    if not own:
        return {"append": _plain_append, "gather": _plain_gather, "absorbed": _plain_absorbed,
                "expanded": _plain_expanded}[op](state)
    import fp8_block_scaled_nt_amd as dg
    if op == "append":
        dg.latent_append(state["latent"], state["rope"], state["cache_of"], state["table"], state["ctx"], state["cu"],
                         state["most"], state["angles"], norm=state["w"], eps=EPS, q_rope=state["q_rope"],
                         q_out=state["q_out"], interleaved=state["pairs"])
        return dict(zip(("latent", "rope", "scales"), state["cache_of"]), q=state["q_out"])
    if op == "gather":
        dg.latent_gather(state["cache_of"], state["table"], state["cu"], state["rows"], state["rope_rows"])
        return {"rows": state["rows"], "rope_rows": state["rope_rows"]}
    if op == "absorbed":
        dg.latent_attention(state["q"], state["q_rope"], state["cache_of"], state["table"], state["kv_lens"], state["cu"],
                            state["most"], state["out"], state["lse"], scale=state["scale"])
    else:
        dg.latent_expanded_attention(state["q"], state["kv_up"], state["k_rope"], state["cu"], state["cu_kv"],
                                     state["most"], state["out"], state["lse"], scale=state["scale"])
    return {"out": state["out"], "lse": state["lse"]}


# ---- the definitions in 64 bits

def _exact_rotation(x, angles, pairs):
    """x [..., P] in 64 bits as complex numbers times e^(i angle)."""
    half = x.shape[-1] // 2
    turn = torch.complex(angles[..., :half].double(), angles[..., half:].double())
    z = torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous()) if pairs else torch.complex(x[..., :half], x[..., half:])
    z = torch.view_as_real(z * turn)
    return z.flatten(-2) if pairs else torch.cat((z[..., 0], z[..., 1]), -1)


def _exact_attention(q, k, v, scale):
    """q [n, d] over k, v [m, ...], the queries last of the m positions."""
    n, m = q.shape[0], k.shape[0]
    x = q @ k.t() * scale
    if n > 1:
        x.masked_fill_(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1), -math.inf)
    return torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, L = case["op"], case["L"]
    new, kv = _lens(case)
    cu = s["cu"].tolist()
    if op == "expanded":
        d, out, lse = L // 4, [], []
        if 2 * case["h"] * (2 * d + L // 8) * sum(n * t for n, t in zip(new, kv)) > 4e13:
            return None
        cu_kv = s["cu_kv"].tolist()
        for i in range(case["b"]):
            rows, keys = slice(cu[i], cu[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
            r, heads = s["k_rope"][keys].double(), []
            for j in range(case["h"]):
                k = torch.cat((s["kv_up"][keys, j, :d].double(), r), 1)
                heads.append(_exact_attention(s["q"][rows, j].double(), k, s["kv_up"][keys, j, d:].double(), s["scale"]))
            out.append(torch.stack([x for x, _ in heads], 1))
            lse.append(torch.stack([x for _, x in heads], 1))
        return {"out": torch.cat(out), "lse": torch.cat(lse)}
    pages, block = s["table"].tolist(), case["block"]
    latent, rope, scales = s["cache_of"]
    if op == "append":
        latent, rope = latent.double(), rope.double()
        scales = None if scales is None else scales.double()
        for i in range(case["b"]):
            ctx = kv[i] - new[i]
            for j in range(ctx // block, -(-kv[i] // block)):
                lo, hi = max(j * block, ctx), min((j + 1) * block, kv[i])
                rows, slots, page = slice(cu[i] + lo - ctx, cu[i] + hi - ctx), slice(lo - j * block, hi - j * block), pages[i][j]
                y = s["latent"][rows].double()
                if s["w"] is not None:
                    y = y / (y.square().mean(1, keepdim=True) + EPS).sqrt() * s["w"].double()
                if scales is not None:
                    g = y.view(y.shape[0], -1, 128)
                    sc = torch.exp2(torch.ceil(torch.log2(g.abs().amax(2).clamp(min=AMAX_FLOOR) / 448)))
                    z = g / sc.unsqueeze(2)
                    # the e4m3 grid: 4 significant bits down to 2^-6, steps of 2^-9 below
                    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
                    y = (torch.round(z / step) * step).clamp(-448, 448).view(y.shape)
                    scales[page, slots] = sc
                latent[page, slots] = y
                rope[page, slots] = _exact_rotation(s["rope"][rows].double(), s["angles"][lo:hi], case["pairs"])
        where = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, kv)])
        q = _exact_rotation(s["q_rope"].double(), s["angles"][where].unsqueeze(1), case["pairs"])
        return {"latent": latent, "rope": rope, "scales": scales, "q": q}
    if op == "gather":
        rows, ropes = [], []
        for i in range(case["b"]):
            own_pages = torch.tensor(pages[i][:-(-kv[i] // block)], device="cuda")
            x = torch.stack([latent[p].double() for p in own_pages.tolist()]).reshape(-1, L)[:kv[i]]
            if scales is not None:
                x = x * scales[own_pages].double().reshape(-1, L // 128)[:kv[i]].repeat_interleave(128, 1)
            rows.append(x)
            ropes.append(rope[own_pages].double().reshape(-1, L // 8)[:kv[i]])
        return {"rows": torch.cat(rows), "rope_rows": torch.cat(ropes)}
    out, lse = [], []
    for i in range(case["b"]):
        own_pages = torch.tensor(pages[i][:-(-kv[i] // block)], device="cuda")
        c = torch.stack([latent[p].double() for p in own_pages.tolist()]).reshape(-1, L)[:kv[i]]
        if scales is not None:
            c = c * scales[own_pages].double().reshape(-1, L // 128)[:kv[i]].repeat_interleave(128, 1)
        k = torch.cat((c, rope[own_pages].double().reshape(-1, L // 8)[:kv[i]]), 1)
        heads = [_exact_attention(torch.cat((s["q"][cu[i]:cu[i + 1], j], s["q_rope"][cu[i]:cu[i + 1], j]), 1).double(), k, c,
                                  s["scale"]) for j in range(case["h"])]
        out.append(torch.stack([x for x, _ in heads], 1))
        lse.append(torch.stack([x for _, x in heads], 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
