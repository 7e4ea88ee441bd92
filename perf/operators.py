"""What is measured of the block-scaled serving operators, and in what form.

Four operators that serve a model from 4-bit weights and an 8-bit key/value
cache.  Each case names one of them and its sizes; `run` computes it with
elementary torch operations in fp32 (own = False) or by the library's entry
points (own = True), on the same inputs.

  w4_gemm    d[m, n] = sum_k a[m, k] * s[n, k/group] * (c[n, k] - z[n, k/group])
             a bf16, 4-bit codes two per byte (element 2i in the low nibble of
             byte i), one bf16 scale per weight row and group of K.  fmt "e2m1":
             c is the e2m1 value of the code and z = 0; fmt "u4": c is the
             code 0..15 and z an integer 0..15 for each row and group.
  w4_quant   the weights' way into that form (codes, scales, zeros) and back
             (the bf16 values they stand for).
  kv_append  new keys and values of every sequence into a paged e4m3 cache with
             one power-of-two fp32 scale for each block of tokens and head.  A
             block whose scale has to grow has its older codes rounded anew.
  kv_attn    attention of new queries over that cache (their own keys are in
             it already), grouped heads, causal, optionally a sliding window;
             output bf16 and the natural log of the sum of exponentials.

Cache layout: keys [num_blocks, h_kv, block, d], values [num_blocks, h_kv, d, block].
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-4


def listed():
    return [
        # one token through the decode shape's projection: latency
        {"name": "w4_token_2112x7168", "op": "w4_gemm", "m": 1, "n": 2112, "k": 7168, "fmt": "e2m1", "group": 128},
        # a handful of sequences, integer codes with zero points
        {"name": "w4_batch8_4096x7168", "op": "w4_gemm", "m": 8, "n": 4096, "k": 7168, "fmt": "u4", "group": 64},
        # a small layer with an odd number of outputs and a K that fills no whole 128
        {"name": "w4_odd_5x1001x1056", "op": "w4_gemm", "m": 5, "n": 1001, "k": 1056, "fmt": "u4", "group": 32},
        # a full decode batch through the largest weight
        {"name": "w4_batch64_7168x16384", "op": "w4_gemm", "m": 64, "n": 7168, "k": 16384, "fmt": "e2m1", "group": 128},
        # laying out one projection's weights
        {"name": "w4_quant_2112x7168", "op": "w4_quant", "n": 2112, "k": 7168, "fmt": "e2m1", "group": 128, "x": "bf16"},
        # laying out the largest weight from fp32, with zero points
        {"name": "w4_quant_7168x16384", "op": "w4_quant", "n": 7168, "k": 16384, "fmt": "u4", "group": 64, "x": "fp32"},
        # one decode step's keys and values of a batch
        {"name": "append_tokens_64", "op": "kv_append", "b": 64, "h_kv": 8, "d": 128, "block": 64, "new": 1, "ctx": 1500,
         "ragged": True},
        # prompts of different lengths, after a cached prefix
        {"name": "append_prompts_4", "op": "kv_append", "b": 4, "h_kv": 8, "d": 128, "block": 64, "new": 4096, "ctx": 300,
         "ragged": True},
        # one short sequence, one key/value head: latency
        {"name": "attn_token_777", "op": "kv_attn", "b": 1, "h_q": 8, "h_kv": 1, "d": 64, "block": 16, "new": 1, "kv": 777,
         "ragged": False, "window": 0},
        # a decode step of a ragged batch
        {"name": "attn_batch32_4096", "op": "kv_attn", "b": 32, "h_q": 32, "h_kv": 8, "d": 128, "block": 64, "new": 1,
         "kv": 4096, "ragged": True, "window": 0},
        # a few long sequences
        {"name": "attn_long_65536", "op": "kv_attn", "b": 4, "h_q": 64, "h_kv": 8, "d": 128, "block": 128, "new": 1,
         "kv": 65536, "ragged": False, "window": 0},
        # prompt chunks with a cached prefix, causal
        {"name": "attn_prompts_2048", "op": "kv_attn", "b": 4, "h_q": 32, "h_kv": 8, "d": 128, "block": 64, "new": 2048,
         "kv": 4096, "ragged": True, "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _held(case):
    """Scores, and cached values of the padded batch, that the plain form of an attention case holds."""
    if case["op"] != "kv_attn":
        return 0, 0
    return case["b"] * case["h_q"] * case["new"] * case["kv"], case["b"] * case["h_kv"] * case["d"] * case["kv"]


def _within(case):
    """Costs no more than the operator's largest listed case."""
    cost = [tuple(work(c).values()) + _held(c) for c in listed() if c["op"] == case["op"]]
    return all(x <= max(top) for x, top in zip(tuple(work(case).values()) + _held(case), zip(*cost)))


def draw(rng):
    op = rng.choice(("w4_gemm", "w4_gemm", "w4_quant", "kv_append", "kv_attn", "kv_attn", "kv_attn"))
    while True:
        if op in ("w4_gemm", "w4_quant"):
            group = rng.choice((32, 64, 128))
            case = {"op": op, "n": _log(rng, 64, 16384), "k": max(1, _log(rng, 256, 16384) // group) * group,
                    "fmt": rng.choice(("e2m1", "u4")), "group": group}
            if op == "w4_gemm":
                case["m"] = _log(rng, 1, 64)
            else:
                case["x"] = rng.choice(("bf16", "fp32"))
        else:
            case = {"op": op, "b": _log(rng, 1, 128), "h_kv": rng.choice((1, 2, 4, 8)), "d": rng.choice((64, 128, 256)),
                    "block": rng.choice((16, 32, 64, 128)), "ragged": rng.random() < 0.7}
            case["new"] = 1 if rng.random() < 0.6 else _log(rng, 2, 2048)
            if op == "kv_append":
                case["ctx"] = rng.choice((0, _log(rng, 1, 2048)))
            else:
                case["h_q"] = case["h_kv"] * rng.choice((1, 2, 4, 5, 8, 16))
                case["kv"] = case["new"] + _log(rng, 1, 65536)
                case["window"] = _log(rng, 16, 4096) if rng.random() < 0.2 else 0
        if _within(case):
            return case


# ---- sizes that follow from a case alone

def _spread(most, i, b, ragged, least=1):
    """Length of sequence i of b: between a quarter of `most` and `most`."""
    if not ragged or b == 1:
        return most
    return max(least, most - (3 * most // 4) * ((i * 5 + 2) % b) // b)


def _lens(case):
    """(new tokens, tokens in the cache after them) of every sequence."""
    b, ragged = case["b"], case["ragged"]
    new = [_spread(case["new"], i, b, ragged) for i in range(b)]
    if case["op"] == "kv_append":
        return new, [n + (_spread(case["ctx"], b - 1 - i, b, ragged) if case["ctx"] else 0) for i, n in enumerate(new)]
    return new, [max(n, _spread(case["kv"], b - 1 - i, b, ragged)) for i, n in enumerate(new)]


def _seen(new, kv, window):
    """Pairs of a query and a key it sees, and keys that any query sees, of one sequence."""
    if window:
        pairs = sum(min(window, kv - new + i + 1) for i in range(new))
        return pairs, min(kv, window + new - 1)
    return new * (kv - new) + new * (new + 1) // 2, kv


def work(case):
    op = case["op"]
    if op in ("w4_gemm", "w4_quant"):
        n, k, groups = case["n"], case["k"], case["k"] // case["group"]
        packed = n * k // 2 + n * groups * (2 + (case["fmt"] == "u4"))
        if op == "w4_gemm":
            return {"bytes": packed + 2 * case["m"] * (n + k), "flops": 2 * case["m"] * n * k}
        return {"bytes": n * k * (2 if case["x"] == "bf16" else 4) + 2 * packed + 2 * n * k, "flops": 6 * n * k}
    new, kv = _lens(case)
    h, d, block = case["h_kv"], case["d"], case["block"]
    if op == "kv_append":
        tiles = sum(-(-t // block) - (t - n) // block for n, t in zip(new, kv))
        values = 2 * h * d * sum(new)
        return {"bytes": 3 * values + 2 * 4 * h * tiles, "flops": 4 * values}
    pairs, keys = (sum(x) for x in zip(*(_seen(n, t, case["window"]) for n, t in zip(new, kv))))
    rows = sum(new) * case["h_q"]
    return {"bytes": 2 * h * keys * d + 8 * h * (keys // block + 1) + rows * (4 * d + 4),
            "flops": 4 * case["h_q"] * d * pairs}


# ---- 4-bit and 8-bit formats in elementary operations (inputs, and the plain form)

def _unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _w4_values(codes, scales, zeros, dtype=torch.float32):
    """The values that packed codes [n, k/2] stand for."""
    n, groups = scales.shape
    c = _unpack(codes).view(n, groups, -1)
    if zeros is None:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
        c = table[c.int()]
    else:
        c = c.to(dtype) - zeros.to(dtype).unsqueeze(-1)
    return (c * scales.to(dtype).unsqueeze(-1)).view(n, -1)


def _w4_quantize(x, fmt, group):
    """fp32 [n, k] -> packed codes, bf16 scales, zeros (None for e2m1)."""
    n, k = x.shape
    g = x.view(n, k // group, group)
    if fmt == "e2m1":
        # by a tensor: a division by a Python number may be done as a product with its rounded reciprocal
        s = (g.abs().amax(-1).clamp(min=AMAX_FLOOR) / torch.full((), 6.0, device=x.device)).bfloat16()
        y = g / s.float().unsqueeze(-1)
        a = y.abs()
        # nearest value, ties to the even code: how many midpoints are passed
        c = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
             + torch.signbit(y).byte() * 8)
        zeros = None
    else:
        lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
        s = ((hi - lo).clamp(min=AMAX_FLOOR) / torch.full((), 15.0, device=x.device)).bfloat16()
        zeros = torch.round(-lo / s.float()).clamp(max=15)
        c = (torch.round(g / s.float().unsqueeze(-1)) + zeros.unsqueeze(-1)).clamp(0, 15).byte()
        zeros = zeros.byte()
    c = c.view(n, k // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), s, zeros


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (fp32, amax floored)."""
    f, e = torch.frexp(amax.clamp(min=AMAX_FLOOR))
    return torch.ldexp(torch.ones_like(f), e - torch.where(f <= 0.875, 9, 8))


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


# ---- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(n, k, gen):
    """Like a trained projection: small, with a few heavier input channels."""
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    return w * (1 + 3 * (torch.rand(k, generator=gen, device="cuda") < 0.01))


def _keys_values(shape, gen, offset):
    """bf16 [..., h_kv, d] keys or values: unit size, a few channels with an offset."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x + offset * (torch.arange(shape[-1], device="cuda") % 32 == 5)).bfloat16()


def _pages(lens, block, gen, spare=3):
    """(block table [b, most], blocks in the pool): blocks handed out in no order."""
    need = [-(-t // block) for t in lens]
    most, total = max(max(need), 1), sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").int()
    need = torch.tensor(need, device="cuda")
    slot = torch.arange(most, device="cuda")
    at = (need.cumsum(0) - need).unsqueeze(1) + slot
    return torch.where(slot < need.unsqueeze(1), order[at.clamp(max=total - 1)], -1).int().contiguous(), total


def prepare(case, seed):
    gen = _generator(seed)
    op, state = case["op"], dict(case)
    if op in ("w4_gemm", "w4_quant"):
        n, k = case["n"], case["k"]
        w = _weights(n, k, gen)
        if op == "w4_quant":
            state["w"] = w.bfloat16() if case["x"] == "bf16" else w
        else:
            state["weight"] = _w4_quantize(w, case["fmt"], case["group"])
            state["a"] = torch.randn(case["m"], k, generator=gen, device="cuda").bfloat16()
            state["out"] = torch.empty(case["m"], n, dtype=torch.bfloat16, device="cuda")
        return state
    b, h, d, block = case["b"], case["h_kv"], case["d"], case["block"]
    new, kv = _lens(case)
    table, blocks = _pages(kv, block, gen)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    state.update(table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), most=max(new),
                 kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                 ctx=torch.tensor([t - x for x, t in zip(new, kv)], dtype=torch.int32, device="cuda"))
    # what the pool holds before the call, one block of a head at a time in its own scale
    k_codes = torch.empty(blocks, h, block, d, dtype=torch.float8_e4m3fn, device="cuda")
    v_codes = torch.empty(blocks, h, d, block, dtype=torch.float8_e4m3fn, device="cuda")
    k_scale, v_scale = (torch.empty(blocks, h, device="cuda") for _ in range(2))
    step = max(1, (1 << 26) // (h * block * d))
    for at in range(0, blocks, step):
        part = slice(at, min(at + step, blocks))
        size = part.stop - at
        x = _keys_values((size, block, h, d), gen, 4.0).transpose(1, 2).float()
        k_scale[part] = _pow2_scale(x.abs().amax((2, 3)))
        k_codes[part] = _e4m3(x / k_scale[part, :, None, None])
        x = _keys_values((size, block, h, d), gen, 0.0).permute(0, 2, 3, 1).float()
        v_scale[part] = _pow2_scale(x.abs().amax((2, 3)))
        v_codes[part] = _e4m3(x / v_scale[part, :, None, None])
    state["cache"] = (k_codes, v_codes, k_scale, v_scale)
    if op == "kv_append":
        # slices of one projection's output, as a model has them: the rows are further apart than h_kv * d
        both = torch.cat((_keys_values((cu[-1], h, d), gen, 4.0), _keys_values((cu[-1], h, d), gen, 0.0)), 1)
        state["k"], state["v"] = both[:, :h], both[:, h:]
    else:
        state["q"] = torch.randn(cu[-1], case["h_q"], d, generator=gen, device="cuda").bfloat16()
        state["out"] = torch.empty_like(state["q"])
        state["lse"] = torch.empty(cu[-1], case["h_q"], device="cuda")
        state["scale"] = d ** -0.5
    return state


# ---- the plain form

def _plain_gemm(s):
    return torch.matmul(s["a"].float(), _w4_values(*s["weight"]).t()).bfloat16()


def _plain_quant(s):
    codes, scales, zeros = _w4_quantize(s["w"].float(), s["fmt"], s["group"])
    return {"values": _w4_values(codes, scales, zeros).bfloat16(), "scales": scales, "zeros": zeros}


def _merge_tiles(pool, scale, at, old, fresh, is_old, is_new):
    """Puts new tokens into tiles of the pool (tokens first, then d): `old` codes stay at `is_old`, rounded anew
    where the scale grows, and `fresh` values go to `is_new`."""
    live = is_new.any(-1)[:, None]
    amax = (fresh.abs() * is_new[:, None, :, None]).amax((2, 3))
    was = torch.where(is_old.any(-1)[:, None], scale[at], 0)
    now = torch.maximum(was, _pow2_scale(amax))
    keep = _e4m3(old.float() * (was / now)[:, :, None, None])
    code = torch.where(is_new[:, None, :, None], _e4m3(fresh / now[:, :, None, None]).float(),
                       torch.where(is_old[:, None, :, None], keep.float(), old.float()))
    return code.to(torch.float8_e4m3fn), torch.where(live, now, scale[at])


def _plain_append(s):
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    block, cu, ctx = s["block"], s["cu"].long(), s["ctx"].long()
    new = cu[1:] - cu[:-1]
    slots = (s["most"] + block - 2) // block + 1
    # every sequence's blocks from its first new token's on; those that take none stay as they are
    at_block = ctx[:, None] // block + torch.arange(slots, device="cuda")
    pos = at_block[..., None] * block + torch.arange(block, device="cuda")
    is_new = (pos >= ctx[:, None, None]) & (pos < (ctx + new)[:, None, None])
    is_old = pos < ctx[:, None, None]
    row = (cu[:-1, None, None] + pos - ctx[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    page = torch.gather(s["table"].long(), 1, at_block.clamp(max=s["table"].shape[1] - 1))
    pick = is_new.any(-1)
    page, row, is_new, is_old = page[pick], row[pick], is_new[pick], is_old[pick]
    fresh = s["k"].float()[row].transpose(1, 2)
    codes, scale = _merge_tiles(k_codes, k_scale, page, k_codes[page], fresh, is_old, is_new)
    k_codes[page], k_scale[page] = codes, scale
    fresh = s["v"].float()[row].transpose(1, 2)
    codes, scale = _merge_tiles(v_codes, v_scale, page, v_codes[page].transpose(2, 3), fresh, is_old, is_new)
    v_codes[page], v_scale[page] = codes.transpose(2, 3).contiguous(), scale
    return {"k_codes": k_codes, "v_codes": v_codes, "k_scale": k_scale, "v_scale": v_scale}


def _plain_attn(s):
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    b, hq, h, d, most = s["b"], s["h_q"], s["h_kv"], s["d"], s["most"]
    table = s["table"].long().clamp(min=0)
    k = (k_codes[table].float() * k_scale[table][..., None, None]).transpose(1, 2).reshape(b, h, -1, d)
    v = (v_codes[table].float() * v_scale[table][..., None, None]).permute(0, 2, 1, 4, 3).reshape(b, h, -1, d)
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device="cuda")
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]              # [b, most, hq, d]
    q = q.view(b, most, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(b, h, hq // h, most, -1) * s["scale"]
    at = (kv - new)[:, None] + i                                                      # where each query stands
    j = torch.arange(x.shape[-1], device="cuda")
    sees = j <= at[..., None]
    if s["window"]:
        sees = sees & (j > at[..., None] - s["window"])
    x = torch.where(sees[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, h, -1, p.shape[-1]), v).view(b, h, hq // h, most, d) / total
    out = torch.where(total > 0, out, 0)
    lse = (top + torch.log(total)).squeeze(-1)
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    out, lse = (y.flatten(1, 2)[seq, :, t - cu[seq]] for y in (out, lse))
    return {"out": out.bfloat16(), "lse": lse}


def run(state):
    op = state["op"]
    if not own:
        return {"w4_gemm": _plain_gemm, "w4_quant": _plain_quant, "kv_append": _plain_append, "kv_attn": _plain_attn}[op](state)
    import fp8_block_scaled_nt_amd as dg
    if op == "w4_gemm":
        return dg.bf16_w4_gemm_nt(state["a"], state["weight"], state["out"])
    if op == "w4_quant":
        codes, scales, zeros = dg.quantize_b_w4(state["w"], state["fmt"], state["group"])
        return {"values": dg.dequantize_b_w4((codes, scales, zeros)), "scales": scales, "zeros": zeros}
    if op == "kv_append":
        dg.kv8_append(state["k"], state["v"], state["cache"], state["table"], state["ctx"], state["cu"], state["most"])
        return dict(zip(("k_codes", "v_codes", "k_scale", "v_scale"), state["cache"]))
    dg.kv8_attention(state["q"], state["cache"], state["table"], state["kv_lens"], state["cu"], state["most"],
                     state["out"], state["lse"], scale=state["scale"], window=state["window"])
    return {"out": state["out"], "lse": state["lse"]}


# ---- the definitions in 64 bits

def _exact_e4m3(x):
    """x rounded onto the e4m3 grid: 4 significant bits down to 2^-6, steps of 2^-9 below."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_scale(amax):
    return 2.0 ** math.ceil(math.log2(max(amax, AMAX_FLOOR) / 448))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "w4_gemm":
        codes, scales, zeros = s["weight"]
        a, rows = s["a"].double(), []
        for at in range(0, case["n"], 1024):
            part = slice(at, at + 1024)
            c = torch.empty(codes[part].shape[0], case["k"], dtype=torch.long, device="cuda")
            c[:, 0::2], c[:, 1::2] = codes[part].long() % 16, codes[part].long() // 16
            if zeros is None:
                e, f = c % 8 // 2, c % 2                   # 2-bit exponent, 1-bit fraction
                w = torch.where(e > 0, (1 + f / 2.0).double() * 2.0 ** (e - 1), f / 2.0) * (1 - 2.0 * (c // 8))
            else:
                w = (c - zeros[part].long().repeat_interleave(case["group"], 1)).double()
            rows.append(a @ (w * scales[part].double().repeat_interleave(case["group"], 1)).t())
        return torch.cat(rows, 1)
    if op == "w4_quant":
        values, all_scales = [], []
        for at in range(0, case["n"], 1024):
            x = s["w"][at:at + 1024].double()
            g = x.view(x.shape[0], -1, case["group"])
            if case["fmt"] == "e2m1":
                sc = (g.abs().amax(2) / 6).clamp(min=AMAX_FLOOR / 6).bfloat16().double()[..., None]
                y = (g / sc).clamp(-6, 6)
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1))) - 1)
                w = torch.round(y / step) * step * sc
            else:
                lo, hi = g.amin(2).clamp(max=0), g.amax(2).clamp(min=0)
                sc = ((hi - lo).clamp(min=AMAX_FLOOR) / 15).bfloat16().double()[..., None]
                z = torch.round(-lo[..., None] / sc).clamp(max=15)
                w = ((torch.round(g / sc) + z).clamp(0, 15) - z) * sc
            values.append(w.view(x.shape))
            all_scales.append(sc.squeeze(-1))
        return {"values": torch.cat(values), "scales": torch.cat(all_scales), "zeros": None}
    new, kv = _lens(case)
    h, d, block = case["h_kv"], case["d"], case["block"]
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    pages, cu = s["table"].tolist(), s["cu"].tolist()
    if op == "kv_append":
        if sum(-(-t // block) - (t - n) // block for n, t in zip(new, kv)) > 4000:
            return None
        k_codes, v_codes = k_codes.double(), v_codes.double().transpose(2, 3)
        k_scale, v_scale = k_scale.double(), v_scale.double()
        for codes, scales, x in ((k_codes, k_scale, s["k"].double()), (v_codes, v_scale, s["v"].double())):
            for i in range(case["b"]):
                ctx = kv[i] - new[i]
                for j in range(ctx // block, -(-kv[i] // block)):
                    lo, hi = max(j * block, ctx), min((j + 1) * block, kv[i])
                    page, before = pages[i][j], max(0, ctx - j * block)
                    fresh = x[cu[i] + lo - ctx:cu[i] + hi - ctx].transpose(0, 1)      # [h, tokens, d]
                    amax = fresh.abs().amax((1, 2)).clamp(min=AMAX_FLOOR)
                    sc = torch.exp2(torch.ceil(torch.log2(amax / 448)))
                    if before:
                        sc = torch.maximum(sc, scales[page])
                        codes[page, :, :before] = _exact_e4m3(codes[page, :, :before] * (scales[page] / sc)[:, None, None])
                    codes[page, :, lo - j * block:hi - j * block] = _exact_e4m3(fresh / sc[:, None, None])
                    scales[page] = sc
        return {"k_codes": k_codes, "v_codes": v_codes.transpose(2, 3).contiguous(), "k_scale": k_scale, "v_scale": v_scale}
    hq = case["h_q"]
    if 4 * hq * d * sum(_seen(n, t, 0)[0] for n, t in zip(new, kv)) > 6e12:
        return None
    out, lse = [], []
    for i in range(case["b"]):
        own_pages = torch.tensor(pages[i][:-(-kv[i] // block)], device="cuda")
        at = torch.arange(kv[i] - new[i], kv[i], device="cuda")[:, None]
        j = torch.arange(kv[i], device="cuda")
        sees = (j <= at) & (j > at - (case["window"] or kv[i] + 1))
        heads, sums = [], []
        for head in range(hq):
            c = head * h // hq
            k = (k_codes[own_pages, c].double() * k_scale[own_pages, c].double()[:, None, None]).reshape(-1, d)[:kv[i]]
            v = (v_codes[own_pages, c].double() * v_scale[own_pages, c].double()[:, None, None])
            v = v.transpose(1, 2).reshape(-1, d)[:kv[i]]
            x = (s["q"][cu[i]:cu[i + 1], head].double() @ k.t() * s["scale"]).masked_fill(~sees, -math.inf)
            heads.append(torch.softmax(x, -1) @ v)
            sums.append(torch.logsumexp(x, -1))
        out.append(torch.stack(heads, 1))
        lse.append(torch.stack(sums, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
