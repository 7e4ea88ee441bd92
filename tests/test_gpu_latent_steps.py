"""Absorbed attention where a workgroup takes many steps: shares that begin and
end inside a tile, hold whole tiles of several steps, and scores whose reference
moves in every step, for every compiled form.

All sequences share one sequence's pages, so the oracle reads its tokens once.
Bounds as derived in test_gpu_latent, with e = 50 2^-24 S for S the largest scale
sum |q||k| of the inputs: 2^-8 |r| + (2^-8 + 2 e) W for out, e + 2^-20 |r| for lse
and two roundings of its parts, 2^-22."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import latent as R
from tests import test_gpu_latent as T
from tests.test_gpu_kv8 import i32, running
from tests.test_gpu_latent_forms import queries

pytestmark = pytest.mark.gpu


def shared_ref(q, qr, c, r, lens, new, scale, causal):
    """(out, mean |c|, lse, S) of sequences that are prefixes of the tokens c, r; float64."""
    total, heads, L = q.shape
    out, size, lse, largest = np.zeros((total, heads, L)), np.zeros((total, heads, L)), np.zeros((total, heads)), 0.0
    row = 0
    for n, m in zip(new, lens):
        for i in range(n):
            hi = max(m - n + i + 1, 0) if causal else m
            assert hi > 0
            x = scale * (q[row].astype(np.float64) @ c[:hi].T + qr[row].astype(np.float64) @ r[:hi].T)
            largest = max(largest, scale * (np.abs(q[row]).astype(np.float64) @ np.abs(c[:hi]).T
                                            + np.abs(qr[row]).astype(np.float64) @ np.abs(r[:hi]).T).max())
            top = x.max(1, keepdims=True)
            p = np.exp(x - top)
            norm = p.sum(1, keepdims=True)
            out[row], size[row], lse[row] = p @ c[:hi] / norm, p @ np.abs(c[:hi]) / norm, (top + np.log(norm))[:, 0]
            row += 1
    return out, size, lse, largest


def shares(form, heads, new, lens):
    """(share, sets of what happens to tiles) by the rule that the kernel's comment states."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    rows, most = int(form[len("latent_rows"):]), max(new)
    tiles = -(-most * heads // rows)
    together = tiles if most * len(new) == sum(new) and tiles <= 8 else 1
    steps = [s for n, m in zip(new, lens) for s in [-(-m // 64)] * (1 if together > 1 else -(-n * heads // rows))]
    share = -(-sum(steps) // (cus // together))
    seen, at = set(), 0
    for s in steps:
        for begin in range(at - at % share, at + s, share):
            lo, hi = max(begin, at), min(begin + share, at + s)
            if lo == at and hi == at + s and s > 1:
                seen.add("whole tile of several steps")
            if lo > at and hi - lo > 1:
                seen.add("begins inside a tile")
            if lo == at and hi < at + s and hi - lo > 1:
                seen.add("ends inside a tile")
            if lo == at and lo > begin:
                seen.add("a second tile")
        at += s
    return share, seen


EVERYTHING = {"whole tile of several steps", "begins inside a tile", "ends inside a tile", "a second tile"}


def check(gpu, monkeypatch, form, L, f8, heads, new, lens, block, scale, causal, bend=None):
    share, seen = shares(form, heads, new, lens)
    print(f"[case] steps {form} {L} {f8} {heads} {len(lens)} share {share}", flush=True)
    assert share > 1 and seen == EVERYTHING
    monkeypatch.setenv("DG_FORCE_CONFIG", form)
    rng = np.random.default_rng(L + heads + len(lens))
    cache, table = T.filled(rng, [max(lens)], block, L, f8)
    q, qr = queries(rng, sum(new), heads, L)
    if bend is not None:
        q[..., 0], qr[..., 0] = 0, 1
        for t in range(max(lens)):
            cache[1][table[0, t // block], t % block, 0] = bend(t)
    c, r, there = R.tokens_of(cache, table, 0, 0, max(lens))
    assert there.all()
    on, t = T.upload(cache, gpu), i32(table, gpu).expand(len(lens), -1).contiguous()
    total = sum(new)
    qd, qrd = T.dev_bf16(q, gpu), T.dev_bf16(qr, gpu)
    outs = [torch.full((total, heads, L), float("nan"), dtype=torch.bfloat16, device=gpu) for _ in range(2)]
    lses = [torch.full((total, heads), float("nan"), device=gpu) for _ in range(2)]
    for o, s in zip(outs, lses):
        dg.latent_attention(qd, qrd, on, t, i32(lens, gpu), i32(running(new), gpu), max(new), o, s, scale=scale, causal=causal)
    assert torch.equal(*outs) and torch.equal(*lses)
    want, w, l, largest = shared_ref(q, qr, c, r, lens, new, scale, causal)
    e = 50 * 2.0 ** -24 * largest
    off = np.abs(T.host(outs[0]) - want)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * e) * w
    assert (off <= bound).all(), f"{np.max(off / bound)} of the bound"
    assert (np.abs(lses[0].cpu().numpy() - l) <= e + 2.0 ** -20 * np.abs(l) + 2.0 ** -22).all()


FORMS = ["latent_rows16", "latent_rows32", "latent_rows64"]


def lengths(n, most):
    """n lengths between 1 and most, short ones among them."""
    return [1 + (i * 7919 + 13) % (150 if i % 3 == 0 else most) for i in range(n)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,f8", [(512, False), (512, True), (256, False), (256, True)])
@pytest.mark.parametrize("heads", [13, 40])
def test_single_tokens(gpu, monkeypatch, form, L, f8, heads):
    # 40 heads: neighbouring workgroups take one tile each
    check(gpu, monkeypatch, form, L, f8, heads, [1] * 128, lengths(128, 1400), 64, (L * 3 / 8) ** -0.5, True)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,f8", [(512, False), (512, True), (256, True)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens_of_each(gpu, monkeypatch, form, L, f8, causal):
    # uneven numbers of queries: no neighbours on one sequence, several tiles of some
    new = [1 + i % 4 for i in range(96)]
    lens = [max(n, m) for n, m in zip(new, lengths(96, 1400))]
    check(gpu, monkeypatch, form, L, f8, 21, new, lens, 32, (L * 3 / 8) ** -0.5, causal)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,f8", [(512, False), (512, True), (256, False)])
@pytest.mark.parametrize("way", ["climb", "fall", "both"])
def test_the_reference_moves_in_every_step(gpu, monkeypatch, form, L, f8, way):
    # each 64 tokens lie 8 to 13 or more in log2 apart, by the rope part, whose products are exact:
    # past the 8 that the reference leads by, so u and l are scaled in every step of a climb
    bend = {"climb": lambda t: 32.0 * (t // 16), "fall": lambda t: -32.0 * (t // 16),
            "both": lambda t: 32.0 * abs(t // 16 - 16)}[way]
    scale = (L * 3 / 8) ** -0.5
    assert 128 * scale * np.log2(np.e) > 8
    lens = [max(m, 30) for m in lengths(160, 600)]
    check(gpu, monkeypatch, form, L, f8, 16, [2] * 80 + [1] * 80, lens, 64, scale, True, bend)
