"""Every compiled form of absorbed attention, and what can go wrong around the
latent operators: masked places, missing blocks, lengths, strides, streams,
graphs, refusals (bounds as derived in test_gpu_latent)."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import latent as R
from tests import gpu_harness as H
from tests import test_gpu_latent as T
from tests.test_gpu_kv8 import bf16, i32, running

pytestmark = pytest.mark.gpu
ROWS = ["latent_rows16", "latent_rows32", "latent_rows64"]


@pytest.fixture(params=ROWS)
def rows(request, monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", request.param)
    return request.param


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("L,f8,block,heads,new,lens", T.ABSORBED)
def test_absorbed(rows, gpu, L, f8, block, heads, new, lens, causal):
    T.test_absorbed(gpu, L, f8, block, heads, new, lens, causal)


def attend(gpu, q, qr, cache, table, lens, cu, scale=None, causal=True, most=None):
    """(out, lse) of absorbed attention on host arrays, as tensors."""
    total, heads, L = q.shape
    out = torch.full((total, heads, L), float("nan"), dtype=torch.bfloat16, device=gpu)
    lse = torch.full((total, heads), float("nan"), device=gpu)
    n = max(b - a for a, b in zip(cu[:-1], cu[1:])) if most is None else most
    dg.latent_attention(T.dev_bf16(q, gpu), T.dev_bf16(qr, gpu), T.upload(cache, gpu), i32(table, gpu), i32(lens, gpu), i32(cu, gpu),
                        int(n), out, lse, scale=scale, causal=causal)
    return out, lse


def queries(rng, total, heads, L):
    return bf16(rng.standard_normal((total, heads, L))), bf16(rng.standard_normal((total, heads, L // 8)))


@pytest.mark.parametrize("L,f8", [(512, False), (256, True)])
def test_missing_blocks_and_lengths_past_the_table(rows, gpu, L, f8):
    rng = np.random.default_rng(1)
    cache, table = T.filled(rng, [200, 70, 40], 16, L, f8)
    table[0, 2], table[0, 4:8], table[1, 0] = -1, 10 ** 6, cache[0].shape[0]
    table[2] = -5                                                            # nothing of sequence 2 is there
    lens, new = [230, 70, 40], [3, 9, 2]                                     # 230: past the table's 208
    q, qr = queries(rng, sum(new), 7, L)
    want = R.attention_ref(q, qr, cache, table, lens, running(new), (L * 3 / 8) ** -0.5)
    out, lse = attend(gpu, q, qr, cache, table, lens, running(new))
    T.check_out(out, lse, want)
    assert (T.host(out)[-2:] == 0).all() and (lse[-2:].cpu().numpy() == -np.inf).all()


def test_sequences_without_tokens_and_queries_before_the_first(rows, gpu):
    rng = np.random.default_rng(2)
    lens, new = [0, 5, 0, 100, 64], [2, 9, 1, 0, 70]
    cache, table = T.filled(rng, lens, 32, 512, True)
    q, qr = queries(rng, sum(new), 3, 512)
    want = R.attention_ref(q, qr, cache, table, lens, running(new), 192 ** -0.5)
    out, lse = attend(gpu, q, qr, cache, table, lens, running(new))
    T.check_out(out, lse, want)
    assert (T.host(out)[:2] == 0).all() and (T.host(out)[2:6] == 0).all()


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("part", ["latent", "rope"])
def test_what_is_not_finite_reaches_no_row_that_does_not_see_it(rows, gpu, what, part):
    # drafted tokens: the last of the queries' own tokens is seen by the last query alone
    rng = np.random.default_rng(3)
    cache, table = T.filled(rng, [130], 64, 512, False)
    x = cache[0] if part == "latent" else cache[1]
    x[table[0, 129 // 64], 129 % 64, 5] = what
    q, qr = queries(rng, 4, 20, 512)
    out, lse = attend(gpu, q, qr, cache, table, [130], [0, 4])
    clean = [np.nan_to_num(y, nan=0, posinf=0, neginf=0) for y in cache[:2]]
    want = R.attention_ref(q, qr, (*clean, None), table, [130], [0, 4], 192 ** -0.5)
    T.check_out(out[:3], lse[:3], [w[:3] for w in want])
    # and with the token before every query, all rows see it
    if np.isnan(what):
        x[table[0, 0], 3, 7] = what
        assert np.isnan(T.host(attend(gpu, q, qr, cache, table, [130], [0, 4])[0])).all()


def test_a_query_that_is_not_finite_stays_in_its_row(rows, gpu):
    rng = np.random.default_rng(4)
    cache, table = T.filled(rng, [150], 16, 256, True)
    q, qr = queries(rng, 1, 40, 256)
    want = R.attention_ref(q, qr, cache, table, [150], [0, 1], 96 ** -0.5)
    q[0, 11, 3], qr[0, 30, 1] = np.nan, np.inf
    out, lse = attend(gpu, q, qr, cache, table, [150], [0, 1])
    others = [h for h in range(40) if h not in (11, 30)]
    T.check_out(out[:, others], lse[:, others], [w[:, others] for w in want])
    assert np.isnan(T.host(out)[0, [11, 30]]).all()


@pytest.mark.parametrize("step", [0.5, -0.5])
def test_scores_that_climb_or_fall(rows, gpu, step):
    # 300 tokens whose scores move by up to 9 in log2 every 16 tokens: the reference moves again and again
    rng = np.random.default_rng(5)
    cache, table = T.filled(rng, [300], 64, 256, False)
    for t in range(300):
        cache[0][table[0, t // 64], t % 64, :8] = bf16(step * (t // 4))
    q, qr = queries(rng, 1, 17, 256)
    q[:, :, :8] = np.array([1, 0.25] * 8 + [0])[None, :, None]
    out, lse = attend(gpu, q, qr, cache, table, [300], [0, 1], scale=0.2)
    want = R.attention_ref(q, qr, cache, table, [300], [0, 1], 0.2)
    # scores of up to 300: scale sum |q||k| < 360, five times what the bound of lse and of 2^-11 W counts on
    r, w, l = want
    assert (np.abs(T.host(out) - r) <= 2.0 ** -8 * np.abs(r) + (2.0 ** -8 + 2.0 ** -8) * w).all()
    assert (np.abs(lse.cpu().numpy() - l) <= 2.0 ** -9 + 2.0 ** -20 * np.abs(l)).all()


def test_scale_of_zero(rows, gpu):
    rng = np.random.default_rng(6)
    cache, table = T.filled(rng, [70, 20], 16, 256, False)
    q, qr = queries(rng, 5, 6, 256)
    out, lse = attend(gpu, q, qr, cache, table, [70, 20], [0, 2, 5], scale=0.0)
    T.check_out(out, lse, R.attention_ref(q, qr, cache, table, [70, 20], [0, 2, 5], 0.0))


def test_scales_far_apart(rows, gpu):
    # e4m3 tokens of sizes from 2^-20 to 2^20: the values are exact in bf16, whatever their scales
    rng = np.random.default_rng(7)
    cache, table = T.filled(rng, [100], 16, 512, True)
    for t in range(100):
        at = (table[0, t // 16], t % 16)
        cache[0][at], cache[2][at] = R.quantise(bf16(rng.standard_normal(512) * np.exp2(rng.integers(-20, 20, 4)).repeat(128)))
    q, qr = queries(rng, 1, 18, 512)
    q = bf16(q * 2.0 ** -24)
    out, lse = attend(gpu, q, qr, cache, table, [100], [0, 1])
    T.check_out(out, lse, R.attention_ref(q, qr, cache, table, [100], [0, 1], 192 ** -0.5))


def test_strides(rows, gpu):
    # queries and outputs as the products of heads leave them: [heads, tokens, L]
    rng = np.random.default_rng(8)
    cache, table = T.filled(rng, [90, 33], 32, 512, False)
    q, qr = queries(rng, 3, 10, 512)
    want = R.attention_ref(q, qr, cache, table, [90, 33], [0, 1, 3], 192 ** -0.5)
    by_head = T.dev_bf16(q.transpose(1, 0, 2), gpu).transpose(0, 1)
    wide = torch.zeros((3, 10, 192), dtype=torch.bfloat16, device=gpu)
    wide[..., 128:] = T.dev_bf16(qr, gpu)
    out = torch.full((10, 4, 520), float("nan"), dtype=torch.bfloat16, device=gpu)
    view = out[:, :3, :512].transpose(0, 1)
    lse = torch.empty((3, 10), device=gpu)
    dg.latent_attention(by_head, wide[..., 128:], T.upload(cache, gpu), i32(table, gpu), i32([90, 33], gpu), i32([0, 1, 3], gpu), 2,
                        view, lse)
    T.check_out(view, lse, want)
    assert torch.isnan(out[:, 3]).all() and torch.isnan(out[..., 512:]).all()


def test_more_queries_than_the_longest(rows, gpu):
    # rows past max_q are left alone, the others stand where the lengths say
    rng = np.random.default_rng(9)
    cache, table = T.filled(rng, [60], 16, 256, False)
    q, qr = queries(rng, 5, 4, 256)
    out, lse = attend(gpu, q, qr, cache, table, [60], [0, 5], most=3)
    want = R.attention_ref(q, qr, cache, table, [60], [0, 5], 96 ** -0.5)
    T.check_out(out[:3], lse[:3], [w[:3] for w in want])
    assert torch.isnan(out[3:]).all() and torch.isnan(lse[3:]).all()


@pytest.mark.parametrize("f8", [False, True])
def test_many_sequences(gpu, f8):
    # more than one pass of a workgroup over the lengths takes, some empty, some of several tiles
    rng = np.random.default_rng(10)
    lens = [int(x) for x in rng.integers(0, 40, 600)]
    lens[300], lens[599] = 1500, 0
    new = [1] * 600
    new[7], new[300] = 30, 12
    cache, table = T.filled(rng, lens, 16, 256, f8)
    q, qr = queries(rng, sum(new), 5, 256)
    out, lse = attend(gpu, q, qr, cache, table, lens, running(new))
    T.check_out(out, lse, R.attention_ref(q, qr, cache, table, lens, running(new), 96 ** -0.5))


def test_same_bits_and_two_streams(rows, gpu):
    rng = np.random.default_rng(11)
    lens = [700, 130, 400]
    cache, table = T.filled(rng, lens, 64, 512, True)
    q, qr = queries(rng, 3, 64, 512)
    args = [T.dev_bf16(q, gpu), T.dev_bf16(qr, gpu), T.upload(cache, gpu), i32(table, gpu), i32(lens, gpu), i32([0, 1, 2, 3], gpu), 1]
    outs = [torch.empty((3, 64, 512), dtype=torch.bfloat16, device=gpu) for _ in range(9)]
    dg.latent_attention(*args, outs[0])
    side = [T.OwnStream(), T.OwnStream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for i, o in enumerate(outs[1:]):
        with torch.cuda.stream(side[i % 2]):
            dg.latent_attention(*args, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_past_four_gib(gpu):
    rng = np.random.default_rng(12)
    own, table = T.filled(rng, [300], 128, 512, False)
    blocks = (1 << 32) // (128 * 1024) + 6
    pool = dg.empty_latent_cache(blocks, 512, 128, "bf16", gpu)
    take = [blocks - 1, blocks - 3, blocks - 2]
    for j, page in enumerate(take):
        pool[0][page] = T.dev_bf16(own[0][table[0, j]], gpu)
        pool[1][page] = T.dev_bf16(own[1][table[0, j]], gpu)
    q, qr = queries(rng, 1, 20, 512)
    out, lse = torch.empty((1, 20, 512), dtype=torch.bfloat16, device=gpu), torch.empty((1, 20), device=gpu)
    t, cu = i32([take], gpu), i32([0, 1], gpu)
    dg.latent_attention(T.dev_bf16(q, gpu), T.dev_bf16(qr, gpu), pool, t, i32([300], gpu), cu, 1, out, lse)
    T.check_out(out, lse, R.attention_ref(q, qr, own, table, [300], [0, 1], 192 ** -0.5))
    an = T.angles(rng, 301, 64)
    x = T.dev_bf16(rng.standard_normal((1, 576)), gpu)
    dg.latent_append(x[:, :512], x[:, 512:], pool, t, i32([300], gpu), cu, 1, H.f32_to_device(an, gpu))
    rows, rope = torch.empty((301, 512), dtype=torch.bfloat16, device=gpu), torch.empty((301, 64), dtype=torch.bfloat16, device=gpu)
    dg.latent_gather(pool, t, i32([0, 301], gpu), rows, rope)
    c, r, _ = R.tokens_of(own, table, 0, 0, 300)
    assert np.array_equal(T.host(rows)[:300], c) and np.array_equal(T.host(rope)[:300], r) and torch.equal(rows[300:], x[:, :512])


def test_expanded_rows_far_apart(gpu):
    # rows of keys and values further apart than 32-bit offsets reach over a step
    rng = np.random.default_rng(13)
    D, heads, keys = 64, 2, 70
    q, kv, r = (bf16(rng.standard_normal(s)) for s in ((6, heads, 96), (keys, heads, 128), (keys, 32)))
    far = torch.empty((keys, (1 << 26) - 8), dtype=torch.bfloat16, device=gpu)
    far[:, :256], far[:, 256:288] = T.dev_bf16(kv, gpu).flatten(1), T.dev_bf16(r, gpu)
    out, lse = torch.empty((6, heads, D), dtype=torch.bfloat16, device=gpu), torch.empty((6, heads), device=gpu)
    dg.latent_expanded_attention(T.dev_bf16(q, gpu), far[:, :256].unflatten(1, (heads, 128)), far[:, 256:288], i32([0, 6], gpu),
                                 i32([0, keys], gpu), 6, out, lse)
    T.check_out(out, lse, R.expanded_ref(q, kv, r, [0, 6], [0, keys], 96 ** -0.5))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_expanded_values_that_are_not_finite(gpu, D, what):
    rng = np.random.default_rng(14)
    keys, heads = 150, 2
    q, kv, r = (bf16(rng.standard_normal(s)) for s in ((keys, heads, D * 3 // 2), (keys, heads, 2 * D), (keys, D // 2)))
    want = R.expanded_ref(q, kv, r, [0, keys], [0, keys], (D * 1.5) ** -0.5)
    kv[100, 1, D + 5] = what                                                 # a value: queries from 100 on, that dimension
    kv[140, 0, 3] = what                                                     # a key: queries from 140 on see it
    out, lse = torch.empty((keys, heads, D), dtype=torch.bfloat16, device=gpu), torch.empty((keys, heads), device=gpu)
    dg.latent_expanded_attention(T.dev_bf16(q, gpu), T.dev_bf16(kv, gpu), T.dev_bf16(r, gpu), i32([0, keys], gpu), i32([0, keys], gpu),
                                 keys, out, lse)
    got = T.host(out)
    assert not np.isfinite(got[100:, 1, 5]).any()
    kept = np.ones(got.shape, bool)
    kept[100:, 1, 5] = kept[140:, 0] = False
    bound = 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -8 + 2.0 ** -11) * want[1]
    assert (np.abs(got - want[0])[kept] <= bound[kept]).all()


def test_expanded_many_prompts(gpu):
    rng = np.random.default_rng(15)
    new = [int(x) for x in rng.integers(0, 30, 60)]
    new[9] = 140
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 50, 60))]
    lens[11] = new[11] // 2
    q, kv, r = (bf16(rng.standard_normal(s)) for s in ((sum(new), 2, 96), (sum(lens), 2, 128), (sum(lens), 32)))
    out, lse = torch.empty((sum(new), 2, 64), dtype=torch.bfloat16, device=gpu), torch.empty((sum(new), 2), device=gpu)
    dg.latent_expanded_attention(T.dev_bf16(q, gpu), T.dev_bf16(kv, gpu), T.dev_bf16(r, gpu), i32(running(new), gpu),
                                 i32(running(lens), gpu), max(new), out, lse)
    T.check_out(out, lse, R.expanded_ref(q, kv, r, running(new), running(lens), 96 ** -0.5))


def test_expanded_same_bits(gpu):
    rng = np.random.default_rng(16)
    q, kv, r = (T.dev_bf16(rng.standard_normal(s), gpu) for s in ((700, 8, 192), (700, 8, 256), (700, 64)))
    outs = [torch.empty((700, 8, 128), dtype=torch.bfloat16, device=gpu) for _ in range(6)]
    for o in outs:
        dg.latent_expanded_attention(q, kv, r, i32([0, 300, 700], gpu), i32([0, 300, 700], gpu), 400, o)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_decode_loop_in_a_graph(rows, gpu):
    # append and attention captured once, replayed as the sequences grow, with eager work between
    rng = np.random.default_rng(17)
    L, P, heads, block, steps = 256, 32, 6, 16, 40
    kv = [130, 3]
    before, table = T.filled(rng, [x + steps for x in kv], block, L, True)
    an = T.angles(rng, 200, P)
    cache, t, on = T.upload(before, gpu), i32(table, gpu), H.f32_to_device(an, gpu)
    ctx, lens, cu = i32(kv, gpu), i32(kv, gpu), i32([0, 1, 2], gpu)
    x = torch.zeros((2, L + P), dtype=torch.bfloat16, device=gpu)
    q = torch.zeros((2, heads, L + P), dtype=torch.bfloat16, device=gpu)
    turned = torch.zeros((2, heads, P), dtype=torch.bfloat16, device=gpu)
    out, lse = torch.empty((2, heads, L), dtype=torch.bfloat16, device=gpu), torch.empty((2, heads), device=gpu)

    def step():
        lens.copy_(ctx + 1)
        dg.latent_append(x[:, :L], x[:, L:], cache, t, ctx, cu, 1, on, q_rope=q[..., L:], q_out=turned)
        dg.latent_attention(q[..., :L], turned, cache, t, lens, cu, 1, out, lse)
        ctx.copy_(lens)

    side = T.OwnStream()
    dg.reserve_workspace(dg.latent_attention_workspace_size(L, 1, heads), side)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    want = before
    for i in range(steps):
        wide, wq = bf16(rng.standard_normal((2, L + P))), bf16(rng.standard_normal((2, heads, L + P)))
        x.copy_(T.dev_bf16(wide, gpu))
        q.copy_(T.dev_bf16(wq, gpu))
        graph.replay()
        torch.cuda.synchronize()
        now = [a + i for a in kv]
        want, _ = R.append_ref(wide[:, :L], wide[:, L:], want, table, now, [0, 1, 2], an)
        if i % 8 == 0 or i == steps - 1:
            held = (want[0], T.host(cache[1]), want[2])                      # rope parts as they were rounded
            assert np.array_equal(cache[0].view(torch.uint8).cpu().numpy(), want[0])
            T.check_out(out, lse, R.attention_ref(wq[..., :L], T.host(turned), held, table, [a + 1 for a in now], [0, 1, 2],
                                                  96 ** -0.5))
            eager, eager_lse = torch.empty_like(out), torch.empty_like(lse)
            dg.latent_attention(q[..., :L], turned, cache, t, lens, cu, 1, eager, eager_lse)
            assert torch.equal(eager, out) and torch.equal(eager_lse, lse)


def test_capture_needs_a_reserved_workspace(gpu):
    rng = np.random.default_rng(18)
    cache, table = T.filled(rng, [40], 16, 256, False)
    q, qr = (T.dev_bf16(y, gpu) for y in queries(rng, 1, 4, 256))
    out, c, t, kv, cu = torch.empty_like(q), T.upload(cache, gpu), i32(table, gpu), i32([40], gpu), i32([0, 1], gpu)
    side = T.OwnStream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with pytest.raises(dg.DGError) as refused:
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            dg.latent_attention(q, qr, c, t, kv, cu, 1, out)
    assert refused.value.status == 7
    torch.cuda.synchronize()


def test_workspace_covers_every_form(gpu, monkeypatch):
    for rows in [""] + ROWS:
        monkeypatch.setenv("DG_FORCE_CONFIG", rows)
        assert dg.latent_attention_workspace_size(512, 1, 128) >= dg.latent_attention_workspace_size(256, 1, 128) > 0
    monkeypatch.setenv("DG_FORCE_CONFIG", "")
    # whatever form a call takes by its table, the size without one is enough
    sizes = []
    for rows in ROWS:
        monkeypatch.setenv("DG_FORCE_CONFIG", rows)
        sizes.append(dg.latent_attention_workspace_size(512, 1, 64))
    monkeypatch.setenv("DG_FORCE_CONFIG", "")
    assert dg.latent_attention_workspace_size(512, 1, 64) == max(sizes)


def test_nothing_to_do(gpu):
    cache = dg.empty_latent_cache(2, 256, 16, "bf16", gpu)
    none = torch.empty((0, 4, 256), dtype=torch.bfloat16, device=gpu)
    t, cu, zero = torch.empty((0, 3), dtype=torch.int32, device=gpu), i32([0], gpu), torch.empty(0, dtype=torch.int32, device=gpu)
    assert dg.latent_attention(none, none[..., :32], cache, t, zero, cu, 0, none).shape == (0, 4, 256)
    dg.latent_append(none[:, 0], none[:, 0, :32], cache, t, zero, cu, 0, torch.empty((4, 32), device=gpu))
    dg.latent_gather(cache, t, cu, none[:, 0].contiguous(), none[:, 0, :32].contiguous())
    of = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=gpu)  # noqa: E731
    dg.latent_expanded_attention(of(0, 4, 96), of(0, 4, 128), of(0, 32), cu, cu, 0, of(0, 4, 64))
    # no blocks at all: queries see nothing, and rope parts of queries are turned all the same
    empty = dg.empty_latent_cache(0, 256, 16, "e4m3", gpu)
    q = torch.ones((2, 4, 256), dtype=torch.bfloat16, device=gpu)
    out = torch.full_like(q, float("nan"))
    dg.latent_attention(q, q[..., :32], empty, i32([[0], [0]], gpu), i32([5, 7], gpu), i32([0, 1, 2], gpu), 1, out)
    assert (out == 0).all()
    an = torch.cat((torch.zeros((9, 16)), torch.ones((9, 16))), 1).to(gpu)   # a quarter turn
    turned = torch.zeros((2, 4, 32), dtype=torch.bfloat16, device=gpu)
    dg.latent_append(q[:, 0], q[:, 0, :32], empty, i32([[0], [0]], gpu), i32([5, 7], gpu), i32([0, 1, 2], gpu), 1, an,
                     q_rope=q[..., :32], q_out=turned)
    assert (turned[..., 0::2] == -1).all() and (turned[..., 1::2] == 1).all()


def test_binding_refuses(gpu):
    cache, wide = dg.empty_latent_cache(4, 256, 16, "bf16", gpu), dg.empty_latent_cache(4, 256, 16, "e4m3", gpu)
    t, lens, cu = i32([[0, 1]], gpu), i32([3], gpu), i32([0, 1], gpu)
    c = torch.zeros((1, 256), dtype=torch.bfloat16, device=gpu)
    r, an = c[:, :32], torch.zeros((8, 32), device=gpu)
    q = torch.zeros((1, 4, 256), dtype=torch.bfloat16, device=gpu)
    out, two = torch.empty_like(q), torch.zeros((2, 256), dtype=torch.bfloat16, device=gpu)
    for i, (error, call) in enumerate([
        (TypeError, lambda: dg.latent_append(c.float(), r, cache, t, lens, cu, 1, an)),
        (ValueError, lambda: dg.latent_append(c, r[:, :16], cache, t, lens, cu, 1, an)),
        (ValueError, lambda: dg.latent_append(c, c[:, :64:2], cache, t, lens, cu, 1, an)),
        (ValueError, lambda: dg.latent_append(c, r, (cache[0], cache[1][:, :8], None), t, lens, cu, 1, an)),
        (TypeError, lambda: dg.latent_append(c, r, (wide[0], wide[1], None), t, lens, cu, 1, an)),
        (TypeError, lambda: dg.latent_append(c, r, (cache[0], cache[1], wide[2]), t, lens, cu, 1, an)),
        (ValueError, lambda: dg.latent_append(c, r, (wide[0], wide[1], wide[2][:2].contiguous()), t, lens, cu, 1, an)),
        (ValueError, lambda: dg.latent_append(c, r, cache, t, lens, i32([0, 1, 1], gpu), 1, an)),
        (ValueError, lambda: dg.latent_append(c, r, cache, t, i32([3, 3], gpu), cu, 1, an)),
        (ValueError, lambda: dg.latent_append(c, r, cache, t, lens, cu, 1, an[:, :16].contiguous())),
        (TypeError, lambda: dg.latent_append(c, r, cache, t, lens, cu, 1, an.double())),
        (ValueError, lambda: dg.latent_append(c, r, cache, t, lens, cu, 1, an, norm=c[0, :128].contiguous())),
        (ValueError, lambda: dg.latent_append(c, r, cache, t, lens, cu, 1, an, q_out=q[..., :32])),
        (ValueError, lambda: dg.latent_append(c, r, cache, t, lens, cu, 1, an, q_rope=q[..., :64])),
        (dg.DGError, lambda: dg.latent_append(c, r, cache, t, lens, cu, -1, an)),
        (dg.DGError, lambda: dg.latent_append(c, r, cache, t, lens, cu, 1, an, q_rope=q[..., 4:36])),     # 8 bytes off
        (ValueError, lambda: dg.latent_gather(cache, t, cu, two, two[:, :32])),                           # rope rows not packed
        (ValueError, lambda: dg.latent_gather(cache, t, cu, c, c[:, :64].contiguous())),
        (ValueError, lambda: dg.latent_gather(cache, t, cu, c, r.contiguous(), starts=i32([0, 0], gpu))),
        (ValueError, lambda: dg.latent_attention(q, q[..., :64], cache, t, lens, cu, 1, out)),
        (ValueError, lambda: dg.latent_attention(q, q[:, :2, :32], cache, t, lens, cu, 1, out)),
        (ValueError, lambda: dg.latent_attention(q, q[..., :32], cache, t, lens, cu, 1, out[..., :128])),
        (TypeError, lambda: dg.latent_attention(q, q[..., :32], cache, t.long(), lens, cu, 1, out)),
        (ValueError, lambda: dg.latent_attention(q, q[..., :32], cache, t, lens, cu, 1, out, torch.empty((1, 3), device=gpu))),
        (dg.DGError, lambda: dg.latent_attention(q, q[..., :32], cache, t, lens, cu, -1, out)),
        (dg.DGError, lambda: dg.latent_attention(q, q[..., :32], cache, t, lens, cu, 1, out, scale=-1.0)),
        (dg.DGError, lambda: dg.latent_attention(q, q[..., :32], cache, t, lens, cu, 1, out, scale=float("nan"))),
        (ValueError, lambda: dg.latent_expanded_attention(q[..., :96].contiguous(), q[..., :64], r, cu, cu, 1, out[..., :64].contiguous())),
        (ValueError, lambda: dg.latent_expanded_attention(q[..., :96], q[..., :128].contiguous(), r, cu, cu, 1, out[..., :64].contiguous())),
        (dg.DGError, lambda: dg.latent_expanded_attention(q[..., :48].contiguous(), q[..., :64].contiguous(), r[:, :16], cu, cu, 1,
                                                          out[..., :32].contiguous())),
        (ValueError, lambda: dg.empty_latent_cache(2, fmt="fp16")),
    ]):
        print("[case]", i, flush=True)
        with pytest.raises(error):
            call()
    odd = dg.empty_latent_cache(4, 384, 16, "bf16", gpu)
    d = torch.zeros((1, 384), dtype=torch.bfloat16, device=gpu)
    with pytest.raises(dg.DGError):
        dg.latent_append(d, d[:, :48], odd, t, lens, cu, 1, torch.zeros((8, 48), device=gpu))
    with pytest.raises(dg.DGError):
        dg.latent_gather(dg.empty_latent_cache(4, 256, 24, "bf16", gpu), t, cu, c, r.contiguous())
