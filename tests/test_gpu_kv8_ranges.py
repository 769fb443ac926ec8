"""The 8-bit paged KV cache's attention where magnitudes lie far apart: logits that outgrow the running reference
inside a tile of keys, V scales of blocks that are far from one another.  Every channel is held to its own bound (kv8_ref.py), so what a few tokens give to a channel
of their own counts, however small it is beside the others.  Needs a GPU."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as R
from test_gpu_kv8 import BF16, FP16, World, _check_attn, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    from sparse_attention_decode_csa2_gb300 import build
    build.build()
    from sparse_attention_decode_csa2_gb300 import csa2
    return csa2


def _tokens(w, s, k, v):
    """Codes of sequence s from values k, v [tokens][H_kv][D]."""
    for j in range(len(k)):
        p = w.table[s, j // w.page]
        w.k[p, :, j % w.page], w.v[p, :, j % w.page] = R.encode(k[j]), R.encode(v[j])


def _steps_of_logits(C, D, page, tokens, powers):
    """One sequence whose keys' logits are powers[token] (in powers of two) for queries of 1 in channel 0, and
    whose V has 1 in channel token // 64."""
    w = World(C, 81, [tokens], 1, D, page)
    k, v = np.zeros((tokens, 1, D)), np.zeros((tokens, 1, D))
    for j in range(tokens):
        k[j, 0, 0] = powers[j]
        v[j, 0, j // 64] = 1.0
    _tokens(w, 0, k, v)
    used = w.table[0]
    w.ks[used], w.vs[used] = 1.0, 1.0
    return w


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 128)])
@pytest.mark.parametrize("rows", [1, 40])
def test_attn_reference_that_moves_in_both_halves_of_every_tile(C, dtype, D, page, rows):
    # the logits grow by 11 powers of two every 64 keys: the reference moves in the first and in the second half
    # of each tile, and what was summed before is scaled down each time (2^-99 in the end, which bf16 keeps)
    n, step = (640, 11.0) if dtype == BF16 else (128, 9.0)
    w = _steps_of_logits(C, D, page, n, [step * (j // 64) for j in range(n)])
    q = torch.zeros((rows, 1, D), dtype=dtype)
    q[:, 0, 0] = 1.0
    _check_attn(C, w, q, None, causal=False, scale=math.log(2.0))


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("rows", [4, 40])
def test_attn_weights_that_the_reference_leaves_behind_keep_their_bits(C, D, page, rows):
    # the last token of a tile outgrows the others by 2^10 .. 2^20: their weights, formed before, are scaled down.
    # They alone reach channel 0, where they keep the bound of weights rounded once (the least is 2^-13, normal)
    w = World(C, 82, [128], 1, D, page)
    k, v = np.zeros((128, 1, D)), np.zeros((128, 1, D))
    k[:64, 0, 0] = np.arange(64) % 8 / 64
    k[127, 0, 0] = 1.0
    v[:64, 0, 0], v[64:, 0, 1] = 448.0, 1.0
    _tokens(w, 0, k, v)
    used = w.table[0]
    w.ks[used], w.vs[used] = 1.0, 2.0 ** 6
    q = torch.zeros((rows, 1, D), dtype=FP16)
    q[:, 0, 0] = torch.linspace(10.0, 19.75, rows)
    out, _ = _check_attn(C, w, q, None, causal=False, scale=math.log(2.0))
    assert (out[:, 0, 0] > 0.5).all()


# ------------------------------------------------------------------ V scales far apart

def _fill(w, v_of, ks=2.0 ** -8):
    """Codes and scales of every token: K at random, V and its block's scale from v_of(sequence, columns, codes):
    columns [tokens] of the block table, random codes' values [tokens][H_kv][D] -> (values, scales [columns])."""
    for s, L in enumerate(w.lens):
        if L == 0:
            continue
        j = np.arange(L)
        p, r = w.table[s, j // w.page], j % w.page
        w.k[p, :, r] = R.encode(60.0 * w.rng.standard_normal((L, w.Hk, w.D)))
        v, vs = v_of(s, j // w.page, 60.0 * w.rng.standard_normal((L, w.Hk, w.D)))
        w.v[p, :, r] = R.encode(v)
        used = w.table[s, :-(-L // w.page)]
        w.ks[used] = ks
        w.vs[used] = np.asarray(vs)[:, None]
    return w


def _queries(w, T, H, dtype):
    return torch.tensor(w.rng.standard_normal((T, H, w.D)) * 1.5, dtype=torch.float32).to(dtype)


FEW = [(1, 4), (6, 2), (13, 2)]   # rows of a sequence, query heads of a KV head: 4, 12 and 26 rows a unit


@pytest.mark.parametrize("n,G", FEW)
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 128), (64, 32)])
@pytest.mark.parametrize("apart", [6, 10, 20, 24, 28, 32, 40, 54])
@pytest.mark.parametrize("dtype,code", [(BF16, 100.0), (FP16, 0.0)])
def test_attn_blocks_with_an_outlier_leave_the_others_their_output(C, n, G, D, page, apart, dtype, code):
    _outlier_blocks(C, n, G, D, page, apart, dtype, code)


def _outlier_blocks(C, n, G, D, page, apart, dtype, code):
    # some blocks have a scale 2^apart times the others' and one channel (fp16: none) that is not zero there: the
    # other channels come from the small blocks alone.  They are the first block, the last, one between, every other
    last = lambda c: c == c.max()
    where = [lambda c: c == 0, last, lambda c: c == c.max() // 2, lambda c: c % 2 == 1]

    def v_of(s, col, v):
        big = where[s](np.arange(col.max() + 1))
        v[big[col]] = 0.0
        v[big[col], :, 5] = code
        return v, np.where(big, 2.0 ** (apart - 8), 2.0 ** -8)

    w = _fill(World(C, 83 + apart, [300, 333, 290, 512], 2, D, page), v_of)
    _check_attn(C, w, _queries(w, 4 * n, 2 * G, dtype), None)


@pytest.mark.parametrize("n,G", FEW)
@pytest.mark.parametrize("D", [64, 128])
def test_attn_outlier_blocks_in_other_parts_of_a_long_context(C, n, G, D):
    _outlier_parts(C, n, G, D)


def _outlier_parts(C, n, G, D):
    # a context that is split over the grid: runs of small blocks and runs with an outlier, 2^40 apart
    def v_of(s, col, v):
        big = np.arange(col.max() + 1) // 9 % 2 == 1
        v[big[col]] = 0.0
        v[big[col], :, 5] = 100.0
        return v, np.where(big, 2.0 ** 32, 2.0 ** -8)

    w = _fill(World(C, 84, [9001], 1, D, 64), v_of)
    q = _queries(w, n, G, BF16)
    a = _check_attn(C, w, q, None)
    b = _check_attn(C, w, q, None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,G", FEW)
@pytest.mark.parametrize("big", [2.0 ** -8, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("lens,page", [([200, 130, 64, 333], 16), ([200, 130, 64, 333], 128), ([7001], 64)])
def test_attn_blocks_of_zeros_count_in_the_sum(C, n, G, big, lens, page):
    _zero_blocks(C, n, G, big, lens, page)


def _zero_blocks(C, n, G, big, lens, page):
    # blocks of zeros, which append gives the scale 2^-100, beside others up to 2^200 above: in a tile, in the tiles
    # of other warps, in other parts
    def v_of(s, col, v):
        zero = (np.arange(col.max() + 1) + s) // 2 % 2 == 0
        v[zero[col]] = 0.0
        return v, np.where(zero, 2.0 ** -100, big)

    w = _fill(World(C, 85, lens, 2, 64, page), v_of)
    _check_attn(C, w, _queries(w, n * len(lens), 2 * G, BF16), None)


@pytest.mark.parametrize("n,G", FEW)
def test_attn_a_head_without_values_has_a_finite_lse(C, n, G):
    _no_values(C, n, G)


def _no_values(C, n, G):
    # every block of V is zeros (scale 2^-100) and all logits are zero, over more than 2^22 tokens.  The sum of the
    # weights, all one power of two, is exact
    D, page, tokens = 64, 128, (1 << 22) + 333
    P = -(-tokens // page)
    z = lambda: torch.zeros((P, 1, page, D), dtype=torch.uint8, device="cuda")
    cache = C.Kv8Cache(z(), z(), torch.ones((P, 1), device="cuda"), torch.full((P, 1), 2.0 ** -100, device="cuda"))
    i = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    batch = C.Kv8Batch(torch.randperm(P).to(torch.int32).cuda().reshape(1, P), i([tokens]), n)
    out, lse = C.kv8_attn(torch.ones((n, G, D), dtype=BF16).cuda(), cache, batch)
    assert (out == 0).all()
    want = torch.log(torch.arange(tokens - n + 1, tokens + 1, dtype=torch.float64))[:, None]
    assert (lse.cpu().double() - want).abs().max() <= 2.0 ** -20 * 16


@pytest.mark.parametrize("n,G", FEW)
@pytest.mark.parametrize("page", [16, 64])
def test_attn_scales_past_2_to_60_apart_lose_only_what_is_that_small(C, n, G, page):
    _past_range(C, n, G, page)


def _past_range(C, n, G, page):
    # scales from 2^-90 to 2^90, every channel of every block: lse as ever, out to 2^-51 of the largest scale
    # that the sequence has, beside the bound
    rng = np.random.default_rng(88)
    w = _fill(World(C, 87, [400, 90, 250], 1, 64, page),
              lambda s, col, v: (v, 2.0 ** rng.integers(-90, 91, col.max() + 1)))
    q = _queries(w, 3 * n, G, BF16)
    cache, batch = w.cache(), w.batch(3 * n)
    out, lse = C.kv8_attn(q.cuda(), cache, batch)
    ref = R.attention(q.double().numpy(), (w.k, w.v, w.ks, w.vs), w.table, w.lens, R.rows_of(3 * n, 3, None), page,
                      True, 0, 1 / 8)
    tol_o, tol_l = R.attention_bounds(*ref, 64, 400, BF16)
    for s, L in enumerate(w.lens):
        tol_o[s * n:s * n + n] += 2.0 ** -51 * w.vs[w.table[s, :-(-L // page)]].max()
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol_o).all()
    got, none = lse.double().cpu().numpy(), np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(got), none)
    assert (np.abs(got[~none] - ref[1][~none]) <= tol_l[~none]).all()



@pytest.mark.parametrize("n,G", FEW)
@pytest.mark.parametrize("page", [16, 128])
def test_attn_a_block_of_nan_is_seen_beside_large_ones(C, n, G, page):
    _nan_block(C, n, G, page)


def _nan_block(C, n, G, page):
    # append gives a block without a number the least scale; its NaN reach the rows that see it all the same
    w = _fill(World(C, 89, [400, 300], 1, 64, page), lambda s, col, v: (v, np.full(col.max() + 1, 2.0 ** -8)))
    p = w.table[0, 128 // page]
    w.v[p, :, :, 3], w.vs[p] = 0x7F, 2.0 ** -100
    q = _queries(w, 2 * n, G, BF16)
    out, lse = C.kv8_attn(q.cuda(), w.cache(), w.batch(2 * n))
    assert torch.isnan(out[:n, :, 3]).all() and torch.isfinite(out[n:]).all() and torch.isfinite(lse[n:]).all()


# The same of prompts: units of one and of two row tiles.
MANY = [(40, 2), (150, 1)]


@pytest.mark.parametrize("n,G", MANY)
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 128), (64, 32), (128, 16)])
@pytest.mark.parametrize("apart", [6, 10, 20, 24, 28, 32, 40, 54])
@pytest.mark.parametrize("dtype,code", [(BF16, 100.0), (FP16, 0.0)])
def test_prompts_blocks_with_an_outlier_leave_the_others_their_output(C, n, G, D, page, apart, dtype, code):
    _outlier_blocks(C, n, G, D, page, apart, dtype, code)


@pytest.mark.parametrize("n,G", MANY)
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_outlier_blocks_in_other_parts_of_a_long_context(C, n, G, D):
    _outlier_parts(C, n, G, D)


@pytest.mark.parametrize("n,G", MANY)
@pytest.mark.parametrize("big", [2.0 ** -8, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("lens,page", [([200, 160, 333], 16), ([200, 160, 333], 128), ([7001], 64)])
def test_prompts_blocks_of_zeros_count_in_the_sum(C, n, G, big, lens, page):
    _zero_blocks(C, n, G, big, lens, page)


def test_prompts_a_head_without_values_has_a_finite_lse(C):
    _no_values(C, 40, 1)


@pytest.mark.parametrize("n,G", MANY)
@pytest.mark.parametrize("page", [16, 64])
def test_prompts_scales_past_2_to_60_apart_lose_only_what_is_that_small(C, n, G, page):
    _past_range(C, n, G, page)


@pytest.mark.parametrize("n,G", MANY)
@pytest.mark.parametrize("page", [16, 128])
def test_prompts_a_block_of_nan_is_seen_beside_large_ones(C, n, G, page):
    _nan_block(C, n, G, page)


@pytest.mark.parametrize("n,G", FEW + MANY)
@pytest.mark.parametrize("page", [16, 32])
def test_attn_scales_that_change_with_every_block(C, n, G, page):
    # eight scales in turn, 2^8 apart, in tiles of several blocks; the logits grow, so that the reference moves too
    def v_of(s, col, v):
        return v, 2.0 ** (8.0 * (np.arange(col.max() + 1) * 5 % 8) - 30)

    w = _fill(World(C, 90, [700, 300], 1, 128, page), v_of)
    for s, L in enumerate(w.lens):
        j = np.arange(L)
        w.k[w.table[s, j // page], 0, j % page, 0] = R.encode(np.minimum(0.6 * j, 448.0))
    q = _queries(w, 2 * n, G, BF16)
    q[:, :, 0] = 4.0
    _check_attn(C, w, q, None, scale=0.3 / 8)


@pytest.mark.parametrize("n,G", FEW + MANY)
def test_attn_an_infinite_value_without_weight_stays_out_of_a_long_context(C, n, G):
    # append stores infinities as 448 at a scale of 2^120, past fp32.  A run of them, which fills the parts of several
    # CTAs, has logits 250 powers of two below the rest (softmax weights of zero): no NaN, and lse as ever
    def v_of(s, col, v):
        big = (np.arange(col.max() + 1) >= 40) & (np.arange(col.max() + 1) < 80)
        v[big[col]] = 0.0
        v[big[col], :, 5] = 448.0
        return v, np.where(big, 2.0 ** 120, 2.0 ** -8)

    w = _fill(World(C, 92, [9001], 1, 64, 64), v_of)
    j = np.arange(9001)
    w.k[w.table[0, j // 64], 0, j % 64, 0] = R.encode(np.where((j // 64 >= 40) & (j // 64 < 80), -448.0, 448.0))
    q = _queries(w, n, G, BF16)
    q[:, :, 0] = 400.0
    cache, batch = w.cache(), w.batch(n)
    out, lse = C.kv8_attn(q.cuda(), cache, batch, causal=False)
    ref = R.attention(q.double().numpy(), (w.k, w.v, w.ks, w.vs), w.table, w.lens, R.rows_of(n, 1, None), 64, False,
                      0, 1 / 8)
    _, tol_l = R.attention_bounds(*ref, 64, 9001, BF16)
    assert torch.isfinite(out).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_l).all()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_append_an_infinity_beside_finite_values(C, D, page):
    # the whole block goes to the largest scale, older rows too, until its page starts anew
    Hk, steps = 2, [page + 5, 1, 2, page, page]
    w = World(C, 93, [sum(steps)], Hk, D, page)
    cache, length = w.cache(), 0
    for i, n in enumerate(steps):
        length += n
        k, v = (_rows(w.rng, n, Hk, D, FP16, 3.0) for _ in range(2))
        if i == 1:
            k[0, 0, 3], v[0, 1, 7], v[0, 1, 8] = math.inf, -math.inf, math.nan
        C.kv8_append(cache, w.batch(n, None, [length]), k.cuda(), v.cuda())
        for codes, sc, x in ((w.k, w.ks, k), (w.v, w.vs, v)):
            R.append(codes, sc, x.double().numpy(), w.table, [length], [(0, n)], page)
        w.same(cache)
    assert w.ks[w.table[0, 1], 0] == 2.0 ** 120 and w.ks[w.table[0, 2], 0] < 1.0


@pytest.mark.parametrize("n,G", FEW + MANY)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("causal,window", [(True, 90), (False, 0)])
@pytest.mark.parametrize("apart", [30, 54])
def test_attn_outlier_blocks_and_rows_that_do_not_see_them(C, n, G, D, page, causal, window, apart):
    # every third block has an outlier; through the window some rows of a unit see it and others do not
    def v_of(s, col, v):
        big = np.arange(col.max() + 1) % 3 == s
        v[big[col]] = 0.0
        v[big[col], :, 5] = 100.0
        return v, np.where(big, 2.0 ** (apart - 8), 2.0 ** -8)

    w = _fill(World(C, 94, [600, 431, 150], 1, D, page), v_of)
    _check_attn(C, w, _queries(w, 3 * n, G, BF16), None, causal, window)
