"""The 8-bit paged KV cache on the GPU: writer and reader bit for bit, attention within the bounds that
kv8_ref.py derives, at sizes and masks where they can go wrong.  Needs a GPU."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as R

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def C():
    from sparse_attention_decode_csa2_gb300 import build
    build.build()
    from sparse_attention_decode_csa2_gb300 import csa2
    return csa2


class World:
    """A cache with pages in random order, its host copy, and the sequences' block table."""

    def __init__(self, C, seed, lens, Hk, D, page, spare=3, wide=None):
        self.C, self.rng = C, np.random.default_rng(seed)
        self.Hk, self.D, self.page = Hk, D, page
        need = [-(-L // page) for L in lens]
        P = sum(need) + spare
        # every byte and scale that no token owns is a NaN: it must never reach a result
        self.k = np.full((P, Hk, page, D), 0x7F, np.uint8)
        self.v = np.full((P, Hk, page, D), 0xFF, np.uint8)
        self.ks, self.vs = (np.full((P, Hk), np.nan, np.float32) for _ in range(2))
        order, at = self.rng.permutation(P), 0
        self.table = np.full((len(lens), wide or max(1, max(need))), -1, np.int32)
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        self.lens = list(lens)

    def fill(self, span=3):
        """Every token's codes and its block's scale."""
        for s, L in enumerate(self.lens):
            for j in range(L):
                p = self.table[s, j // self.page]
                for c in (self.k, self.v):
                    c[p, :, j % self.page] = R.encode(60.0 * self.rng.standard_normal((self.Hk, self.D)))
                if j % self.page == 0:
                    self.ks[p] = 2.0 ** self.rng.integers(-8, -8 + span, self.Hk)
                    self.vs[p] = 2.0 ** self.rng.integers(-8, -8 + span, self.Hk)
        return self

    def cache(self):
        f = lambda a: torch.from_numpy(a.copy()).cuda()
        return self.C.Kv8Cache(f(self.k), f(self.v), f(self.ks), f(self.vs))

    def batch(self, rows, cu=None, lens=None, extra=0):
        i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32).cuda()
        return self.C.Kv8Batch(i(self.table), i(self.lens if lens is None else lens), rows + extra,
                               None if cu is None else i(cu))

    def same(self, cache):
        for got, ref in ((cache.k, self.k), (cache.v, self.v)):
            g = got.cpu().numpy()
            assert (g == ref).all(), np.argwhere(g != ref)[:4]
        for got, ref in ((cache.k_scale, self.ks), (cache.v_scale, self.vs)):
            assert np.array_equal(got.cpu().numpy(), ref, equal_nan=True)


def _rows(rng, T, H, D, dtype, gain):
    x = rng.standard_normal((T, H, D)) * gain
    return torch.tensor(x, dtype=FP32).to(dtype)


# ------------------------------------------------------------------ writer

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D,page,Hk", [(128, 64, 2), (64, 16, 3), (128, 128, 1), (64, 128, 2), (128, 32, 1)])
def test_append_over_several_steps_is_bit_exact(C, dtype, D, page, Hk):
    # prompt, then single tokens and short drafts whose magnitudes grow and shrink, so that scales grow in
    # partly filled pages; lengths cross page borders
    S, steps = 5, [None, 1, 1, 3, 1, page + 3, 1]
    prompt = [1, page - 1, page, page + 1, 2 * page + 5]
    total = sum(n for n in steps if n)
    w = World(C, 7, [L + total for L in prompt], Hk, D, page)
    cache, lens = w.cache(), [0] * S
    gains = [1.0, 4.0, 0.01, 100.0, 1.0, 1e-4, 3000.0]
    for n, gain in zip(steps, gains):
        if n is None:
            cu = np.concatenate([[0], np.cumsum(prompt)])
            T, add = int(cu[-1]), prompt
        else:
            cu, T, add = None, n * S, [n] * S
        lens = [a + b for a, b in zip(lens, add)]
        k, v = (_rows(w.rng, T, Hk, D, dtype, gain) for _ in range(2))
        k[0, 0, 0], v[-1, -1, -1] = 0.0, -0.0
        C.kv8_append(cache, w.batch(T, cu, lens), k.cuda(), v.cuda())
        shares = R.rows_of(T, S, None if cu is None else cu.tolist())
        R.append(w.k, w.ks, k.double().numpy(), w.table, lens, shares, page)
        R.append(w.v, w.vs, v.double().numpy(), w.table, lens, shares, page)
        w.same(cache)


def test_append_strided_rows_of_a_joint_projection(C):
    S, Hk, D, page = 3, 2, 128, 32
    w = World(C, 1, [70, 33, 9], Hk, D, page)
    cu = [0, 70, 103, 112]
    qkv = _rows(w.rng, 112, 9, D, BF16, 1.0)
    cache = w.cache()
    dev = qkv.cuda()
    C.kv8_append(cache, w.batch(112, cu), dev[:, 5:7], dev[:, 7:9])
    for codes, sc, x in ((w.k, w.ks, qkv[:, 5:7]), (w.v, w.vs, qkv[:, 7:9])):
        R.append(codes, sc, x.double().numpy(), w.table, w.lens, R.rows_of(112, S, cu), page)
    w.same(cache)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_append_extreme_values(C, dtype):
    # blocks of zeros, infinities, NaN, the largest and the smallest numbers, midpoints between codes
    D, page, big = 64, 16, float(torch.finfo(dtype).max)
    rows = [np.zeros(D), np.full(D, big), np.full(D, -np.inf), np.full(D, 1e-38), np.full(D, 448.0)]
    mid = np.array([(R.E4M3[i] + R.E4M3[i + 1]) / 2 for i in range(0, 126)])
    rows += [np.concatenate([[448.0], mid[:63]]), np.concatenate([[-448.0], -mid[63:126]])]
    nan = np.linspace(-3, 3, D)
    nan[5] = np.nan
    rows += [nan, np.concatenate([np.full(D - 1, 1.0), [449.0]]), np.full(D, 2.0 ** -110)]
    S = len(rows)
    x = torch.tensor(np.stack(rows)[:, None], dtype=FP32).to(dtype)
    w = World(C, 3, [1] * S, 1, D, page)
    cache = w.cache()
    C.kv8_append(cache, w.batch(S), x.cuda(), (-x).cuda())
    for codes, sc, y in ((w.k, w.ks, x), (w.v, w.vs, -x)):
        R.append(codes, sc, y.double().numpy(), w.table, w.lens, R.rows_of(S, S, None), page)
    w.same(cache)


def test_append_leaves_idle_slots_and_later_rows_alone(C):
    # idle sequences (no tokens), sequences shorter than their share, rows of no sequence
    Hk, D, page = 2, 128, 16
    w = World(C, 5, [0, 2, 40, 17], Hk, D, page).fill()
    lens, cache = [0, 2, 40, 17], w.cache()
    k, v = (_rows(w.rng, 12, Hk, D, FP16, 50.0) for _ in range(2))
    C.kv8_append(cache, w.batch(12), k.cuda(), v.cuda())  # three rows each: sequence 1 has two tokens
    for codes, sc, x in ((w.k, w.ks, k), (w.v, w.vs, v)):
        R.append(codes, sc, x.double().numpy(), w.table, lens, R.rows_of(12, 4, None), page)
    w.same(cache)
    cu = [0, 0, 1, 3, 3]
    C.kv8_append(cache, w.batch(3, cu, extra=9), k.cuda(), v.cuda())
    for codes, sc, x in ((w.k, w.ks, k), (w.v, w.vs, v)):
        R.append(codes, sc, x.double().numpy(), w.table, lens, R.rows_of(3, 4, cu), page)
    w.same(cache)


def test_append_many_sequences_with_uneven_rows(C):
    # more sequences than one search round covers, with runs of empty ones
    rng = np.random.default_rng(11)
    S, Hk, D, page = 1100, 1, 64, 16
    n = rng.integers(0, 4, S) * (rng.random(S) < 0.6) + 40 * (rng.random(S) < 0.02)
    lens = (n + rng.integers(0, 20, S)).tolist()
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    w = World(C, 12, lens, Hk, D, page).fill()
    cache = w.cache()
    k, v = (_rows(w.rng, cu[-1], Hk, D, BF16, 2.0) for _ in range(2))
    C.kv8_append(cache, w.batch(cu[-1], cu), k.cuda(), v.cuda())
    for codes, sc, x in ((w.k, w.ks, k), (w.v, w.vs, v)):
        R.append(codes, sc, x.double().numpy(), w.table, lens, R.rows_of(cu[-1], S, cu), page)
    w.same(cache)


# ------------------------------------------------------------------ reader

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D,page,Hk,cu", [(128, 64, 2, [0, 130, 131, 131, 200]), (64, 16, 3, [0, 3, 50, 67, 67]),
                                          (128, 128, 1, None), (64, 32, 5, None)])
def test_read_is_bit_exact(C, dtype, D, page, Hk, cu):
    lens = [130, 77, 0, 300]
    w = World(C, 21, lens, Hk, D, page).fill(span=9)
    T = cu[-1] if cu else 4 * 65
    k, v = C.kv8_read(w.cache(), w.batch(T, cu), dtype)
    for got, codes, sc in ((k, w.k, w.ks), (v, w.v, w.vs)):
        ref = torch.zeros((T, Hk, D), dtype=torch.float64)
        for s, (r0, n) in enumerate(R.rows_of(T, 4, cu)):
            lo = max(0, lens[s] - n)
            if lens[s] > lo:
                ref[r0 + n - (lens[s] - lo):r0 + n] = torch.from_numpy(
                    R.gather(codes, sc, w.table[s], lo, lens[s], page))
        assert torch.equal(got.cpu(), ref.to(dtype))


def test_read_leaves_rows_of_no_sequence(C):
    w = World(C, 22, [9, 20], 2, 64, 16).fill()
    out_k, out_v = (torch.full((40, 2, 64), 7.0, dtype=FP16, device="cuda") for _ in range(2))
    C.kv8_read(w.cache(), w.batch(29, [0, 9, 29], extra=11), FP16, out_k, out_v)
    assert (out_k[29:] == 7).all() and (out_v[29:] == 7).all()
    assert not (out_k[:29] == 7).all(dim=(1, 2)).any()


# ------------------------------------------------------------------ attention

def _check_attn(C, w, q, cu, causal=True, window=0, scale=None, lens=None, extra=0, **kw):
    T, H, D = q.shape
    T -= extra
    lens = w.lens if lens is None else lens
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    cache, batch = w.cache(), w.batch(T, cu, lens, extra)
    ws = C.make_kv8_workspace(cache, batch, H)
    out, lse = C.kv8_attn(q.cuda(), cache, batch, causal, window, scale, ws=ws, **kw)
    assert C.read_status(ws) == (0, 0)
    shares = R.rows_of(T, len(lens), cu)
    ref = R.attention(q[:T].double().numpy(), (w.k, w.v, w.ks, w.vs), w.table, lens, shares, w.page, causal,
                      window, scale)
    tol_o, tol_l = R.attention_bounds(*ref, D, max(1, max(lens)), q.dtype)
    got_o, got_l = out[:T].double().cpu().numpy(), lse[:T].double().cpu().numpy()
    empty = np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(got_l), empty)
    assert (got_o[empty] == 0).all()
    off = np.abs(got_o - ref[0]) - tol_o
    assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:4])
    off = np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, ref[1])) - tol_l
    assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:4])
    return out, lse


def _q(rng, T, H, D, dtype, gain=1.5):
    return torch.tensor(rng.standard_normal((T, H, D)) * gain, dtype=FP32).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 16), (64, 128), (128, 32), (128, 128)])
@pytest.mark.parametrize("Hk,G", [(2, 1), (1, 8), (3, 5), (1, 16)])
def test_attn_single_tokens(C, dtype, D, page, Hk, G):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257, 700]
    w = World(C, D + page + G, lens, Hk, D, page).fill()
    _check_attn(C, w, _q(w.rng, len(lens), Hk * G, D, dtype), None)


@pytest.mark.parametrize("n", [2, 3, 8])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (False, 0)])
@pytest.mark.parametrize("D,page,Hk,G", [(128, 64, 1, 4), (64, 32, 2, 7)])
def test_attn_drafted_tokens(C, n, causal, window, D, page, Hk, G):
    # sequences shorter than their share: their first rows see nothing
    lens = [1, n, n + 1, 64, 130, 0, 333]
    w = World(C, n + window, lens, Hk, D, page).fill()
    _check_attn(C, w, _q(w.rng, n * len(lens), Hk * G, D, BF16), None, causal, window)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
@pytest.mark.parametrize("D,page,Hk,G", [(128, 64, 1, 4), (64, 128, 2, 3), (128, 16, 1, 1), (64, 64, 1, 16)])
def test_attn_prompts_of_uneven_lengths(C, dtype, causal, window, D, page, Hk, G):
    n = [1, 130, 0, 47, 129]
    lens = [5, 130, 64, 300, 500]
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    w = World(C, 31, lens, Hk, D, page).fill()
    _check_attn(C, w, _q(w.rng, cu[-1], Hk * G, D, dtype), cu, causal, window)


@pytest.mark.parametrize("D,page,G,n", [(128, 64, 17, 1), (64, 16, 32, 1), (128, 32, 33, 2), (128, 64, 64, 1),
                                        (64, 64, 65, 1), (128, 128, 100, 2), (64, 32, 256, 1), (128, 16, 129, 1)])
def test_attn_many_query_heads_per_kv_head(C, D, page, G, n):
    lens = [1, 33, 0, 200, 385]
    w = World(C, 32 + G, lens, 1, D, page).fill()
    _check_attn(C, w, _q(w.rng, n * len(lens), G, D, BF16), None)


@pytest.mark.parametrize("D,page,window", [(128, 64, 0), (64, 16, 0), (128, 16, 700)])
def test_attn_chunk_over_a_long_context_is_split(C, D, page, window):
    # two units over a long context: the tokens are split over every CTA and joined
    w = World(C, 33, [6001], 2, D, page).fill()
    q = _q(w.rng, 67, 4, D, BF16)
    a = _check_attn(C, w, q, None, True, window)
    b = _check_attn(C, w, q, None, True, window)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D", [64, 128])
def test_attn_prompt_rows_with_growing_logits(C, D):
    # logits that grow along the keys: the running maximum moves in every tile, past a lazy margin
    L = 700
    w = World(C, 34, [L], 1, D, 64).fill(span=1)
    for j in range(L):
        p = w.table[0, j // 64]
        w.k[p, 0, j % 64] = R.encode(R.E4M3[w.k[p, 0, j % 64]] * 0.02)
        w.k[p, 0, j % 64, 0] = R.encode(np.array(0.6 * j))
        w.ks[p] = 2.0 ** -3
    q = _q(w.rng, 140, 1, D, BF16, 0.2)
    q[:, 0, 0] = 4.0
    _check_attn(C, w, q, None, scale=0.3)


@pytest.mark.parametrize("wide", [None, 40])
@pytest.mark.parametrize("S,G,choices", [(300, 1, [1]), (300, 4, [0, 1, 1, 1, 2, 5, 20]), (560, 16, [0, 1, 2, 3, 4, 30])])
def test_attn_many_sequences(C, S, G, choices, wide):
    # more sequences than the warps of a CTA look at in one step, some of several blocks of rows
    rng = np.random.default_rng(S + G)
    n = rng.choice(choices, S)
    lens = [int(m + x) for m, x in zip(n, rng.integers(0, 60, S))]
    w = World(C, 71, lens, 1, 64, 16, wide=wide).fill()
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    _check_attn(C, w, _q(w.rng, cu[-1], G, 64, BF16), cu)


@pytest.mark.parametrize("n", [1, 50])
def test_attn_sequences_may_share_pages(C, n):
    # a prefix that two sequences share, and a page that one of them has twice
    w = World(C, 72, [160, 160, 100], 2, 64, 32).fill()
    w.table[1, :3] = w.table[0, :3]
    w.table[2, 1] = w.table[2, 0]
    _check_attn(C, w, _q(w.rng, 3 * n, 4, 64, BF16), None)


def test_attn_long_context_split_over_the_grid(C):
    # two sequences, one head: the tokens are split over every CTA and joined
    lens = [5000, 3001]
    w = World(C, 41, lens, 1, 128, 64).fill()
    q = _q(w.rng, 2, 8, 128, BF16)
    a = _check_attn(C, w, q, None)
    b = _check_attn(C, w, q, None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits twice


def test_attn_scales_far_apart(C):
    # block scales from 2^-60 to 2^60: weights and scales must not overflow or vanish together
    w = World(C, 42, [200, 400], 2, 64, 16).fill()
    for sc in (w.ks, w.vs):
        ok = ~np.isnan(sc)
        sc[ok] = 2.0 ** np.where(w.rng.random(ok.sum()) < 0.1, -60, w.rng.integers(-8, -4, ok.sum()))
    w.vs[w.table[0, 0]] = 2.0 ** 60
    w.ks[w.table[0, 0]] = 2.0 ** -9
    _check_attn(C, w, _q(w.rng, 2, 8, 64, BF16), None)


def test_attn_queries_of_extreme_magnitude(C):
    w = World(C, 43, [100] * 4, 1, 128, 64).fill()
    q = _q(w.rng, 4, 4, 128, BF16)
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2] = 0
    q[3, :, 7] *= 3e4
    # row 0: logits of about 1e30; only its finiteness and its largest token are defined
    w2 = World(C, 43, [100] * 4, 1, 128, 64).fill()
    cache, batch = w2.cache(), w2.batch(4)
    out, lse = C.kv8_attn(q.cuda(), cache, batch)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    z = R.gather(w.k, w.ks, w.table[0], 0, 100, 64)[:, 0] @ q[0].double().numpy().T
    V = R.gather(w.v, w.vs, w.table[0], 0, 100, 64)[:, 0]
    for h in range(4):
        assert torch.equal(out[0, h].cpu(), torch.from_numpy(V[z[:, h].argmax()]).to(BF16))
    ref = R.attention(q[1:].double().numpy(), (w.k, w.v, w.ks, w.vs), w.table[1:], [100] * 3,
                      R.rows_of(3, 3, None), 64, True, 0, 1 / math.sqrt(128))
    tol_o, tol_l = R.attention_bounds(*ref, 128, 100, BF16)
    assert (np.abs(out[1:].double().cpu().numpy() - ref[0]) <= tol_o).all()
    assert (np.abs(lse[1:].double().cpu().numpy() - ref[1]) <= tol_l).all()


def test_attn_prompt_queries_of_extreme_magnitude(C):
    # as above for prompts: logits of 1e30 (only the largest token counts), 1e5, 1e-30 and 0
    n, D = 80, 128
    w = World(C, 47, [300] * 3, 1, D, 64).fill()
    q = _q(w.rng, 3 * n, 2, D, BF16)
    q[:n:2] *= 1e30
    q[1:n:2] *= 1e5
    q[n:2 * n:2] *= 1e-30
    q[n + 1:2 * n:2] = 0
    cache, batch = w.cache(), w.batch(3 * n)
    out, lse = C.kv8_attn(q.cuda(), cache, batch)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    V = R.gather(w.v, w.vs, w.table[0], 0, 300, 64)[:, 0]
    z = R.gather(w.k, w.ks, w.table[0], 0, 300, 64)[:, 0] @ q[:n].double().numpy().transpose(0, 2, 1)  # [n][300][2]
    for i in range(0, n, 2):
        for h in range(2):
            best = z[i, :300 - n + i + 1, h].argmax()
            assert torch.equal(out[i, h].cpu(), torch.from_numpy(V[best]).to(BF16)), (i, h)
    ref = R.attention(q[n:].double().numpy(), (w.k, w.v, w.ks, w.vs), w.table[1:], [300] * 2,
                      R.rows_of(2 * n, 2, None), 64, True, 0, 1 / math.sqrt(D))
    tol_o, tol_l = R.attention_bounds(*ref, D, 300, BF16)
    assert (np.abs(out[n:].double().cpu().numpy() - ref[0]) <= tol_o).all()
    assert (np.abs(lse[n:].double().cpu().numpy() - ref[1]) <= tol_l).all()


def test_attn_a_long_tail_of_small_weights_is_not_lost(C):
    # one token with weight near 1 and 4096 tokens 2^-20 below it that all share a direction
    D, L = 64, 4097
    w = World(C, 44, [L], 1, D, 64)
    codes = np.zeros((L, D))
    codes[0, 0], codes[1:, 1] = 1.0, 256.0
    kk = np.zeros((L, D))
    kk[0, 0] = 20 * math.log(2) * 8
    for j in range(L):
        p = w.table[0, j // 64]
        w.k[p, 0, j % 64], w.v[p, 0, j % 64] = R.encode(kk[j]), R.encode(codes[j])
        w.ks[p], w.vs[p] = 1.0, 1.0
    q = torch.zeros((1, 1, D), dtype=BF16)
    q[0, 0, 0] = 1.0
    out, _ = _check_attn(C, w, q, None, scale=1.0 / 8)
    assert out[0, 0, 1] > 0.5


def test_attn_strided_queries_and_padded_rows(C):
    cu = [0, 3, 60]
    w = World(C, 45, [40, 200], 2, 64, 16).fill()
    q = _q(w.rng, 75, 12, 64, FP16)
    out = torch.full((75, 8, 64), 3.0, dtype=FP16, device="cuda")
    lse = torch.full((75, 8), 5.0, device="cuda")
    _check_attn(C, w, q[:, 2:10], cu, extra=15, out=out, lse=lse)
    assert (out[60:] == 3).all() and (lse[60:] == 5).all()


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("G,n,window", [(4, [4, 4, 4], 0), (4, [8, 8, 8], 0), (2, [6, 6, 6], 40), (3, [10, 10, 10], 33),
                                        (4, [150, 60, 300], 0), (3, [150, 70, 300], 50), (16, [5, 9, 17], 0)])
def test_attn_nan_of_a_token_stays_with_the_rows_that_see_it(C, D, page, G, n, window):
    Hk, lens = 2, [150, 73, 409]
    w = World(C, 48 + G, lens, Hk, D, page).fill()
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    q = _q(w.rng, cu[-1], Hk * G, D, BF16)
    # a NaN in V of head 0 of some tokens of this step (and one before it), in K of head 1 of another
    k, v = w.k.copy(), w.v.copy()
    vs_, ks_ = [], []
    for s, L in enumerate(lens):
        for j in (L - 2, L - n[s] + n[s] // 2, max(0, L - n[s] - 20)):
            vs_.append((s, j, int(w.rng.integers(D))))
        ks_.append((s, L - 1 - n[s] // 3))
    for s, j, c in vs_:
        v[w.table[s, j // page], 0, j % page, c] = 0x7F if j & 1 else 0xFF
        w.v[w.table[s, j // page], 0, j % page, c] = 0
    for s, j in ks_:
        k[w.table[s, j // page], 1, j % page, 3] = 0x7F
        w.k[w.table[s, j // page], 1, j % page, 3] = 0
    f = lambda a: torch.from_numpy(a.copy()).cuda()
    cache, batch = C.Kv8Cache(f(k), f(v), f(w.ks), f(w.vs)), w.batch(cu[-1], cu)
    out, lse = C.kv8_attn(q.cuda(), cache, batch, True, window)
    shares = R.rows_of(cu[-1], 3, cu)
    ref = R.attention(q.double().numpy(), (w.k, w.v, w.ks, w.vs), w.table, lens, shares, page, True, window,
                      1 / math.sqrt(D))
    tol_o, tol_l = R.attention_bounds(*ref, D, max(lens), BF16)
    got_o, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    clean = np.ones((cu[-1], Hk * G), bool)
    for s, (r0, m) in enumerate(shares):
        pos = lens[s] - m + np.arange(m)
        sees = lambda j: (pos >= j) & ((pos - j < window) if window else True)
        for t, j, c in vs_:
            if t == s:
                rows = r0 + np.flatnonzero(sees(j))
                assert np.isnan(got_o[rows, :G, c]).all()
                clean[rows, :G] = False
        for t, j in ks_:
            if t == s:
                rows = r0 + np.flatnonzero(sees(j))
                assert np.isnan(got_o[rows, G:]).all() and np.isnan(got_l[rows, G:]).all()
                clean[rows, G:] = False
    assert clean.any() and not clean.all()
    assert (np.abs(got_o - ref[0]) <= tol_o)[clean].all()
    assert (np.abs(got_l - ref[1]) <= tol_l)[clean].all()


def test_attn_without_a_causal_mask_takes_more_rows_than_tokens(C):
    w = World(C, 49, [3, 0, 17], 2, 64, 16).fill()
    _check_attn(C, w, _q(w.rng, 15, 4, 64, FP16), None, causal=False)
    _check_attn(C, w, _q(w.rng, 165, 4, 64, FP16), None, causal=False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_attn_window_of_whole_units(C, D, n):
    # up to 512 visible tokens a unit stays with one CTA, past it units are cut: the same sums either way
    w = World(C, 50 + n, [1400, 30], 1, D, 32).fill()
    for window in (512, 513, (1 << 31) - 1):
        _check_attn(C, w, _q(w.rng, 2 * n, 4, D, BF16), None, True, window)


@pytest.mark.parametrize("rows", [1, 70])
def test_sequences_without_tokens_pages_or_rows(C, rows):
    i = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    for pages, width in ((4, 2), (4, 0), (0, 2), (0, 0)):
        cache = C.Kv8Cache.empty(pages, 2, 16, 64)
        table = torch.full((3, width), -1, dtype=torch.int32).cuda()
        batch = C.Kv8Batch(table, i([0, 0, 0]), 3 * rows)
        q, x = torch.ones((3 * rows, 4, 64), dtype=BF16).cuda(), torch.ones((3 * rows, 2, 64), dtype=BF16).cuda()
        ws = C.make_kv8_workspace(cache, batch, 4)
        before = cache.k.clone()
        C.kv8_append(cache, batch, x, x, ws=ws)
        assert torch.equal(cache.k, before)
        for causal in (True, False):
            out, lse = C.kv8_attn(q, cache, batch, causal, ws=ws)
            assert (out == 0).all() and torch.isneginf(lse).all()
        k, v = C.kv8_read(cache, batch, BF16, ws=ws)
        assert (k == 0).all() and (v == 0).all() and C.read_status(ws) == (0, 0)
    none = C.Kv8Batch(table, i([0, 0, 0]), 0)
    out, lse = C.kv8_attn(q[:0], cache, none)
    C.kv8_append(cache, none, x[:0], x[:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_attn_window_never_reads_pages_behind_it(C):
    # pages behind every row's window have been given away: their table entries are -1
    w = World(C, 46, [1000, 513], 1, 128, 64).fill()
    ref_table = w.table.copy()
    w.table[0, :(1000 - 4 - 128 + 1) // 64] = -1
    w.table[1, :(513 - 4 - 128 + 1) // 64] = -1
    q = _q(w.rng, 8, 4, 128, BF16)
    out, lse = _check_attn(C, w, q, None, True, 128)
    w.table = ref_table
    out2, lse2 = _check_attn(C, w, q, None, True, 128)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_bad_entries_are_skipped_and_reported(C):
    Hk, D, page = 1, 64, 16
    w = World(C, 51, [40, 40, 40], Hk, D, page).fill()
    q = _q(w.rng, 3, 2, D, BF16)
    good, _ = _check_attn(C, w, q, None)
    n_pages = w.k.shape[0]

    def run(table, lens, cu=None, T=3):
        i = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32).cuda()
        cache, batch = w.cache(), C.Kv8Batch(i(table), i(lens), T, None if cu is None else i(cu))
        ws = C.make_kv8_workspace(cache, batch, 2)
        out, lse = C.kv8_attn(q.cuda(), cache, batch, ws=ws)
        st = [C.read_status(ws)[0]]
        k, v = C.kv8_read(cache, batch, FP32, ws=ws)
        st.append(C.read_status(ws)[0])
        x = _rows(w.rng, T, Hk, D, BF16, 1.0).cuda()
        before = cache.k.clone()
        C.kv8_append(cache, batch, x, x, ws=ws)
        st.append(C.read_status(ws)[0])
        return out, k, (cache.k != before), st

    table = w.table.copy()
    table[1, 2] = n_pages          # the page of the last token is outside the cache
    out, k, changed, st = run(table, [40, 40, 40])
    assert st == [5, 5, 5]
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and torch.isfinite(out).all()
    assert (k[1] == 0).all() and (k[0] != 0).any()
    assert not changed[w.table[1, :3]].any() and changed[w.table[0, 2]].any()
    table = w.table.copy()
    table[2, 0] = -1               # an unused entry in the visible range
    out, _, _, st = run(table, [40, 40, 40])
    assert st[0] == 5 and torch.equal(out[:2], good[:2]) and torch.isfinite(out).all()
    # lengths past the table (its tokens 40 .. 47 were never written: NaN is right for row 1), and below zero
    out, k, changed, st = run(w.table, [40, 49, -3])
    assert st == [5, 5, 5] and torch.equal(out[0], good[0])
    assert (k[1:] == 0).all() and (out[2] == 0).all()
    # row offsets that decrease or leave the step's rows
    out, _, _, st = run(w.table, [40, 40, 40], [0, 1, 0, 0])
    assert st == [5, 5, 5] and torch.equal(out[0], good[0])
    out, _, _, st = run(w.table, [40, 40, 40], [0, 1, 2, 9])
    assert st == [5, 5, 5] and torch.equal(out[:2], good[:2])


# ------------------------------------------------------------------ together

def test_a_layer_over_prompt_drafts_and_decode_steps(C):
    # append and attend as a layer does, with the reference appending to its own copy
    Hk, G, D, page = 2, 4, 128, 32
    prompt, steps = [70, 1, 33], [1, 1, 4, 1]
    w = World(C, 61, [L + sum(steps) for L in prompt], Hk, D, page)
    cache, lens = w.cache(), [0, 0, 0]
    for step, n in enumerate([None] + steps):
        add = prompt if n is None else [n] * 3
        cu = np.concatenate([[0], np.cumsum(add)]).tolist()
        lens = [a + b for a, b in zip(lens, add)]
        T = cu[-1]
        qkv = _rows(w.rng, T, Hk * (G + 2), D, BF16, 1.0 + step)
        dev = qkv.cuda()
        batch = w.batch(T, cu if n is None else None, lens)
        ws = C.make_kv8_workspace(cache, batch, Hk * G)
        C.kv8_append(cache, batch, dev[:, Hk * G:Hk * (G + 1)], dev[:, Hk * (G + 1):], ws=ws)
        out, lse = C.kv8_attn(dev[:, :Hk * G], cache, batch, ws=ws)
        shares = R.rows_of(T, 3, cu)
        for codes, sc, x in ((w.k, w.ks, qkv[:, Hk * G:Hk * (G + 1)]), (w.v, w.vs, qkv[:, Hk * (G + 1):])):
            R.append(codes, sc, x.double().numpy(), w.table, lens, shares, page)
        w.same(cache)
        ref = R.attention(qkv[:, :Hk * G].double().numpy(), (w.k, w.v, w.ks, w.vs), w.table, lens, shares, page,
                          True, 0, 1 / math.sqrt(D))
        tol_o, tol_l = R.attention_bounds(*ref, D, max(lens), BF16)
        assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol_o).all()
        assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_l).all()
        k, v = C.kv8_read(cache, batch, FP32, ws=ws)
        last = R.gather(w.k, w.ks, w.table[0], lens[0] - 1, lens[0], page)[0]
        assert torch.equal(k[cu[1] - 1].cpu(), torch.from_numpy(last).float())
        assert C.read_status(ws) == (0, 0)


def test_a_captured_step_follows_the_batch_it_was_captured_with(C):
    # the graph holds pointers: lengths, block table and rows may change between replays
    Hk, G, D, page = 2, 4, 64, 16
    w = World(C, 62, [200, 90], Hk, D, page).fill()
    cache = w.cache()
    batch = w.batch(2, None, [100, 50])
    q = torch.zeros((2, Hk * G, D), dtype=BF16, device="cuda")
    k, v = (torch.zeros((2, Hk, D), dtype=BF16, device="cuda") for _ in range(2))
    ws = C.make_kv8_workspace(cache, batch, Hk * G)

    def step():
        C.kv8_append(cache, batch, k, v, ws=ws)
        return C.kv8_attn(q, cache, batch, ws=ws)

    step()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = step()
    for lens in ([200, 1], [17, 90], [129, 64]):
        fresh = w.cache()
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(cache, name).copy_(getattr(fresh, name))
        hq, hk, hv = (_rows(w.rng, 2, h, D, BF16, 1.0) for h in (Hk * G, Hk, Hk))
        q.copy_(hq), k.copy_(hk), v.copy_(hv)
        batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        b2 = w.batch(2, None, lens)
        C.kv8_append(fresh, b2, k, v)
        want, want_lse = C.kv8_attn(q, fresh, b2)
        assert torch.equal(cache.k, fresh.k) and torch.equal(cache.v_scale[w.table[0]], fresh.v_scale[w.table[0]])
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_graphs_that_share_a_workspace_replay_in_turn(C):
    # few rows and many rows, both of them cut into parts: each replay leaves the other's results alone
    w = World(C, 65, [3000, 1700], 2, 64, 64).fill()
    cache = w.cache()
    calls = []
    for n, H in ((1, 8), (100, 4)):
        q, batch = _q(w.rng, 2 * n, H, 64, BF16).cuda(), w.batch(2 * n)
        calls.append((q, batch, C.kv8_attn(q, cache, batch)))
    ws = max((C.make_kv8_workspace(cache, b, q.shape[1]) for q, b, _ in calls), key=lambda t: t.numel())
    graphs = []
    for q, batch, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, C.kv8_attn(q, cache, batch, ws=ws)))
    for order in ((0, 1), (1, 0, 1), (0, 0, 1, 1)):
        for k in order:
            for t in graphs[k][1]:
                t.fill_(7)
            graphs[k][0].replay()
    torch.cuda.synchronize()
    for (_, got), (_, _, want) in zip(graphs, calls):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert C.read_status(ws) == (0, 0)


def test_binding_refusals(C):
    cache = C.Kv8Cache.empty(4, 2, 16, 64)
    i = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    batch = C.Kv8Batch(i([[0, 1], [2, 3]]), i([20, 5]), 4)
    q, x = torch.zeros((4, 4, 64), dtype=BF16).cuda(), torch.zeros((4, 2, 64), dtype=BF16).cuda()
    ws = C.make_kv8_workspace(cache, batch, 4)
    bad = [
        lambda: C.kv8_append(cache, batch, x[:3], x), lambda: C.kv8_append(cache, batch, x, x.half()),
        lambda: C.kv8_append(cache, batch, x.double(), x.double()), lambda: C.kv8_append(cache, batch, x.cpu(), x),
        lambda: C.kv8_append(cache, batch, x, x[:, :1]), lambda: C.kv8_append(cache, batch, x[..., :32], x),
        lambda: C.kv8_append(cache, batch, x[:1].expand(4, 2, 64), x),
        lambda: C.kv8_append(cache, batch, x.transpose(1, 2).contiguous().transpose(1, 2), x),
        lambda: C.kv8_append(cache, batch, x[0], x), lambda: C.kv8_append(cache, batch, x, x, ws=ws.cpu()),
        lambda: C.kv8_read(cache, batch, torch.float64), lambda: C.kv8_read(cache, batch, BF16, out_k=x.float()),
        lambda: C.kv8_read(cache, batch, BF16, out_v=x[:2]), lambda: C.kv8_attn(q.float(), cache, batch),
        lambda: C.kv8_attn(q, cache, batch, window=-1), lambda: C.kv8_attn(q, cache, batch, window=1 << 32),
        lambda: C.kv8_attn(q, cache, batch, out=q.half()), lambda: C.kv8_attn(q, cache, batch, lse=q[:, :, 0]),
        lambda: C.kv8_attn(q.cpu(), cache, batch), lambda: C.kv8_attn(q[:, :, ::2], cache, batch),
        lambda: C.Kv8Batch(i([[0, 1], [2, 3]]), i([20, 5]), 3), lambda: C.Kv8Batch(i([0, 1]), i([20, 5]), 2),
        lambda: C.Kv8Batch(i([[0, 1], [2, 3]]), i([20]), 4), lambda: C.Kv8Batch(i([[0], [2]]), i([1, 1]), 4, i([0, 4])),
        lambda: C.Kv8Batch(i([[0], [2]]).long(), i([1, 1]), 4), lambda: C.Kv8Batch(i([[0], [2]]), i([1, 1]), -2),
        lambda: C.Kv8Cache(cache.k[0], cache.v[0], cache.k_scale, cache.v_scale),
        lambda: C.Kv8Cache(cache.k, cache.v[:2], cache.k_scale, cache.v_scale),
        lambda: C.Kv8Cache(cache.k, cache.v, cache.k_scale[:, :1], cache.v_scale),
        lambda: C.Kv8Cache(cache.k, cache.v, cache.k_scale, cache.v_scale.double()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: C.kv8_attn(q[:, :3], cache, batch), lambda: C.kv8_attn(q, cache, batch, ws=ws[:256]),
                 lambda: C.kv8_attn(q, cache, batch, causal=False, window=3),
                 lambda: C.kv8_attn(q, cache, batch, softmax_scale=0.0),
                 lambda: C.kv8_append(cache, batch, x, x, ws=ws[:128]),
                 lambda: C.kv8_append(C.Kv8Cache.empty(4, 2, 24, 64), batch, x, x)):
        with pytest.raises(C.Csa2Error):
            call()


def test_calls_on_two_streams_with_their_own_workspaces(C):
    w = World(C, 63, [3000, 2500, 2000], 2, 128, 64).fill()
    cache, batch = w.cache(), w.batch(3)
    qs = [_q(w.rng, 3, 8, 128, BF16).cuda() for _ in range(2)]
    want = [C.kv8_attn(q, cache, batch) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = C.kv8_attn(qs[i], cache, batch)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_positions_past_32_bits_of_bytes(C):
    # a cache of more than 2^32 bytes: blocks at its far end are read and written
    Hk, D, page = 8, 128, 64
    P = (1 << 32) // (Hk * D * page) + 8
    k, v = (torch.empty((P, Hk, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = C.Kv8Cache(k, v, torch.ones((P, Hk), device="cuda"), torch.ones((P, Hk), device="cuda"))
    small = World(C, 64, [150], Hk, D, page)
    i = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    far, near = [P - 1, P - 3, P - 2], [0, 1, 2]
    x, y = (_rows(small.rng, 150, Hk, D, BF16, 1.0).cuda() for _ in range(2))
    q = _q(small.rng, 1, 16, D, BF16).cuda()
    res = []
    for pages in (far, near):
        C.kv8_append(cache, C.Kv8Batch(i([pages]), i([150]), 150), x, y)
        res.append(C.kv8_attn(q, cache, C.Kv8Batch(i([pages]), i([150]), 1)))
    assert torch.equal(k[P - 1], k[0]) and torch.equal(v[P - 3], v[1])
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert torch.isfinite(res[0][0]).all()
