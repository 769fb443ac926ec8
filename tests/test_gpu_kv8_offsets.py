"""The 8-bit paged KV cache with row offsets that make no sense: a bad entry costs its own sequence its rows and no
other.  Needs a GPU."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as R
from test_gpu_kv8 import BF16, FP16, World, _q, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    from sparse_attention_decode_csa2_gb300 import build
    build.build()
    from sparse_attention_decode_csa2_gb300 import csa2
    return csa2


def _shares(cu, T):
    return [(a, b - a) if 0 <= a <= b <= T else (0, 0) for a, b in zip(cu[:-1], cu[1:])]


def _many(S, page):
    """Offsets of many sequences, some of them broken: more than one round of the search."""
    rng = np.random.default_rng(S)
    n = rng.integers(0, 3 * page, S)
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1])
    for i, x in zip(rng.choice(S - 1, 4, replace=False) + 1, (-1, T + 7, 0, T)):
        cu[i] = x
    return cu.tolist(), T


MANY, MANY_T = _many(70, 16)
CASES = [
    # the offsets, the step's rows, page, D, H_kv
    ([0, 100, 50, 150], 150, 16, 64, 1),
    ([0, 100, 200, 300, 400, -1, 500], 500, 16, 64, 2),
    ([0, 100, 0, 100], 100, 16, 128, 1),
    ([0, 90, 700, 300, 400, 500], 500, 32, 64, 1),
    ([0, 300, -5, 300, 700], 700, 128, 128, 1),
    ([-3, 200, 400], 400, 64, 128, 2),
    ([2 ** 31 - 1, -2 ** 31, 0, 60], 60, 16, 64, 1),
    (MANY, MANY_T, 16, 64, 1),
]


@pytest.mark.parametrize("cu,T,page,D,Hk", CASES)
def test_bad_offsets_cost_their_own_sequence_alone(C, cu, T, page, D, Hk):
    S, shares = len(cu) - 1, _shares(cu, T)
    claims = np.zeros(T, int)
    for r0, n in shares:
        claims[r0:r0 + n] += 1
    lens = [n + (15, 7, 12, 22)[s % 4] for s, (_, n) in enumerate(shares)]
    w = World(C, 91 + T, lens, Hk, D, page).fill()
    cache, batch = w.cache(), w.batch(T, cu)
    ws = C.make_kv8_workspace(cache, batch, 2 * Hk)

    k, v = (_rows(w.rng, T, Hk, D, BF16, 2.0) for _ in range(2))
    C.kv8_append(cache, batch, k.cuda(), v.cuda(), ws=ws)
    assert C.read_status(ws)[0] == 5
    for codes, sc, x in ((w.k, w.ks, k), (w.v, w.vs, v)):
        R.append(codes, sc, x.double().numpy(), w.table, lens, shares, page)
    w.same(cache)

    out_k, out_v = (torch.full((T, Hk, D), 7.0, dtype=FP16, device="cuda") for _ in range(2))
    C.kv8_read(cache, batch, FP16, out_k, out_v, ws=ws)
    assert C.read_status(ws)[0] == 5
    for got, codes, sc in ((out_k, w.k, w.ks), (out_v, w.v, w.vs)):
        want = [set() for _ in range(T)]
        for s, (r0, n) in enumerate(shares):
            x = torch.from_numpy(R.gather(codes, sc, w.table[s], lens[s] - n, lens[s], page)).to(FP16).numpy()
            for i in range(n):
                want[r0 + i].add(x[i].tobytes())
        none = np.full((Hk, D), 7.0, np.float16).tobytes()
        got = got.cpu().numpy()
        assert all(got[r].tobytes() in (want[r] or {none}) for r in range(T))

    q = _q(w.rng, T, 2 * Hk, D, BF16)
    out, lse = C.kv8_attn(q.cuda(), cache, batch, ws=ws)
    assert C.read_status(ws)[0] == 5
    ref = R.attention(q.double().numpy(), (w.k, w.v, w.ks, w.vs), w.table, lens, shares, page, True, 0,
                      1 / math.sqrt(D))
    tol_o, tol_l = R.attention_bounds(*ref, D, max(lens), BF16)
    one = claims == 1
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol_o)[one].all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_l)[one].all()
