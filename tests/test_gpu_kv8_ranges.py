"""The 8-bit paged KV cache's attention where magnitudes lie far apart: logits that outgrow the running reference
inside a tile of keys.  Every channel is held to its own bound (kv8_ref.py), so what a few tokens give to a channel
of their own counts, however small it is beside the others.  Needs a GPU."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as R
from test_gpu_kv8 import BF16, FP16, World, _check_attn

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
