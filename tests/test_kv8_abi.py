"""The 8-bit paged KV cache's refusals (no GPU: validation comes before any device work), and its reference."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_ref as R

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def C():
    from sparse_attention_decode_csa2_gb300 import build
    build.build()
    from sparse_attention_decode_csa2_gb300 import csa2
    return csa2


def _structs(C, **kw):
    g = lambda name, d: kw.get(name, d)
    cache = C.Csa2Kv8Cache(g("k", FAKE), g("v", FAKE), g("ks", FAKE), g("vs", FAKE), g("n_pages", 10),
                           g("H_kv", 8), g("page", 64), g("D", 128))
    batch = C.Csa2Kv8Batch(g("table", FAKE), g("kv_len", FAKE), g("cu", None), g("S", 2), g("T", 2),
                           g("max_pages", 4))
    return ctypes.byref(cache), ctypes.byref(batch)


def _append(C, **kw):
    c, b = _structs(C, **kw)
    return C.lib.csa2_kv8_append(c, b, kw.get("x", FAKE), kw.get("y", FAKE), kw.get("type", 0),
                                 kw.get("x_stride", 1024), kw.get("y_stride", 1024), kw.get("ws", FAKE),
                                 kw.get("ws_bytes", 256), None)


def _read(C, **kw):
    c, b = _structs(C, **kw)
    return C.lib.csa2_kv8_read(c, b, kw.get("x", FAKE), kw.get("y", FAKE), kw.get("type", 0),
                               kw.get("ws", FAKE), kw.get("ws_bytes", 256), None)


def _attn(C, **kw):
    c, b = _structs(C, **kw)
    return C.lib.csa2_kv8_attn(kw.get("q", FAKE), kw.get("type", 0), kw.get("q_stride", 4096), kw.get("H", 32), c, b,
                               kw.get("causal", 1), kw.get("window", 0), kw.get("scale", 0.1),
                               kw.get("out", FAKE), None, kw.get("ws", FAKE), kw.get("ws_bytes", 1 << 40), None)


BAD_FOR_ALL = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(k=FAKE + 8), 1),
    (dict(table=None), 1), (dict(kv_len=None), 1), (dict(S=-1), 1), (dict(T=-1), 1), (dict(max_pages=-1), 1),
    (dict(n_pages=-1), 1), (dict(H_kv=0), 1), (dict(T=3), 1), (dict(S=0), 1),
    (dict(D=96), 2), (dict(D=256), 2), (dict(page=48), 2), (dict(page=8), 2), (dict(page=256), 2),
    (dict(max_pages=1 << 25), 2), (dict(n_pages=1 << 31), 2), (dict(T=1 << 29), 2),
    (dict(type=3), 1), (dict(type=-1), 1),
    (dict(ws=None), 3), (dict(ws_bytes=255), 3),
]


@pytest.mark.parametrize("kw,code", BAD_FOR_ALL)
def test_bad_arguments_are_refused(C, kw, code):
    assert _append(C, **kw) == code
    assert _read(C, **kw) == code
    assert _attn(C, **kw) == code


def test_row_arguments_are_refused(C):
    for f in (_append, _read):
        assert f(C, x=None) == 1 and f(C, y=None) == 1
        assert f(C, x=FAKE + 4) == 1 and f(C, y=FAKE + 8) == 1
    assert _append(C, x_stride=1023) == 1        # tokens overlap
    assert _append(C, y_stride=1028) == 1        # bf16 rows 8 bytes off a 16-byte vector
    assert _append(C, type=2, x_stride=1026) == 1
    assert _attn(C, q=None) == 1 and _attn(C, q=FAKE + 2) == 1 and _attn(C, out=None) == 1
    assert _attn(C, out=FAKE + 8) == 1
    assert _attn(C, q_stride=4095) == 1 and _attn(C, q_stride=4100) == 1
    assert _attn(C, type=2) == 1                 # no fp32 queries
    assert _attn(C, H=0) == 1 and _attn(C, H=12) == 1
    assert _attn(C, window=-1) == 1 and _attn(C, causal=0, window=5) == 1
    assert _attn(C, H=8 * 257, q_stride=1 << 20) == 2
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert _attn(C, scale=scale) == 1
    assert _attn(C, ws=FAKE + 4) == 3


@pytest.mark.parametrize("name", ["ks", "vs", "table", "kv_len", "cu"])
def test_words_off_their_alignment_are_refused(C, name):
    for f in (_append, _read, _attn):
        assert f(C, **{name: FAKE + 2}) == 1


def test_a_workspace_or_lse_off_its_alignment_is_refused(C):
    assert _append(C, ws=FAKE + 2) == 3 and _read(C, ws=FAKE + 2) == 3
    c, b = _structs(C)
    assert C.lib.csa2_kv8_attn(FAKE, 0, 4096, 32, c, b, 1, 0, 0.1, FAKE, FAKE + 2, FAKE, 1 << 40, None) == 1


def test_empty_batches_do_nothing(C):
    none = dict(S=0, T=0, table=None, kv_len=None)
    for kw in (none, dict(T=0)):
        assert _append(C, x=None, y=None, **kw) == 0
        assert _read(C, x=None, y=None, **kw) == 0
        assert _attn(C, q=None, out=None, **kw) == 0


def test_workspace_size(C):
    c, b = _structs(C)
    assert C.lib.csa2_kv8_workspace_size(c, b, 0) == 256
    assert C.lib.csa2_kv8_workspace_size(c, b, 32) > 256
    n = C.lib.csa2_kv8_workspace_size(c, b, 32)
    assert _attn(C, ws_bytes=n - 1) == 3
    for kw in (dict(H_kv=0), dict(S=0, T=0), dict(T=0)):  # nothing to attend with: the status alone
        assert C.lib.csa2_kv8_workspace_size(*_structs(C, **kw), 32) == 256
    assert C.lib.csa2_kv8_workspace_size(None, b, 32) == 256


def test_binding_refuses_host_tensors(C):
    k = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    s = torch.ones((4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        C.Kv8Cache(k, k, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        C.Kv8Batch(torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1)


# ---- the reference itself

def test_reference_codes_agree_with_torch():
    vals = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, R.E4M3, equal_nan=True)
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * 10.0 ** rng.integers(-4, 3, 20000)).clip(-448, 448).astype(np.float32)
    mids = ((R.E4M3[:126] + R.E4M3[1:127]) / 2).astype(np.float32)
    x = np.concatenate([x, mids, -mids])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (R.encode(x) == want).all()
    assert R.encode(np.array([np.inf, -np.inf, np.nan, 1e9])).tolist() == [126, 254, 127, 126]


def test_reference_scale_is_the_least_power_of_two():
    for amax in (448.0, 448.0000001, 1.0, 1.75, 1.7500001, 3e38, 1e-27):
        s = R.need_scale(amax)
        assert amax <= 448 * s and not amax <= 448 * (s / 2)
    assert R.need_scale(0.0) == 2.0 ** -100 and R.need_scale(np.inf) == 2.0 ** 120


def test_reference_attention_agrees_with_torch():
    rng = np.random.default_rng(1)
    P, Hk, page, D, L, n = 4, 2, 16, 64, 50, 3
    k, v = (R.encode(40 * rng.standard_normal((P, Hk, page, D))) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-7, -4, (P, Hk)).astype(np.float64) for _ in range(2))
    table = np.array([[2, 0, 3, 1]])
    q = rng.standard_normal((n, 4, D))
    out, lse, *_ = R.attention(q, (k, v, ks, vs), table, [L], [(0, n)], page, True, 20, 0.125)
    K, V = (torch.from_numpy(R.gather(c, s, table[0], 0, L, page)).repeat_interleave(2, dim=1)
            for c, s in ((k, ks), (v, vs)))
    i, j = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
    mask = (j <= i) & (j > i - 20)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), K.transpose(0, 1), V.transpose(0, 1), mask, scale=0.125)
    assert np.allclose(out, want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


def test_reference_appends_as_one_write_where_no_scale_grows():
    rng = np.random.default_rng(2)
    page, D = 16, 64
    x = rng.standard_normal((20, 1, D))
    x[0, 0, 0] = 6.0
    x[16, 0, 0] = 6.0   # each page's largest value comes first
    one = np.zeros((2, 1, page, D), np.uint8), np.ones((2, 1))
    two = np.zeros((2, 1, page, D), np.uint8), np.ones((2, 1))
    R.append(*one, x, [[1, 0]], [20], [(0, 20)], page)
    for i in range(20):
        R.append(*two, x[i:i + 1], [[1, 0]], [i + 1], [(0, 1)], page)
    assert (one[0] == two[0]).all() and (one[1] == two[1]).all()
