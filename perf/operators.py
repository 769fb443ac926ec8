"""The operators of the 8-bit paged KV cache: their cases, their plain forms and their definition in 64 bits.

A layer's cache holds E4M3 codes ``k``, ``v`` [n_pages][kv_heads][page][dim] with one fp32 scale per page and
head.  A step's batch is a block table, the sequences' lengths after the step and the number of rows that each
sequence has in it.  Three operators work on them:

* append: quantises the step's new K and V rows into the pages (a page's scale only grows while it fills, and
  the rows it holds are requantised when it does);
* read: values of the step's rows, read back from the pages;
* attn: attention of the step's queries over their sequences' pages.

``own`` false: the operators from elementary torch operations.  ``own`` true: the framework's kernels.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EMIN, _EMAX = -100, 120


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# op, seqs: sequences; rows: rows of the step, for each sequence ("each") or in all, spread unevenly; ctx: the
# longest sequence after the step (lengths are spread over [ctx / 2, ctx], "even": all have ctx); heads,
# kv_heads, dim, page, type.  A sequence of length 0 is among them where "empty" is true.

def _case(name, op, seqs, rows, each, ctx, kv_heads, dim, page, dtype, heads=0, causal=True, window=0, even=False,
          empty=False):
    return {"name": name, "op": op, "seqs": seqs, "rows": rows, "each": each, "ctx": ctx, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "type": dtype, "causal": causal, "window": window,
            "even": even, "empty": empty}


def listed():
    return [
        # one user's next token: nothing but latency
        _case("append 1 token", "append", 1, 1, True, 1000, 8, 128, 64, "bf16"),
        # a served batch's next tokens, each in its sequence's last, partly filled page
        _case("append 256 x 1 token", "append", 256, 1, True, 4096, 8, 128, 64, "bf16"),
        # prompts of several users written at once, of uneven lengths, rows not split into heads evenly
        _case("append prompts 20011", "append", 7, 20011, False, 16384, 8, 128, 64, "bf16"),
        # fp32 rows of a small model with short pages
        _case("append fp32 5000 d64", "append", 13, 5000, False, 2048, 3, 64, 16, "fp32"),
        # a short prefix read back for a check
        _case("read 37 tokens", "read", 1, 37, False, 37, 4, 64, 16, "fp16"),
        # whole sequences read back, to be moved or requantised elsewhere
        _case("read 8 x 16k", "read", 8, 16384, True, 16384, 8, 128, 64, "bf16", even=True),
        # one user's next token over a short context: nothing but latency
        _case("attn 1 token 333", "attn", 1, 1, True, 333, 8, 128, 64, "bf16", heads=32),
        # the headline decode batch of this framework (32 sequences, 64K tokens, 64 heads), lengths uneven
        _case("attn decode 32 x 64k", "attn", 32, 1, True, 65536, 8, 128, 64, "bf16", heads=64),
        # a small model's decode batch: five heads to a KV head, short pages, one sequence without tokens
        _case("attn decode 17 x 9k g5 d64", "attn", 17, 1, True, 9001, 8, 64, 16, "fp16", heads=40, empty=True),
        # four drafted tokens of each sequence checked at once
        _case("attn draft 24 x 4 16k", "attn", 24, 4, True, 16384, 4, 128, 32, "bf16", heads=32),
        # a prompt chunk of 4096 tokens behind a long context
        _case("attn chunk 4096 of 16k", "attn", 1, 4096, True, 16384, 8, 128, 64, "bf16", heads=32, even=True),
        # prompts of uneven lengths through a sliding-window layer of a small model
        _case("attn prompts 10007 w1024 d64", "attn", 9, 10007, False, 2500, 4, 64, 128, "fp16", heads=16,
              window=1024),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "attn"])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8])
    if op != "attn":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        seqs = _spread(rng, 1, 200)
        if rng.random() < 0.5:
            rows, each = rng.choice([1, 1, 2, 5]), True
            ctx = _spread(rng, max(8, 2 * rows), 8192)
        else:
            rows, each = _spread(rng, seqs, 20000), False
            ctx = 2 * rows // seqs + 2 + _spread(rng, 1, 2000)
        return _case(None, op, seqs, rows, each, ctx, kv_heads, dim, page, dtype) | {"name": ""}
    dtype, group = rng.choice(["bf16", "fp16"]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    kind = rng.choice(["decode", "decode", "draft", "chunk", "prompts"])
    window = rng.choice([0, 0, 0, 128, 1000])
    if kind in ("decode", "draft"):
        rows, each = (1, True) if kind == "decode" else (rng.randint(2, 8), True)
        ctx = _spread(rng, 16, 60000)
        seqs = _spread(rng, 1, max(1, min(128, 1_000_000 // ctx)))
    elif kind == "chunk":
        seqs, rows, each = rng.randint(1, 2), _spread(rng, 30, 4000), True
        ctx = rows + _spread(rng, 1, 16000 if rows * kv_heads * group < 65536 else 2000)
    else:
        seqs, each = rng.randint(2, 8), False
        rows = _spread(rng, 4 * seqs, 1200 * seqs)
        ctx = 2 * rows // seqs + 2 + _spread(rng, 1, 500)
    causal = window > 0 or rng.random() < 0.8
    return _case(None, "attn", seqs, rows, each, ctx, kv_heads, dim, page, dtype, heads=kv_heads * group,
                 causal=causal, window=window) | {"name": ""}


def _geometry(case):
    """Rows and lengths of the case's sequences, as lists of whole numbers: the same for every seed."""
    S, ctx = case["seqs"], case["ctx"]
    if case["each"]:
        n = [case["rows"]] * S
    else:  # uneven shares of the rows, one at least
        share = [1.0 + 0.9 * math.sin(2.3 * s + 1.0) for s in range(S)]
        n = [max(1, int(case["rows"] * x / sum(share))) for x in share]
        n[0] += case["rows"] - sum(n)
    spread = [0.0 if case["even"] else 0.5 * (0.5 + 0.5 * math.sin(1.7 * s + 0.4)) for s in range(S)]
    length = [max(k, int(ctx * (1.0 - x))) for k, x in zip(n, spread)]
    if case["empty"]:
        length[S // 2] = 0
    return n, length


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    n, length = _geometry(case)
    S, page, Hk, D = case["seqs"], case["page"], case["kv_heads"], case["dim"]
    dtype = _TYPES[case["type"]]
    pages = [-(-x // page) for x in length]
    wide = max(1, max(pages))
    n_pages = sum(pages) + 3  # a few pages that no sequence has
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((S, wide), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(pages):
        table[s, :k] = order[at:at + k]
        at += k
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    st = {"case": case, "table": table, "n_rows": cu[-1],
          "kv_len": torch.tensor(length, dtype=torch.int32, device=dev),
          "cu": None if case["each"] else torch.tensor(cu, dtype=torch.int32, device=dev)}

    # what the layer before has left in the cache: channels of uneven size, blocks of uneven scale
    chan = torch.exp(0.5 * torch.randn((2, Hk, 1, D), generator=g, device=dev))
    codes = []
    for i in range(2):
        c = torch.empty((n_pages, Hk, page, D), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (Hk * page * D))
        for p in range(0, n_pages, step):
            x = torch.randn((min(step, n_pages - p), Hk, page, D), generator=g, device=dev)
            c[p:p + step] = (48.0 * x * chan[i]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(c)
    st["k"], st["v"] = codes
    for name in ("k_scale", "v_scale"):
        e = torch.randint(-7, -4, (n_pages, Hk), generator=g, device=dev)
        st[name] = _pow2(e)

    T = cu[-1]
    if case["op"] == "append":
        # K and V are slices of one projection's output, so their rows are further apart than their size
        qkv = torch.randn((T, 3 * Hk, D), generator=g, device=dev)
        qkv[:, Hk:2 * Hk] *= chan[0, :, 0]
        qkv[:, 2 * Hk:] *= torch.exp(0.7 * torch.randn((T, 1, 1), generator=g, device=dev))
        qkv = qkv.to(dtype)
        st["new_k"], st["new_v"] = qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
    elif case["op"] == "attn":
        H = case["heads"]
        st["q"] = torch.randn((T, H, D), generator=g, device=dev).to(dtype)
        st["scale"] = 1.0 / math.sqrt(D)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _pow2(e):
    """2^e in fp32 for whole e of [-126, 127], from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _rows(st):
    """Sequence, position and table column of each row of the step."""
    case, dev = st["case"], st["table"].device
    T, S = st["n_rows"], case["seqs"]
    cu = st["cu"] if st["cu"] is not None else torch.arange(S + 1, device=dev, dtype=torch.int32) * case["rows"]
    row = torch.arange(T, device=dev)
    s = torch.searchsorted(cu.long(), row, right=True) - 1
    n = (cu[1:] - cu[:-1]).long()
    i = row - cu.long()[s]
    return s, i, n, st["kv_len"].long()[s] - n[s] + i


def _plain_append_one(st, x, codes, scale, s, pos, n):
    page, D = st["case"]["page"], st["case"]["dim"]
    T, Hk = x.shape[0], x.shape[1]
    col = pos // page
    pid = st["table"][s, col].long()
    # the pages of the step, each once, and what is written there
    pages, inv = torch.unique(pid, return_inverse=True)
    P = pages.numel()
    amax = torch.zeros((P, Hk), device=x.device)
    amax.index_reduce_(0, inv, x.float().abs().amax(dim=2), "amax")
    first = torch.full((P,), page, device=x.device, dtype=torch.int64)
    first.index_reduce_(0, inv, pos % page, "amin")
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), _EMIN).clamp(_EMIN, _EMAX)
    need = _pow2(e)
    old = scale[pages]
    new = torch.where((first > 0)[:, None], torch.maximum(old, need), need)
    # rows that the pages held, where the scale grew
    held = codes[pages]
    val = held.view(torch.float8_e4m3fn).float() * (old / new)[:, :, None, None]
    again = val.to(torch.float8_e4m3fn).view(torch.uint8)
    move = (torch.arange(page, device=x.device)[None, :] < first[:, None])[:, None, :] & (new > old)[:, :, None]
    codes[pages] = torch.where(move[..., None], again, held)
    scale[pages] = new
    q = (x.float() / new[inv][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[pid, :, pos % page] = q


def _plain_append(st):
    s, _, n, pos = _rows(st)
    _plain_append_one(st, st["new_k"], st["k"], st["k_scale"], s, pos, n)
    _plain_append_one(st, st["new_v"], st["v"], st["v_scale"], s, pos, n)


def _plain_read(st):
    s, _, _, pos = _rows(st)
    page, dtype = st["case"]["page"], _TYPES[st["case"]["type"]]
    pid = st["table"][s, pos // page].long()
    k = st["k"][pid, :, pos % page].view(torch.float8_e4m3fn).float() * st["k_scale"][pid][..., None]
    v = st["v"][pid, :, pos % page].view(torch.float8_e4m3fn).float() * st["v_scale"][pid][..., None]
    return k.to(dtype), v.to(dtype)


def _plain_sequences(codes, scale, table):
    """fp32 values [S][kv_heads][tokens][dim] of the sequences' pages."""
    pid = table.clamp(min=0).long()
    x = codes[pid].view(torch.float8_e4m3fn).float() * scale[pid][..., None, None]
    S, W, Hk, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(S, Hk, W * page, D)


def _plain_attn(st):
    case = st["case"]
    S, Hk, D, H = case["seqs"], case["kv_heads"], case["dim"], case["heads"]
    G = H // Hk
    s, i, n, pos = _rows(st)
    k = _plain_sequences(st["k"], st["k_scale"], st["table"])
    v = _plain_sequences(st["v"], st["v_scale"], st["table"])
    Q = int(case["rows"]) if case["each"] else int(n.max())
    L = k.shape[2]
    dev = k.device
    q = torch.zeros((S, Q, H, D), device=dev)
    q[s, i] = st["q"].float()
    q = q.reshape(S, Q, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * Q, D)
    logit = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    j = torch.arange(L, device=dev)
    length = st["kv_len"].long()
    at = (length - n)[:, None] + torch.arange(Q, device=dev)[None, :]
    seen = (j[None, None, :] < length[:, None, None]).expand(S, Q, L)
    if case["causal"]:
        seen = seen & (j[None, None, :] <= at[:, :, None])
    if case["window"] > 0:
        seen = seen & (j[None, None, :] > at[:, :, None] - case["window"])
    logit.view(S, Hk, G, Q, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = logit.amax(dim=3, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    logit = logit.sub_(top).exp_()
    total = logit.sum(dim=3, keepdim=True)
    out = torch.matmul(logit, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    out = out.reshape(S, Hk, G, Q, D).permute(0, 3, 1, 2, 4).reshape(S, Q, H, D)[s, i]
    lse = lse.reshape(S, Hk, G, Q).permute(0, 3, 1, 2).reshape(S, Q, H)[s, i]
    return out.to(st["q"].dtype), lse


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _handles(st):
    """The cache, the batch and the workspace that a serving loop keeps: they name the state's buffers."""
    if "handles" not in st:
        from sparse_attention_decode_csa2_gb300 import csa2
        cache = csa2.Kv8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        batch = csa2.Kv8Batch(st["table"], st["kv_len"], st["n_rows"], st["cu"])
        ws = csa2.make_kv8_workspace(cache, batch, st["case"]["heads"])
        st["handles"] = csa2, cache, batch, ws
    return st["handles"]


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        csa2, cache, batch, ws = _handles(st)
        if op == "append":
            csa2.kv8_append(cache, batch, st["new_k"], st["new_v"], ws=ws)
        elif op == "read":
            k, v = csa2.kv8_read(cache, batch, _TYPES[case["type"]], ws=ws)
        else:
            out, lse = csa2.kv8_attn(st["q"], cache, batch, causal=case["causal"], window=case["window"],
                                     softmax_scale=st["scale"], ws=ws)
    else:
        if op == "append":
            _plain_append(st)
        elif op == "read":
            k, v = _plain_read(st)
        else:
            out, lse = _plain_attn(st)
    if op == "append":  # the codes as the numbers that they are, in units of their block's scale
        return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
                "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    return {"k": k, "v": v} if op == "read" else {"out": out, "lse": lse}


def _pairs(case, n, length):
    """Visible (row, token) pairs of one head, and tokens that some row of their sequence sees."""
    pairs = tokens = 0
    w = case["window"]
    for k, L in zip(n, length):
        if L == 0:
            continue
        if not case["causal"]:
            pairs, tokens = pairs + k * L, tokens + L
            continue
        p0, p1 = L - k, L - 1  # positions of the rows
        if w == 0:
            pairs += (p0 + 1 + p1 + 1) * k // 2
            tokens += L
        else:
            short = max(0, min(p1, w - 2) - p0 + 1)  # rows that see fewer than w tokens
            pairs += short * (2 * p0 + short + 1) // 2 + (k - short) * w
            tokens += L - max(0, p0 - w + 1)
    return pairs, tokens


def work(case):
    n, length = _geometry(case)
    T, Hk, D, page = sum(n), case["kv_heads"], case["dim"], case["page"]
    b = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    pages = sum(-(-L // page) - (L - k) // page for k, L in zip(n, length) if L)
    if case["op"] == "append":  # new rows in, codes out, the pages' scales in and out
        return {"bytes": 2 * T * Hk * D * (b + 1) + 2 * pages * Hk * 8, "flops": 4 * T * Hk * D}
    if case["op"] == "read":
        return {"bytes": 2 * T * Hk * D * (b + 1) + 2 * pages * Hk * 4, "flops": 2 * T * Hk * D}
    pairs, tokens = _pairs(case, n, length)
    H = case["heads"]
    return {"bytes": 2 * tokens * Hk * D + 2 * T * H * D * b + T * H * 4, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_values(dev):
    """The value of each of the 256 E4M3 codes."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if b >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _two(e):
    """2^e in float64, from a table."""
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=e.device)[e.long() + 160]


def _e4m3_round(x):
    """float64 values (|x| <= 448) to the nearest E4M3 value, ties to the even one."""
    unit = _two(torch.frexp(x)[1].clamp(min=-5) - 4)  # last place: 2^(floor(log2 |x|) - 3), 2^-9 at least
    return torch.round(x / unit) * unit


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["table"].device
    val = _e4m3_values(dev)
    n, length = _geometry(case)
    page, Hk, D = case["page"], case["kv_heads"], case["dim"]
    table = st["table"].cpu().tolist()
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)

    if case["op"] == "append":
        if cu[-1] // page + 2 * len(n) > 4000:
            return None
        res = {}
        for name, x in (("k", st["new_k"]), ("v", st["new_v"])):
            codes = val[st[name].long()]
            scale = st[name + "_scale"].double()
            for s, (k, L) in enumerate(zip(n, length)):
                pos = L - k
                while pos < L and L > 0:
                    a = pos % page
                    rows = min(page - a, L - pos)
                    p = table[s][pos // page]
                    r = cu[s] + pos - (L - k)
                    new = x[r:r + rows].double().permute(1, 0, 2)  # [Hk][rows][D]
                    amax = new.abs().amax(dim=(1, 2))
                    e = torch.ceil(torch.log2(amax / 448.0)).clamp(_EMIN, _EMAX)
                    e = torch.where(amax > 448.0 * _two(e), e + 1, e)  # log2 may round across a power
                    e = torch.where(amax <= 224.0 * _two(e), e - 1, e).clamp(_EMIN, _EMAX)
                    sc = _two(e)
                    if a > 0:
                        grown = torch.maximum(scale[p], sc)
                        moved = _e4m3_round(codes[p, :, :a] * (scale[p] / grown)[:, None, None])
                        codes[p, :, :a] = moved
                        sc = grown
                    codes[p, :, a:a + rows] = _e4m3_round(new / sc[:, None, None])
                    scale[p] = sc
                    pos += rows
            res[name], res[name + "_scale"] = codes, scale
        return res

    def rows_of(name, s, lo, hi):
        """float64 [Hk][hi - lo][D]: tokens lo .. hi - 1 of sequence s."""
        j = torch.arange(lo, hi, device=dev)
        p = st["table"][s].long()[j // page]
        x = val[st[name][p, :, j % page].long()] * st[name + "_scale"][p].double()[..., None]
        return x.permute(1, 0, 2)

    if case["op"] == "read":
        k = [rows_of("k", s, L - c, L).permute(1, 0, 2) for s, (c, L) in enumerate(zip(n, length))]
        v = [rows_of("v", s, L - c, L).permute(1, 0, 2) for s, (c, L) in enumerate(zip(n, length))]
        return {"k": torch.cat(k), "v": torch.cat(v)}

    H = case["heads"]
    G = H // Hk
    out = torch.zeros((cu[-1], H, D), dtype=torch.float64, device=dev)
    lse = torch.full((cu[-1], H), -math.inf, dtype=torch.float64, device=dev)
    for s, (c, L) in enumerate(zip(n, length)):
        if L == 0:
            continue
        k, v = rows_of("k", s, 0, L), rows_of("v", s, 0, L)
        for i0 in range(0, c, 512):
            i1 = min(c, i0 + 512)
            q = st["q"][cu[s] + i0:cu[s] + i1].double().reshape(i1 - i0, Hk, G, D)
            z = torch.einsum("ihgd,hjd->hgij", q, k) * st["scale"]
            i = L - c + torch.arange(i0, i1, device=dev)
            j = torch.arange(L, device=dev)
            if case["causal"]:
                z.masked_fill_(j[None, :] > i[:, None], -math.inf)
            if case["window"] > 0:
                z.masked_fill_(j[None, :] <= i[:, None] - case["window"], -math.inf)
            w = torch.logsumexp(z, dim=3)
            o = torch.einsum("hgij,hjd->ihgd", torch.exp(z - w[..., None]), v)
            out[cu[s] + i0:cu[s] + i1] = o.reshape(i1 - i0, H, D)
            lse[cu[s] + i0:cu[s] + i1] = w.permute(2, 0, 1).reshape(i1 - i0, H)
    return {"out": out, "lse": lse}
