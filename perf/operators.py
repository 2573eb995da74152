"""The 8-bit serving operators as they are measured: cases, plain forms and exact values.

Four operators of one decode or prefill step with 8-bit weights and an 8-bit
key/value cache:

  quant   bf16 / fp32 values -> e4m3 with one fp32 scale per 1 x 128 (tokens)
          or 128 x 128 (weights) block:
              a = max(max |x| over the block's finite values, 448 * 2^-64)
              scale = fl(a / 448),  q = e4m3(sat(fl(x * fl(448 / a))))
  matmul  Y[m][n] = sum_b sx[m][b] sw[n/128][b] sum_{k in b} xq[m][k] wq[n][k]
          with X given in bf16 (quantised as above inside the call) or in e4m3
  append  new keys and values written to a paged cache of 8-bit values with one
          scale per page and head, the scale a power of two that grows with the
          page's largest value (the page's earlier values are rescaled then)
  attend  softmax attention of a few (or many) new queries over that cache,
          causal, with an optional sliding window and first tokens that stay
          visible (sinks)

``own`` selects the library's calls (sparse_weight_b200.hyb) or the plain form
in elementary torch operations.
"""
import math
import random

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
MIN_AMAX = 448.0 * 2.0 ** -64   # smaller blocks quantise as if their largest value were this
MIN_EXP, MAX_EXP = -40, 60      # exponents of a cache scale
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through a grouped key (or value) projection: the smallest product of a
        # decode step, where the launch and the first bytes' latency count
        dict(name="matmul b1 1024x4096", op="matmul", m=1, n=1024, k=4096, x="bf16", out="f32"),
        # the widest decode batch through a down projection: bound by the weight's bytes
        dict(name="matmul b16 4096x14336", op="matmul", m=16, n=4096, k=14336, x="bf16", out="bf16"),
        # a short prompt through a matrix whose sides are no multiples of the blocks
        dict(name="matmul 45 ragged 1000x4100", op="matmul", m=45, n=1000, k=4100, x="e4m3", out="f32"),
        # a prompt's block of tokens through a gate (or up) projection: bound by arithmetic
        dict(name="matmul 2048 14336x4096", op="matmul", m=2048, n=14336, k=4096, x="bf16", out="bf16"),
        # the input of a prompt's down projection, quantised once
        dict(name="quant tokens 2048x14336", op="quant", rows=2048, cols=14336, x="bf16", block_rows=1),
        # a ragged weight in 32 bits, quantised when it is loaded
        dict(name="quant weight 1000x4100", op="quant", rows=1000, cols=4100, x="f32", block_rows=128),
        # one decode step's new keys and values of a batch
        dict(name="append b64 x1", op="append", batch=64, q=1, ragged=False, max_len=1024, kv_heads=8, dim=128,
             page=16, type="e4m3"),
        # prompts of different lengths written at once
        dict(name="append b3 x2048 ragged", op="append", batch=3, q=2048, ragged=True, max_len=4096, kv_heads=8,
             dim=128, page=64, type="i8"),
        # one short sequence: latency
        dict(name="attend b1 short", op="attend", batch=1, q=1, ragged=False, max_len=300, heads=32, kv_heads=8,
             dim=128, page=16, type="e4m3", window=0, sinks=0),
        # a full decode batch of sequences of all lengths, one slot empty: bound by the cache's bytes
        dict(name="attend b32 to 8192", op="attend", batch=32, q=1, ragged=False, max_len=8192, heads=64, kv_heads=8,
             dim=128, page=64, type="e4m3", window=0, sinks=0),
        # drafted tokens of long conversations checked at once, a window with sinks
        dict(name="attend b8 x4 window of 65536", op="attend", batch=8, q=4, ragged=False, max_len=65536, heads=32,
             kv_heads=8, dim=128, page=32, type="i8", window=4096, sinks=4),
        # prompts' chunks over what came before, with a window: bound by arithmetic
        dict(name="attend b2 x1024 window of 5120", op="attend", batch=2, q=1024, ragged=True, max_len=5120, heads=32,
             kv_heads=8, dim=128, page=64, type="e4m3", window=2048, sinks=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "quant", "append", "attend", "attend"])
    if op == "matmul":
        while True:
            m, n, k = _log(rng, 1, 2048), _log(rng, 64, 14336), _log(rng, 128, 14336)
            if m * n * k <= 2048 * 14336 * 4096:
                break
        return dict(op=op, m=m, n=n, k=k, x=rng.choice(["bf16", "e4m3"]), out=rng.choice(["f32", "bf16"]))
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 2048), cols=_log(rng, 16, 14336), x=rng.choice(["bf16", "f32"]),
                    block_rows=rng.choice([1, 128]))
    kv_heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64])
    cache = dict(kv_heads=kv_heads, dim=dim, page=page, type=rng.choice(["e4m3", "i8"]))
    if op == "append":
        q = rng.choice([1, _log(rng, 1, 2048)])
        batch = _log(rng, 1, max(1, min(64, 6144 // q)))
        return dict(op=op, batch=batch, q=q, ragged=rng.random() < 0.5, max_len=max(q, _log(rng, 16, 4096)), **cache)
    q = rng.choice([1, 1, _log(rng, 1, 16), _log(rng, 16, 1024)])
    max_len = max(q, _log(rng, 16, 65536 if q <= 16 else 5120))
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    most = min(64, 2 ** 19 // max_len, max(1, 2 * 32 * 1024 * 5120 // (heads * q * max_len)))
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    return dict(op=op, batch=_log(rng, 1, max(1, most)), q=q, ragged=q > 1 and rng.random() < 0.5, max_len=max_len,
                heads=heads, window=window, sinks=rng.choice([0, 4, 20]) if window else 0, **cache)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _values(gen, rows, cols, std):
    """Normal values with one in a hundred twenty times as large, as outlier channels are."""
    x = torch.randn(rows, cols, generator=gen, device=DEV) * std
    big = torch.rand(cols, generator=gen, device=DEV) < 0.01
    return torch.where(big, 20 * x, x)


def _lengths(case):
    """(new tokens, length after them) per sequence, the same for every seed: the longest is the case's, one slot of a
    batch is empty."""
    rng = random.Random("lengths %d %d %d" % (case["batch"], case["q"], case["max_len"]))
    B, q, most = case["batch"], case["q"], case["max_len"]
    new = [rng.randint(1, q) if case["ragged"] else q for _ in range(B)]
    new[0] = q
    if most >= 65536:
        lens = [rng.randint(most // 2, most) for _ in range(B)]
    else:
        lens = [max(n, round(math.exp(rng.uniform(math.log(max(1, most // 8)), math.log(most))))) for n in new]
    lens[0] = most
    if case["op"] == "attend" and B >= 8:
        lens[B // 2] = 0
    return new, [max(n, t) if t else 0 for n, t in zip(new, lens)]


def _pages(case, lens, seed):
    """A page table in which every sequence's pages lie scattered over the cache."""
    P = case["page"]
    need = [-(-t // P) for t in lens]
    width = max(1, -(-case["max_len"] // P))
    total = sum(need) + 3
    gen = torch.Generator().manual_seed(seed + 17)
    order = torch.randperm(total, generator=gen, dtype=torch.int64)
    table = torch.zeros(case["batch"], width, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c].to(torch.int32)
        at += c
    return table.to(DEV), total


def _cache(case, gen, pages):
    """A filled cache: values of bf16 size in pages, each page and head with its own power-of-two scale."""
    H, P, D = case["kv_heads"], case["page"], case["dim"]
    most = 127.0 if case["type"] == "i8" else E4M3_MAX
    parts = []
    for std in (1.5, 0.7):
        q = torch.empty(pages, H, P, D, dtype=torch.int8 if case["type"] == "i8" else torch.float8_e4m3fn, device=DEV)
        s = torch.empty(pages, H, device=DEV)
        chunk = max(1, 2 ** 26 // (H * P * D))
        channel = 0.5 + torch.rand(H, 1, D, generator=gen, device=DEV)
        for i in range(0, pages, chunk):
            x = torch.randn(min(chunk, pages - i), H, P, D, generator=gen, device=DEV) * channel * std
            e = torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / most))
            sc = torch.exp2(e)
            y = x / sc[:, :, None, None]
            q[i:i + chunk] = (y.round().clamp(-127, 127) if case["type"] == "i8" else y.clamp(-most, most)).to(q.dtype)
            s[i:i + chunk] = sc
        parts += [q, s]
    return dict(k=parts[0], k_scale=parts[1], v=parts[2], v_scale=parts[3])


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "quant":
        x = _values(gen, case["rows"], case["cols"], 1.0)
        st["x"] = x.to(torch.bfloat16) if case["x"] == "bf16" else x
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        ld = -(-k // 16) * 16  # rows start on 16 bytes
        wq, st["ws"] = _quant_plain(_values(gen, n, k, 0.02), 128)
        x = _values(gen, m, ld, 1.0).to(torch.bfloat16)[:, :k]
        st["wq"] = _padded(wq, ld)
        if case["x"] == "bf16":
            st["x"], st["xs"] = x, None
        else:
            xq, st["xs"] = _quant_plain(x, 1)
            st["x"] = _padded(xq, ld)
    else:
        new, lens = _lengths(case)
        st["table"], pages = _pages(case, lens, seed)
        st.update(_cache(case, gen, pages))
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        off = [0]
        for c in new:
            off.append(off[-1] + c)
        st["off"] = torch.tensor(off, dtype=torch.int32, device=DEV) if case["ragged"] else None
        rows, D = off[-1], case["dim"]
        if case["op"] == "append":
            # keys and values are slices of the rows of one projection's output
            kv = _values(gen, rows, 2 * case["kv_heads"] * D, 1.0).to(torch.bfloat16)
            kv = kv.view(rows, 2 * case["kv_heads"], D)
            st["new_k"], st["new_v"] = kv[:, :case["kv_heads"]], kv[:, case["kv_heads"]:]
        else:
            st["q"] = _values(gen, rows, case["heads"] * D, 1.0).to(torch.bfloat16).view(rows, case["heads"], D)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from sparse_weight_b200 import hyb
        if case["op"] == "matmul":
            st["A"] = hyb.Fp8Matrix(case["n"], case["k"], st["wq"], st["ws"])
            st["work"] = hyb.new_workspace(hyb.fp8_workspace_bytes(case["m"], case["n"], case["k"]), DEV)
        elif case["op"] == "quant":
            st["work"] = hyb.new_workspace(hyb.fp8_quant_workspace_bytes(), DEV)
        else:
            st["cache"] = hyb.Cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
            st["work"] = hyb.new_workspace(
                hyb.cache_append_workspace_bytes() if case["op"] == "append" else
                hyb.cache_attention_workspace_bytes(st["cache"], case["batch"], case["heads"], case["q"],
                                                    st["table"].shape[1] * case["page"]), DEV)
    return st


def _padded(q, ld):
    """The rows of q at a row stride of ld, with zeros behind them."""
    out = torch.zeros(q.shape[0], ld, dtype=q.dtype, device=q.device)
    out[:, :q.shape[1]] = q
    return out[:, :q.shape[1]]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "quant":
        return _quant_plain(state["x"], c["block_rows"])
    if c["op"] == "matmul":
        return _matmul_plain(c, state)
    return _append_plain(c, state) if c["op"] == "append" else _attend_plain(c, state)


def _run_own(c, st):
    from sparse_weight_b200 import hyb
    if c["op"] == "quant":
        return hyb.quant_fp8(st["x"], block_rows=c["block_rows"], ws=st["work"])
    if c["op"] == "matmul":
        return hyb.matmul_fp8(st["A"], st["x"], xs=st["xs"], ydt=hyb.HYB_F32 if c["out"] == "f32" else hyb.HYB_BF16,
                              ws=st["work"])
    if c["op"] == "append":
        hyb.cache_append(st["cache"], st["new_k"], st["new_v"], st["table"], st["lens"], off=st["off"], max_new=c["q"],
                         ws=st["work"])
        return st["k"], st["v"], st["k_scale"], st["v_scale"]
    return hyb.cache_attention(st["cache"], st["q"], st["table"], st["lens"], off=st["off"], max_new=c["q"],
                               window=c["window"], sinks=c["sinks"], return_lse=True, ws=st["work"])


def _blocks(x, block_rows):
    """x in 32 bits, padded with zeros to whole blocks: [row blocks, block rows, column blocks, 128]."""
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    p = torch.nn.functional.pad(x.float(), (0, cb * BLOCK - cols, 0, rb * block_rows - rows))
    return p.view(rb, block_rows, cb, BLOCK)


def _quant_plain(x, block_rows):
    rows, cols = x.shape
    p = _blocks(x, block_rows)
    a = torch.where(torch.isfinite(p), p.abs(), 0.0).amax(dim=(1, 3)).clamp(min=MIN_AMAX)
    # true 32-bit divisions: by a tensor, since one by a number may become a product with its reciprocal
    top = torch.full_like(a, E4M3_MAX)
    q = (p * (top / a)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(p.shape[0] * block_rows, -1)[:rows, :cols].contiguous().view(torch.float8_e4m3fn)
    return q, a / top


def _matmul_plain(c, st):
    m, n, k = c["m"], c["n"], c["k"]
    x, xs = (st["x"], st["xs"]) if st["xs"] is not None else _quant_plain(st["x"], 1)
    xd = x.float() * xs.repeat_interleave(BLOCK, 1)[:, :k]
    wd = st["wq"].float() * st["ws"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    y = xd @ wd.t()
    return y if c["out"] == "f32" else y.to(torch.bfloat16)


def _rows(c, st):
    """For every new row: its sequence and its place among that sequence's new tokens; new tokens per sequence."""
    B, q = c["batch"], c["q"]
    rows = st["q"].shape[0] if c["op"] == "attend" else st["new_k"].shape[0]
    r = torch.arange(rows, device=DEV)
    if st["off"] is None:
        return r // q, r % q, torch.full((B,), q, device=DEV)
    off = st["off"].long()
    b = torch.searchsorted(off, r, right=True) - 1
    return b, r - off[b], off[1:] - off[:-1]


def _append_plain(c, st):
    P, B, H, D = c["page"], c["batch"], c["kv_heads"], c["dim"]
    i8 = c["type"] == "i8"
    most = 127.0 if i8 else E4M3_MAX
    b, i, new = _rows(c, st)
    lens = st["lens"].long()
    start = lens - new
    pos = start[b] + i                                                     # place of every new row
    first = start // P                                                     # first page that each sequence writes
    touched = (c["q"] + P - 2) // P + 1                                    # most pages that one sequence writes
    slot = first[:, None] + torch.arange(touched, device=DEV)              # [B, touched] pages in the table
    live = (slot * P < lens[:, None]) & (new[:, None] > 0)
    page = st["table"].long().gather(1, slot.clamp(max=st["table"].shape[1] - 1))
    ids = page[live]                                                       # pages that are written
    at = (torch.cumsum(live.flatten().long(), 0) - 1).view(B, touched)     # their number among the written ones
    row = at[b, pos // P - first[b]]
    inside = pos % P
    tok = slot[live][:, None] * P + torch.arange(P, device=DEV)            # place of each token of those pages
    owner = torch.arange(B, device=DEV)[:, None].expand(B, touched)[live]
    old = (tok < start[owner][:, None])[:, None, :, None]
    for x, q, s in ((st["new_k"], st["k"], st["k_scale"]), (st["new_v"], st["v"], st["v_scale"])):
        x = torch.nan_to_num(x.float(), nan=0.0, posinf=math.inf, neginf=-math.inf)
        fresh = torch.zeros(ids.numel(), H, P, D, device=DEV)
        fresh[row, :, inside] = x
        written = torch.zeros(ids.numel(), P, dtype=torch.bool, device=DEV)
        written[row, inside] = True
        amax = torch.where(torch.isfinite(fresh), fresh.abs(), 0.0).amax(dim=(2, 3))
        # the smallest 2^e that holds amax: from the mantissa and exponent, exactly
        mant, e = torch.frexp(amax)
        mm, me = math.frexp(most)
        e = torch.where(mant <= mm, e - me, e - me + 1)
        e = torch.where(amax > 0, e, MIN_EXP).clamp(MIN_EXP, MAX_EXP)
        need = torch.ldexp(torch.ones_like(amax), e)
        had = torch.where(old.any(dim=2)[:, :, 0], s[ids], torch.zeros_like(need))
        scale = torch.maximum(need, had)
        kept = _take(q, ids)
        again = kept * (had / scale)[:, :, None, None]
        y = fresh / scale[:, :, None, None]
        if i8:
            again, y = again.round(), y.round()
        z = torch.where(written[:, None, :, None], y.clamp(-most, most), torch.where(old, again, kept))
        q.view(torch.uint8)[ids] = z.to(q.dtype).view(torch.uint8)
        s[ids] = scale
    return st["k"], st["v"], st["k_scale"], st["v_scale"]


def _take(q, ids):
    """The pages `ids` of 8-bit values, in 32 bits."""
    return q.view(torch.uint8)[ids].view(q.dtype).float()


def _attend_plain(c, st):
    B, H, D, P, q = c["batch"], c["kv_heads"], c["dim"], c["page"], c["q"]
    G, L = c["heads"] // H, st["table"].shape[1] * P
    b, i, new = _rows(c, st)
    lens, table = st["lens"].long(), st["table"].long()
    Q = torch.zeros(B, q, c["heads"], D, device=DEV)
    Q[b, i] = st["q"].float()
    Q = Q.view(B, q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * q, D)

    def dense(x, s):
        y = _take(x, table) * s[table][..., None, None]                   # [B, pages, H, P, D]
        return y.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)

    S = (Q @ dense(st["k"], st["k_scale"]).transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, H, G, q, L)
    place = (lens - new)[:, None] + torch.arange(q, device=DEV)            # [B, q]
    t = torch.arange(L, device=DEV)
    seen = (t <= place[:, :, None]) & (t < lens[:, None, None])
    if c["window"]:
        seen &= (t > place[:, :, None] - c["window"]) | (t < c["sinks"])
    S.masked_fill_(~seen[:, None, None], -math.inf)
    top = S.amax(dim=4, keepdim=True)
    S = S.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    den = S.sum(dim=4)
    live = (torch.arange(L, device=DEV) < lens[:, None])[:, None, :, None]
    O = S.view(B, H, G * q, L) @ torch.where(live, dense(st["v"], st["v_scale"]), 0.0)
    O = (O.view(B, H, G, q, D) / torch.where(den > 0, den, 1.0)[..., None]).permute(0, 3, 1, 2, 4)
    lse = (torch.log(den) + top[..., 0]).permute(0, 3, 1, 2)
    return O.reshape(B, q, c["heads"], D)[b, i].to(torch.bfloat16), lse.reshape(B, q, c["heads"])[b, i].contiguous()


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _visible(c, lens, new):
    """(query, key) pairs seen and tokens read, over all sequences."""
    pairs = tokens = 0
    for n, t in zip(new, lens):
        if not t:
            continue
        w, s = c["window"], c["sinks"]
        if not w:
            tokens += t
            pairs += n * t - n * (n - 1) // 2
            continue
        lowest = max(0, t - n - w + 1)                                     # first token that the window reaches
        tokens += t - lowest + min(s, lowest)
        for i in range(n):
            p = t - n + i
            low = max(0, p - w + 1)
            pairs += p - low + 1 + min(s, low)
    return pairs, tokens


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        x = 2 * m * k if case["x"] == "bf16" else m * k + 4 * m * kb
        return {"bytes": x + n * k + 4 * -(-n // BLOCK) * kb + m * n * (4 if case["out"] == "f32" else 2),
                "flops": 2 * m * n * k}
    if case["op"] == "quant":
        r, k = case["rows"], case["cols"]
        return {"bytes": r * k * ((2 if case["x"] == "bf16" else 4) + 1) + 4 * -(-r // case["block_rows"]) * -(-k // BLOCK),
                "flops": 3 * r * k}
    new, lens = _lengths(case)
    H, D = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        pages = sum(-(-t // case["page"]) - (t - n) // case["page"] for n, t in zip(new, lens))
        old = sum((t - n) % case["page"] for n, t in zip(new, lens))
        return {"bytes": 2 * H * D * (3 * sum(new) + old) + 8 * H * pages, "flops": 6 * H * D * sum(new)}
    pairs, tokens = _visible(case, lens, new)
    pages = -(-tokens // case["page"])
    return {"bytes": 2 * tokens * H * D + 8 * H * pages + 4 * pages + sum(new) * case["heads"] * (4 * D + 4),
            "flops": 4 * pairs * case["heads"] * D}


# ---------------------------------------------------------------------------
# exact values, in 64 bits
# ---------------------------------------------------------------------------

def _to_e4m3(y):
    """y (64 bits) to the nearest e4m3 value, ties to even, saturating: steps of 2^(e-3), 2^-9 below 2^-6."""
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_quant(x, block_rows):
    """The values that q stands for and the scales; the two 32-bit roundings of the definition are made in order."""
    rows, cols = x.shape
    cb = -(-cols // 128)
    q = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    s = torch.empty(-(-rows // block_rows), cb, dtype=torch.float64, device=x.device)
    for j in range(cb):
        part = x[:, 128 * j:128 * j + 128].double()
        big = part.abs().amax(dim=1)
        if block_rows > 1:
            big = torch.stack([p.amax() for p in big.split(block_rows)])
        big = big.clamp(min=MIN_AMAX)
        s[:, j] = big / 448.0
        inv = (448.0 / big).float().double().repeat_interleave(block_rows)[:rows, None]
        q[:, 128 * j:128 * j + 128] = _to_e4m3((part * inv).float().double())
    return q, s


def _exact_attend(c, st):
    H, D, P = c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // H
    out, lse, at = [], [], 0
    off = st["off"].tolist() if st["off"] is not None else [c["q"] * j for j in range(c["batch"] + 1)]
    for b, t in enumerate(st["lens"].tolist()):
        n = off[b + 1] - off[b]
        Q = st["q"][off[b]:off[b + 1]].double().view(n, H, G, D)
        if t == 0:
            out.append(torch.zeros(n, H * G, D, dtype=torch.float64, device=DEV))
            lse.append(torch.full((n, H * G), -math.inf, dtype=torch.float64, device=DEV))
            continue
        place = torch.arange(t - n, t, device=DEV)
        ids = st["table"][b, :-(-t // P)].long()
        # only the tokens that some query sees
        tok = torch.arange(t, device=DEV)
        if c["window"]:
            tok = tok[(tok > t - n - c["window"]) | (tok < c["sinks"])]
        seen = tok[None] <= place[:, None]
        if c["window"]:
            seen &= (tok[None] > place[:, None] - c["window"]) | (tok[None] < c["sinks"])
        o_b = torch.empty(n, H, G, D, dtype=torch.float64, device=DEV)
        l_b = torch.empty(n, H, G, dtype=torch.float64, device=DEV)
        for h in range(H):
            k, v = ((st[w].view(torch.uint8)[ids[tok // P], h, tok % P].view(st[w].dtype).double()
                     * st[w + "_scale"][ids[tok // P], h, None].double()) for w in "kv")
            for g in range(G):
                z = Q[:, h, g] @ k.t() / math.sqrt(D)
                z = z.masked_fill(~seen, -math.inf)
                l_b[:, h, g] = torch.logsumexp(z, dim=1)
                o_b[:, h, g] = torch.softmax(z, dim=1) @ v
        out.append(o_b.view(n, H * G, D))
        lse.append(l_b.view(n, H * G))
    return torch.cat(out), torch.cat(lse)


def _exact_append(c, st):
    """The cache after the append, page by page: the values that are stored, and the scales."""
    P, i8 = c["page"], c["type"] == "i8"
    most = 127.0 if i8 else 448.0
    got = {w: st[w].double() for w in ("k", "v", "k_scale", "v_scale")}
    lens, table = st["lens"].tolist(), st["table"].tolist()
    off = st["off"].tolist() if st["off"] is not None else [c["q"] * j for j in range(c["batch"] + 1)]
    for b, t in enumerate(lens):
        start = t - (off[b + 1] - off[b])
        for j in range(start // P, -(-t // P)):
            page, lo, hi = table[b][j], max(start, j * P), min(t, j * P + P)
            for w in "kv":
                x = st["new_" + w][off[b] + lo - start:off[b] + hi - start].double().transpose(0, 1)  # [H, tokens, D]
                e = torch.ceil(torch.log2(x.abs().amax(dim=(1, 2)) / most)).clamp(MIN_EXP, MAX_EXP)
                scale, old = torch.exp2(e), lo - j * P
                if old:
                    had = got[w + "_scale"][page]
                    scale = torch.maximum(scale, had)
                    y = got[w][page, :, :old] * (had / scale)[:, None, None]
                    got[w][page, :, :old] = torch.round(y) if i8 else _to_e4m3(y)
                y = x / scale[:, None, None]
                got[w][page, :, old:hi - j * P] = torch.round(y).clamp(-127, 127) if i8 else _to_e4m3(y)
                got[w + "_scale"][page] = scale
    return got["k"], got["v"], got["k_scale"], got["v_scale"]


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "quant":
        return _exact_quant(st["x"], case["block_rows"])
    if case["op"] == "attend":
        return _exact_attend(case, st)
    q, s = (st["x"].double(), st["xs"].double()) if st["xs"] is not None else _exact_quant(st["x"], 1)
    if st["xs"] is None:
        s = s.float().double()  # the scales are held in 32 bits
    y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
    for j in range(s.shape[1]):
        w = st["wq"][:, 128 * j:128 * j + 128].double()
        sw = st["ws"][:, j].double().repeat_interleave(128)[:case["n"]]
        y += (q[:, 128 * j:128 * j + 128] * s[:, j, None]) @ (w * sw[:, None]).t()
    return y
