"""Cases of the 4-bit KV cache: rows stored and read back, and the attention that reads it.

The self-decoder's full-attention layer writes one key and one value row per
token; every cross-attention layer reads all of them for every generated
token.  In the 4-bit cache a row of ``head_dim`` values is kept in blocks of
16:  x ~ 2^e * s * c,  with c one of the 4-bit values 0, .5, 1, 1.5, 2, 3, 4, 6
(and their negatives), s an 8-bit scale (e4m3, the block's largest value over
6), and e a whole number per KV head for K and for V.

Kinds of case:

  store   K and V rows of new tokens are quantised into the cache's pages and
          read back as the values they stand for
  read    rows that are in the cache are read back
  attend  queries of the newest tokens attend over what is cached
"""

import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def _case(name, kind, batch, tokens, past, kv_heads, head_dim, page, io, q_heads=0, ragged=False, fused=False):
    """tokens: new tokens of a call; past: cached tokens before them (attend: cached tokens, the new ones among them)."""
    return dict(name=name, kind=kind, batch=batch, tokens=tokens, past=past, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, io=io, ragged=ragged, fused=fused)


def listed():
    return [
        # one decode step of 64 sequences after a 2048-token prompt: K and V are slices of a fused projection's rows
        _case("store_step_b64", "store", 64, 1, 2048, 20, 64, 64, "bf16", fused=True),
        # the prompt of the headline workload
        _case("store_prompt_b1_l2048", "store", 1, 2048, 0, 20, 64, 64, "bf16"),
        # a padded batch of prompt pieces of different lengths that go on at odd positions, small pages, f32
        _case("store_ragged_b7_f32", "store", 7, 777, 1003, 8, 128, 16, "f32", ragged=True),
        # the long prefill: 4 prompts of 32768 tokens
        _case("store_prompt_b4_l32768", "store", 4, 32768, 0, 20, 64, 64, "bf16"),
        # one sequence's rows handed over to a bf16 reader
        _case("read_b1_l2048", "read", 1, 2048, 0, 20, 64, 64, "bf16"),
        # a batch of different lengths read back in f32
        _case("read_ragged_b16_f32", "read", 16, 4097, 0, 8, 128, 32, "f32", ragged=True),
        # the smallest call: the first tokens of one sequence
        _case("attend_b1_n64", "attend", 1, 1, 64, 20, 64, 64, "bf16", q_heads=40),
        # the decode workload: 64 sequences at 2048 cached tokens
        _case("attend_b64_n2048", "attend", 64, 1, 2048, 20, 64, 64, "bf16", q_heads=40),
        # 16 sequences at the end of a 2048 + 32768 token generation
        _case("attend_b16_n34816", "attend", 16, 1, 34816, 20, 64, 64, "bf16", q_heads=40),
        # a serving batch of very different lengths, wide heads, small pages
        _case("attend_ragged_b37", "attend", 37, 1, 5000, 8, 128, 16, "bf16", q_heads=40, ragged=True),
        # four drafted tokens of each sequence checked at once
        _case("attend_draft_b8_n4097", "attend", 8, 4, 4097, 20, 64, 64, "bf16", q_heads=40),
        # one KV head for all query heads, f32, few sequences
        _case("attend_b3_n8191_f32", "attend", 3, 1, 8191, 1, 128, 128, "f32", q_heads=16),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("store", "read", "attend", "attend"))
    kv_heads, head_dim = rng.choice((1, 2, 4, 5, 8, 20)), rng.choice((64, 128))
    batch = _spread(rng, 1, 64)
    page, io, ragged = rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.5
    row = kv_heads * head_dim * batch
    if kind == "attend":
        most = min(34816, 4 * 10 ** 8 // row)
        tokens = rng.choice((1, 1, 1, 2, 3, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 8, 16))
        past = max(tokens, _spread(rng, 1, most))
        return {k: v for k, v in _case("", kind, batch, tokens, past, kv_heads, head_dim, page, io, heads, ragged).items() if k != "name"}
    tokens = 1 if rng.random() < 0.3 else _spread(rng, 1, min(32768, 6 * 10 ** 7 // row))
    past = _spread(rng, 1, 4096) - 1
    return {k: v for k, v in _case("", kind, batch, tokens, past, kv_heads, head_dim, page, io, 0, ragged,
                                   kind == "store" and rng.random() < 0.5).items() if k != "name"}


def _counts(case):
    """New rows of each sequence (store, read), or its cached tokens (attend): a property of the case, not of the seed."""
    B, most = case["batch"], case["past"] if case["kind"] == "attend" else case["tokens"]
    if not case["ragged"]:
        return [most] * B
    # spread over 0 .. most; the first sequence is full, and one is empty where there are several
    return [most if b == 0 else 0 if b == 1 else int(most * ((b * 0.6180339887) % 1.0)) for b in range(B)]


def _starts(case):
    """Cached tokens of each sequence before the rows of store and read."""
    past = case["past"]
    return [past - (b * 7) % (past + 1) if case["ragged"] else past for b in range(case["batch"])]


def work(case):
    row = case["kv_heads"] * case["head_dim"]
    io, packed = (2 if case["io"] == "bf16" else 4), 0.5 + 1 / 16
    rows = sum(_counts(case))
    if case["kind"] == "attend":
        q = case["batch"] * case["tokens"] * case["q_heads"] * case["head_dim"]
        return {"bytes": rows * row * 2 * packed + 2 * q * io, "flops": 4 * rows * case["tokens"] * case["q_heads"] * case["head_dim"]}
    if case["kind"] == "read":
        return {"bytes": rows * row * 2 * (packed + io), "flops": 2 * rows * row}
    # stored, and read back
    return {"bytes": rows * row * 2 * (2 * packed + 2 * io), "flops": 6 * rows * row}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """(rows of K, of V, exponents of K, of V, queries): rows [B, tokens or cached tokens, Hkv, dh]."""
    g = torch.Generator("cuda").manual_seed(int(seed))
    B, H, D = case["batch"], case["kv_heads"], case["head_dim"]
    dtype = torch.bfloat16 if case["io"] == "bf16" else torch.float32
    n = case["past"] if case["kind"] == "attend" else case["tokens"]
    if case["fused"]:  # a fused projection's rows: [q | k | v]
        both = torch.randn(B, n, 4 * H * D, generator=g, device="cuda", dtype=dtype)
        K, V = (both[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in (2, 3))
    else:
        K, V = (torch.randn(B, n, H, D, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    # keys have channels that are larger than the rest; values are small
    wide = torch.exp2(torch.randn(H, D, generator=g, device="cuda")).to(dtype)
    K.mul_(wide)
    V.mul_(0.0625)
    # per head, so that the largest block scale is inside e4m3's upper half
    ek = torch.ceil(torch.log2(8.0 * wide.float().amax(-1) / 2688.0)).to(torch.int32)
    ev = torch.full((H,), -12, device="cuda", dtype=torch.int32)
    q = torch.randn(B, case["tokens"], case["q_heads"], D, generator=g, device="cuda", dtype=dtype) if case["q_heads"] else None
    return K, V, ek, ev, q


def _pages(case, seed):
    """(table [B, pages a sequence], pages of the pool): every page at a place of its own in the pool, in no order."""
    P, B = case["page"], case["batch"]
    each = -(-(case["past"] + (0 if case["kind"] == "attend" else case["tokens"])) // P)
    pool = B * each + 3
    g = torch.Generator("cuda").manual_seed(int(seed) + 1)
    return torch.randperm(pool, generator=g, device="cuda")[:B * each].view(B, each).to(torch.int32), pool


def prepare(case, seed):
    """Inputs, and the program's cache: filled where the case reads it."""
    K, V, ek, ev, q = _inputs(case, seed)
    table, pool = _pages(case, seed)
    B, H, D, P = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
    attend = case["kind"] == "attend"
    whole = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    s = dict(kind=case["kind"], count=whole(_counts(case)), start=whole([0] * B if attend else _starts(case)), ek=ek, ev=ev, tokens=case["tokens"])
    if own:
        from gated_memory_sharing_b200 import abi
        from gated_memory_sharing_b200.layers import KV4Cache
        cache = KV4Cache(B, H, D, table.shape[1] * P, page_tokens=P, io=abi.BF16 if case["io"] == "bf16" else abi.F32,
                         num_pages=pool, table=table, k_exp=ek, v_exp=ev)
    else:
        # one page more than the pool has: rows that are none go there
        cache = dict(table=table, page=P, **{n: torch.zeros(pool + 1, H, P, w, device="cuda", dtype=torch.uint8)
                                             for n, w in (("k", D // 2), ("v", D // 2), ("ks", D // 16), ("vs", D // 16))})
    s["cache"] = cache
    if attend:
        s.update(q=q, out=torch.empty_like(q))
    if case["kind"] != "store":
        if own:
            cache.write(K, V, s["start"], s["count"])
        else:
            _write(s, K, V)
    else:
        s.update(K=K, V=V)
    if not attend:
        s.update(Ko=torch.zeros(K.shape, device="cuda", dtype=K.dtype), Vo=torch.zeros(K.shape, device="cuda", dtype=K.dtype))
    return s


# ------------------------------------------------------------------ the plain form

def _block_scale(amax):
    """e4m3(amax / 6), to nearest even, at most 448: the number of borders that amax reaches, as e4m3's codes count up."""
    codes = torch.arange(127, device=amax.device, dtype=torch.uint8)
    values = codes.view(torch.float8_e4m3fn).float()
    border = 6.0 * 0.5 * (values[1:] + values[:-1])          # exact in 32 bits
    # on a border the even code is taken: the upper one if its number is even
    border = torch.where(codes[1:] % 2 == 0, border, torch.nextafter(border, torch.full_like(border, math.inf)))
    return torch.bucketize(amax, border, right=True).to(torch.uint8)


def _quantise(x, e):
    """x [..., H, D] in 32 bits -> (codes, two a byte [..., H, D / 2], scales as e4m3's codes [..., H, D / 16])."""
    x = torch.ldexp(x.float(), -e[:, None]).unflatten(-1, (-1, 16))
    ax = x.abs()
    sc = _block_scale(ax.amax(-1))
    s = sc.view(torch.float8_e4m3fn).float()[..., None]
    c = ((ax > 0.25 * s).to(torch.uint8) + (ax >= 0.75 * s) + (ax > 1.25 * s) + (ax >= 1.75 * s) + (ax > 2.5 * s)
         + (ax >= 3.5 * s) + (ax > 5.0 * s))
    c = ((c + 8 * (x < 0)) * (s > 0)).to(torch.uint8).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], sc


def _values(codes, scales):
    """The values that codes [..., D / 2] and scales [..., D / 16] stand for, before the head's power of two."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    c = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return (c.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _rows(s, n):
    """(page, place in it, whether the row is one) of the rows start .. start + n of each sequence; no row: the page behind the pool."""
    c = s["cache"]
    t = torch.arange(n, device="cuda")
    at = s["start"][:, None].long() + t
    real = t < s["count"][:, None]
    page = torch.gather(c["table"].long(), 1, torch.clamp(at // c["page"], max=c["table"].shape[1] - 1))
    return torch.where(real, page, c["k"].shape[0] - 1), at % c["page"], real


def _write(s, K, V):
    page, place, _ = _rows(s, K.shape[1])
    c = s["cache"]
    for x, e, codes, scales in ((K, s["ek"], "k", "ks"), (V, s["ev"], "v", "vs")):
        c[codes][page, :, place], c[scales][page, :, place] = _quantise(x, e)


def _read(s, Ko, Vo):
    page, place, real = _rows(s, Ko.shape[1])
    c = s["cache"]
    for out, e, codes, scales in ((Ko, s["ek"], "k", "ks"), (Vo, s["ev"], "v", "vs")):
        x = torch.ldexp(_values(c[codes][page, :, place], c[scales][page, :, place]), e[:, None])
        out.copy_(torch.where(real[..., None, None], x, out.float()))


def _attend(s):
    c, q = s["cache"], s["q"]
    B, T, Hq, D = q.shape
    H = c["k"].shape[1]
    n = c["table"].shape[1] * c["page"]
    pages = c["table"].long()
    whole = lambda codes, scales: _values(c[codes][pages], c[scales][pages]).transpose(1, 2).reshape(B, H, n, D)  # noqa: E731
    # rows of a KV head: its query heads, for each of the new tokens
    rows = torch.ldexp(q.float().unflatten(2, (H, -1)), s["ek"][:, None, None]).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    S = torch.matmul(rows, whole("k", "ks").transpose(2, 3)) / math.sqrt(D)
    # the newest query sees count cached tokens, the one before it one fewer
    sees = s["count"][:, None] - (T - 1 - torch.arange(T, device="cuda"))
    sees = sees[:, None, None, :].expand(B, H, Hq // H, T).reshape(B, H, -1, 1)
    S = torch.where(torch.arange(n, device="cuda") < sees, S, -math.inf)
    top = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(torch.isfinite(top), top, 0.0))
    del S
    o = torch.matmul(p, whole("v", "vs")) / torch.clamp(p.sum(-1, keepdim=True), min=1e-30)  # no token: 0
    o = torch.ldexp(o, s["ev"][:, None, None])
    s["out"].copy_(o.view(B, H, Hq // H, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D))


def run(s):
    kind = s["kind"]
    if own:
        cache = s["cache"]
        if kind == "attend":
            return cache.attend(s["q"], s["count"], out=s["out"])
        if kind == "store":
            cache.write(s["K"], s["V"], s["start"], s["count"])
        return cache.read(s["start"], s["tokens"], s["count"], K=s["Ko"], V=s["Vo"])
    if kind == "attend":
        _attend(s)
        return s["out"]
    if kind == "store":
        _write(s, s["K"], s["V"])
    _read(s, s["Ko"], s["Vo"])
    return s["Ko"], s["Vo"]


# ------------------------------------------------------------------ the definition in 64 bits

def _nearest(y, bits, lowest, most):
    """y >= 0 to the nearest value with `bits` bits after the leading one (exponents from `lowest` up), ties to even, at most `most`."""
    e = torch.clamp(torch.frexp(y).exponent - 1, min=lowest) - bits
    return torch.clamp(torch.ldexp(torch.round(torch.ldexp(y, -e)), e), max=most)


def _as_kept(x, e):
    """x [..., H, D] as the cache's values, in 64 bits."""
    x = torch.ldexp(x.double(), -e[:, None]).unflatten(-1, (-1, 16))
    s = _nearest(x.abs().amax(-1, keepdim=True) / 6.0, 3, -6, 448.0)
    c = _nearest(x.abs() / torch.where(s > 0, s, 1.0), 1, 0, 6.0)
    return torch.ldexp((torch.sign(x) * c * s).flatten(-2), e[:, None])


def exact(case, seed):
    K, V, ek, ev, q = _inputs(case, seed)
    counts = _counts(case)
    if case["kind"] != "attend":
        real = torch.arange(case["tokens"], device="cuda") < torch.tensor(counts, device="cuda")[:, None]
        return tuple(torch.where(real[..., None, None], _as_kept(x, e), 0.0) for x, e in ((K, ek), (V, ev)))
    B, T, Hq, D = q.shape
    H = case["kv_heads"]
    out = torch.zeros(B, T, Hq, D, device="cuda", dtype=torch.float64)
    for b in range(B):
        if counts[b] == 0:
            continue
        k, v = (_as_kept(x[b, :counts[b]], e).transpose(0, 1) for x, e in ((K, ek), (V, ev)))     # [H, n, D]
        for t in range(T):
            n = counts[b] - (T - 1 - t)
            if n > 0:
                w = torch.softmax(q[b, t].double().view(H, Hq // H, D) @ k[:, :n].transpose(1, 2) / math.sqrt(D), -1)
                out[b, t] = (w @ v[:, :n]).view(Hq, D)
    return out
