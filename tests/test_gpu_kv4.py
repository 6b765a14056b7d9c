"""GPU parity of the 4-bit KV cache: rows written and read back bit for bit
against the oracle, the attention over it within bounds worked out per element,
and both together as a prompt and its decode steps use them."""

import numpy as np
import pytest
import torch

from gated_memory_sharing_b200 import abi
from gated_memory_sharing_b200.layers import KV4Cache
from oracle.kv4_ref import kv4_attention_ref, kv4_kept

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_memory_sharing_b200 import build
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    abi.load()
    torch.cuda.set_device(0)
    yield
    assert abi.sambay_device_status() == 0


BF16, F32 = torch.bfloat16, torch.float32


def io_of(dtype):
    return abi.BF16 if dtype == BF16 else abi.F32


def rows(seed, *shape, dtype=BF16, scale=1.0):
    """Rows with channels of different sizes, on the device."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * torch.exp2(torch.randn(shape[-2:], generator=g, device="cuda"))
    return (x * scale).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def make(batch, heads, dh, max_tokens, page, dtype=BF16, spare=3, shuffled=True, k_exp=None, v_exp=None):
    """A cache whose pages lie in the pool in no order, over bytes that are not zeros."""
    each = -(-max_tokens // page)
    pool = batch * each + spare
    g = torch.Generator().manual_seed(batch * 131 + each)
    order = torch.randperm(pool, generator=g)[:batch * each] if shuffled else torch.arange(batch * each)
    c = KV4Cache(batch, heads, dh, max_tokens, page_tokens=page, io=io_of(dtype), num_pages=pool,
                 table=order.view(batch, each).to(torch.int32).cuda(), k_exp=k_exp, v_exp=v_exp)
    c.pages.fill_(0xFF)          # scales of NaN wherever nothing is written
    return c


def same(got, want):
    """Equal values, NaN where NaN."""
    return np.array_equal(got, want, equal_nan=True)


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,dh,page,T,starts,counts", [
    (1, 1, 64, 16, 1, [0], None),
    (1, 20, 64, 64, 100, [0], None),
    (3, 2, 64, 16, 37, [0, 5, 130], [37, 0, 21]),
    (2, 3, 128, 32, 1, [31, 32], None),
    (5, 4, 128, 128, 64, [1, 2, 15, 16, 127], [64, 63, 1, 17, 48]),
    (2, 5, 64, 1024, 333, [700, 0], [333, 332]),
])
def test_rows_come_back_as_kept(B, H, dh, page, T, starts, counts, dtype):
    ek, ev = i32([(-9, 2, 0, -3)[i % 4] for i in range(H)]), i32([(-10, 1)[i % 2] for i in range(H)])
    c = make(B, H, dh, max(starts) + T, page, dtype, k_exp=ek, v_exp=ev)
    K, V = rows(1, B, T, H, dh, dtype=dtype), rows(2, B, T, H, dh, dtype=dtype, scale=0.1)
    pos, count = i32(starts), None if counts is None else i32(counts)
    c.write(K, V, pos, count)
    Ko, Vo = torch.full_like(K, 7.0), torch.full_like(V, 7.0)
    assert c.read(pos, T, count, K=Ko, V=Vo)[0] is Ko
    real = np.arange(T) < np.array(counts if counts else [T] * B)[:, None]
    for got, x, e in ((Ko, K, ek), (Vo, V, ev)):
        want = np.where(real[..., None, None], kv4_kept(f64(x), e.cpu().numpy()), 7.0)
        assert same(f64(got), want)


def test_special_values():
    """Borders, zeros, values past the scale's range, NaN and infinities, tiny values."""
    H, dh = 1, 64
    x = np.zeros((12, 4, 16), dtype=np.float64)
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i, s in enumerate((1.0, 0.5625, 448.0, 2.0 ** -9, 1.875 * 2.0 ** -6)):       # every border of e2m1, up to 6 s
        x[i, :, :8], x[i, :, 8:] = grid * s, -grid * s
        x[i, 1:, 0] += s / 64 * np.array([1, -1, 0])
    for i in range(4):                                                                # borders of the scale
        x[5, i, 3] = 6 * 2 * (1 + (2 * i + 1) / 16)
        x[6, i, 3] = 6 * 2.0 ** -9 * (i + 0.5)
    x[7, 0, 2], x[7, 1, 0], x[7, 2, 5], x[7, 3, 9] = np.nan, np.inf, -np.inf, 3e38
    x[8, 0, 0], x[8, 1, 0], x[8, 2, 0], x[8, 3, 0] = 2.0 ** -11, 6 * 2.0 ** -10, 6.1 * 2.0 ** -10, 1e-40
    x[9, 0, :], x[9, 1, 4] = -0.0, 1e30
    x[10] = np.random.default_rng(5).integers(-127, 128, (4, 16)) / 8
    for dtype in (BF16, F32):
        t = torch.from_numpy(x.reshape(1, 12, H, dh)).to(dtype).cuda()
        c = make(1, H, dh, 16, 16, dtype)
        c.write(t, t, i32([2]))
        K, V = c.read(i32([2]), 12)
        want = kv4_kept(f64(t))
        assert same(f64(K), want) and same(f64(V), want)
        assert np.isnan(want[0, 7, 0]).sum() == 48 and np.abs(want[0, 7, 0, 48:]).max() == 2688


def test_rows_of_a_fused_projection():
    B, T, H, dh = 3, 19, 4, 64
    both = rows(6, B, T, 4 * H, dh)
    K, V = both[:, :, 2 * H:3 * H], both[:, :, 3 * H:]
    c = make(B, H, dh, 64, 16)
    c.write(K, V, i32([0, 9, 45]))
    Ko, Vo = c.read(i32([0, 9, 45]), T)
    assert same(f64(Ko), kv4_kept(f64(K))) and same(f64(Vo), kv4_kept(f64(V)))
    # one token of several sequences: the stride between sequences
    step = rows(7, B, 1, 4 * H, dh)
    c.write(step[:, :, :H], step[:, :, H:2 * H], i32([63, 0, 20]))
    Ko, Vo = c.read(i32([63, 0, 20]), 1)
    assert same(f64(Ko), kv4_kept(f64(step[:, :, :H]))) and same(f64(Vo), kv4_kept(f64(step[:, :, H:2 * H])))


def test_a_write_changes_only_its_positions():
    B, H, dh, page = 2, 3, 128, 32
    c = make(B, H, dh, 96, page)
    K, V = rows(8, B, 96, H, dh), rows(9, B, 96, H, dh)
    c.write(K, V, i32([0, 0]))
    before = c.pages.clone()
    k0, v0 = c.read(i32([0, 0]), 96)
    K2, V2 = rows(10, B, 7, H, dh), rows(11, B, 7, H, dh)
    c.write(K2, V2, i32([30, 89]), i32([5, 7]))
    k1, v1 = c.read(i32([0, 0]), 96)
    for b, (s, n) in enumerate(((30, 5), (89, 7))):
        for old, new, rows2 in ((k0, k1, K2), (v0, v1, V2)):
            want = f64(old[b])
            want[s:s + n] = kv4_kept(f64(rows2[b, :n]))
            assert same(f64(new[b]), want)
    # the same rows again: the same bytes, in pages of the table and outside it
    c.write(K[:, 30:37].contiguous(), V[:, 30:37].contiguous(), i32([30, 30]), i32([5, 0]))
    c.write(K[:, 89:96].contiguous(), V[:, 89:96].contiguous(), i32([89, 89]), i32([0, 7]))
    assert torch.equal(before, c.pages)


# ------------------------------------------------------------------ attention

def bound(ref, spread, logit, dtype, dh, n):
    """How far an output may be from the float64 value, per element.

    The output's own rounding: eps / 2 of it.  The rest is relative to
    sum_j p_j |v_j|: each probability's rounding (f16: 2^-11; a pair of f16:
    2^-22) and ex2's error (2 ulp: 2^-22), twice (numerator and denominator),
    with the logits' error, which moves every p by at most e^(2 d) - 1:
    d = (dh + 4) roundings of the sum |q k| (2^-23, the tensor cores truncate),
    and for f32 the pair of f16 that q is (2^-22); and the sums over n tokens, 16
    a step, at 2^-23 each, with 64 more for joining warps and splits."""
    half = torch.finfo(dtype).eps / 2
    p = 2.0 ** -11 if dtype == BF16 else 2.0 ** -22
    q = 0.0 if dtype == BF16 else 2.0 ** -22
    d = logit * ((dh + 4) * 2.0 ** -23 + q)
    rel = 2 * (p + 2.0 ** -22) + np.expm1(2 * d) + (n / 16 + 64) * 2.0 ** -23
    return half * np.abs(ref) + rel[..., None] * spread * (1 + half) + 1e-30


def check(out, q, K, V, lens, count=None, scale=None, what=""):
    ref, spread, logit = kv4_attention_ref(f64(q), K, V, lens, count, scale)
    got = f64(out)
    live = ~np.isnan(logit)
    lim = bound(ref, spread, logit, out.dtype, q.shape[-1], max(lens))
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got[live])), what
    worst = np.max((err / lim)[live]) if live.any() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"
    return worst


def filled(B, H, dh, page, lens, dtype, seed=20, **kw):
    """A cache with lens[b] rows of each sequence, and what it keeps."""
    n = max(max(lens), 1)
    K, V = rows(seed, B, n, H, dh, dtype=dtype), rows(seed + 1, B, n, H, dh, dtype=dtype)
    c = make(B, H, dh, n, page, dtype, **kw)
    c.write(K, V, i32([0] * B), i32(lens))
    e = [None if t is None else t.cpu().numpy() for t in (c.k_exp, c.v_exp)]
    return c, kv4_kept(f64(K), e[0]), kv4_kept(f64(V), e[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hkv,dh,page,lens", [
    (1, 2, 1, 64, 16, [1]),
    (4, 4, 2, 64, 16, [0, 1, 15, 16]),
    (4, 4, 2, 64, 64, [17, 63, 64, 65]),
    (3, 6, 2, 128, 32, [300, 257, 0]),
    (2, 16, 1, 64, 128, [1000, 129]),        # 16 query heads share one
    (2, 15, 1, 128, 64, [700, 5]),
    (1, 9, 9, 64, 16, [333]),                # none share
    (1, 8, 1, 128, 16, [5000]),              # few sequences, many tokens
    (33, 10, 5, 64, 64, [(37 * i) % 200 for i in range(33)]),
    (70, 4, 2, 128, 16, [(i * i * 31) % 1500 for i in range(70)]),
    (40, 3, 3, 64, 16, [3000 if i == 7 else i % 3 for i in range(40)]),      # one long among short ones
])
def test_attention(B, Hq, Hkv, dh, page, lens, dtype):
    c, K, V = filled(B, Hkv, dh, page, lens, dtype)
    q = rows(30, B, 1, Hq, dh, dtype=dtype)
    out = c.attend(q, i32(lens))
    check(out, q, K, V, lens, what=f"{dtype} B{B} Hq{Hq} Hkv{Hkv} dh{dh}")
    assert torch.equal(out[:, 0], c.attend(q[:, 0].contiguous(), i32(lens)))     # and the same bits again
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.all(out[b] == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,Hq,Hkv,dh,lens,count", [
    (4, 4, 2, 64, [100, 4, 3, 1], None),               # the first queries of short sequences see nothing
    (5, 6, 2, 128, [64, 65, 0, 200], [5, 3, 2, 0]),
    (16, 16, 1, 64, [70, 600, 16, 17], None),          # several row tiles
    (3, 8, 2, 128, [1500, 33, 2, 48], [1, 2, 3, 3]),
])
def test_attention_of_several_tokens(T, Hq, Hkv, dh, lens, count, dtype):
    B = len(lens)
    c, K, V = filled(B, Hkv, dh, 32, lens, dtype, seed=40)
    q = rows(50, B, T, Hq, dh, dtype=dtype)
    out = torch.full_like(q, 7.0)
    c.attend(q, i32(lens), None if count is None else i32(count), out=out)
    check(out, q, K, V, lens, count, what=f"{dtype} T{T}")
    for b, n in enumerate(count or []):
        assert torch.all(out[b, n:] == 7.0)                                       # rows that are none: left as they were


@pytest.mark.parametrize("dtype,Hq,Hkv,dh,page", [(BF16, 16, 8, 64, 32), (F32, 8, 8, 128, 16), (BF16, 128, 8, 64, 128)])
def test_many_long_and_short_sequences(dtype, Hq, Hkv, dh, page):
    """Warps' shares that are long (where changing to another sequence counts in
    them), with runs of empty and short sequences; some sequences against the oracle."""
    lens = [3000 - i if i % 9 == 0 else (0, 1, 64, 700, 65, 2000, 0, 5)[i % 8] for i in range(120)]
    B = len(lens)
    assert Hkv * sum(max(1, -(-n * dh // 4096)) for n in lens) >= 4 * 148 * 3 * 4
    K, V = rows(55, B, max(lens), Hkv, dh, dtype=dtype), rows(56, B, max(lens), Hkv, dh, dtype=dtype)
    c = make(B, Hkv, dh, max(lens), page, dtype)
    c.write(K, V, i32([0] * B), i32(lens))
    q = rows(57, B, 1, Hq, dh, dtype=dtype)
    out = c.attend(q, i32(lens))
    some = [0, 1, 3, 5, 8, 9, 40, 63, 90, 112, 117, 119]
    at = torch.tensor(some, device="cuda")
    check(out[at], q[at], kv4_kept(f64(K[at])), kv4_kept(f64(V[at])), [lens[i] for i in some], what="long and short")
    assert torch.isfinite(out).all() and torch.all(out[i32([i for i in range(B) if lens[i] == 0]).long()] == 0)
    assert torch.equal(out, c.attend(q, i32(lens)))
    # a sequence alone: other shares, the same bound
    kk, vv = kv4_kept(f64(K[at])), kv4_kept(f64(V[at]))
    for j in (0, 2, 8):
        one = i32([lens[some[j]] if i == some[j] else 0 for i in range(B)])
        alone = c.attend(q, one)
        check(alone[at][j:j + 1], q[at][j:j + 1], kk[j:j + 1], vv[j:j + 1], [lens[some[j]]], what="alone")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("G,T,Hkv", [
    (5, 1, 8),       # 8 columns: 4 rows and one more
    (7, 1, 8),       # ... and three more
    (11, 1, 5),      # 16 columns, three more than 8
    (5, 2, 5),       # rows of two tokens, 10 in all
    (7, 3, 3),       # two tiles of rows, 16 and 5
    (1, 4, 8),       # just 4
])
def test_rows_joined_four_at_a_time(G, T, Hkv, dh, dtype):
    """Many pairs of few parts each, the last columns of a pair among them."""
    rows_, B = G * T, 126
    lens = [(0, 3, 900, 64, 333, 128, 1, 517, 250)[i % 9] + i for i in range(B)]
    tiles, wide = -(-rows_ // (8 if rows_ <= 8 else 16)), 8 if rows_ <= 8 else 16
    pairs, warps = B * Hkv * tiles, 4 * 148 * (3 if wide == 8 else 2)
    assert warps <= 2 * pairs and min(rows_, wide) >= 4          # this form's condition
    K, V = rows(61, B, max(lens), Hkv, dh, dtype=dtype), rows(62, B, max(lens), Hkv, dh, dtype=dtype)
    c = make(B, Hkv, dh, max(lens), 64, dtype)
    c.write(K, V, i32([0] * B), i32(lens))
    q = rows(63, B, T, Hkv * G, dh, dtype=dtype)
    out = torch.full_like(q, 7.0)
    counts = [T - (i % 5 == 4) for i in range(B)]
    c.attend(q, i32(lens), i32(counts), out=out)
    some = [0, 1, 2, 4, 7, 11, 65, 101, 120, 125]
    at = torch.tensor(some, device="cuda")
    check(out[at], q[at], kv4_kept(f64(K[at])), kv4_kept(f64(V[at])), [lens[i] for i in some],
          [counts[i] for i in some], what=f"G{G} T{T}")
    assert torch.isfinite(out).all()
    for i, n in enumerate(counts):
        assert torch.all(out[i, n:] == 7.0)
    again = torch.full_like(q, 7.0)
    assert torch.equal(out, c.attend(q, i32(lens), i32(counts), out=again))


def test_many_sequences():
    """More sequences than a warp's lanes have looked through so far, up to the most that a call takes."""
    for B, n, page in ((5000, 200, 32), (65535, 80, 16)):
        lens = np.random.default_rng(B).integers(0, n + 1, B)
        lens[B // 2], lens[-1] = n, n
        K, V = rows(64, B, n, 1, 64), rows(65, B, n, 1, 64)
        c = make(B, 1, 64, n, page)
        L = torch.from_numpy(lens.astype(np.int32)).cuda()
        c.write(K, V, torch.zeros_like(L), L)
        q = rows(66, B, 1, 2, 64)
        out = c.attend(q, L)
        some = [0, 1, 31, 32, 2047, 2048, B // 2, B - 2, B - 1] + list(range(100, B, B // 13))
        at = torch.tensor(some, device="cuda")
        check(out[at], q[at], kv4_kept(f64(K[at])), kv4_kept(f64(V[at])), [int(lens[i]) for i in some], what=f"B{B}")
        assert torch.isfinite(out).all() and torch.all(out[L == 0] == 0) and torch.all(out[L > 0].abs().amax((1, 2, 3)) > 0)
        del K, V, c, out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hkv,dh", [
    (150, 4, 2, 64),          # 1 or 4 warps join a row, by how many rows there are
    (301, 2, 1, 128),
    (600, 2, 2, 64),
    (130, 48, 3, 64),
])
def test_one_long_sequence_among_many_empty(B, Hq, Hkv, dh, dtype):
    """Rows of many parts beside rows of none, in batches of many rows."""
    n, at = 2500, B // 2
    lens = [n if b == at else (0, 0, 1, 0)[b % 4] for b in range(B)]
    K, V = rows(58, 1, n, Hkv, dh, dtype=dtype), rows(59, 1, n, Hkv, dh, dtype=dtype)
    c = make(B, Hkv, dh, n, 64, dtype)
    c.write(K.expand(B, -1, -1, -1).contiguous(), V.expand(B, -1, -1, -1).contiguous(), i32([0] * B), i32(lens))
    q = rows(60, B, 1, Hq, dh, dtype=dtype)
    out = c.attend(q, i32(lens))
    kk, vv = kv4_kept(f64(K)), kv4_kept(f64(V))
    check(out[at:at + 1], q[at:at + 1], kk, vv, [n], what="long")
    one = [b for b in range(B) if lens[b] == 1]
    sel = torch.tensor(one, device="cuda")
    rep = lambda x: np.repeat(x[:, :1], len(one), axis=0)
    check(out[sel], q[sel], rep(kk), rep(vv), [1] * len(one), what="one token")
    assert torch.all(out[torch.tensor([b for b in range(B) if lens[b] == 0], device="cuda")] == 0)
    assert torch.equal(out, c.attend(q, i32(lens)))


def test_exponents_and_scale():
    B, H, dh, lens = 2, 4, 64, [130, 77]
    Kr, Vr = rows(60, B, 130, H, dh, scale=2.0 ** -20), rows(61, B, 130, H, dh, scale=2.0 ** 13)
    ek, ev = KV4Cache.exponents(Kr), KV4Cache.exponents(Vr)
    for e, x in ((ek, Kr), (ev, Vr)):
        top = f64(x.abs().amax((0, 1, 3)).float()) / 2.0 ** e.cpu().double().numpy()
        assert np.all(top <= 2688) and np.all(top > 1344)
    c = make(B, H, dh, 130, 16, k_exp=ek, v_exp=ev)
    c.write(Kr, Vr, i32([0, 0]), i32(lens))
    q = rows(62, B, 1, 8, dh, scale=2.0 ** 20)
    out = c.attend(q, i32(lens), scale=0.3)
    check(out, q, kv4_kept(f64(Kr), ek.cpu().numpy()), kv4_kept(f64(Vr), ev.cpu().numpy()), lens, scale=0.3)


def test_dominant_and_equal_logits():
    """Logits far apart (one token takes all) and all equal (a mean of values); queries of zeros; tiny and huge rows."""
    c, K, V = filled(1, 1, 64, 64, [500], F32, seed=70)
    q = rows(71, 1, 1, 8, 64, dtype=F32)
    q[0, 0, 0] *= 300.0
    q[0, 0, 1] = 0.0
    q[0, 0, 2] *= 2.0 ** -100
    q[0, 0, 3, 1:] = 0.0
    check(c.attend(q, i32([500])), q, K, V, [500], what="logits far apart and equal")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 16, 2), (2, 16, 1)])       # 8 columns; 16, and two tiles of rows
@pytest.mark.parametrize("keys", ["top", "least negative", "equal"])
def test_large_logits(keys, T, Hq, Hkv, dh, dtype):
    """Logits (in base 2) of 2^20 to 2^101: one key above the others, whose value
    is the output, or all keys the same, whose mean value it is.

    Rows of keys are +-1, +-.25 or +-2 (kept as 1.03125 times that), and queries
    have the signs of the top key: the other logits are at least 3/4 of the top
    one's size below it.  Both may be off by dh + 4 roundings of 2^-23, below 2^-15
    of their size, so the others weigh less than 2^-100 from 2^20 on, and the bound
    has no part of the logits' errors.  Equal keys give equal sums, whatever they
    are off by."""
    lens = [2, 33, 700, 5000]                   # one tile; several; pairs that several warps share
    B, n = len(lens), max(lens)
    g = torch.Generator("cuda").manual_seed(dh + T)
    signs = lambda *shape: 2.0 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1.0  # noqa: E731
    u = signs(1, 1, Hkv, dh)
    at = [0, 20, 123, 3456]
    K = {"top": 0.25 * signs(B, n, Hkv, dh), "least negative": -2.0 * u.expand(B, n, -1, -1),
         "equal": u.expand(B, n, -1, -1)}[keys].to(dtype).contiguous()
    for b, j in enumerate(at):
        if keys != "equal":
            K[b, j] = (u if keys == "top" else -u)[0, 0].to(dtype)
    V = rows(73, B, n, Hkv, dh, dtype=dtype)
    c = make(B, Hkv, dh, n, 64, dtype)
    c.write(K, V, i32([0] * B), i32(lens))
    kept = np.repeat(kv4_kept(f64(V)), Hq // Hkv, axis=2)                    # [B, n, Hq, dh]
    want, spread = np.zeros((B, T, Hq, dh)), np.zeros((B, T, Hq, dh))
    for b, j in enumerate(at):
        for t in range(T):
            seen = slice(0, lens[b] - (T - 1 - t)) if keys == "equal" else slice(j, j + 1)
            want[b, t], spread[b, t] = kept[b, seen].mean(0), np.abs(kept[b, seen]).mean(0)
    lim = bound(want, spread, np.zeros((B, T, Hq)), dtype, dh, n)
    wrong = {}
    for log2 in (20, 24, 25, 26, 27, 28, 30, 45, 60, 100):
        for scale in (None, 1e4):
            size = 2.0 ** log2 * np.log(2.0) / (dh * (scale or dh ** -0.5))
            q = size * (1 + torch.rand(B, T, Hq, dh, generator=g, device="cuda", dtype=torch.float64))
            q = (q.view(B, T, Hkv, -1, dh) * u[:, :, :, None].double()).view(B, T, Hq, dh).to(dtype)
            off = (np.abs(f64(c.attend(q, i32(lens), scale=scale or 0.0)) - want) / lim).max(-1)
            if not np.all(off <= 1.0):
                wrong[log2, scale] = np.mean(~(off <= 1.0))
    assert not wrong, f"shares of rows that are off, by log2 of the logits and scale: {wrong}"


def test_what_is_not_the_sequences_is_not_read():
    """NaN in every byte behind the last token, in the spare pages, and in another sequence's tokens."""
    for dh, n in ((64, 50), (128, 17)):
        c, K, V = filled(2, 2, dh, 16, [n, 0], BF16, seed=80)
        q = rows(81, 2, 1, 4, dh)
        bad = torch.full((2, 16 - n % 16, 2, dh), float("nan"), device="cuda", dtype=BF16)
        c.write(bad, bad, i32([n, 0]), i32([14 if 16 - n % 16 >= 14 else 16 - n % 16, 5]))
        check(c.attend(q, i32([n, 0])), q, K, V, [n, 0], what="NaN behind the end")
    # a NaN that belongs to the sequence is seen
    c.write(bad[:, :1].contiguous(), bad[:, :1].contiguous(), i32([3, 0]), i32([1, 0]))
    assert torch.isnan(c.attend(q, i32([n, 0]))[0]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_nan_reaches_only_the_queries_that_see_it(dtype):
    """Rows of NaN and infinity at newer tokens: older queries of the same call do not see them."""
    for dh, n, T, at in ((64, 70, 4, 68), (128, 40, 6, 35), (64, 64, 3, 63), (128, 16, 2, 15)):
        c, K, V = filled(1, 2, dh, 16, [n], dtype, seed=85)
        q = rows(86, 1, T, 6, dh, dtype=dtype)
        want = c.attend(q, i32([n]))
        k, v = rows(85, 1, n, 2, dh, dtype=dtype)[:, at:at + 1].clone(), rows(86, 1, n, 2, dh, dtype=dtype)[:, at:at + 1].clone()
        v[0, 0, 1, 20] = float("inf")              # one block of one head's V
        c.write(k, v, i32([at]))
        out = c.attend(q, i32([n]))
        first = at - (n - T)                       # the first query that sees token `at`
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[0, first:, 3:, 16:32] = True
        assert torch.equal(torch.isnan(out), hit)
        assert torch.equal(out[:, :first], want[:, :first])
        k[0, 0, 0, 3] = float("nan")               # and one of the other head's K
        c.write(k, v, i32([at]))
        hit[0, first:, :3] = True
        out = c.attend(q, i32([n]))
        assert torch.equal(torch.isnan(out), hit)
        assert torch.equal(out[:, :first], want[:, :first])


def test_pages_outside_the_pool_are_skipped_and_recorded():
    c, K, V = filled(2, 2, 64, 16, [100, 100], BF16, seed=90)
    q = rows(91, 2, 1, 4, 64)
    good = c.attend(q, i32([100, 100]))
    assert abi.sambay_device_status() == 0
    keep = c.table.clone()
    for page in (-1, c.dims.num_pages, 2 ** 31 - 1, -2 ** 31):
        c.table.copy_(keep)
        c.table[0, 2] = page
        out = c.attend(q, i32([100, 100]))
        assert abi.sambay_device_status() == 1
        assert torch.equal(out[1], good[1])
        left = [j for j in range(100) if not 32 <= j < 48]        # the others' tokens are attended to
        check(out[:1], q[:1], K[:1, left], V[:1, left], [len(left)], what="a page that is none")
        x = rows(92, 2, 20, 2, 64)
        before = c.pages.clone()
        c.write(x, x, i32([30, 0]), i32([20, 0]))
        assert abi.sambay_device_status() == 1
        Ko = torch.full_like(x, 7.0)
        c.read(i32([30, 0]), 20, i32([20, 0]), K=Ko, V=torch.empty_like(x))
        assert abi.sambay_device_status() == 1
        want = kv4_kept(f64(x))
        assert same(f64(Ko[0, :2]), want[0, :2]) and torch.all(Ko[0, 2:18] == 7.0) and same(f64(Ko[0, 18:]), want[0, 18:])
        c.pages.copy_(before)
    c.table.copy_(keep)
    # lengths, positions and counts outside the table or the call
    q3 = rows(93, 2, 3, 4, 64)
    cap = c.table.shape[1] * 16
    for lens, count in (([cap + 1, 100], None), ([-5, 100], None), ([100, 100], [4, 3]), ([100, 100], [-1, 3])):
        c.attend(q3, i32(lens), None if count is None else i32(count))
        assert abi.sambay_device_status() == 1
    x = rows(94, 2, 3, 2, 64)
    before = c.pages.clone()
    for pos, count in (([cap, -3], None), ([2 ** 31 - 1, cap + 5], None), ([-2 ** 31, -9], None), ([0, 0], [0, -2])):
        c.write(x, x, i32(pos), None if count is None else i32(count))
        assert abi.sambay_device_status() == 1
    assert torch.equal(before, c.pages)


def test_cache_past_32_bits():
    """A pool of more than 4 GB: the last page's rows."""
    H, dh, page = 8, 128, 1024
    pool = (1 << 32) // (H * page * dh * 9 // 8) + 40
    c = KV4Cache(2, H, dh, 2 * page, page_tokens=page, num_pages=pool,
                 table=i32([[pool - 1, 0], [1, pool - 2]]))
    assert c.pages.numel() > 1 << 32
    K, V = rows(100, 2, 1100, H, dh), rows(101, 2, 1100, H, dh)
    c.write(K, V, i32([0, 300]))
    Ko, Vo = c.read(i32([0, 300]), 1100)
    assert same(f64(Ko), kv4_kept(f64(K))) and same(f64(Vo), kv4_kept(f64(V)))
    q = rows(102, 2, 1, H, dh)
    first = i32([1100, 0])
    check(c.attend(q, first), q, kv4_kept(f64(K)), kv4_kept(f64(V)), [1100, 0])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_and_decode_steps(dtype):
    """A padded batch of prompts, then decode steps: each writes one row a sequence and attends, two layers reading it."""
    B, Hq, H, dh, page, T = 3, 8, 4, 64, 16, 45
    lens = [45, 30, 1]
    ek, ev = i32([-8] * H), i32([-9] * H)
    c = make(B, H, dh, T + 6, page, dtype, k_exp=ek, v_exp=ev)
    K = np.full((B, T + 6, H, dh), np.nan)
    V = K.copy()
    k, v = rows(110, B, T, H, dh, dtype=dtype), rows(111, B, T, H, dh, dtype=dtype)
    c.write(k, v, i32([0] * B), i32(lens))
    e = [ek.cpu().numpy(), ev.cpu().numpy()]
    for b in range(B):
        K[b, :lens[b]], V[b, :lens[b]] = kv4_kept(f64(k[b, :lens[b]]), e[0]), kv4_kept(f64(v[b, :lens[b]]), e[1])
    pos = i32(lens)
    for step in range(6):
        k, v = rows(120 + step, B, 1, H, dh, dtype=dtype), rows(130 + step, B, 1, H, dh, dtype=dtype)
        c.write(k, v, pos)
        pos += 1
        for b in range(B):
            K[b, lens[b]], V[b, lens[b]] = kv4_kept(f64(k[b, 0]), e[0]), kv4_kept(f64(v[b, 0]), e[1])
            lens[b] += 1
        for layer in range(2):
            q = rows(140 + 2 * step + layer, B, 1, Hq, dh, dtype=dtype)
            check(c.attend(q, pos), q, K, V, lens, what=f"step {step} layer {layer}")


def test_streams_and_graphs():
    """Calls on two streams at once, on an explicit stream, and two captured graphs of one cache replayed together."""
    lens = [900, 333]
    c, K, V = filled(2, 4, 64, 64, lens, BF16, seed=150)
    n = i32(lens)
    qs = [rows(160 + i, 2, 1, 8, 64) for i in range(2)]
    want = [c.attend(q, n) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(c.attend(qs[i], n, stream=s))
    raw = c.attend(qs[0], n, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in got[i]) and torch.equal(raw, want[0])
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.attend(q, n))
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # a captured decode step follows the lengths it reads on the device
    x = rows(170, 2, 1, 4, 64)
    pos, after = i32([100, 20]), i32([101, 21])
    out = torch.empty_like(qs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.write(x, x, pos)
        c.attend(qs[0], after, out=out)
    for step in range(3):
        pos.fill_(100 + 7 * step)
        after.copy_(pos + 1)
        g.replay()
        want = out.clone()
        assert torch.equal(c.attend(qs[0], after), want)
        assert same(f64(c.read(pos, 1)[0]), kv4_kept(f64(x)))


def test_the_default_stream_by_its_handle():
    """The handle 0 is the default stream's: calls given it follow what was queued there."""
    assert torch.cuda.default_stream().cuda_stream == 0
    lens = [200, 77]
    c, _, _ = filled(2, 4, 64, 16, lens, BF16, seed=185)
    n, pos = i32(lens), i32([199, 76])
    src, xs = rows(186, 2, 1, 8, 64), rows(187, 2, 1, 4, 64)
    assert c._on(0)[0] == 0
    x, q = torch.zeros_like(xs), torch.zeros_like(src)
    torch.cuda._sleep(20_000_000)              # about 10 ms in front of the copies
    x.copy_(xs)
    q.copy_(src)
    c.write(x, x, pos, stream=0)
    out = c.attend(q, n, stream=torch.cuda.default_stream().cuda_stream)
    Ko, _ = c.read(pos, 1, stream=0)
    assert same(f64(Ko), kv4_kept(f64(xs)))
    assert torch.equal(out, c.attend(src, n))


def test_after_other_work_in_a_graph():
    """Captured behind a copy, a fill, and a join with another stream: each call still follows what was queued before it."""
    lens = [200, 77]
    c, _, _ = filled(2, 4, 64, 16, lens, BF16, seed=190)
    n = i32(lens)
    src, q, x, xs = rows(191, 2, 1, 8, 64), rows(192, 2, 1, 8, 64), rows(193, 2, 1, 4, 64), rows(194, 2, 1, 4, 64)
    wants = []
    for k in range(3):
        src.copy_(rows(195 + k, 2, 1, 8, 64))
        xs.copy_(rows(198 + k, 2, 1, 4, 64))
        c.write(xs, xs, i32([199, 76]))
        wants.append(c.attend(src, n))
    side, out = torch.cuda.Stream(), torch.empty_like(q)
    pos = i32([199, 76])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.copy_(src)
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x.copy_(xs)
        torch.cuda.current_stream().wait_stream(side)
        c.write(x, x, pos)
        c.attend(q, n, out=out)
        Ko, _ = c.read(pos, 1)
    for k in range(3):
        src.copy_(rows(195 + k, 2, 1, 8, 64))
        xs.copy_(rows(198 + k, 2, 1, 4, 64))
        g.replay()
        assert torch.equal(out, wants[k]) and same(f64(Ko), kv4_kept(f64(xs)))


def test_the_table_changes_in_place_only():
    lens = [100, 60]
    c, K, V = filled(2, 2, 64, 16, lens, BF16, seed=175)
    q = rows(176, 2, 1, 4, 64)
    want = c.attend(q, i32(lens))
    moved = c.table.clone()
    moved[0, 0], moved[0, 1] = c.table[0, 1], c.table[0, 0]        # 16 tokens before the 16 in front of them
    with pytest.raises(ValueError):
        c.table = moved
    assert torch.equal(c.attend(q, i32(lens)), want)
    table = c.table
    c.table += 0
    c.table[:] = moved
    assert c.table is table
    for x in (K, V):
        x[0, :32] = np.concatenate([x[0, 16:32], x[0, :16]])
    check(c.attend(q, i32(lens)), q, K, V, lens, what="pages exchanged")
    Ko, Vo = c.read(i32([0, 0]), 60)
    assert same(f64(Ko), K[:, :60]) and same(f64(Vo), V[:, :60])


def test_layer_refusals():
    c = KV4Cache(2, 4, 64, 100, page_tokens=16)
    k = rows(180, 2, 5, 4, 64)
    pos = i32([0, 0])
    for bad in (lambda: c.write(k.float(), k, pos), lambda: c.write(k[:1], k[:1], pos), lambda: c.write(k, k[:, :3], pos),
                lambda: c.write(k.transpose(1, 2), k, pos), lambda: c.write(k[..., ::2], k, pos),
                lambda: c.write(k, k, pos.long()), lambda: c.write(k, k, pos.cpu()), lambda: c.write(k, k, i32([0])),
                lambda: c.write(k.cpu(), k, pos), lambda: c.write(k, k, pos, i32([1, 2, 3])),
                lambda: c.write(rows(181, 2, 10, 4, 64)[:, ::2].expand(2, 5, 4, 64)[:, :, :, :32], k, pos),
                lambda: c.write(k[:, :1].expand(2, 5, 4, 64), k, pos), lambda: c.write(k, k[:1].expand(2, 5, 4, 64), pos),
                lambda: c.write(k[:, :0], k[:, :0], pos), lambda: c.read(pos, 0), lambda: c.attend(k[:, :0], pos),
                lambda: c.read(pos, 5, K=k.float()), lambda: c.read(pos, 4, K=k), lambda: c.read(pos.float(), 4),
                lambda: c.attend(k, pos.long()), lambda: c.attend(k.float(), pos), lambda: c.attend(k, pos, out=k[:, :2]),
                lambda: c.attend(k.transpose(0, 1), pos), lambda: c.attend(k[:, :, :, :32], pos)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.attend(rows(182, 2, 1, 6, 64), pos), lambda: c.attend(rows(183, 2, 17, 4, 64), pos),
                lambda: c.attend(k, pos, out=k), lambda: c.attend(k, pos, scale=-1.0)):
        with pytest.raises(abi.SambayError):
            bad()
    for kw in (dict(head_dim=96), dict(page_tokens=24), dict(num_pages=3), dict(table=i32([[0, 1]])),
               dict(table=i32([[0, 1], [1, 2]]).long(), num_pages=9), dict(k_exp=i32([0] * 3))):
        with pytest.raises(ValueError):
            KV4Cache(**{**dict(batch=2, kv_heads=4, head_dim=64, max_tokens=100, page_tokens=16), **kw})
