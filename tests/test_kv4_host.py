"""Host-side checks of the 4-bit KV cache's entry points that need no GPU: every
case is built so that validation fails before the library touches a device."""

import pytest
import torch

from gated_memory_sharing_b200 import abi, build
from gated_memory_sharing_b200.layers import KV4Cache


class _Ptr:
    """A pointer that is only looked at."""

    def __init__(self, address, nbytes=0):
        self.address, self.nbytes = address, nbytes

    def data_ptr(self):
        return self.address

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


def dims(batch=2, kv_heads=4, head_dim=64, page_tokens=64, num_pages=8, table_pages=4, io=abi.BF16):
    return abi.Kv4Dims(batch, kv_heads, head_dim, page_tokens, num_pages, table_pages, io)


P = [_Ptr(0x10000 * i) for i in range(1, 12)]
PAGES, TABLE, K, V, POS, COUNT, Q, OUT, LENS, WS, EXP = P


def cache(pages=PAGES, table=TABLE, k_exp=None, v_exp=None):
    return abi.make_kv4_cache(pages, table, k_exp, v_exp)


BAD_DIMS = [
    (dict(batch=0), 1), (dict(kv_heads=0), 1), (dict(head_dim=0), 1), (dict(page_tokens=0), 1),
    (dict(num_pages=0), 1), (dict(table_pages=0), 1), (dict(io=7), 1), (dict(batch=-1), 1),
    (dict(head_dim=96), 2), (dict(page_tokens=8), 2), (dict(page_tokens=48), 2), (dict(page_tokens=2048), 2),
    (dict(page_tokens=1024, table_pages=(1 << 20) + 1), 2), (dict(batch=65536), 2), (dict(kv_heads=65536), 2),
]


def refused(code, fn, *args, **kw):
    with pytest.raises(abi.SambayError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.code == code


def test_cache_bytes():
    # 4.5 bits an element: 18 dh bytes for 16 tokens of a head
    assert abi.sambay_kv4_cache_bytes(dims()) == 8 * 4 * 64 * 64 * 9 // 8
    assert abi.sambay_kv4_cache_bytes(dims(head_dim=128, page_tokens=16, num_pages=1, kv_heads=1)) == 2304
    # past 32 bits
    assert abi.sambay_kv4_cache_bytes(dims(num_pages=1 << 20, kv_heads=20)) == (1 << 20) * 20 * 4608


@pytest.mark.parametrize("bad,code", BAD_DIMS)
def test_bad_sizes(bad, code):
    d = dims(**bad)
    assert abi.sambay_kv4_cache_bytes(d) == 0
    assert abi.sambay_cross_attn_decode_kv4_workspace(d, 8, 1) == 0
    refused(code, abi.sambay_kv4_write, cache(), d, 1, K, V, POS)
    refused(code, abi.sambay_kv4_read, cache(), d, 1, K, V, POS)
    refused(code, abi.sambay_cross_attn_decode_kv4, cache(), d, 8, 1, Q, OUT, LENS, None, 0.0, WS)


@pytest.mark.parametrize("fn", [abi.sambay_kv4_write, abi.sambay_kv4_read])
def test_rows_refusals(fn):
    d = dims()
    refused(1, fn, cache(), d, 0, K, V, POS)
    refused(1, fn, cache(), d, -3, K, V, POS)
    refused(1, fn, cache(pages=None), d, 1, K, V, POS)
    refused(1, fn, cache(table=None), d, 1, K, V, POS)
    refused(1, fn, cache(), d, 1, None, V, POS)
    refused(1, fn, cache(), d, 1, K, None, POS)
    refused(1, fn, cache(), d, 1, K, V, None)
    refused(1, fn, cache(), d, 1, PAGES, V, POS)
    refused(2, fn, cache(pages=_Ptr(0x10008)), d, 1, K, V, POS)
    refused(2, fn, cache(table=_Ptr(0x10002)), d, 1, K, V, POS)
    refused(2, fn, cache(k_exp=_Ptr(0x10001)), d, 1, K, V, POS)
    refused(2, fn, cache(v_exp=_Ptr(0x10001)), d, 1, K, V, POS)
    refused(2, fn, cache(), d, 1, _Ptr(0x10004), V, POS)
    refused(2, fn, cache(), d, 1, K, V, _Ptr(0x10002))
    refused(2, fn, cache(), d, 1, K, V, POS, _Ptr(0x10002))
    refused(2, fn, cache(), dims(batch=65535, kv_heads=64), 1 << 30, K, V, POS)


def test_write_strides():
    d = dims()
    refused(1, abi.sambay_kv4_write, cache(), d, 2, K, V, POS, None, 255, 0)
    refused(1, abi.sambay_kv4_write, cache(), d, 2, K, V, POS, None, 0, -256)
    refused(2, abi.sambay_kv4_write, cache(), d, 2, K, V, POS, None, 260, 0)
    refused(2, abi.sambay_kv4_write, cache(), dims(io=abi.F32), 2, K, V, POS, None, 0, 258)
    refused(1, abi.sambay_kv4_read, cache(), d, 2, K, K, POS)


def test_attention_refusals():
    d = dims(table_pages=64)
    fn = abi.sambay_cross_attn_decode_kv4
    need = abi.sambay_cross_attn_decode_kv4_workspace(d, 8, 1)
    assert need > 0 and need % 256 == 0
    ok = _Ptr(0xA0000, need)
    for heads, tokens, code in ((0, 1, 1), (8, 0, 1), (6, 1, 2), (68, 1, 2), (8, 17, 2), (8, -1, 1)):
        refused(code, fn, cache(), d, heads, tokens, Q, OUT, LENS, None, 0.0, ok)
        assert abi.sambay_cross_attn_decode_kv4_workspace(d, heads, tokens) == 0
    refused(1, fn, cache(), d, 8, 1, None, OUT, LENS, None, 0.0, ok)
    refused(1, fn, cache(), d, 8, 1, Q, None, LENS, None, 0.0, ok)
    refused(1, fn, cache(), d, 8, 1, Q, OUT, None, None, 0.0, ok)
    refused(1, fn, cache(), d, 8, 1, Q, Q, LENS, None, 0.0, ok)
    refused(1, fn, cache(), d, 8, 1, Q, PAGES, LENS, None, 0.0, ok)
    refused(2, fn, cache(), d, 8, 1, _Ptr(0x10008), OUT, LENS, None, 0.0, ok)
    refused(2, fn, cache(), d, 8, 1, Q, OUT, _Ptr(0x10001), None, 0.0, ok)
    refused(2, fn, cache(), d, 8, 1, Q, OUT, LENS, _Ptr(0x10001), 0.0, ok)
    for scale in (float("nan"), -1.0, 2e4):
        refused(1, fn, cache(), d, 8, 1, Q, OUT, LENS, None, scale, ok)
    refused(3, fn, cache(), d, 8, 1, Q, OUT, LENS, None, 0.0, None)
    refused(3, fn, cache(), d, 8, 1, Q, OUT, LENS, None, 0.0, _Ptr(0xA0000, need - 1))
    refused(3, fn, cache(), d, 8, 1, Q, OUT, LENS, None, 0.0, _Ptr(0xA0010, need))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_exponents_of_rows_with_infinities_and_nan(dtype):
    x = torch.zeros(3, 5, 4, 64, dtype=dtype)
    x[1, 2, 0, 7], x[0, 0, 1, 0], x[2, 4, 2, 63] = 2688.0, -2689.0 - 11, 2.0 ** -9     # bf16: 2704
    want = torch.tensor([0, 1, -20, -64], dtype=torch.int32)
    assert torch.equal(KV4Cache.exponents(x), want)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[0, 1, :, 5] = bad                     # one in every head
        assert torch.equal(KV4Cache.exponents(y), want)
    # nothing but these, and past what an exponent of 64 holds
    assert torch.equal(KV4Cache.exponents(torch.full((2, 1, 16), float("nan"), dtype=dtype)), torch.tensor([-64], dtype=torch.int32))
    assert KV4Cache.exponents(torch.full((2, 1, 16), 3e38, dtype=dtype)).item() == 64


@pytest.mark.parametrize("name", ["table", "k_exp", "v_exp", "pages"])
def test_the_layers_tensors_cannot_be_exchanged(name):
    """Calls use the addresses that the cache was made with: a new tensor in its place would not be seen."""
    c = KV4Cache.__new__(KV4Cache)
    old = torch.zeros(4, dtype=torch.int32)
    c._own = {name: old}
    with pytest.raises(ValueError):
        setattr(c, name, old.clone())
    with pytest.raises(ValueError):
        setattr(c, name, None)
    assert getattr(c, name) is old
    setattr(c, name, old.add_(1))               # what an operation in place does
    assert getattr(c, name) is old and old[0] == 1


def test_outputs_that_share_memory_with_other_rows():
    """Not only the same address: any byte in common.  (Where they have none, a short workspace keeps the call from a launch.)"""
    d = dims(table_pages=64)
    n = 2 * 3 * 4 * 64 * 2                       # bytes of K and of V, 3 tokens
    for io, size in ((abi.BF16, n), (abi.F32, 2 * n)):
        d.io = io
        for off in (0, 16, size - 16, -16, 16 - size):
            refused(1, abi.sambay_kv4_read, cache(), d, 3, K, _Ptr(K.address + off), POS)
    d.io = abi.BF16
    need = abi.sambay_cross_attn_decode_kv4_workspace(d, 8, 3)
    short, n = _Ptr(0xA0000, need - 1), 2 * n    # 8 query heads
    for off in (0, 16, n - 16, -16, 16 - n):
        refused(1, abi.sambay_cross_attn_decode_kv4, cache(), d, 8, 3, Q, _Ptr(Q.address + off), LENS, None, 0.0, short)
    for off in (n, -n):                          # one behind the other: the next check's turn
        refused(3, abi.sambay_cross_attn_decode_kv4, cache(), d, 8, 3, Q, _Ptr(Q.address + off), LENS, None, 0.0, short)
