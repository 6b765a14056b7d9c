"""The 4-bit cache's oracle against values worked out by hand, torch's e4m3
conversion, and the dense attention oracle."""

import numpy as np
import pytest
import torch

from oracle import sambay_ref as ref
from oracle.kv4_ref import E2M1, E4M3, kv4_attention_ref, kv4_kept, nearest_code


def test_scale_values_are_torch_e4m3():
    got = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3, got)


def test_scale_rounding_is_torch_e4m3():
    x = np.random.default_rng(0).uniform(0, 448, 20000).astype(np.float32)
    x = np.concatenate([x, np.exp2(np.random.default_rng(1).uniform(-14, 8, 20000)).astype(np.float32),
                        0.5 * (E4M3[1:] + E4M3[:-1]).astype(np.float32)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3[nearest_code(x, E4M3)], want)


@pytest.mark.parametrize("x,want", [(0.24, 0.0), (0.25, 0.0), (0.26, 0.5), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0),
                                    (2.5, 2.0), (2.51, 3.0), (3.5, 4.0), (5.0, 4.0), (5.01, 6.0), (7.0, 6.0)])
def test_codes_go_to_the_nearest_and_half_way_to_the_even(x, want):
    assert E2M1[nearest_code(x, E2M1)] == want


def test_a_block_by_hand():
    # max 12 -> scale 2; the values over 2: 6, -1.25 (half way: 1), .75 (half way: 1), 2.5 (half way: 2), ...
    row = np.zeros((1, 16))
    row[0, :6] = [12.0, -2.5, 1.5, 5.0, 0.5, -0.51]
    want = np.zeros((1, 16))
    want[0, :6] = [12.0, -2.0, 2.0, 4.0, 0.0, -1.0]
    assert np.array_equal(kv4_kept(row), want)
    # times 2^e, exactly
    assert np.array_equal(kv4_kept(row * 2.0 ** -9, [-9]), want * 2.0 ** -9)
    # past what the scale holds: 448 * 6; a NaN or an infinity takes its block, not the next one
    row = np.ones((1, 32))
    row[0, 0], row[0, 16] = 1e6, np.inf
    kept = kv4_kept(row)
    assert kept[0, 0] == 2688 and np.all(kept[0, 1:16] == 0) and np.all(np.isnan(kept[0, 16:]))


def test_attention_of_one_token_is_the_dense_oracle():
    r = np.random.default_rng(3)
    q, K, V = r.normal(size=(2, 4, 16)), r.normal(size=(2, 9, 2, 16)), r.normal(size=(2, 9, 2, 16))
    out, spread, logit = kv4_attention_ref(q[:, None], K, V, [9, 5])
    want = ref.cross_attention_decode_ref(q, K, V)
    assert np.allclose(out[0, 0], want[0], atol=1e-14)
    assert np.allclose(out[1, 0], ref.cross_attention_decode_ref(q[1:], K[1:, :5], V[1:, :5])[0], atol=1e-14)
    assert np.all(spread + 1e-14 >= np.abs(out)) and np.all(logit > 0)


def test_attention_of_several_tokens_sees_up_to_its_own():
    r = np.random.default_rng(4)
    q, K, V = r.normal(size=(1, 3, 2, 16)), r.normal(size=(1, 6, 2, 16)), r.normal(size=(1, 6, 2, 16))
    out, _, _ = kv4_attention_ref(q, K, V, [6])
    for t, n in enumerate((4, 5, 6)):
        assert np.allclose(out[0, t], ref.cross_attention_decode_ref(q[:, t], K[:, :n], V[:, :n])[0], atol=1e-14)
    out, _, _ = kv4_attention_ref(q, K, V, [2], count=[3])       # the first query sees nothing
    assert np.all(out[0, 0] == 0) and np.allclose(out[0, 1], np.repeat(V[0, :1], 1, 0)[0], atol=1e-14)
    out, _, _ = kv4_attention_ref(q, K, V, [6], count=[2])       # the third row is not one
    assert np.all(np.isnan(out[0, 2])) and np.isfinite(out[0, :2]).all()
