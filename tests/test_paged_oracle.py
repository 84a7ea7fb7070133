"""Pins of the paged cache's float64 oracle (CPU)."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as PO


def test_codes_match_torch_for_every_bf16_up_to_448():
    x = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[(x <= 448) & ~torch.isnan(x)]
    x = torch.cat([x, -x])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(PO.e4m3_code(x.double().numpy()), want)
    back = torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(PO.e4m3_value(want), back)


def test_saturates():
    assert PO.e4m3_value(PO.e4m3_code(np.array([500.0, -1e9]))).tolist() == [448.0, -448.0]


@pytest.mark.parametrize("amax,k", [(0.0, -124), (448.0, 0), (448.0001, 1), (447.9, 0), (224.0, -1), (224.1, 0),
                                    (1.75, -8), (1.7501, -7), (2.0 ** -140, -124), (3.38e38, 119)])
def test_row_exponent(amax, k):
    assert PO.row_exponent(amax) == k


def test_held_values_are_bf16_and_within_half_a_step():
    """code * 2^k is exactly a bf16; a row's values are off by at most half an
    e4m3 step (2^-4 of the value, or half the smallest subnormal).  Past
    448 * 2^119, the largest value held (the next power of two would round
    values near bf16's largest up to infinity), a value is off by what it
    passes it by."""
    rng = np.random.default_rng(5)
    for s in (1e-38, 1e-20, 1.0, 1e20, 1e38):
        x = torch.from_numpy(rng.standard_normal(128) * s).to(torch.bfloat16)
        c, e = PO.quantise_row(x.double().numpy())
        got = PO.dequantise_row(c, e)
        assert np.array_equal(torch.from_numpy(got).to(torch.bfloat16).double().numpy(), got)
        err = np.abs(got - x.double().numpy())
        past = np.maximum(np.abs(x.double().numpy()) - 448 * 2.0 ** 119, 0)
        assert (err <= np.maximum(np.maximum(np.abs(x.double().numpy()) * 2.0 ** -4, 2.0 ** (e - 127 - 10)), past)).all()


def test_attention_against_softmax_of_the_mask():
    rng = np.random.default_rng(6)
    N, R, G = 40, 7, 3
    q, k, v = rng.standard_normal((R, G, 16)), rng.standard_normal((N, 16)), rng.standard_normal((N, 16))
    pos = np.arange(N - R, N)
    for window, sinks in ((0, 0), (1, 0), (5, 2), (5, 50), (100, 3)):
        out, lse = PO.attend_rows(q, k, v, pos, np.ones(N, bool), window, sinks, 0.3)
        for r in range(R):
            for g in range(G):
                z = np.full(N, -np.inf)
                for t in range(N):
                    if t <= pos[r] and (not window or t > pos[r] - window or t < sinks):
                        z[t] = 0.3 * float(q[r, g] @ k[t])
                p = torch.softmax(torch.from_numpy(z), 0).numpy()
                assert np.allclose(out[r, g], p @ v, rtol=0, atol=1e-12)
                assert np.isclose(lse[r, g], torch.logsumexp(torch.from_numpy(z), 0).item(), rtol=1e-12)
                o1, l1 = PO.attend(q[r, g], k, v, np.isfinite(z), 0.3)
                assert np.allclose(o1, out[r, g]) and np.isclose(l1, lse[r, g])


def test_a_row_that_sees_nothing():
    out, lse = PO.attend_rows(np.ones((1, 1, 4)), np.ones((3, 4)), np.ones((3, 4)), [-1], np.ones(3, bool), 0, 0, 1.0)
    assert (out == 0).all() and lse[0, 0] == -np.inf
