"""The attention bounds of the GPU tests, on the CPU: they pass outputs that are only rounded and reject outputs with
a mistake in them.  The mistakes are planted in what the reference computes."""
import pytest
import torch

import attention_bounds as A

BF16, F16 = torch.bfloat16, torch.float16


def case(dtype, n, d=64, hq=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((1, hq, d), generator=g).to(dtype).double()
    k, v = (torch.randn((n, 1, d), generator=g).to(dtype).double() for _ in range(2))
    return q, k, v, torch.ones((1, n), dtype=torch.bool)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 2, 33, 2000, 60001])
@pytest.mark.parametrize("gain", [0.01, 1.0, 12.0])
def test_rounded_outputs_pass(dtype, n, gain):
    for seed in range(3):
        q, k, v, seen = case(dtype, n, seed=seed)
        r = A.reference(q * gain, k, v, 0.125, seen)
        A.check(A.as_computed(q * gain, k, v, 0.125, seen, dtype), r["lse"], r, dtype)


def test_rows_that_see_nothing():
    q, k, v, _ = case(BF16, 5)
    q = q.expand(3, -1, -1)
    seen = torch.tensor([[0, 0, 0, 0, 0], [1, 0, 0, 0, 0], [1, 1, 1, 1, 1]], dtype=torch.bool)
    r = A.reference(q, k, v, 0.125, seen)
    got = A.as_computed(q, k, v, 0.125, seen, BF16)
    A.check(got, r["lse"], r, BF16)
    assert (r["out"][0] == 0).all() and (r["lse"][0] == -float("inf")).all()
    got[0] = 1e-6
    with pytest.raises(AssertionError):
        A.check(got, None, r, BF16)


@pytest.mark.parametrize("dtype,n", [(F16, 60001), (BF16, 20000), (F16, 3000), (BF16, 3000)])
def test_mistakes_are_rejected(dtype, n):
    q, k, v, seen = case(dtype, n, d=64, seed=5)
    r = A.reference(q, k, v, 0.125, seen)
    good = A.as_computed(q, k, v, 0.125, seen, dtype)
    A.check(good, None, r, dtype)

    def rejected(out):
        with pytest.raises(AssertionError):
            A.check(out.to(dtype), None, r, dtype)

    rejected(torch.zeros_like(good))
    rejected(good.double() * 0.5)
    rejected(good.double() * 0.97)
    at = n // 2 // 32 * 32
    for rows in (slice(at, at + 32), slice(n - 32, n)):
        wrong = v.clone()
        wrong[rows] = 0.0                                       # one tile's values dropped
        rejected(A.as_computed(q, k, wrong, 0.125, seen, dtype))
        wrong = v.clone()
        wrong[rows] = v[:32]                                    # one tile's values from another page
        rejected(A.as_computed(q, k, wrong, 0.125, seen, dtype))
        wrong = k.clone()
        wrong[rows] = k[:32]
        rejected(A.as_computed(q, wrong, v, 0.125, seen, dtype))


def test_small_values_have_small_bounds():
    # the bound scales with the values: a loss that is invisible beside values of one shows beside values of 1e-3
    q, k, v, seen = case(F16, 3000, seed=7)
    v = 1e-3 * (1 + 0.1 * v)
    r = A.reference(q, k, v, 0.125, seen)
    good = A.as_computed(q, k, v, 0.125, seen, F16)
    A.check(good, None, r, F16)
    with pytest.raises(AssertionError):
        A.check((good.double() * (1 - 3e-3)).to(F16), None, r, F16)
