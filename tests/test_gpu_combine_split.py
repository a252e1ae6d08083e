"""The combine shares a token's row among several warps where there are few tokens. The sums are per
element and in slot order either way, so a token's row has the same bits in a call of any size."""
import pytest
import torch

from ragged_grouped_gemm_device_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [8, 264, 512, 2048])
@pytest.mark.parametrize("k", [1, 3, 9])
def test_a_row_does_not_depend_on_the_number_of_tokens(lib, k, d):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 64 * sms + 300  # one warp a token
    g = torch.Generator("cuda").manual_seed(k + d)
    y = torch.randn(T * k, d, generator=g, device="cuda").to(torch.bfloat16)
    inv = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    inv[torch.rand(T, k, generator=g, device="cuda") < 0.1] = -1
    w = torch.rand(T, k, generator=g, device="cuda")

    def combine(first, n):
        out = torch.full((n, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        rows = inv[first:first + n]
        mine = y[rows.clamp(min=0).view(-1).long()]  # the rows of these tokens, in slot order
        at = torch.arange(n * k, dtype=torch.int32, device="cuda").view(n, k).where(rows >= 0, torch.full_like(rows, -1))
        _lib.moe_unpermute_combine(mine, at, w[first:first + n], n, k, d, out)
        return out

    whole = combine(0, T)
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for j in range(k):
        on = inv[:, j] >= 0
        ref[on] += w[on, j, None].double() * y[inv[on, j].long()].double()
    # fp32 sums of k terms, then one bf16 rounding of at most 2^-8 of the value
    assert ((whole.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 2.0 ** -20 * k * 5).all()
    for first, n in ((0, 1), (5, 37), (17, 32 * sms), (0, 64 * sms - 1), (3, 64 * sms + 1)):
        assert torch.equal(combine(first, n), whole[first:first + n]), n
