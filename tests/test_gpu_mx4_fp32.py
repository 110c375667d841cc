"""fp32 gradients of the 4-bit layer keep what fp32 holds, whatever dx's type:
data whose sums are known."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


def ones_layer(dbf, M, N):
    return dbf.Mx4Layer.quantize(torch.ones(N, M, device="cuda"))


@pytest.mark.parametrize("T,M,N", [(1, 32, 8), (3, 100, 64), (70, 300, 1000), (300, 96, 513)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_what_cancels_leaves_the_last_bits(dbf, T, M, N, out):
    """Rows of v, -v (1 - 2^-20) and zeros against weights of one: dx is v 2^-20, v = 1.5 (24 bits of the second value
    are needed: 1.5 - 1.5 * 2^-20). All sums are exact, in any order: multiples of 1.5 * 2^-20 below 2^24 of them. bf16
    holds the result too."""
    L = ones_layer(dbf, M, N)
    dy = torch.zeros(T, N, device="cuda")
    dy[:, 0], dy[:, N - 1] = 1.5, -1.5 * (1 - 2.0 ** -20)
    assert dy[0, N - 1].item() == -1.5 + 1.5 * 2.0 ** -20
    dx = dbf.mx4_backward(L, dy, dx_dtype=out)
    assert (dx.double() == 1.5 * 2.0 ** -20).all().item()


@pytest.mark.parametrize("T,M,N", [(2, 64, 40), (130, 200, 264), (33, 95, 255)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_what_cancels_in_the_gated_gradient(dbf, T, M, N, out):
    """At g = 64 the sigmoid is 1 in fp32 (e^-64 < 2^-25), so with u = 64 SiLU hands on dg = du = 64 dh, and dx is 128
    times the sum of dh's row: 2^-13 here. All sums are exact, in any order: multiples of 2^-14 up to 128."""
    L = ones_layer(dbf, M, N)
    saved = tuple(dbf.act8_save(torch.full((T, N), v, device="cuda")) for v in (64.0, 64.0))
    dh = torch.zeros(T, N, device="cuda")
    dh[:, 0], dh[:, N - 1] = 1.0, -1.0 + 2.0 ** -20
    dx, dg, du = dbf.mx4_gated_backward(L, L, dh, saved, dx_dtype=out)
    assert torch.equal(dg, 64 * dh) and torch.equal(du, 64 * dh)
    assert (dx.double() == 2.0 ** -13).all().item()
