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


# v has a bit in each of its pieces: 1, 2^-9 and 2^-18. All terms of dx are v (weights of one), so dx = n v for n terms.
# The tensor cores add 16 terms of a piece at a time and truncate the sum to fp32. Added first, the small pieces' sums
# are exact: n 2^-18 needs log2 n bits, n 2^-9 beside it 9 more. Then the sum grows by 16 a step: what it holds below its
# last place is cut once for each power of two that it passes, all these cuts together below 2 units of the last place of
# the whole (2^-23 of it each). A contraction in parts (16 at most) is the same in each part, and adding these rounds to
# half a unit each. Adding the smallest piece last instead loses it: 16 2^-18 is no unit of a sum past 2^9 or so, and
# n 2^-18 is 2^-18 of the result.
V = 1 + 2.0 ** -9 + 2.0 ** -18
WITHIN = (4 + 15) * 2.0 ** -24


@pytest.mark.parametrize("T,M,N", [(2048, 4096, 11008), (16, 64, 11008), (600, 300, 4095), (1, 32, 8192)])
def test_small_pieces_are_not_lost_in_a_long_sum(dbf, T, M, N):
    L = ones_layer(dbf, M, N)
    dy = torch.full((T, N), V, device="cuda")
    assert dy[0, 0].item() == V
    dx = dbf.mx4_backward(L, dy, dx_dtype=torch.float32).double()
    assert ((dx - N * V).abs() <= WITHIN * N * V).all().item()


@pytest.mark.parametrize("T,M,N", [(2048, 4096, 11008), (600, 300, 4095)])
def test_small_pieces_of_both_gated_gradients(dbf, T, M, N):
    """g = u = 64: dg = du = 64 dh (above), twice as many terms."""
    L = ones_layer(dbf, M, N)
    saved = tuple(dbf.act8_save(torch.full((T, N), 64.0, device="cuda")) for _ in range(2))
    dx = dbf.mx4_gated_backward(L, L, torch.full((T, N), V / 64, device="cuda"), saved, dx_dtype=torch.float32)[0].double()
    assert ((dx - 2 * N * V).abs() <= WITHIN * 2 * N * V).all().item()
