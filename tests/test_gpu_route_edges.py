"""Routing at the ends of its range, against the definition in 64 bits (the reference and the tolerances are those of the
other tests of the route): biases of the type's lowest value, sums of two of them as the scores of groups,
sums that cancel."""
import pytest
import torch

from gpu_helpers import nv
from test_gpu_route import INF, _bias, _logits, check

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


def _masked_bias(E, left, seed, value=LOWEST):
    """A balance bias that switches all experts but `left` of them off."""
    bias = _bias(E, seed)
    off = torch.randperm(E, generator=torch.Generator().manual_seed(seed))[left:]
    bias[off] = value
    return bias


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(7, 4), (16, 4), (24, 5), (30, 8), (31, 31), (32, 8), (33, 8), (64, 6), (256, 8)])
def test_experts_switched_off_by_the_lowest_bias(E, k, sigmoid):
    """c = s + the lowest number is that number, in 64 bits too: eligible, all alike, chosen by index where fewer than k experts are
    left.  The last token's logits end where the buffer does."""
    x = _logits(70, E, E)
    gone = x.clone()
    gone[::2, ::3] = -INF                  # never chosen
    gone[5] = -INF
    for left in (0, 1, k - 1, k):
        bias = _masked_bias(E, left, left)
        for logits in (x, gone, x.bfloat16()):
            check(logits, k, sigmoid=sigmoid, bias=bias)
        check(x[:1], k, sigmoid=sigmoid, bias=bias, renormalize=False)
    near = _masked_bias(E, 1, 3)
    near[near == LOWEST] = torch.tensor(LOWEST).nextafter(torch.tensor(0.0))   # and next to it
    near[0] = LOWEST
    check(gone, k, sigmoid=sigmoid, bias=near)
    never = _masked_bias(E, 2, 4)
    never[1::4] = -INF                     # beside biases that may not be chosen
    check(gone, k, sigmoid=sigmoid, bias=never)


# with lanes or whole groups of lanes that have no expert
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top_groups", [(30, 8, 5, 2), (64, 8, 8, 3), (24, 6, 3, 2), (20, 6, 10, 4), (63, 12, 9, 5), (96, 9, 32, 6)])
def test_groups_with_experts_switched_off_by_the_lowest_bias(E, k, groups, top_groups, sigmoid):
    x = _logits(70, E, E)
    x[::3, ::4] = -INF
    for left in (0, 2, k, E // 2):
        check(x, k, sigmoid=sigmoid, bias=_masked_bias(E, left, left), groups=groups, top_groups=top_groups)


def _masked_groups(E, groups, left, seed, value=LOWEST):
    """A balance bias that switches all groups but `left` off."""
    bias = _bias(E, seed).view(groups, -1)
    bias[torch.randperm(groups, generator=torch.Generator().manual_seed(seed))[left:]] = value
    return bias.flatten()


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [LOWEST, -LOWEST], ids=["lowest", "largest"])
@pytest.mark.parametrize("E,k,groups,top_groups", [(64, 12, 8, 3), (30, 8, 5, 2), (24, 24, 4, 4), (256, 8, 8, 4), (63, 12, 9, 5), (64, 9, 32, 6)])
def test_groups_whose_two_largest_add_to_more_than_fp32_holds(E, k, groups, top_groups, value, sigmoid):
    """Twice the lowest number is above -inf in 64 bits: such a group stays, behind the others and the lowest index first."""
    x = _logits(70, E, E)
    gone = x.clone()
    gone[::2, ::3] = -INF
    gone[5] = -INF
    for left in range(top_groups + 1):
        bias = _masked_groups(E, groups, left, left, value)
        for logits in (x, gone):
            check(logits, k, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=top_groups, group_top=2)
        bias.view(groups, -1)[:, 0] = 0.125        # one expert of each is left: sums of the number itself
        check(gone, k, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=top_groups, group_top=2)
        bias[E // 2:] = -INF                       # and groups that cannot stay
        check(gone, k, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [(32, 8, 4), (96, 6, 2), (64, 32, 9)])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e30])
def test_groups_whose_two_largest_cancel(size, E, groups, top_groups, sigmoid):
    """A large bias on one expert of each group and its opposite on the others: the sum has the size of the scores, its error in
    fp32 that of the biases."""
    x = _logits(2000, E, groups)
    bias = torch.full((groups, E // groups), -size)
    bias[:, 1] = size
    for k in (1, top_groups):
        check(x, k, sigmoid=sigmoid, bias=bias.flatten(), groups=groups, top_groups=top_groups, group_top=2)
    bias[1::2] = _bias(E // 2, 1).view(-1, E // groups)          # beside groups of ordinary biases
    check(x, top_groups, sigmoid=sigmoid, bias=bias.flatten(), groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_more_choices_than_a_block_keeps(sigmoid):
    """A long packed batch: 1352 tokens x 8 of each of 148 blocks, whose ranks go through `rows` (a block's shared memory keeps 8192)."""
    T, E, k = 200000, 16, 8
    valid = torch.arange(T) % 7 != 3
    valid[150000:160000] = False
    check(_logits(T, E, 1), k, sigmoid=sigmoid, valid=valid, bias=_bias(E, 1))


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top_groups", [(256, 20, 1, 1), (256, 24, 1, 1), (256, 32, 1, 1), (64, 32, 1, 1), (512, 8, 8, 1), (1024, 32, 4, 2)])
def test_more_candidates_than_lanes(E, k, groups, top_groups, sigmoid):
    """Many choices of few values a lane: most tokens have more than 32 values above the bound."""
    for n, (dtype, bias) in enumerate([(torch.float32, True), (torch.bfloat16, False)]):
        check(_logits(300, E, E + n, dtype), k, sigmoid=sigmoid, bias=_bias(E, n) if bias else None, groups=groups, top_groups=top_groups, group_top=2)
