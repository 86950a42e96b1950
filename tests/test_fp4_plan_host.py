"""The sizes of the GPU tests reach every variant of the 4-bit kernels, whatever a new measurement makes of the plan."""
import itertools

import pytest

import fp4_plans as plans

FORMATS = (0, 1)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_pair_kernel_is_tested(fmt):
    seen = set()
    for M, N, K, first, behind in plans.PAIRS:
        assert M > plans.library().small_tokens()
        aligned = first == 0 and (N + behind) % 8 == 0
        seen.add((*plans.pair_plan(M, N, K, fmt, aligned), aligned))
    one = set(itertools.product((384, 256, 192, 128, 64), (1,), (False, True), (False, True)))
    shared = set(itertools.product((128, 64), (2, 4), (False,), (False, True)))
    assert seen == one | shared


def test_every_split_of_few_tokens_is_tested():
    seen = {(16 if M <= 16 else 32 if M <= 32 else 64, plans.library().split(M, N, K)) for M, N, K in plans.FEW}
    assert seen == set(itertools.product((16, 32, 64), (1, 2, 4, 8)))
    assert all(M <= plans.library().small_tokens() for M, _, _ in plans.FEW)


def test_patches_of_64_rows_are_tested():
    assert all(plans.library().patch_rows(rows, K) == 64 for rows, K, _ in plans.PATCHES)
    assert plans.library().patch_rows(300, 640) == 32


def test_the_split_follows_from_the_sizes():
    """What groups the sums is the same for every alignment of y."""
    for fmt, M, N, K in itertools.product(FORMATS, (65, 200, 513, 2048), (64, 300, 2560, 13824), (128, 2560, 6912, 20000)):
        splits = {plans.pair_plan(M, N, K, fmt, aligned)[1] for aligned in (False, True)}
        assert len(splits) == 1, (fmt, M, N, K)
