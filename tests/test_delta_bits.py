"""The bound of the gated delta rule's bf16 outputs, on the CPU: a model with two parts of every factor keeps it, and one that
loses the second part of any of them does not."""
import numpy as np
import pytest

from tests import delta_bits as bits


def _block(seed, C, dk, dv, strong):
    r = np.random.RandomState(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    q, k = (bits.parts(unit(r.randn(C, dk)), 1)[0] for _ in range(2))
    return q, k, bits.parts(r.randn(C, dv), 1)[0], -r.rand(C) * (3.0 if strong else 0.05), r.rand(C), r.randn(dk, dv)


def _over(args, **n):
    """By how much the worst output passes its share of the terms and one rounding to bf16."""
    got, want, terms = bits.outputs(*args, **n)
    out = bits.parts(got, 1)[0]
    return (np.abs(out - want) / (bits.SHARE * terms + 2.0 ** -8 * np.abs(want))).max()


@pytest.mark.parametrize("C,dk,dv", [(1, 64, 64), (7, 128, 64), (64, 128, 128), (64, 64, 64)])
@pytest.mark.parametrize("strong", [False, True])
def test_two_parts_keep_the_bound(C, dk, dv, strong):
    assert _over(_block(1, C, dk, dv, strong)) <= 1


@pytest.mark.parametrize("lost", ["n_state", "n_weights", "n_u"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_a_lost_second_part_passes_it(lost, dk, dv):
    assert _over(_block(2, 64, dk, dv, False), **{lost: 1}) > 4
