"""Paged attention at sizes where its reckoning takes more than one step: more than 256 sequences, and
one cache whose parts are joined in several rounds."""
import pytest

from test_paged_gpu import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("B,T", [(300, 1), (600, 2)])
def test_more_sequences_than_are_kept(B, T, d, dtype):
    """Mixed lengths, some empty, a long one behind number 256, empty ones at the end."""
    lens = [(11 * i) % 47 for i in range(B)]
    lens[7] = 900
    lens[B - 20] = 6000
    lens[-3:] = [0, 0, 0]
    _run(lens, 2, 1, T, 16, d, dtype, cap=20.0, seed=B)
    q_lens = [i % 3 for i in range(B)] if T > 1 else None
    _run(lens, 2, 1, T, 16, d, dtype, alibi=True, q_lens=q_lens, seed=B + 1)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("lens,H,T", [([40000], 1, 1), ([41111], 4, 3), ([20, 70001, 0, 5], 3, 7)])
def test_more_parts_than_one_round_joins(lens, H, T, d, dtype):
    """One key head: its cache alone is shared by up to all CTAs, 64 parts a round."""
    _run(lens, H, 1, T, 64, d, dtype, cap=30.0, alibi=True, seed=d)
    _run(lens, H, 1, T, 64, d, dtype, seed=d + 1)
