"""Key lengths of the scored calls: what is copied is said to be (CPU only)."""
import torch

import exact_io_aware_23_gb300 as fa


def test_a_copy_of_the_lengths_is_handed_on():
    q = torch.zeros(3, 2, 8, 64)
    lens = torch.tensor([1, 2, 3], dtype=torch.int32)
    assert fa._kv_lens(None, 3, -1, q) == (None, None)
    got, new = fa._kv_lens(lens, 3, lens.get_device(), q)
    assert got is lens and new is None
    wide = torch.arange(6, dtype=torch.int32)[::2]
    got, new = fa._kv_lens(wide, 3, wide.get_device(), q)
    assert new is got and got.is_contiguous() and got.tolist() == [0, 2, 4]
