"""Sizes at which the write into pages and the assignment of pages take their rarer ways: pages of more tokens than a block
holds, calls sized for nearly 2^31 tokens, more sequences than blocks that place tokens."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
import test_page_choice_gpu as choice
import test_page_store_gpu as store_tests
from page_reference import LARGEST, power
from test_paged_gpu import _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store,bounds", [("int8", True), ("e4m3", True), ("int8", False), ("16", True)])
@pytest.mark.parametrize("d,page,T", [(128, 1024, 1300), (64, 1024, 1030), (64, 4096, 4500)])
def test_large_pages(store, bounds, d, page, T):
    store_tests.test_append_is_exact(store, bounds, "bf16", d, page, T)


@pytest.mark.parametrize("store,bounds", [("int8", True), ("e4m3", False), ("16", True)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,page,T,lens,new", [(128, 128, 1024, 1500, [1500, 30, 1900], [1500, 7, 1100]),
                                                   (64, 32, 1024, 1200, [1200, 2, 1500], [1200, 9, 900]),
                                                   (64, 64, 4096, 2000, [2000, 500, 4500], [2000, 500, 1999])])
def test_large_pages_of_turned_keys(store, bounds, interleaved, d, rot, page, T, lens, new):
    store_tests.test_append_turns_keys_and_queries(store, bounds, interleaved, d, rot, page, T, lens, new)


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 4000])
def test_a_call_sized_for_many_tokens_writes_the_few_there_are(T):
    """Keys seen T times, of which q_lens says that three are real."""
    kc, vc = (torch.zeros((2, 1, 4096, 64), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((2, 1), device="cuda") for _ in range(2))
    k = torch.randn((1, 1, 1, 64), device="cuda").to(torch.bfloat16)
    many = k.expand(1, 1, T, 64)
    fa.append_paged(many, many, kc, vc, _i32([[1, 0]]), _i32([4097]), q_lens=_i32([3]), k_scales=ks, v_scales=vs)
    assert fa.check_device_status() == 0
    two = power(float(k.abs().max()), LARGEST["int8"])
    codes = torch.round(k[0, 0, 0].float() / two)
    assert ks[:, 0].tolist() == [two, two] and vs[:, 0].tolist() == [two, two]
    for c in (kc, vc):
        assert torch.equal(c[1, 0, 4094:].float(), codes.expand(2, 64)) and torch.equal(c[0, 0, 0].float(), codes)
        assert not bool(c[1, 0, :4094].any()) and not bool(c[0, 0, 1:].any())


@pytest.mark.parametrize("B,T", [(4097, 1), (5000, 40), (20000, 9), (65535, 3)])
def test_more_sequences_than_blocks_place(B, T):
    choice.test_pages_are_assigned([(7 * i) % 90 for i in range(B)], [(11 * i) % 90 for i in range(B)], 16, T)
    choice.test_pages_are_assigned([(5 * i) % 40 for i in range(B)], [(5 * i) % 40 + i % (T + 2) for i in range(B)], 16, T)
