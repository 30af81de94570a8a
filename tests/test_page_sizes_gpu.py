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


@pytest.mark.parametrize("kind,d,H,T", [("int8", 64, 4, 1), ("int8", 64, 24, 1), ("e4m3", 128, 4, 2), ("bf16", 64, 4, 1), ("bf16", 128, 4, 1)])
def test_lengths_up_to_the_last_ones_of_31_bits(kind, d, H, T):
    """2^31 - 16 keys and a few less, one page of 4096 named again and again: each of its keys counts as often as it is
    seen.  A lane adds the sums of at most 2^31 / (32 * 608) = 110000 tiles in turn (152 SMs, 4 warps each at least):
    2^-24 of the sum each time, 0.7 % in all."""
    g = torch.Generator(device="cuda").manual_seed(d + H)
    raw = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16}[kind]
    kc, vc = ((torch.randint(-60, 61, (1, 1, 4096, d), generator=g, device="cuda") / (64 if kind == "bf16" else 1)).to(raw) for _ in range(2))
    scales = {} if kind == "bf16" else dict(zip(("k_scales", "v_scales"), torch.full((2, 1, 1), 1 / 64, device="cuda")))
    table = torch.zeros((1, 2 ** 31 // 4096), dtype=torch.int32, device="cuda")
    q = torch.randn((1, H, T, d), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (c[0, 0].double() / (1 if kind == "bf16" else 64) for c in (kc, vc))
    for length in (2 ** 31 - 16, 2 ** 31 - 17, 2 ** 31 - 64, 2 ** 31 - 2100):
        o, lse = fa.forward_paged(q, kc, vc, table, _i32([length]), **scales)
        assert fa.check_device_status() == 0
        for t in range(T):
            seen = length - T + t + 1
            times = torch.where(torch.arange(4096, device="cuda") < seen % 4096, seen // 4096 + 1, seen // 4096).double()
            x = q[0, :, t].double() @ k.T / d ** 0.5 + torch.log(times)
            want = torch.logsumexp(x, -1)
            p = torch.exp(x - want[:, None])
            assert bool(((lse[0, :, t].double() - want).abs() <= 8e-3).all())
            assert bool(((o[0, :, t].double() - p @ v).abs() <= 2.0 ** -8 * (p @ v).abs() + 0.02 * (p @ v.abs())).all())


def test_choices_of_two_host_threads():
    """Small and large tables chosen from at once, on streams of their own: each thread's kernels find the shared memory that
    they ask for."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(5)
    work = []
    for length in (16 * 600, 16 * 40000, 16 * 30, 16 * 9000):
        table, n = choice._table([length], 16, g)
        bounds, unit = choice._bounds(n, 1, 64, g)
        q = torch.randn((1, 20, 1, 64), generator=g, device="cuda").to(torch.float16)      # 20 rows: kernels that few calls use
        work.append((q, bounds, unit, table, _i32([length]), choice._want(q, bounds, unit, table, [length], 12, 16, 1, 1)))
    torch.cuda.synchronize()
    wrong = []

    def run(order):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for i in order * 30:
                q, bounds, unit, table, lens, want = work[i]
                try:
                    if not torch.equal(fa.select_pages(q, bounds, unit, table, lens, 12, 16), want):
                        wrong.append(i)
                except fa.FaError as e:
                    wrong.append(str(e))

    threads = [threading.Thread(target=run, args=(order,)) for order in ([0, 2, 1, 3], [1, 3, 0, 2], [3, 0, 2, 1])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [] and fa.check_device_status() == 0
