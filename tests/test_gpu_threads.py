"""Calls from several host threads at once: what a launcher sets on a kernel for
one thread's sizes may not take another's launch away."""
import threading

import pytest
import torch

import int8_w8a8_scaled_gb300 as w8

pytestmark = pytest.mark.gpu


def at_once(*calls, times=2000):
    """Each call repeated by a thread of its own, all starting together."""
    errors, gate = [], threading.Barrier(len(calls))

    def work(call):
        try:
            gate.wait()
            for _ in range(times):
                call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


def tables(batch):
    ints = lambda *n, fill=0: torch.full(n, fill, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, new, free = ints(batch, fill=3), ints(batch, fill=1), torch.arange(batch + 5, dtype=torch.int32, device="cuda")
    out = (ints(batch, 4, fill=-1), 16, ints(batch + 1), ints(batch), torch.zeros(batch, dtype=torch.int64, device="cuda"), ints(batch), ints(1))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    return lambda: w8.build_block_tables(ctx, new, free, free[-1:], *out, stream=stream)


def test_block_tables_of_small_and_large_batches():
    at_once(tables(8), tables(1000), tables(12000))


def test_a_thread_whose_first_cuda_call_is_a_matmul():
    a, b = (torch.full((n, 512), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for n in (256, 128))
    one, out = torch.ones(1, device="cuda"), torch.empty(256, 128, dtype=torch.bfloat16, device="cuda")
    at_once(lambda: w8.scaled_mm(a, b, one, one, out), times=1)
    assert (out == 512).all()


def rows_of(cols):
    x = torch.randn(3, cols, device="cuda").bfloat16()
    q, s = torch.empty(3, cols, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    return lambda: w8.scaled_quant(x, q, s)


def test_quantisers_of_shorter_and_longer_rows():
    at_once(rows_of(30000), rows_of(65536))


def product(stages):
    a, b = (torch.zeros(n, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for n in (256, 128))
    one, out = torch.ones(1, device="cuda"), torch.empty(256, 128, dtype=torch.bfloat16, device="cuda")
    cfg = {"swap_ab": 0, "block_n": 64, "split_k": 1, "stages": stages}
    return lambda: w8.scaled_mm(a, b, one, one, out, config=cfg)


def test_matmuls_with_fewer_and_more_stages():
    at_once(product(3), product(0))
