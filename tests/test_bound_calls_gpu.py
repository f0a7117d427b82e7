"""The calls of csrc/bind.cpp as a program with several threads makes them."""

import threading
import time

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["norm_rope", "norm_rope_bwd", "norm_rope_append_paged", "prefix_fwd_paged"])
def test_other_threads_run_while_a_launch_waits(cuda_ok, name):
    # the stream is busy for about a second and takes some thousand launches; the next one waits, without the interpreter's lock
    import torch

    import split_kv_decode_bsr_gb300 as sta

    dev = torch.device("cuda", 0)
    i32 = dict(device=dev, dtype=torch.int32)
    q, k = (torch.randn(2, h, 64, device=dev).bfloat16() for h in (4, 2))
    pages = torch.zeros(2, 16, 2, 64, device=dev, dtype=torch.bfloat16)
    v_pages = torch.zeros_like(pages)
    lists = (torch.arange(3, **i32), torch.arange(2, **i32))
    qi, ki = torch.arange(3, **i32), torch.tensor([0, 1, 2], **i32)
    pos, rope = torch.zeros(2, **i32), sta.Rope(64)
    out, dk = torch.empty_like(q), torch.empty_like(k)
    lse, ws = torch.empty(2, 4, device=dev), torch.empty(1 << 20, device=dev, dtype=torch.uint8)
    calls = dict(
        norm_rope=lambda: sta.sta_norm_rope(q, None, pos, rope, q_out=out),
        norm_rope_bwd=lambda: sta.sta_norm_rope_bwd(q, k, q, k, pos, rope, dq=out, dk=dk, workspace=ws),
        norm_rope_append_paged=lambda: sta.sta_norm_rope_append_paged(q, k, k, pages, v_pages, *lists, qi, ki, rope, q_out=out),
        prefix_fwd_paged=lambda: sta.sta_prefix_fwd_paged(q, pages, pages, *lists, qi, [0, 1, 2], ki, [0, 1, 2], [0, 2], [0], o=out, lse=lse,
                                                          workspace=ws))
    call = calls[name]
    call()
    torch.cuda.synchronize()
    longest, done = 0.0, threading.Event()

    def watch():
        nonlocal longest
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            longest, last = max(longest, now - last), now

    other = threading.Thread(target=watch)
    other.start()
    torch.cuda._sleep(2_000_000_000)
    slowest = 0.0
    for _ in range(3000):
        t = time.perf_counter()
        call()
        slowest = max(slowest, time.perf_counter() - t)
    done.set()
    other.join()
    torch.cuda.synchronize()
    print(f"{name}: longest call {slowest:.3f} s, longest pause of the other thread {longest:.3f} s")
    assert longest < 0.25, f"{longest:.3f} s of another thread's time within a call of {slowest:.3f}"
    assert sta.sta_device_error(reset=True) == 0
