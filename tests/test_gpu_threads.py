"""The calls on tensors leave the interpreter to other threads while the CUDA runtime works on them."""
import threading
import time

import pytest
import torch

import reduce_residual_rmsnorm_gb300 as pkg

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_launch_waits():
    """A launch that waits for room in its stream's queue (behind a kernel of about a second) stops only its own thread."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    dev = torch.device("cuda:0")
    ids = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    rows = pkg.ts_moe_sort(ids, 1)
    y = torch.ones(1, 8, dtype=torch.bfloat16, device=dev)
    out = pkg.ts_moe_combine(y, rows)
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def watch():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    other = threading.Thread(target=watch)
    other.start()
    try:
        torch.cuda._sleep(1_900_000_000)
        longest = 0.0
        for _ in range(20000):  # a queue holds about a thousand launches
            t = time.perf_counter()
            pkg.ts_moe_combine(y, rows, out=out)
            longest = max(longest, time.perf_counter() - t)
            if longest > 0.2:
                break
    finally:
        stop.set()
        other.join()
        torch.cuda.synchronize()
    print("longest call %.3f s, longest pause of the other thread %.3f s" % (longest, max(gaps)))
    assert longest > 0.2, "no launch had to wait"
    assert max(gaps) < longest / 2


def test_calls_from_several_threads():
    """Every thread's calls, on its own stream and with new outputs, give the results of calls one after the other; a
    refusal in one thread is raised there with its own detail."""
    import __graft_entry__

    __graft_entry__.build()
    dev = torch.device("cuda:0")
    torch.manual_seed(0)
    g = torch.ones(1, device=dev)
    sets = []
    for i in range(4):
        x = torch.randn(64 + i, 256, device=dev).bfloat16()
        ids = torch.randint(0, 7, (64 + i, 3), dtype=torch.int32, device=dev)
        rows = pkg.ts_moe_sort(ids, 7)
        w = torch.rand(64 + i, 3, device=dev)
        q, s = pkg.ts_nvfp4_quantize(x, g, sf_layout=0)
        y = pkg.ts_moe_dispatch(x, rows)
        sets.append((x, ids, w, [q, pkg.ts_nvfp4_gemm(q, s, q[:64].contiguous(), s, g), *rows, y, pkg.ts_moe_combine(y, rows, w)]))
    torch.cuda.synchronize()
    wrong = []

    def work(x, ids, w, want):
        try:
            torch.cuda.set_device(dev)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(200):
                    q, s = pkg.ts_nvfp4_quantize(x, g, sf_layout=0)
                    out = pkg.ts_nvfp4_gemm(q, s, q[:64].contiguous(), s, g)
                    rows = pkg.ts_moe_sort(ids, 7)
                    y = pkg.ts_moe_dispatch(x, rows)
                    with pytest.raises(pkg.TsError, match="K = 250" if x.shape[0] % 2 else "x is not"):
                        pkg.ts_nvfp4_quantize(x[:, :250] if x.shape[0] % 2 else x[:, 4:20], g)
                    got = [q, out, *rows, y, pkg.ts_moe_combine(y, rows, w)]
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
        except BaseException as e:  # noqa: BLE001 (raised in the test's thread below)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=z) for z in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
