"""Two host threads call the operators that take a workspace, on one stream: the results are those of
serial calls, bit for bit (the workspaces come from an allocator that both threads share)."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_two_threads_on_one_stream():
    import fp4_block_scaled_tensor_amd as fp4
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def weight(n, k):
        q = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8, device="cuda")
        s = torch.randint(122, 131, (n, k // 32), generator=g, dtype=torch.uint8, device="cuda")
        return fp4.QTensor(q, s, torch.ones(1, device="cuda"), fp4.E8M0, 32, fp4.FP4_SCALES_1D, n, k)

    def work(seed):
        """One thread's calls: a float32 product, one with a split K (equal sizes in both threads, so that
        their workspaces are interchangeable blocks) and a sort over several workgroups."""
        x = torch.randn(40, 2048, generator=g, device="cuda") * seed
        y = torch.randn(9, 2048, generator=g, device="cuda") * seed
        w = weight(512, 2048)
        ids = torch.randint(-1, 70, (9000, 3), generator=g, dtype=torch.int32, device="cuda")

        def run():
            p = fp4.expert_sort(ids, 64)
            return [fp4.linear(x, w), fp4.linear(y, w), fp4.linear(x.to(torch.bfloat16), w), p.order, p.pos, p.offsets]
        return run
    runs = [work(1.0), work(3.0)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    start, wrong, errors = threading.Barrier(2), [0, 0], []

    def body(i):
        try:
            start.wait(timeout=30)
            for _ in range(60):
                got = runs[i]()
                wrong[i] += sum(not torch.equal(a.view(torch.int16) if a.dtype is torch.bfloat16 else a.view(torch.int32),
                                                b.view(torch.int16) if b.dtype is torch.bfloat16 else b.view(torch.int32))
                                for a, b in zip(got, want[i]))
        except Exception as e:  # reported in the main thread
            errors.append(e)
    threads = [threading.Thread(target=body, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert wrong == [0, 0]
