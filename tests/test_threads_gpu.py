"""Calls of several host threads at once, each on a stream of its own: the same
kernels with different amounts of shared memory in one process."""
import threading

import pytest
import torch

from gated_delta_rule_156_b200 import kda as K

pytestmark = pytest.mark.gpu
DEV = "cuda"


def problem(d, dtype, seed, T=130, H=2):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=DEV)
    q, k = (torch.nn.functional.normalize(randn(1, T, H, d), dim=-1)
            for _ in range(2))
    return dict(q=(q * d ** -0.5).to(dtype), k=k.to(dtype),
                v=randn(1, T, H, d).to(dtype),
                log_alpha=-0.1 * torch.rand(1, T, H, d, generator=g,
                                            device=DEV),
                beta=torch.rand(1, T, H, generator=g, device=DEV),
                d_out=randn(1, T, H, d).to(dtype))


def backward(p, chunk):
    return K.chunk_bwd(p["q"], p["k"], p["v"], p["log_alpha"], p["beta"],
                       None, None, p["d_out"], chunk=chunk)


def forward(p, chunk):
    return K.chunk_fwd(p["q"], p["k"], p["v"], p["log_alpha"], p["beta"],
                       chunk=chunk)


@pytest.mark.parametrize("call,dtype,sizes", [
    # one shape: its products contract over 64 and over 128
    (backward, torch.bfloat16, [(128, 64)] * 4),
    (backward, torch.float32, [(64, 64), (128, 32)] * 2),
    (forward, torch.float32, [(64, 64), (128, 32)] * 2)])
def test_threads(call, dtype, sizes):
    problems = [problem(d, dtype, i) for i, (d, _) in enumerate(sizes)]
    want = [call(p, c) for p, (_, c) in zip(problems, sizes)]
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(sizes))

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            with torch.cuda.stream(stream):
                for _ in range(300):
                    got = call(problems[i], sizes[i][1])
            stream.synchronize()
            assert all(a is None or torch.equal(a, b)
                       for a, b in zip(got, want[i]))
        except Exception as e:  # the thread's failure is the test's
            failed.append(f"{sizes[i]}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,))
               for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
