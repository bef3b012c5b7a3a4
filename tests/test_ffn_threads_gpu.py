"""Products called by two threads at once, each on a stream of its own: bit for bit as one after the other."""
import threading

import pytest
import torch

from moe_matmul_amd import ffn
from test_ffn_gpu import announce, rng, same  # noqa: F401

pytestmark = pytest.mark.gpu


def test_few_rows_of_long_and_short_k():
    """The kernel of few rows with as much shared memory as it ever takes in one thread, with less in the other."""
    ks = [(16384, 8192), (4104, 5120, 64)]
    r = rng(21)
    data = {k: (r(8, k).bfloat16(), (r(96, k) * k ** -0.5).bfloat16()) for k in sum(ks, ())}
    want = {k: (ffn.linear(*d), ffn.gated(*d)) for k, d in data.items()}
    torch.cuda.synchronize()
    got, ready = {}, threading.Barrier(2)

    def work(mine):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ready.wait()
            for _ in range(20):
                for k in mine:
                    got[k] = ffn.linear(*data[k]), ffn.gated(*data[k])
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(mine,)) for mine in ks]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert got.keys() == want.keys()
    for k in want:
        for a, b in zip(got[k], want[k]):
            same(a, b)
