"""The Python entry points as a program with threads meets them."""

import sys
import threading

import pytest
import torch

from paged_latent_attention_mla_gb300 import cache_copy
from paged_latent_attention_mla_gb300 import _native as n
from paged_latent_attention_mla_gb300 import build as nbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()
    n.load()


def pools(pages=8, P=16):
    return (torch.zeros((pages, P, 512), dtype=torch.bfloat16, device="cuda"),
            torch.zeros((pages, P, 64), dtype=torch.bfloat16, device="cuda"))


def test_other_threads_run_while_a_call_is_launched():
    """A launch can wait for room in the GPU's queue: the interpreter is not held meanwhile.  With a
    switch interval of minutes a thread that waits for the interpreter only gets it where it is given up."""
    ckv, kpe = pools()
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [2, 3]))
    cache_copy(ckv, kpe, src, dst)
    torch.cuda.synchronize()
    go, ran = threading.Event(), []

    def other():
        go.wait()
        ran.append(1)

    t = threading.Thread(target=other)
    t.start()
    old = sys.getswitchinterval()
    sys.setswitchinterval(600.0)
    try:
        go.set()
        for _ in range(5000):
            cache_copy(ckv, kpe, src, dst)
            if ran:
                break
        got = len(ran)
    finally:
        sys.setswitchinterval(old)
    t.join()
    torch.cuda.synchronize()
    assert got == 1
