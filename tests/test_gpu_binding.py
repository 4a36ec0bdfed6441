"""The Python entry points as a program with threads and little memory meets them."""

import sys
import threading

import pytest
import torch

from paged_latent_attention_mla_gb300 import PagedMlaDecoder, cache_copy
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


def test_outputs_that_do_not_fit_raise_the_out_of_memory_error():
    """The outputs a call makes are torch's: so is the error when there is no memory for them."""
    B, H, P = 512, 128, 16
    ckv, kpe = pools(P=P)
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    ql = torch.zeros((B, 1, H, 512), dtype=torch.bfloat16, device="cuda")
    qr = torch.zeros((B, 1, H, 64), dtype=torch.bfloat16, device="cuda")
    dec = PagedMlaDecoder(H=H, seq_len_q=1, num_pages=8, page_table_stride=1, qkv_dtype=torch.bfloat16, page_size=P)
    dec.plan([1] * B)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-9)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            dec(ql, qr, ckv, kpe, table, lens, 1.0)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    out, _ = dec(ql, qr, ckv, kpe, table, lens, 1.0)
    assert out.shape == (B, 1, H, 512)
