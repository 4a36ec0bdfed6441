"""Captured decodes replayed: every replay writes its outputs, for inputs that change in place."""

import pytest
import torch
from test_gpu_features import compare, host

import oracle
from paged_latent_attention_mla_gb300 import _native as n
from paged_latent_attention_mla_gb300 import build as nbuild
from paged_latent_attention_mla_gb300 import decoder_for
from paged_latent_attention_mla_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()
    n.load()


@pytest.mark.parametrize("options", [dict(num_clusters=40, combine_in_kernel=True), dict(num_clusters=40),
                                     dict(num_clusters=3, combine_in_kernel=True, partial_fp16=False), {}])
def test_replays_write_their_outputs(options):
    """Two graphs over one workspace, replayed in turn, with an eager call between; rows cut into many pieces."""
    probs = [wl.make_problem("uniform", seed=s, H=128, Sq=2, causal=True, seq_lens=[5000, 300, 2048, 9, 0]) for s in (71, 72, 73)]
    want = [oracle.decode(p.host_inputs()) for p in probs]
    d = probs[0].device_inputs("cuda")
    dec = decoder_for(probs[0], **options)
    outs = [torch.empty((5, 2, 128, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.empty((5, 2, 128), device="cuda") for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    decode = lambda out, lse: dec(d["q_latent"], d["q_rope"], d["ckv"], d["kpe"], d["page_table"], d["seq_lens"], d["scale"],  # noqa: E731
                                  out=out, lse=lse)
    decode(outs[0], lses[0])
    torch.cuda.synchronize()
    for g, o, l in zip(graphs, outs, lses):
        with torch.cuda.graph(g):
            decode(o, l)

    def load(i):
        other = probs[i].device_inputs("cuda")
        for k in ("q_latent", "q_rope", "ckv", "kpe", "page_table"):
            d[k].copy_(other[k])

    for step, (i, which) in enumerate([(0, 0), (1, 0), (2, 0), (0, 1), (1, 1), (2, 0), (1, 0)]):
        load(i)
        if step == 3:
            decode(outs[0], lses[0])
        outs[which].fill_(float("nan"))
        lses[which].fill_(float("nan"))
        graphs[which].replay()
        torch.cuda.synchronize()
        assert dec.status() == n.MLA_OK
        compare("bf16", *host(outs[which], lses[which]), *want[i])
