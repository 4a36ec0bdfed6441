"""The cache calls' refusals, without a GPU: the C entries reject bad arguments before anything
launches, and the Python wrappers reject what the C side cannot see (types, shapes, strides)."""

import ctypes

import pytest
import torch

from paged_latent_attention_mla_gb300 import _native as n
from paged_latent_attention_mla_gb300 import build as nbuild
from paged_latent_attention_mla_gb300 import cache_append, cache_compact, cache_copy, cache_fork

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return n.load()


def layout(num_pages=64, page_size=64, stride=8, dtype=n.MLA_BF16):
    return ctypes.byref(n.MlaCache(num_pages, page_size, stride, dtype))


BAD_LAYOUTS = [
    (dict(num_pages=0), n.MLA_ERR_INVALID_ARG),
    (dict(stride=0), n.MLA_ERR_INVALID_ARG),
    (dict(dtype=n.MLA_F32), n.MLA_ERR_INVALID_ARG),
    (dict(page_size=48), n.MLA_ERR_UNSUPPORTED),
    (dict(page_size=4), n.MLA_ERR_UNSUPPORTED),
    (dict(page_size=2048), n.MLA_ERR_UNSUPPORTED),
    (dict(page_size=1024, stride=(1 << 20) + 1), n.MLA_ERR_UNSUPPORTED),
]


def append_status(lib, cache=None, **over):
    a = dict(c=0x10000, cs=512, k=0x20000, ks=64, start=0, N=6, pt=0x30000, sl=0x40000, B=2, ckv=0x50000, kpe=0x60000,
             status=0, opts={})
    a.update(over)
    o = dict(in_dtype=n.MLA_BF16, kv_descale=1.0)
    o.update(a["opts"])
    return lib.mla_cache_append(a["c"], a["cs"], a["k"], a["ks"], a["start"], a["N"], a["pt"], a["sl"], a["B"], a["ckv"],
                                a["kpe"], cache or layout(), ctypes.byref(n.MlaAppend(**o)), a["status"], 0)


@pytest.mark.parametrize("over,status", [
    (dict(N=-1), n.MLA_ERR_INVALID_ARG),
    (dict(B=-1), n.MLA_ERR_INVALID_ARG),
    (dict(B=0), n.MLA_ERR_INVALID_ARG),  # tokens of no rows and no token_start
    (dict(B=16385, start=0x70000), n.MLA_ERR_UNSUPPORTED),
    (dict(N=7), n.MLA_ERR_INVALID_ARG),  # 7 tokens of 2 rows and no token_start
    (dict(c=0x10008), n.MLA_ERR_INVALID_ARG),
    (dict(cs=511), n.MLA_ERR_INVALID_ARG),
    (dict(cs=516), n.MLA_ERR_INVALID_ARG),  # rows not 16-byte aligned
    (dict(ks=63), n.MLA_ERR_INVALID_ARG),
    (dict(c=0), n.MLA_ERR_INVALID_ARG),
    (dict(ckv=0x50008), n.MLA_ERR_INVALID_ARG),
    (dict(sl=0), n.MLA_ERR_INVALID_ARG),
    (dict(start=0x70002), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(in_dtype=n.MLA_E4M3)), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(kv_descale=0.5)), n.MLA_ERR_INVALID_ARG),  # a bf16 cache takes no scale
    (dict(opts=dict(kv_descale=float("nan"))), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(norm_weight=0x80000, norm_eps=-1.0)), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(norm_weight=0x80008)), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(rope_table=0x80000, rope_positions=0)), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(rope_interleaved=2)), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(cp_world=2, cp_rank=2, global_seq_lens=0x90000)), n.MLA_ERR_INVALID_ARG),
    (dict(opts=dict(cp_world=2, cp_rank=1)), n.MLA_ERR_INVALID_ARG),  # whole lengths missing
])
def test_append_rejects(lib, over, status):
    assert append_status(lib, **over) == status


def test_append_of_no_tokens_launches_nothing(lib):
    assert append_status(lib, N=0, c=0, k=0) == n.MLA_OK
    assert append_status(lib, N=0, B=0, c=0, k=0, pt=0, sl=0) == n.MLA_OK
    assert append_status(lib, B=0, start=0x70000, pt=0, sl=0) == n.MLA_OK  # all padding


@pytest.mark.parametrize("over", [dict(kv_descale=0.0), dict(kv_descale=-2.0), dict(kv_descale=1e-45),
                                  dict(kv_descale=float("inf"))])
def test_append_rejects_scales_of_an_e4m3_cache(lib, over):
    assert append_status(lib, cache=layout(dtype=n.MLA_E4M3), opts=over) == n.MLA_ERR_INVALID_ARG


def fork_status(lib, cache=None, **over):
    a = dict(pt=0x100000, sl=0x10000, B=4, par=0x20000, add=0x30000, N=4, ref=0x40000, ckv=0x50000, kpe=0x60000, window=-1,
             sinks=0, pto=0x200000, slo=0x70000, refo=0x80000, ws=0x400000, wsb=1 << 30, status=0)
    a.update(over)
    return lib.mla_cache_fork(a["pt"], a["sl"], a["B"], a["par"], a["add"], a["N"], a["ref"], a["ckv"], a["kpe"],
                              cache or layout(), a["window"], a["sinks"], a["pto"], a["slo"], a["refo"], a["ws"], a["wsb"],
                              a["status"], 0)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), n.MLA_ERR_INVALID_ARG),
    (dict(N=16385), n.MLA_ERR_UNSUPPORTED),
    (dict(window=-2), n.MLA_ERR_INVALID_ARG),
    (dict(sinks=-1), n.MLA_ERR_INVALID_ARG),
    (dict(pt=0), n.MLA_ERR_INVALID_ARG),
    (dict(par=0x20001), n.MLA_ERR_INVALID_ARG),
    (dict(ckv=0), n.MLA_ERR_INVALID_ARG),
    (dict(ws=0x400080), n.MLA_ERR_INVALID_ARG),
    (dict(wsb=128), n.MLA_ERR_WORKSPACE_TOO_SMALL),
    (dict(pto=0x100000), n.MLA_ERR_INVALID_ARG),  # the table in place, the lengths not
    (dict(pto=0x100020), n.MLA_ERR_INVALID_ARG),  # a row further: overlaps
    (dict(slo=0x10004), n.MLA_ERR_INVALID_ARG),
    (dict(slo=0x10000), n.MLA_ERR_INVALID_ARG),  # the lengths in place, the table not
    (dict(refo=0x40004), n.MLA_ERR_INVALID_ARG),
])
def test_fork_rejects(lib, over, status):
    assert fork_status(lib, **over) == status


@pytest.mark.parametrize("kept", [0x90002, 0x70000, 0x80010, 0x200000, 0x100040])
def test_fork_and_append_reject_misplaced_kept(lib, kept):
    """Not aligned, or over the lengths, counts or table that the fork writes, or the table it reads."""
    cache = ctypes.byref(n.MlaCache(64, 64, 8, n.MLA_BF16, kept))
    assert fork_status(lib, cache=cache) == n.MLA_ERR_INVALID_ARG
    if kept % 4:
        assert append_status(lib, cache=cache) == n.MLA_ERR_INVALID_ARG


def compact_status(lib, cache=None, **over):
    a = dict(pt=0x100000, B=4, ref=0x40000, ckv=0x50000, kpe=0x60000, pto=0x200000, refo=0x80000, map=0x90000, used=0xA0000,
             ws=0x400000, wsb=1 << 30)
    a.update(over)
    return lib.mla_cache_compact(a["pt"], a["B"], a["ref"], a["ckv"], a["kpe"], cache or layout(), a["pto"], a["refo"],
                                 a["map"], a["used"], a["ws"], a["wsb"], 0)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), n.MLA_ERR_INVALID_ARG),
    (dict(B=16385), n.MLA_ERR_UNSUPPORTED),
    (dict(pt=0), n.MLA_ERR_INVALID_ARG),
    (dict(map=0), n.MLA_ERR_INVALID_ARG),
    (dict(used=0xA0002), n.MLA_ERR_INVALID_ARG),
    (dict(pto=0x100010), n.MLA_ERR_INVALID_ARG),
    (dict(refo=0x40010), n.MLA_ERR_INVALID_ARG),
    (dict(map=0x40000), n.MLA_ERR_INVALID_ARG),  # the map over the counts
    (dict(map=0x100000), n.MLA_ERR_INVALID_ARG),  # and over the table
    (dict(wsb=256), n.MLA_ERR_WORKSPACE_TOO_SMALL),
])
def test_compact_rejects(lib, over, status):
    assert compact_status(lib, **over) == status


def copy_status(lib, cache=None, **over):
    a = dict(cs=0x10000, ks=0x20000, pages=9, ckv=0x30000, kpe=0x40000, src=0x50000, dst=0x60000, n=3, status=0)
    a.update(over)
    return lib.mla_cache_copy(a["cs"], a["ks"], a["pages"], a["ckv"], a["kpe"], a["src"], a["dst"], a["n"],
                              cache or layout(), a["status"], 0)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), n.MLA_ERR_INVALID_ARG),
    (dict(pages=0), n.MLA_ERR_INVALID_ARG),
    (dict(cs=0x10004), n.MLA_ERR_INVALID_ARG),
    (dict(src=0), n.MLA_ERR_INVALID_ARG),
    (dict(dst=0x60001), n.MLA_ERR_INVALID_ARG),
    (dict(status=0x70001), n.MLA_ERR_INVALID_ARG),
])
def test_copy_rejects(lib, over, status):
    assert copy_status(lib, **over) == status


def test_copy_of_no_pages_launches_nothing(lib):
    assert copy_status(lib, n=0, src=0, dst=0) == n.MLA_OK


@pytest.mark.parametrize("kw,status", BAD_LAYOUTS)
def test_every_call_rejects_bad_layouts(lib, kw, status):
    c = layout(**kw)
    assert append_status(lib, cache=c) == status
    assert fork_status(lib, cache=c) == status
    assert compact_status(lib, cache=c) == status
    assert copy_status(lib, cache=c) == status
    assert lib.mla_cache_workspace(c, 4, ctypes.byref(ctypes.c_size_t())) == status


def test_workspace_and_status_arguments(lib):
    size = ctypes.c_size_t()
    assert lib.mla_cache_workspace(layout(), -1, ctypes.byref(size)) == n.MLA_ERR_INVALID_ARG
    assert lib.mla_cache_workspace(layout(), 16385, ctypes.byref(size)) == n.MLA_ERR_UNSUPPORTED
    assert lib.mla_cache_workspace(layout(), 4, None) == n.MLA_ERR_INVALID_ARG
    assert lib.mla_cache_workspace(layout(), 4, ctypes.byref(size)) == n.MLA_OK and size.value % 256 == 0
    small = size.value
    assert lib.mla_cache_workspace(layout(num_pages=1 << 20), 4, ctypes.byref(size)) == n.MLA_OK and size.value > small
    assert lib.mla_cache_status(0, 0) == n.MLA_ERR_INVALID_ARG
    assert n.status_string(n.MLA_ERR_NO_PAGES) == "MLA_ERR_NO_PAGES"


# ---------------------------------------------------------------- the Python wrappers
def pools(pages=6, P=16, dtype=BF16):
    return torch.zeros((pages, P, 512), dtype=dtype), torch.zeros((pages, P, 64), dtype=dtype)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def append_args(**over):
    ckv, kpe = pools()
    a = dict(c=torch.zeros((4, 512), dtype=BF16), kpe=torch.zeros((4, 64), dtype=BF16), ckv_cache=ckv, kpe_cache=kpe,
             page_table=i32(2, 3), seq_lens=i32(2))
    a.update(over)
    return a


@pytest.mark.parametrize("over,error", [
    (dict(c=torch.zeros((4, 512), dtype=torch.float16)), TypeError),
    (dict(kpe=torch.zeros((4, 64))), TypeError),  # fp32 beside bf16
    (dict(c=torch.zeros((4, 511), dtype=BF16)), ValueError),
    (dict(kpe=torch.zeros((3, 64), dtype=BF16)), ValueError),
    (dict(c=torch.zeros((512, 4), dtype=BF16).t()), ValueError),
    (dict(kpe_cache=torch.zeros((6, 16, 64), dtype=F8)), TypeError),
    (dict(ckv_cache=torch.zeros((6, 16, 512))), TypeError),
    (dict(kpe_cache=torch.zeros((6, 8, 64), dtype=BF16)), ValueError),
    (dict(page_table=torch.zeros((2, 3), dtype=torch.int64)), TypeError),
    (dict(page_table=i32(3, 3)), ValueError),
    (dict(page_table=i32(2, 6)[:, ::2]), ValueError),
    (dict(token_start=i32(2)), ValueError),
    (dict(norm_weight=torch.zeros(512)), ValueError),  # not of c's type
    (dict(rope_table=torch.zeros((9, 32))), ValueError),
    (dict(global_seq_lens=i32(3)), ValueError),
    (dict(kept=i32(3)), ValueError),
])
def test_append_wrapper_rejects(over, error):
    with pytest.raises(error):
        cache_append(**append_args(**over))


@pytest.mark.parametrize("over,error", [
    (dict(seq_lens=i32(3)), ValueError),
    (dict(parents=i32(2, 1)), ValueError),
    (dict(parents=torch.zeros(2)), TypeError),
    (dict(ref_count=i32(5)), ValueError),
    (dict(new_tokens=i32(3)), ValueError),
    (dict(page_table_out=i32(2, 4)), ValueError),
    (dict(seq_lens_out=i32(1)), ValueError),
    (dict(ref_count_out=i32(7)), ValueError),
    (dict(kept=i32(3)), ValueError),
])
def test_fork_wrapper_rejects(over, error):
    ckv, kpe = pools()
    a = dict(page_table=i32(2, 3), seq_lens=i32(2), parents=i32(2), ref_count=i32(6), ckv_cache=ckv, kpe_cache=kpe,
             workspace=torch.zeros(4096, dtype=torch.uint8))
    a.update(over)
    with pytest.raises(error):
        cache_fork(**a)


def test_compact_and_copy_wrappers_reject():
    ckv, kpe = pools()
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        cache_compact(i32(2, 3), i32(5), ckv, kpe, ws)
    with pytest.raises(ValueError):
        cache_compact(i32(2, 3), i32(6), ckv, kpe, ws, page_table_out=i32(2, 2))
    with pytest.raises(TypeError):
        cache_compact(i32(2, 3), i32(6), ckv, kpe, ws, num_used=torch.zeros(1))
    with pytest.raises(ValueError):
        cache_copy(ckv, kpe, i32(3), i32(2))
    with pytest.raises(ValueError):
        cache_copy(ckv, kpe, i32(3), i32(3), ckv_src=ckv)
    with pytest.raises(ValueError):
        cache_copy(ckv, kpe, i32(3), i32(3), ckv_src=pools(P=8)[0], kpe_src=pools(P=8)[1])


def test_decode_wrapper_rejects_what_does_not_fit_its_config(lib):
    """Before anything launches: sizes below the config's, other element sizes, strided tensors."""
    from paged_latent_attention_mla_gb300 import PagedMlaDecoder

    dec = PagedMlaDecoder(H=16, seq_len_q=1, num_pages=6, page_table_stride=3, qkv_dtype=BF16, page_size=16, num_clusters=4,
                          device="cpu")
    dec.plan([20, 40])
    ckv, kpe = pools()

    def call(**over):
        a = dict(q_latent=torch.zeros((2, 1, 16, 512), dtype=BF16), q_rope=torch.zeros((2, 1, 16, 64), dtype=BF16), ckv=ckv,
                 kpe=kpe, page_table=i32(2, 3), seq_lens=i32(2), scale=1.0)
        a.update(over)
        return dec(**a)

    for over, error in [
        (dict(), ValueError),  # not on a GPU
        (dict(q_latent=torch.zeros((2, 2, 16, 512), dtype=BF16)[:, ::2]), ValueError),
        (dict(q_rope=torch.zeros((2, 1, 8, 64), dtype=BF16)), ValueError),
        (dict(q_rope=torch.zeros((2, 1, 16, 64))), TypeError),
        (dict(ckv=pools(pages=5)[0]), ValueError),
        (dict(page_table=i32(2, 2)), ValueError),
        (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
        (dict(out=torch.zeros((2, 1, 16, 512))), TypeError),
        (dict(lse=torch.zeros(31)), ValueError),
        (dict(local_visible_lens=i32(1)), ValueError),
    ]:
        with pytest.raises(error):
            call(**over)


def test_fork_rejects_tables_whose_entries_pass_32_bits(lib):
    """The pages the rows ask for are summed in 32 bits; no row asks for more than its table row holds."""
    def status(N, stride, page_size=8, **over):
        # arrays far apart; a workspace too small, so that what is accepted launches nothing
        return fork_status(lib, cache=layout(stride=stride, page_size=page_size), N=N, pt=1 << 40, pto=1 << 44, wsb=256, **over)

    assert status(16384, 131072) == n.MLA_ERR_UNSUPPORTED
    assert status(16384, 131071) == n.MLA_ERR_WORKSPACE_TOO_SMALL
    assert status(16, 1 << 27) == n.MLA_ERR_UNSUPPORTED
    assert status(15, 1 << 27) == n.MLA_ERR_WORKSPACE_TOO_SMALL
    assert status(2049, 1 << 20, page_size=1024) == n.MLA_ERR_UNSUPPORTED
    assert status(1, 1 << 27, B=16384) == n.MLA_ERR_WORKSPACE_TOO_SMALL  # the present rows ask for nothing


def test_decode_wrapper_rejects_what_it_would_read_at_the_wrong_place(lib):
    """Tensors large enough but laid out for another config: each is named, not read at the wrong stride."""
    from paged_latent_attention_mla_gb300 import PagedMlaDecoder

    def decoder(dtype=BF16, **over):
        a = dict(H=16, seq_len_q=1, num_pages=6, page_table_stride=3, qkv_dtype=dtype, page_size=16, num_clusters=4, device="cpu")
        a.update(over)
        dec = PagedMlaDecoder(**a)
        dec.plan([20, 40])
        return dec

    def call(dec, dtype=BF16, B=2, Sq=1, **over):
        ckv, kpe = pools(dtype=dtype)
        a = dict(q_latent=torch.zeros((B, Sq, 16, 512), dtype=dtype), q_rope=torch.zeros((B, Sq, 16, 64), dtype=dtype), ckv=ckv,
                 kpe=kpe, page_table=i32(B, 3), seq_lens=i32(B), scale=1.0)
        a.update(over)
        return dec(**a)

    one, two, eight = decoder(), decoder(seq_len_q=2), decoder(F8)
    for dec, over, error, what in [
        (one, dict(page_table=i32(2, 4)), ValueError, "page_table"),
        (one, dict(page_table=torch.zeros((2, 3))), TypeError, "page_table"),
        (one, dict(seq_lens=torch.zeros(2)), TypeError, "seq_lens"),
        (one, dict(Sq=2), ValueError, "q_latent"),
        (two, dict(Sq=2, q_rope=torch.zeros((4, 1, 16, 64), dtype=BF16)), ValueError, "q_rope"),
        (one, dict(q_rope=torch.zeros((2, 1, 64, 16), dtype=BF16)), ValueError, "q_rope"),
        (one, dict(kpe=pools(pages=12, P=8)[1]), ValueError, "kpe"),
        (one, dict(ckv=torch.zeros((6, 16, 1024), dtype=BF16)), ValueError, "ckv"),
        (one, dict(q_latent=torch.zeros((2, 1, 16, 1024), dtype=BF16)), ValueError, "q_latent"),
        (one, dict(ckv=torch.zeros((6, 16, 512), dtype=torch.float16)), TypeError, "ckv"),
        (one, dict(q_latent=torch.zeros((2, 1, 16, 512), dtype=torch.float16)), TypeError, "q_latent"),
        (one, dict(out=torch.zeros((2, 1, 16, 512), dtype=torch.float16)), TypeError, "out"),
        (eight, dict(dtype=F8, kpe=torch.zeros((6, 16, 64), dtype=torch.float8_e5m2)), TypeError, "kpe"),
        (two, dict(Sq=2, local_visible_lens=i32(2, 3)), ValueError, "local_visible_lens"),
        (one, dict(global_seq_lens=torch.zeros(2)), TypeError, "global_seq_lens"),
    ]:
        with pytest.raises(error, match=what):
            call(dec, **over)

    # what is read where the kernels read it passes these checks and is refused for lying on the CPU
    for dec, over in [
        (one, {}), (two, dict(Sq=2, local_visible_lens=i32(2, 2))), (eight, dict(dtype=F8)),
        (one, dict(page_table=i32(5, 3), seq_lens=i32(5))),  # more rows than the batch
        (one, dict(page_table=i32(6), q_rope=torch.zeros(2048, dtype=BF16), lse=torch.zeros(32))),  # flat
        (one, dict(B=1, page_table=i32(1, 9))),  # one row of a wider table
        (one, dict(ckv=pools(pages=9)[0], kpe=pools(pages=7)[1])),  # pools past num_pages
        (one, dict(q_latent=torch.zeros((2, 1, 16, 512), dtype=BF16).view(torch.int16))),  # raw bits
    ]:
        with pytest.raises(ValueError, match="CUDA tensors"):
            call(dec, **over)
