"""Host-side checks of the paged entry points (no compute calls): what the
library refuses before it launches anything, and the binding's own checks."""
import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

FAKE = 4096  # a 16-byte aligned address that no accepted call here gets to use


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build_library()
    return abi.load()


APPEND = dict(latent=FAKE, latent_stride=576, k_rope=FAKE, k_rope_stride=576, norm_weight=None, norm_eps=1e-6,
              q_rope=FAKE, q_tok=8 * 192, q_head=192, q_out=FAKE + 1024, qo_tok=8 * 576, qo_head=576, heads=8,
              rope=FAKE, max_positions=100, style=0, positions=None, indptr=FAKE, lens=FAKE, batch=2, total_q=4,
              table=FAKE, table_stride=4, max_pages=4, cache=FAKE, page_stride=64 * 576, num_pages=10, page_size=64,
              status=None, stream=None)
DECODE = dict(q=FAKE, q_tok=8 * 576, q_head=576, cache=FAKE, page_stride=64 * 576, num_pages=10, page_size=64,
              table=FAKE, table_stride=4, max_pages=4, lens=FAKE, batch=2, heads=8, scale=0.1, out=FAKE, lse=FAKE,
              ws=FAKE, ws_bytes=1 << 40, status=None, stream=None)


def _append(lib, **kw):
    return lib.mla_paged_append(*{**APPEND, **kw}.values())


def _decode(lib, **kw):
    return lib.mla_paged_decode(*{**DECODE, **kw}.values())


BAD_CACHE = [dict(page_size=0), dict(page_size=-64), dict(page_stride=64 * 576 - 8), dict(page_stride=64 * 576 + 4),
             dict(num_pages=-1), dict(max_pages=-1), dict(table_stride=3), dict(cache=FAKE + 8), dict(cache=None),
             dict(max_pages=1 << 26, table_stride=1 << 26), dict(table=None), dict(lens=None), dict(batch=-1),
             dict(num_pages=1 << 31)]


@pytest.mark.parametrize("kw", BAD_CACHE + [
    dict(latent=None), dict(k_rope=None), dict(rope=None), dict(indptr=None), dict(latent=FAKE + 2),
    dict(k_rope=FAKE + 8), dict(rope=FAKE + 4), dict(norm_weight=FAKE + 2), dict(latent_stride=504),
    dict(latent_stride=580), dict(k_rope_stride=56), dict(k_rope_stride=68), dict(norm_eps=-1e-6),
    dict(norm_eps=float("nan")), dict(norm_eps=float("inf")), dict(style=2), dict(style=-1), dict(heads=-1),
    dict(total_q=-1), dict(max_positions=-1), dict(q_rope=None), dict(q_out=None), dict(heads=0),
    dict(q_rope=FAKE + 8), dict(q_out=FAKE + 8), dict(q_tok=-8), dict(q_head=4), dict(qo_tok=4), dict(qo_head=60),
    # outputs that would share elements: heads inside one another, tokens inside one another, tokens between heads
    dict(qo_head=56), dict(qo_tok=7 * 576), dict(qo_tok=0), dict(qo_tok=64, qo_head=128),
    # in place, but through other strides
    dict(q_out=FAKE)])
def test_append_refuses(lib, kw):
    assert _append(lib, **kw) == abi.MT_EINVAL


@pytest.mark.parametrize("kw", BAD_CACHE + [
    dict(q=None), dict(out=None), dict(lse=None), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2),
    dict(q_tok=568), dict(q_head=568), dict(q_tok=8 * 576 + 4), dict(q_head=580), dict(heads=0), dict(heads=-8),
    dict(scale=float("nan")), dict(scale=float("inf"))])
def test_decode_refuses(lib, kw):
    assert _decode(lib, **kw) == abi.MT_EINVAL


def test_decode_workspace(lib):
    for heads in (1, 8, 16, 17, 32, 33, 64, 65, 128, 1000, 4096):
        n = abi.mla_paged_decode_workspace_bytes(3, heads)
        assert n > 0 and n % 256 == 0
        assert _decode(lib, heads=heads, q_tok=heads * 576, ws_bytes=n - 1) == abi.MT_EWORKSPACE
    assert _decode(lib, ws=None) == abi.MT_EWORKSPACE
    assert _decode(lib, ws=FAKE + 16) == abi.MT_EWORKSPACE
    for bad in ((-1, 8), (2, 0), (2, -1), (2, 4097)):
        assert abi.mla_paged_decode_workspace_bytes(*bad) == 0


def test_more_than_supported(lib):
    assert _decode(lib, heads=4097, q_tok=4097 * 576) == abi.MT_EUNSUPPORTED
    assert _decode(lib, batch=65536) == abi.MT_EUNSUPPORTED
    assert _append(lib, heads=4097, q_tok=4097 * 192, qo_tok=4097 * 576) == abi.MT_EUNSUPPORTED
    # more tokens and heads than one grid can take
    assert _append(lib, total_q=(1 << 31) - 1, heads=4096, q_tok=4096 * 192, qo_tok=4096 * 576) == abi.MT_EUNSUPPORTED


def test_empty_calls_launch_nothing(lib):
    assert _append(lib, batch=0) == abi.MT_OK
    assert _append(lib, total_q=0) == abi.MT_OK
    assert _decode(lib, batch=0) == abi.MT_OK


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    bf = torch.bfloat16
    cache, table, lens = z(2, 64, 576, dtype=bf), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32)
    with pytest.raises(abi.MlaTreeError, match="cache must be a CUDA tensor"):
        abi.mla_paged_decode(z(1, 8, 576, dtype=bf), cache, table, lens, 0.1, z(1, 8, 512, dtype=bf), z(1, 8),
                             z(1, dtype=torch.uint8))
    with pytest.raises(abi.MlaTreeError, match="cache must be a CUDA tensor"):
        abi.mla_paged_append(z(1, 512, dtype=bf), z(1, 64, dtype=bf), z(2, dtype=torch.int32), lens, table, cache,
                             z(4, 64))


def test_append_without_indptr_is_one_token_a_request(lib):
    """Refused unless there are as many tokens as requests (nothing to launch where there are none)."""
    for total_q in (1, 3, 4):
        assert _append(lib, indptr=None, total_q=total_q) == abi.MT_EINVAL
    assert _append(lib, indptr=None, total_q=0) == abi.MT_OK
    assert _append(lib, indptr=None, batch=0, total_q=2) == abi.MT_OK
