"""Host-side checks of the entry points around the attention (window decode,
log probabilities, acceptance, compaction, pages): what the library refuses
before it launches anything, and the binding's own checks."""
import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

FAKE = 4096  # a 16-byte aligned address that no accepted call here gets to use
BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build_library()
    return abi.load()


CALLS = {
    "mla_paged_decode_window": dict(
        q=FAKE, q_tok=8 * 576, q_head=576, cache=FAKE, page_stride=64 * 576, num_pages=10, page_size=64, table=FAKE,
        table_stride=4, max_pages=4, lens=FAKE, window=100, sinks=4, batch=2, heads=8, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE,
        ws_bytes=1 << 40, status=None, stream=None),
    "mla_token_logprobs": dict(
        logits=FAKE, type=0, stride=1000, rows=4, vocab=1000, tokens=FAKE, token_stride=2, per_row=2, top_k=5, logprobs=FAKE,
        lse=FAKE, entropy=FAKE, ids=FAKE, top=FAKE, status=None, stream=None),
    "mla_tree_accept": dict(
        parents=FAKE, tokens=FAKE, targets=FAKE, target_stride=1, first=FAKE, indptr=FAKE, lens=FAKE, batch=2, total_q=9,
        most=4, path=FAKE, counts=FAKE, next=FAKE, new_lens=FAKE, status=None, stream=None),
    "mla_paged_compact": dict(
        path=FAKE, path_stride=4, most=4, counts=FAKE, lens=FAKE, batch=2, table=FAKE, table_stride=4, max_pages=4, cache=FAKE,
        page_stride=64 * 576, num_pages=10, page_size=64, layers=3, layer_stride=640 * 576, status=None, stream=None),
    "mla_pages_fork": dict(
        parents=FAKE, lens=FAKE, held=FAKE, table=FAKE, table_stride=4, old=2, max_pages=4, refs=FAKE, num_pages=10,
        new_lens=2 * FAKE, new_held=2 * FAKE, new_table=2 * FAKE, new_stride=4, new=3, status=None, stream=None),
    "mla_pages_fit": dict(
        lens=FAKE, want=FAKE, held=FAKE, table=FAKE, table_stride=4, batch=2, max_pages=4, refs=FAKE, num_pages=10,
        page_size=64, window=0, sinks=0, copies=FAKE, ws=FAKE, ws_bytes=1 << 30, status=None, stream=None),
    "mla_paged_copy": dict(
        copies=FAKE, n=3, cache=FAKE, page_stride=64 * 576, num_pages=10, page_size=64, layers=3, layer_stride=640 * 576,
        status=None, stream=None),
}

BAD_CACHE = [dict(page_size=0), dict(page_stride=64 * 576 - 8), dict(page_stride=64 * 576 + 4), dict(num_pages=-1),
             dict(cache=FAKE + 8), dict(cache=None), dict(num_pages=1 << 31)]
BAD_TABLE = [dict(max_pages=-1), dict(table_stride=3), dict(max_pages=1 << 26, table_stride=1 << 26), dict(table=None),
             dict(batch=-1), dict(lens=None)]
BAD_LAYERS = [dict(layers=-1), dict(layer_stride=-8), dict(layer_stride=640 * 576 + 4),
              # layers inside one another, one page short, between pages that leave no room
              dict(layer_stride=0), dict(layer_stride=639 * 576), dict(layer_stride=9 * 64 * 576),
              dict(layer_stride=64 * 576), dict(layer_stride=64 * 576, page_stride=2 * 64 * 576)]
REFUSED = {
    "mla_paged_decode_window": BAD_CACHE + BAD_TABLE + [
        dict(window=0), dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(lse=None), dict(q=FAKE + 8),
        dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(q_tok=568), dict(q_head=580), dict(heads=0), dict(scale=float("nan"))],
    "mla_token_logprobs": [
        dict(type=3), dict(type=-1), dict(rows=-1), dict(vocab=0), dict(vocab=-5), dict(stride=-1), dict(token_stride=-1),
        dict(per_row=-1), dict(top_k=-1), dict(top_k=3, vocab=2), dict(logits=None), dict(logits=FAKE + 1),
        dict(logits=FAKE + 2, type=2), dict(tokens=None), dict(logprobs=None), dict(per_row=0), dict(ids=None), dict(top_k=0),
        dict(stride=1 << 62), dict(token_stride=1 << 62)],
    "mla_tree_accept": [
        dict(batch=-1), dict(total_q=-1), dict(most=-1), dict(target_stride=-1), dict(target_stride=1 << 62), dict(parents=None),
        dict(tokens=None), dict(targets=None), dict(indptr=None), dict(lens=None), dict(path=None), dict(counts=None),
        dict(next=None), dict(new_lens=None)],
    "mla_paged_compact": BAD_CACHE + BAD_TABLE + BAD_LAYERS + [dict(path=None), dict(counts=None), dict(most=-1), dict(path_stride=3)],
    "mla_pages_fork": [
        dict(old=-1), dict(new=-1), dict(max_pages=-1), dict(table_stride=3), dict(new_stride=3), dict(num_pages=-1),
        dict(num_pages=1 << 31), dict(table_stride=1 << 60), dict(parents=None), dict(lens=None), dict(held=None),
        dict(table=None), dict(refs=None), dict(new_lens=None), dict(new_held=None), dict(new_table=None),
        # the two sides share memory
        dict(new_lens=FAKE), dict(new_held=FAKE + 4), dict(new_table=FAKE), dict(new_table=FAKE + 28), dict(table=2 * FAKE + 44)],
    "mla_pages_fit": [
        dict(batch=-1), dict(max_pages=-1), dict(table_stride=3), dict(num_pages=-1), dict(num_pages=1 << 31), dict(page_size=0),
        dict(max_pages=1 << 26, table_stride=1 << 26), dict(window=-1), dict(sinks=-1), dict(lens=None), dict(want=None),
        dict(held=None), dict(table=None), dict(refs=None), dict(copies=None)],
    "mla_paged_copy": BAD_CACHE + BAD_LAYERS + [dict(n=-1), dict(copies=None)],
}


def call(lib, name, **kw):
    return getattr(lib, name)(*{**CALLS[name], **kw}.values())


@pytest.mark.parametrize("name,kw", [(n, kw) for n, v in REFUSED.items() for kw in v],
                         ids=lambda v: v if isinstance(v, str) else "-".join("%s=%s" % i for i in v.items()))
def test_refuses(lib, name, kw):
    assert call(lib, name, **kw) == abi.MT_EINVAL


def test_workspaces(lib):
    n = abi.mla_pages_fit_workspace_bytes(2, 10)
    assert n > 0
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=n - 1)):
        assert call(lib, "mla_pages_fit", **kw) == abi.MT_EWORKSPACE
    for bad in ((-1, 10), (65536, 10), (2, -1), (2, (1 << 30) + 1), (2, 1 << 31)):
        assert abi.mla_pages_fit_workspace_bytes(*bad) == 0
    n = abi.mla_paged_decode_workspace_bytes(2, 8)
    assert call(lib, "mla_paged_decode_window", ws_bytes=n - 1) == abi.MT_EWORKSPACE


def test_more_than_supported(lib):
    assert call(lib, "mla_paged_decode_window", batch=65536) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_paged_decode_window", heads=4097, q_tok=4097 * 576) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_token_logprobs", top_k=33) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_tree_accept", batch=65536) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_paged_compact", batch=65536) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_pages_fork", old=65536, table=1 << 40) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_pages_fork", new=65536, new_table=1 << 40) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_pages_fit", batch=65536) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_pages_fit", num_pages=(1 << 30) + 1) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_paged_copy", n=1 << 31) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_paged_copy", layers=BIG) == abi.MT_EUNSUPPORTED


def test_columns_that_a_step_of_a_warp_would_pass(lib):
    """Rows of more than 2^30 columns: a lane's next column may be beyond 32 bits."""
    wide = dict(max_pages=(1 << 30) + 1, table_stride=(1 << 30) + 1)
    assert call(lib, "mla_pages_fork", new_stride=(1 << 30) + 1, **wide) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_pages_fit", page_size=1, **wide) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_token_logprobs", per_row=(1 << 30) + 1) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_tree_accept", most=(1 << 30) + 1) == abi.MT_EUNSUPPORTED
    assert call(lib, "mla_paged_compact", most=(1 << 30) + 1, path_stride=(1 << 30) + 1) == abi.MT_EUNSUPPORTED


def test_empty_calls_launch_nothing(lib):
    for name, kw in [("mla_paged_decode_window", dict(batch=0)), ("mla_token_logprobs", dict(rows=0, logits=None, tokens=None,
                                                                                             logprobs=None)),
                     ("mla_tree_accept", dict(batch=0)), ("mla_paged_compact", dict(batch=0)), ("mla_paged_compact", dict(most=0)),
                     ("mla_paged_compact", dict(layers=0)), ("mla_pages_fork", dict(old=0, new=0)), ("mla_pages_fit", dict(batch=0)),
                     ("mla_paged_copy", dict(n=0)), ("mla_paged_copy", dict(layers=0))]:
        assert call(lib, name, **kw) == abi.MT_OK, name


def test_binding_refuses_cpu_tensors():
    z = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros(2, 4, 576, dtype=torch.bfloat16)
    for f, a in [(abi.mla_token_logprobs, (torch.zeros(2, 5),)),
                 (abi.mla_tree_accept, (z(3), z(3), z(3), z(2), z(1), z(1, 2), z(1), z(1), z(1))),
                 (abi.mla_paged_compact, (z(1, 2), z(1), z(1), z(1, 3), cache)),
                 (abi.mla_pages_fork, (z(1), z(1), z(1), z(1, 3), z(9), z(1), z(1), z(1, 3))),
                 (abi.mla_pages_fit, (z(1), z(1), z(1), z(1, 3), z(9), 4, z(1, 3), torch.zeros(99, dtype=torch.uint8))),
                 (abi.mla_paged_copy, (z(1, 3), cache)),
                 (abi.mla_paged_decode_window, (torch.zeros(1, 8, 576, dtype=torch.bfloat16), cache, z(1, 1), z(1), 5, 0, 0.1,
                                                torch.zeros(1, 8, 512, dtype=torch.bfloat16), torch.zeros(1, 8),
                                                torch.zeros(1, dtype=torch.uint8)))]:
        with pytest.raises(abi.MlaTreeError, match="must be a CUDA tensor"):
            f(*a)
        with pytest.raises(abi.MlaTreeError, match="must be a CUDA tensor"):
            f(*(None,) + a[1:])
