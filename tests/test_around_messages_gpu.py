"""What is refused beside an argument of an unusual but allowed stride is named
itself, and not that argument."""
import pytest
import torch

import __graft_entry__
from speculative_decode_mla_tree_gb300 import abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def i(*n):
    return torch.zeros(*n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("targets", [lambda: i(1).expand(6), lambda: i(6, 4)[:, 1]], ids=["one number", "a column"])
def test_accept(targets):
    ok = dict(parents=i(6), tokens=i(6), targets=targets(), qo_indptr=i(3), kv_lens=i(2), path=i(2, 4), counts=i(2), next_tokens=i(2),
              new_lens=i(2))
    abi.mla_tree_accept(**ok)
    for kw, message in [(dict(counts=i(3)), "counts must"), (dict(first=i(1)), "first must"), (dict(status=i(1).float()), "status must"),
                        (dict(qo_indptr=i(2)), "qo_indptr must"), (dict(targets=targets()[:5]), "targets must")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_tree_accept(**{**ok, **kw})


@pytest.mark.parametrize("tokens", [lambda: i(1).expand(6), lambda: i(6, 4)[:, 1]], ids=["one number", "a column"])
def test_logprobs(tokens):
    z = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
    ok = dict(logits=z(6, 50), tokens=tokens(), logprobs=z(6))
    abi.mla_token_logprobs(**ok)
    for kw, message in [(dict(lse=z(5)), "lse must"), (dict(logprobs=z(5)), "logprobs must"), (dict(status=z(1)), "status must"),
                        (dict(tokens=tokens()[:5]), "rows")]:
        with pytest.raises(abi.MlaTreeError, match=message):
            abi.mla_token_logprobs(**{**ok, **kw})
    with pytest.raises(abi.MlaTreeError, match="unit stride"):
        abi.mla_token_logprobs(z(6, 50), i(6, 8)[:, ::2], z(6, 4))
