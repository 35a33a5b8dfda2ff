"""What sessions with drafted trees and limited views refuse (no GPU)."""

import pytest
import torch

from test_streams_host import rec  # noqa: F401  (a fixture)


def session(lengths, n_q, **kw):
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    from mla_absorbed_decode_absorb_gb300.runtime import DecodeSession
    return DecodeSession(W.generate(W.custom("views", lengths, n_q=n_q), seed=3), device="cpu", **kw)


def chain(*shape):
    return torch.arange(-1, shape[-1] - 1, dtype=torch.int32).expand(shape).contiguous()


def test_set_tree_takes_parents_of_every_sequence(rec):  # noqa: F811
    """One row is not every sequence's tree."""
    with rec:
        s = session([5, 70], 3, tree=chain(2, 3))
    before = s.parents.clone()
    for shape in [(3,), (1, 3), (2, 1), (2, 2), (2, 4), (3, 3), (1, 2, 3), ()]:
        rec.log.clear()
        with pytest.raises(ValueError), rec:
            s.set_tree(torch.full(shape, -1, dtype=torch.int32))
        assert torch.equal(s.parents, before) and not any(kind == "launch" for kind, *_ in rec.log)
    with rec:
        s.set_tree(torch.full((2, 3), -1, dtype=torch.int32))
    assert (s.parents == -1).all()


@pytest.mark.parametrize("kw", [{}, {"window": 9}, {"window": 9, "path": "non_absorbed"}])
def test_a_session_without_a_tree_takes_none(rec, kw):  # noqa: F811
    with rec:
        s = session([5], 3, **kw)
    with pytest.raises(ValueError):
        s.set_tree(chain(1, 3))


def test_more_new_tokens_than_the_causal_append_takes_are_refused_at_once(rec):  # noqa: F811
    """The absorbed path of a window appends at most eight tokens a sequence; a chain given as a tree goes further, and so
    does the other path."""
    with pytest.raises(ValueError), rec:
        session([5, 70], 9, window=20, path="absorbed")
    with rec:
        assert session([5, 70], 8, window=20, path="absorbed").path == "absorbed"
        assert session([5, 70], 9, window=20).path == "non_absorbed"
        s = session([5, 70], 9, window=20, tree=chain(2, 9))
        rec.log.clear()
        s.step()
    assert s.path == "absorbed" and [n for kind, n, _ in rec.log if kind == "launch"][0] == "mla_append_absorb_q_tree"
