"""The example decoder's choice of the attention call and of its arguments, without
its layers (no GPU)."""

import inspect

import dequant_matmul_gptq_amd as dq
from examples.decoder import Decoder


def _decoder(pages=64, page_size=4, **kw):
    d = Decoder.__new__(Decoder)
    d.pool, d.device, d.window = dq.PagePool(pages, page_size), "cpu", 0
    for name, value in kw.items():
        setattr(d, name, value)
    d._copy = lambda pairs: None
    d.forward = lambda tokens, positions, slots, where: where
    return d


def _branches(d, tokens, names="ab"):
    d.add(names[0])
    d.step([(names[0], list(range(tokens)))])
    for name in names[1:]:
        d.fork(names[0], name)


def _call(where):
    """The call that forward would make, with no argument that it does not know."""
    call = dq.paged_attention_shared if "shared_len" in where else dq.paged_attention
    inspect.signature(call).bind(None, None, workspace=None, **where)
    return call


def test_sinks_without_a_window_and_shared_pages():
    """Sinks say nothing without a window; sequences that share pages have none in their call."""
    d = _decoder(sinks=3, share=True)
    _branches(d, 9)
    where = d.step([("a", [1]), ("b", [2])])
    assert _call(where) is dq.paged_attention_shared and where["shared_len"].tolist() == [8]
    assert _call(d.step([("a", [1])])) is dq.paged_attention


def test_sinks_with_a_window_share_nothing():
    d = _decoder(sinks=3, share=True, window=5)
    _branches(d, 9)
    where = d.step([("a", [1]), ("b", [2])])
    assert _call(where) is dq.paged_attention and (where["window"], where["sinks"]) == (5, 3)
