"""The example decoder's choice of the attention call and of its arguments, without
its layers (no GPU)."""

import inspect

import dequant_matmul_gptq_amd as dq
from examples import decoder as example
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


def test_shared_only_where_it_gains():
    """share=SHARE_GAINS: eight branches or more of up to four new tokens each on average, behind 4096 shared tokens or
    more."""
    def step(count, tokens, new, **kw):
        d = _decoder(pages=6000, page_size=16, **kw)
        _branches(d, tokens, [chr(97 + i) for i in range(count)])
        where = d.step([(chr(97 + i), [1] * (new if i else 1)) for i in range(count)])
        assert _call(where) is (dq.paged_attention_shared if "shared_len" in where else dq.paged_attention)
        return where["shared_len"].tolist() if "shared_len" in where else None

    gains = dict(share=example.SHARE_GAINS)
    assert step(8, 4100, 1, **gains) == step(8, 4100, 4, **gains) == [4096]
    assert step(20, 9000, 2, **gains) == [8992]
    assert step(7, 4100, 1, **gains) is None            # too few
    assert step(8, 4095, 1, **gains) is None            # behind too little
    assert step(8, 4100, 5, **gains) is None            # prompts gain nothing
    assert step(4, 1000, 1, **gains) is None
    assert step(2, 20, 9, share=True) == [16] and step(8, 4100, 1) is None


def test_each_group_by_itself():
    d = _decoder(pages=3000, page_size=16, share=example.SHARE_GAINS)
    _branches(d, 5000, "abcdefgh")
    _branches(d, 300, "xyz")
    where = d.step([(n, [1]) for n in "xyzabcdefgh"])
    assert where["shared_start"].tolist() == [0, 3, 11] and where["shared_len"].tolist() == [0, 4992]


def test_a_prompt_among_many_single_tokens_shares_with_them():
    d = _decoder(pages=3000, page_size=16, share=example.SHARE_GAINS)
    names = [str(i) for i in range(30)]
    _branches(d, 5000, names)
    where = d.step([(n, [1] * (80 if n == "7" else 1)) for n in names])
    assert where["shared_len"].tolist() == [4992]
    where = d.step([(n, [1] * (100 if n == "7" else 1)) for n in names])
    assert "shared_len" not in where


def test_the_command_shares_where_it_gains():
    assert example.arguments([]).share == example.SHARE_GAINS
    assert example.arguments(["--share", "0"]).share == 0
