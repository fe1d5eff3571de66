"""Prompt processing without a GPU, at the edges that test_prompt_cpu.py leaves out."""
import pytest

from test_abi_cpu import lib  # noqa: F401  (the built library)
from test_prompt_cpu import E, U, _prefill


@pytest.mark.parametrize("kw,code", [
    (dict(causal=0, gseq=18), U), (dict(causal=0, gseq=18, cp=2), U), (dict(causal=0, gseq=None, cp=2), U),
    (dict(causal=1, gseq=18), E), (dict(causal=1, gseq=None, cp=2), E),
])
def test_prefill_global_lengths_play_no_part_where_not_causal(lib, kw, code):  # noqa: F811
    """Not looked at without causal, not even for its alignment: the next check (too many row tiles) refuses
    these calls."""
    assert _prefill(lib, H=1 << 30, T=1 << 10, **kw) == code
