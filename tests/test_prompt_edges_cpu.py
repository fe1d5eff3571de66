"""Prompt processing without a GPU, at the edges that test_prompt_cpu.py leaves out."""
import pytest
import torch
from torch._subclasses import FakeTensorMode

import mla_paged_decode_03_gb300 as M
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


@pytest.mark.parametrize("D,out,lse,what", [
    (512, (3, 4, 128), None, "out must be"), (128, (3, 4, 512), None, "out must be"), (128, (3, 3, 128), None, "out must be"),
    (512, (2, 4, 512), None, "out must be"), (128, (12, 128), None, "out must be"), (512, None, (3, 3), "out_lse must be"),
    (128, (3, 4, 128), (11,), "out_lse must be"),
])
def test_merge_refuses_outputs_that_do_not_fit(lib, D, out, lse, what):  # noqa: F811
    """Rows would be written behind an output of the other width, or of fewer rows.  Tensors without memory,
    so that the checks are reached without a GPU and a call that passes them stops at the null pointers."""
    with FakeTensorMode():
        def cuda(shape, dtype=torch.float32):
            return None if shape is None else torch.empty(shape, dtype=dtype, device="cuda")
        with pytest.raises(ValueError, match=what):
            M.lse_merge(cuda((2, 3, 4, D), torch.bfloat16), cuda((2, 3, 4)), out=cuda(out, torch.bfloat16), out_lse=cuda(lse))
