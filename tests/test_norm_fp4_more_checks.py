"""Further checks of mla_norm_rope's, mla_norm_rope_bwd's and
sparse_mla_decode_fp4's arguments (no GPU): what the binding hands to the
library, and codes of the C entry points."""
import pytest
import torch

import mla_inputs as mi
from tests.test_binding_checks import STREAM, b  # noqa: F401  (the recorder fixture)
from tests.test_norm_fp4_checks import _norm, lib  # noqa: F401


@pytest.fixture
def sent(b, monkeypatch):  # noqa: F811
    """(binding, list of the calls' arguments as the library takes them)."""
    calls = []

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                kinds = b.SIGNATURES[name][1]
                assert len(args) == len(kinds)
                calls.append((name, [k(a).value for k, a in zip(kinds, args)]))
                return 0
            return call

    monkeypatch.setattr(b, "load", lambda path=None: Recorder())
    return b, calls


def test_padding_rows_of_fresh_outputs_are_asked_to_be_zeros(sent):
    binding, calls = sent
    q, kv, _, _ = mi.norm_rows(1, 5, 3)
    pos, cs = torch.arange(5, dtype=torch.int32), mi.rope_table(9)
    cache = torch.zeros(2, 16, 416, dtype=torch.uint8)
    for qo in (None, torch.empty_like(q)):
        for ko in (None, torch.empty_like(kv)):
            binding.mla_norm_rope(q, kv, pos, cs, kv_cache=cache, slots=pos, q_out=qo, kv_out=ko, stream=STREAM)
            form = calls[-1][1][15]
            assert form == 2 | (0x100 if qo is None else 0) | (0x200 if ko is None else 0)


def test_format_codes(lib):  # noqa: F811
    for bad in (dict(form=2 | 0x400), dict(form=3 | 0x100), dict(form=-1), dict(form=1 | 0x100, ks=0.5)):
        assert _norm(lib, **bad) == 1, bad
    for good in (2 | 0x100, 1 | 0x200, 0x300, 2 | 0x300):   # past the checks; no tokens, so that nothing is launched
        assert _norm(lib, form=good, n=0) != 1
