"""The smoke run notices a call that does nothing."""

import pytest

import __graft_entry__ as entry
from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu


def test_smoke_passes():
    entry.smoke()


def test_smoke_notices_that_nothing_was_compacted(monkeypatch):
    monkeypatch.setattr(tl.PagedKVCache, "compact", lambda *args, **more: None)
    with pytest.raises(AssertionError, match="compact"):
        entry.smoke()
