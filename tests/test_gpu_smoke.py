"""smoke() runs every paged call, and early enough for a trace of its first
launches to show them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu


class Launches(TorchDispatchMode):
    """torch operations with a CUDA tensor among what they return, launches at most."""

    count = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        got = func(*args, **(kwargs or {}))
        out = got if isinstance(got, (tuple, list)) else (got,)
        self.count += any(isinstance(t, torch.Tensor) and t.is_cuda for t in out)
        return got


def test_smoke_reaches_every_paged_call_within_500_launches(hd, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__ as entry
    reached = {}
    with Launches() as launches:
        for name in ("rope_append_paged", "attn_paged", "select_pages", "attn_selected_pages"):
            def call(*args, _name=name, _f=getattr(hd, name), **kw):
                reached.setdefault(_name, []).append(launches.count)
                return _f(*args, **kw)
            monkeypatch.setattr(hd, name, call)
        entry.smoke()
    assert set(reached) == {"rope_append_paged", "attn_paged", "select_pages", "attn_selected_pages"}
    # the second batch is single tokens, the first with a chunk: the last calls are the kernel of few rows' and the choice's
    assert max(x[-1] for x in reached.values()) < 500, reached
