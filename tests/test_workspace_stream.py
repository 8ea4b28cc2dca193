"""Whose memory a call's own workspace is (CPU): that of the stream the kernels run on."""
import contextlib

import pytest
import torch

from diffusion_long_context_b200 import build as focus_build


@pytest.fixture(scope="module")
def F():
    focus_build.build()
    from diffusion_long_context_b200 import focus
    return focus


class Recorder:
    """Stands for the stream context, the allocation and the library: notes the stream each ran under."""

    def __init__(self, F, monkeypatch):
        self.current, self.allocated, self.launched = "current", [], []

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s if s is not None else self.current
            yield
            self.current = before

        empty = torch.empty

        def note(n, dtype=None, device=None):
            self.allocated.append(self.current)
            return empty(n, dtype=dtype)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch, "empty", note)


class Side:
    cuda_stream = 4096


def test_a_workspace_belongs_to_the_stream_of_the_call(F, monkeypatch):
    rec, side = Recorder(F, monkeypatch), Side()
    ws, n = F._workspace(512, "cpu", None, side)
    assert rec.allocated == [side] and n == 512 and rec.current == "current"
    F._workspace(512, "cpu", None, None)
    assert rec.allocated[1:] == ["current"]
    mine = ws
    assert F._workspace(512, "cpu", mine, side) == (mine, 512) and len(rec.allocated) == 2
    assert F._workspace(0, "cpu", None, side) == (None, 0)


@pytest.mark.parametrize("name", ["focus_dense_attention", "focus_dense_attention_sinks", "focus_full_refresh",
                                  "focus_sparse_attention", "focus_sparse_attention_fused", "focus_cache_attention",
                                  "focus_cache_sparse_attention"])
def test_every_call_with_a_workspace_passes_its_stream(F, monkeypatch, name):
    side, seen = Side(), []
    monkeypatch.setattr(F, "_need", lambda *a: None)
    monkeypatch.setattr(F, "_here", lambda *a: 0)
    monkeypatch.setattr(F, "_workspace", lambda nbytes, device, ws, stream=None: seen.append(stream) or (None, 0))
    monkeypatch.setattr(F.lib, name, lambda *a: seen.append(a[-1]) or 0)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    Q, K, n = bf(1, 2, 3, 64), bf(1, 2, 64, 64), i32(1)
    sinks, blocks, kbar = i32(1, 2, 4), i32(1, 2, 1), torch.zeros(1, 2, 1, 64)

    class Layer:
        n_mat, n_pages, Hkv, page, d, k, _ref = 1, 4, 2, 16, 64, K, None
    args = dict(focus_dense_attention=(Q, n, K, K, Q), focus_dense_attention_sinks=(Q, n, K, K, Q, torch.zeros(1, 2, 64), sinks),
                focus_full_refresh=(K, K, K, K, 32, 32, kbar), focus_sparse_attention=(Q, n, K, K, sinks, blocks, 32, 32, 32, 64, Q),
                focus_sparse_attention_fused=(Q, n, K, K, kbar, 1, sinks, 32, 32, 32, 64, blocks, Q),
                focus_cache_attention=(Q, n, Layer, i32(1, 4), n, Q),
                focus_cache_sparse_attention=(Q, n, Layer, i32(1, 4), n, n, 32, sinks, blocks, Q))
    getattr(F, name)(*args[name], stream=side)
    assert seen == [side, side.cuda_stream]
