"""The 4-bit product's binding on the CPU: which workspace it takes, and of which device.  The library's calls
are recorded in place of run; plain tensors that say they are on a GPU stand for device tensors."""
import contextlib

import pytest
import torch

import sparse_gemm_02_amd as S


class On(torch.Tensor):
    """A host tensor that says it is on GPU `index`."""
    index = 1

    def get_device(self):
        return self.index


def _on(index, *shape, dtype=torch.uint8):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.index = index
    return t


def test_the_workspace_is_that_of_the_tensors_device(monkeypatch):
    """Its size is asked with the tensors' device current, and kept for each device by itself."""
    current, asked, calls = [0], [], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    def size(T, K, N, out):
        asked.append(current[0])
        out._obj.value = 1000 * (1 + current[0])
        return 0

    class Library:
        slope_spmm_mxfp4_workspace_bytes = staticmethod(size)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(S, "library", lambda: Library)
    monkeypatch.setattr(S, "_on_device", lambda fn, dev, stream, *a: calls.append((fn, dev, a[-1])))
    T, K, N = 3, 128, 64                                             # sizes that nothing else here asks for
    for index in (1, 0, 1, 2, 0):
        args = _on(index, T, 64), _on(index, T, 16), K, _on(index, 3328), N, _on(index, T, N, dtype=torch.float32)
        empty = torch.empty
        monkeypatch.setattr(torch, "empty", lambda n, dtype, device, i=index: _on(i, n))
        S.slope_spmm_mxfp4_packed(*args)
        monkeypatch.setattr(torch, "empty", empty)
        assert calls[-1] == ("slope_spmm_mxfp4_packed", index, 1000 * (1 + index))
    assert asked == [1, 0, 2] and current == [0]
    # a given stream: no workspace is taken; a given workspace is passed on
    args = _on(1, T, 64), _on(1, T, 16), K, _on(1, 3328), N, _on(1, T, N, dtype=torch.float32)
    S.slope_spmm_mxfp4_packed(*args, stream=0)
    assert calls[-1][2] == 0
    S.slope_spmm_mxfp4_packed(*args, stream=0, workspace=_on(1, 77))
    assert calls[-1][2] == 77
