"""Outputs that a caller gives to the MLP layers' calls, on the CPU: one without room for the
result is refused in the binding, before the library is called with its pointer."""
import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture()
def mlp(monkeypatch):
    from dlrm_embedding_bag_b200 import mlp as _mlp

    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or 0

    # placements are checked elsewhere: here CPU tensors stand in
    monkeypatch.setattr(_mlp, "_pitched", lambda t, name, dtype: (64, t.stride(0)))
    monkeypatch.setattr(_mlp, "_planes", lambda t, name: (64, t.stride(1), t.stride(0)))
    monkeypatch.setattr(_mlp.ops, "_lib", Library())
    monkeypatch.setattr(_mlp.ops, "_stream", lambda: 0)
    _mlp.calls = calls
    yield _mlp
    del _mlp.calls


@pytest.mark.parametrize("rows,cols,ok", [(4, 8, True), (5, 16, True), (3, 8, False),
                                          (4, 7, False), (0, 8, False), (8, 4, False)])
def test_outputs_have_room(mlp, rows, cols, ok):
    x = torch.zeros((4, 8))
    a, w = torch.zeros((4, 16), dtype=BF16), torch.zeros((8, 16), dtype=BF16)
    planes = torch.zeros((3, 4, 16), dtype=BF16)
    f32, bf16 = torch.zeros((rows, cols)), torch.zeros((rows, cols), dtype=BF16)
    bf16x3 = torch.zeros((3, rows, cols), dtype=BF16)
    for call in (lambda: mlp.to_bf16(x, bf16), lambda: mlp.split_bf16x3(x, bf16x3),
                 lambda: mlp.linear_bf16(a, w, out_f32=f32),
                 lambda: mlp.linear_bf16(a, w, f32=False, out_bf16=bf16),
                 lambda: mlp.linear_f32a(planes, w, out_f32=f32),
                 lambda: mlp.linear_f32a(planes, w, f32=False, out_planes=bf16x3)):
        n = len(mlp.calls)
        if ok:
            call()
            assert len(mlp.calls) == n + 1
        else:
            with pytest.raises(ValueError, match=r"room for \(4, 8\)"):
                call()
            assert len(mlp.calls) == n
