"""The state of an optimiser step has its own types, whatever torch's default is."""
import pytest
import torch


@pytest.fixture(scope="module")
def optim():
    from dlrm_embedding_bag_b200 import build

    build.build()
    from dlrm_embedding_bag_b200 import optim as _optim

    return _optim


@pytest.mark.parametrize("default", [torch.float32, torch.float64, torch.bfloat16])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_state_under_another_default_type(optim, monkeypatch, default, bits):
    monkeypatch.setattr(optim, "_on", lambda t, name, index: None)  # CPU tensors in place of the device's
    params = [torch.zeros(300, dtype=torch.float32), torch.zeros((4, 5), dtype=torch.bfloat16)]
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        st = optim.adamw_state(params, bits=bits, master=True)
    finally:
        torch.set_default_dtype(before)
    f32 = torch.float32
    want = (f32, f32, None, None) if bits == 32 else (torch.float8_e4m3fn, torch.uint8, f32, f32)
    assert tuple(t if t is None else t.dtype for t in (st.m, st.v, st.m_scale, st.v_scale)) == want
    assert st.master.dtype == f32 and st.step.dtype == torch.int32
