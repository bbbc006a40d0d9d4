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


def test_empty_tensors_cost_no_more_than_others(optim, monkeypatch):
    """Several parameters without an address are no reason to compare each with all before it: a long
    list takes about as long with them (50 times as long when each was compared)."""
    import time

    monkeypatch.setattr(optim, "_on", lambda t, name, index: None)
    monkeypatch.setattr(optim, "_arena", lambda t, name, dtype, n, index: 0)
    seen = []
    monkeypatch.setattr(optim, "_call", lambda fn, name, index, args: seen.append(args))
    st = optim.AdamWState(torch.zeros(1), torch.zeros(1), torch.zeros(2, dtype=torch.int32))

    def fastest(params):
        took = []
        for _ in range(4):
            at = time.perf_counter()
            optim.adamw_step(params, params, st, lr=0.1)
            took.append(time.perf_counter() - at)
        return min(took)

    full = [torch.zeros(1) for _ in range(6000)]
    empty = [torch.zeros(0) for _ in range(3)]
    assert fastest(empty[:1] + full + empty[1:]) < 5 * fastest(full)
    assert len(seen) == 8
    for where in (1, 3000, 5999):
        twice = empty + full + full[where:where + 1]
        with pytest.raises(ValueError, match=r"params\[6003\] is there twice"):
            optim.adamw_step(twice, twice, st, lr=0.1)
