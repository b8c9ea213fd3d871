"""A caller's workspace must lie apart from the operands of its call (host tensors stand in for device ones)."""
import pytest
import torch

from lossless_entropy_coded_ecf8_amd import adapters as A


def test_a_workspace_over_an_operand_is_refused():
    memory = torch.zeros(4096, dtype=torch.uint8)
    x = memory[1024:2048].view(torch.bfloat16).view(16, 32)
    cpu = torch.device("cpu")
    for ws in (memory[:1025], memory[2047:], memory[1500:1600], memory):
        with pytest.raises(ValueError, match="workspace overlaps x"):
            A._scratch(1, ws, cpu, None, [("out", None), ("x", x)])
    for ws in (memory[:1024], memory[2048:], memory[1500:1500]):
        assert A._scratch(1, ws, cpu, None, [("out", None), ("x", x)]) is ws


@pytest.mark.gpu
def test_entry_points_refuse_it():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_entropy_coded_ecf8_amd as E
    d = torch.device("cuda", 0)
    memory = torch.zeros(64 << 20, dtype=torch.uint8, device=d)
    T, K, N, R, L = 40, 8192, 8192, 16, 4
    at = 0

    def of(*shape, dtype=torch.bfloat16):
        nonlocal at
        n = torch.Size(shape).numel() * dtype.itemsize
        at = (at + 255) // 256 * 256
        t = memory[at:at + n].view(dtype).view(shape)
        at += n
        return t

    x, base, out, dy, dx = of(T, K), of(T, N), of(T, N), of(T, N), of(T, K)
    down, up, scaling, index = of(L, R, K), of(L, R, N), of(L, dtype=torch.float32), of(T, dtype=torch.int32)
    plan = E.AdapterPlan(index, L, workspace=of(1 << 16, dtype=torch.uint8))
    rest = memory[(at + 255) // 256 * 256:]
    for over in (x, base, out, down, up, index):
        ws = memory[over.data_ptr() - memory.data_ptr():]
        with pytest.raises(ValueError):
            E.adapter_add(base, x, down, up, scaling, index, out=out, workspace=ws)
    for over in (x, base, out, down, up, plan.workspace):
        with pytest.raises(ValueError):
            E.adapter_add(base, x, down, up, scaling, plan, out=out, workspace=memory[over.data_ptr() - memory.data_ptr():])
    for over in (x, dy, dx, down, up, plan.workspace):
        with pytest.raises(ValueError):
            E.adapter_grads(dy, x, down, up, scaling, plan, dx=dx, workspace=memory[over.data_ptr() - memory.data_ptr():])
    with pytest.raises(ValueError):
        E.AdapterPlan(index, L, workspace=memory)
    w, s = torch.zeros(8192, 256, dtype=torch.uint8, device=d), torch.ones((), device=d)
    with pytest.raises(ValueError):
        E.linear_fp8_input_grad(dy, w, s, workspace=memory)
    E.adapter_add(base, x, down, up, scaling, index, out=out, workspace=rest)
    E.adapter_add(base, x, down, up, scaling, plan, out=out, workspace=rest)
    E.adapter_grads(dy, x, down, up, scaling, plan, dx=dx, workspace=rest)
    E.linear_fp8_input_grad(dy, w, s, workspace=rest)
    torch.cuda.synchronize()
    assert bool((memory[:at][:T * K * 2] == 0).all()) and bool((out == 0).all()) and bool((dx == 0).all())
