"""The example asks every workspace with an error word (the norms' has none) that it used for errors
of the device."""
import os
import sys

import pytest
import torch

import mixture_experts_routed_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import expert_block  # noqa: E402

pytestmark = pytest.mark.gpu
ARGS = ["expert_block.py", "--d", "256", "--f", "128", "--E", "4", "--tokens", "64", "--decode", "2"]


def of_a_run(monkeypatch, error_of):
    """(workspaces by what allocated them, those asked for errors) of one run of main; error_of:
    the kind of workspace whose query answers with an error."""
    made, asked, kinds = {}, [], {}
    for name in ("alloc_workspace", "alloc_fp8_workspace", "alloc_router_loss_workspace",
                 "alloc_mx4_workspace"):
        def alloc(*a, call=getattr(moe, name), name=name, **kw):
            ws = call(*a, **kw)
            made.setdefault(name, []).append(ws)  # (kept, so that no address is used twice)
            kinds[ws.data_ptr()] = name
            return ws
        monkeypatch.setattr(moe, name, alloc)
    query = moe.get_device_error

    def get(ws, *a, **kw):
        asked.append(ws.data_ptr())
        st = query(ws, *a, **kw)
        return moe.MOE_ERR_TIMEOUT if kinds[ws.data_ptr()] == error_of else st

    monkeypatch.setattr(moe, "get_device_error", get)
    monkeypatch.setattr(sys, "argv", ARGS)
    expert_block.main()
    return made, asked


def test_all_of_them(cuda_ok, monkeypatch):
    made, asked = of_a_run(monkeypatch, None)
    for name, some in made.items():
        # (the training steps allocate theirs anew for each repeat: the last one's are asked)
        assert some[-1].data_ptr() in asked, name
    # decode, prefill 2, a step 2, a step with 8-bit experts 3
    assert len(set(asked)) == 8


@pytest.mark.parametrize("kind", ["alloc_fp8_workspace", "alloc_router_loss_workspace"])
def test_an_error_ends_the_run(cuda_ok, monkeypatch, kind):
    with pytest.raises(SystemExit):
        of_a_run(monkeypatch, kind)


def test_a_step_returns_its_workspaces(cuda_ok, monkeypatch):
    made = []
    for name in ("alloc_workspace", "alloc_fp8_workspace", "alloc_router_loss_workspace"):
        def alloc(*a, call=getattr(moe, name), **kw):
            made.append(call(*a, **kw))
            return made[-1]
        monkeypatch.setattr(moe, name, alloc)
    block = expert_block.ExpertBlock(256, 128, 4, 2)
    x = torch.randn((32, 256), device="cuda").bfloat16()
    dout, dnext = torch.randn_like(x), torch.randn((32, 256), device="cuda")
    state = torch.tensor([1, 0], dtype=torch.int64, device="cuda")
    for step in (lambda: block.train_step(x, dout, dnext),
                 lambda: block.train_step_fp8(x, dout, dnext, state)):
        made.clear()
        wss = step()[-1]
        assert {w.data_ptr() for w in wss} == {w.data_ptr() for w in made}
        for ws in wss:
            assert moe.get_device_error(ws) == moe.MOE_OK
