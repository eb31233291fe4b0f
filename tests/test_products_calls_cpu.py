"""The operators' calls without a GPU: a descriptor belongs to the device of its tensors, and so
does the stream that it is queued on; sizes up to the documented limits pass the checks."""

import os

import pytest
import torch

from precision_optimizer_step_amd import opt8, opt8_products as ops

E4, BF = torch.float8_e4m3fn, torch.bfloat16


class Stream:
    def __init__(self, index, handle=64):
        self.device = torch.device("cuda", index)
        self.cuda_stream = handle


@pytest.fixture
def calls(monkeypatch):
    """Descriptors as if their tensors were on cuda:1, and what reaches the library."""
    queued = []
    monkeypatch.setattr(ops, "_placed", lambda names, tensors: 1)
    monkeypatch.setattr(ops, "_fns", {n: (lambda desc, stream, n=n: queued.append((n, stream)) or 0) for n in ops._CALLS})
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    x, w, h = torch.zeros(4, 64, dtype=BF), torch.zeros(16, 64, dtype=BF), torch.zeros(4, 16, dtype=BF)
    q, b = torch.zeros(4, 64, dtype=torch.uint8).view(E4), torch.zeros(16, 64, dtype=torch.uint8).view(E4)
    s, sb = torch.zeros(1, 4), torch.zeros(1, 1)
    work = torch.zeros(1 << 16, dtype=torch.uint8)
    made = {
        "opt8_fp8_quantize": ops.make_fp8_quant(x, q, s),
        "opt8_fp8_matmul": ops.make_fp8_product(q, s, b, sb, h),
        "opt8_gated_ffn_forward": ops.make_gated_ffn(x, w, w, h),
        "opt8_gated_ffn_backward": ops.make_gated_ffn_grad(h, x, w, w, h, h, x, w, w, work),
    }
    return made, queued


@pytest.mark.parametrize("name", list(ops._CALLS))
def test_a_call_on_another_device_is_refused(calls, name, monkeypatch):
    made, queued = calls
    call = getattr(ops, name)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for stream in (None, Stream(1), 64):
        with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
            call(made[name], stream=stream)
    assert queued == []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="stream.*cuda:0"):
        call(made[name], stream=Stream(0))
    assert queued == []
    assert call(made[name]) == 0 and call(made[name], stream=Stream(1)) == 0 and call(made[name], stream=7) == 0
    assert queued == [(name, 101), (name, 64), (name, 7)]


def test_a_struct_filled_by_hand_has_no_device(calls):
    """Its addresses are the caller's business, as in C."""
    _, queued = calls
    assert ops.opt8_fp8_quantize(ops.opt8_fp8_quant(rows=0), stream=9) == 0
    assert queued == [("opt8_fp8_quantize", 9)]


@pytest.mark.parametrize("rows,f", [(1 << 17, (1 << 20) - 8), (1 << 22, 1 << 15), ((1 << 22) - 1, 1 << 15), (1 << 18, 1 << 18)])
def test_the_workspace_of_the_largest_gradients(rows, f):
    """Matrices of up to 2^37 elements are taken; the workspace, four bytes for each and more,
    is no matrix and is not held to that count."""
    if not os.path.exists(opt8.LIB_PATH):
        pytest.fail("libopt8.so is not built (run __graft_entry__.build())")
    if torch.cuda.is_available():
        pytest.skip("the addresses here are made up: checked where no GPU could follow them")
    names = ["dh", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up", "workspace"]
    apart = 1 << 42
    at = {n: apart * (i + 1) for i, n in enumerate(names)}
    need = ops.opt8_gated_ffn_workspace(rows, 8, f)
    assert rows * f <= 1 << 37 < need < apart
    kw = dict(rows=rows, d=8, f=f, ldx=8, ldw=8, lddh=f, ldg=f, lddx=8, lddw=8, type=ops.OPT8_TYPE_BF16)
    rc = ops.opt8_gated_ffn_backward(ops.opt8_gated_ffn_grad(workspace_bytes=need, **at, **kw), stream=0, check=False)
    assert rc in (opt8.OPT8_OK, opt8.OPT8_E_HIP), opt8.opt8_last_error()      # with no device the launch fails
    rc = ops.opt8_gated_ffn_backward(ops.opt8_gated_ffn_grad(workspace_bytes=need - 1, **at, **kw), stream=0, check=False)
    assert rc == opt8.OPT8_E_SIZE
    # its last bytes are checked against the other buffers like any output's
    at["x"] = at["workspace"] + need - 16
    rc = ops.opt8_gated_ffn_backward(ops.opt8_gated_ffn_grad(workspace_bytes=need, **at, **kw), stream=0, check=False)
    assert rc == opt8.OPT8_E_ALIAS
    at["x"] += 16
    rc = ops.opt8_gated_ffn_backward(ops.opt8_gated_ffn_grad(workspace_bytes=need, **at, **kw), stream=0, check=False)
    assert rc in (opt8.OPT8_OK, opt8.OPT8_E_HIP), opt8.opt8_last_error()
