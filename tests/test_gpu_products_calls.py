"""The operators' calls beside what else a program does with the runtime: errors that other
calls left, other devices and their streams."""

import ctypes

import pytest
import torch

from precision_optimizer_step_amd import opt8, opt8_products as ops

pytestmark = pytest.mark.gpu

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def every_call():
    """Each operator's call, its descriptor and the tensors that it writes; what must live beside them."""
    g = torch.Generator().manual_seed(1)
    rows, d, f = 40, 64, 96

    def values(*shape):
        return torch.randn(*shape, generator=g).to(BF).cuda()
    x, wg, wu, h, gate, up, dh = (values(*s) for s in ((rows, d), (f, d), (f, d), (rows, f), (rows, f), (rows, f), (rows, f)))
    q, s = torch.empty(rows, d, dtype=torch.uint8, device="cuda").view(E4), torch.empty(1, rows, device="cuda")
    a, b = values(rows, d).to(E4), values(f, d).to(E4)
    sa, sb = torch.ones(1, rows, device="cuda"), torch.ones(1, 1, device="cuda")
    c = torch.empty(rows, f, dtype=BF, device="cuda")
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    return {
        "quantize": (ops.opt8_fp8_quantize, ops.make_fp8_quant(x, q, s), (q.view(torch.uint8), s)),
        "product": (ops.opt8_fp8_matmul, ops.make_fp8_product(a, sa, b, sb, c), (c,)),
        "gated": (ops.opt8_gated_ffn_forward, ops.make_gated_ffn(x, wg, wu, h), (h,)),
        "gated one row": (ops.opt8_gated_ffn_forward, ops.make_gated_ffn(x[:1], wg, wu, h[:1]), (h[:1],)),
        "gated backward": (ops.opt8_gated_ffn_backward,
                           ops.make_gated_ffn_grad(dh, x, wg, wu, gate, up, dx, dwg, dwu, work), (dx, dwg, dwu)),
    }, (x, wg, wu, gate, up, dh, a, sa, b, sb, work)


def runtime():
    """The HIP runtime that this process has loaded."""
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line)
    return ctypes.CDLL(path)


def test_an_error_that_another_call_left_is_not_the_launch_s():
    """A refused hipSetDevice leaves its error in the runtime until somebody reads it.  The
    operators queue their work and say so, and leave that error to its reader."""
    hip = runtime()
    calls, _keep = every_call()
    for name, (call, desc, outs) in calls.items():
        call(desc)
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        try:
            left = hip.hipSetDevice(9999)
            rc = call(desc, check=False)
            message = opt8.opt8_last_error()
            found = hip.hipGetLastError()
        finally:
            hip.hipGetLastError()
        torch.cuda.synchronize()
        assert left != 0
        assert (rc, message) == (opt8.OPT8_OK, ""), name
        assert found == left, name
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), name


def test_a_call_after_the_current_device_changed(monkeypatch):
    """Descriptors made on cuda:0 are refused while another device is current; nothing is queued."""
    calls, _keep = every_call()
    torch.cuda.synchronize()
    for name, (call, desc, outs) in calls.items():
        for t in outs:
            t.fill_(3)
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "current_device", lambda: 1)
            with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
                call(desc)
        torch.cuda.synchronize()
        assert all(bool((t == 3).all()) for t in outs), name
        assert call(desc) == opt8.OPT8_OK and call(desc, stream=torch.cuda.current_stream()) == opt8.OPT8_OK
        torch.cuda.synchronize()
        assert not all(bool((t == 3).all()) for t in outs), name
