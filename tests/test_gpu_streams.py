"""Calls on a stream of the caller's: their outputs' memory is that stream's."""
import numpy as np
import pytest

import moe_inputs
from gpu_helpers import bf16_tensor, device_bank

pytestmark = pytest.mark.gpu

E, H, I, T, k = 16, 256, 256, 8, 2


def _setup():
    import torch
    import nvfp4_weight_only_top_b200 as moe
    cfg = moe_inputs.LayerConfig("streams", E, k, H, I, T, seed=5)
    buf, bank = device_bank(cfg)
    x, lg = bf16_tensor(moe_inputs.make_x(cfg)), torch.from_numpy(moe_inputs.make_logits(cfg)).cuda()
    router = moe.make_router(groups=4, top_groups=2)
    w = torch.randn(E, 2 * I, H, device="cuda").to(torch.bfloat16)
    route = moe.moe_nvfp4_route(lg, k)
    rows = moe.moe_nvfp4_gather_rows(x, route["perm"], k)
    ids = torch.sort(route["ids"].view(-1)).values
    y = moe.moe_nvfp4_experts(rows, ids, bank)
    q, s = moe.moe_nvfp4_fp8_quantize(x)
    b, sb = moe.moe_nvfp4_fp8_quantize_weights(w)
    off = torch.tensor([0] * E + [T], dtype=torch.int32, device="cuda")
    g, u, d = (torch.randn(2, *n, device="cuda").to(torch.bfloat16) for n in ((I, H), (I, H), (H, I)))
    act = torch.ones(E, 2, device="cuda")
    calls = dict(
        forward=lambda st: moe.moe_nvfp4_forward(x, lg, bank, k, stream=st),
        forward_ex=lambda st: moe.moe_nvfp4_forward_ex(x, lg, bank, k, stream=st),
        forward_noalloc=lambda st: moe.moe_nvfp4_forward_noalloc(x, lg, bank, k, stream=st),
        forward_w4a4=lambda st: moe.moe_nvfp4_forward_w4a4(x, lg, bank, act, k, stream=st),
        forward_scored=lambda st: moe.moe_nvfp4_forward_scored(x, lg, bank, router, k, stream=st),
        route=lambda st: list(moe.moe_nvfp4_route(lg, k, stream=st).values()),
        route_scored=lambda st: list(moe.moe_nvfp4_route_scored(lg, router, k, stream=st).values()),
        experts=lambda st: moe.moe_nvfp4_experts(rows, ids, bank, stream=st),
        gather_rows=lambda st: moe.moe_nvfp4_gather_rows(x, route["perm"], k, stream=st),
        combine=lambda st: moe.moe_nvfp4_combine(y, route["w"], route["inv"], k, stream=st),
        ep_plan=lambda st: moe.moe_nvfp4_ep_plan(route["counts"].view(1, E), 0, T * k, stream=st),
        encode_bank=lambda st: moe.encode_bank(g, u, d, stream=st)[0],
        fp8_quantize=lambda st: moe.moe_nvfp4_fp8_quantize(x, inv=route["inv"], k=k, stream=st),
        fp8_quantize_weights=lambda st: moe.moe_nvfp4_fp8_quantize_weights(w, stream=st),
        fp8_swiglu_quantize=lambda st: moe.moe_nvfp4_fp8_swiglu_quantize(x, stream=st),
        fp8_matmul=lambda st: moe.moe_nvfp4_fp8_matmul(q, s, b, sb, off, stream=st),
    )
    return torch, moe, calls, (buf, bank)


def _tensors(out):
    return list(out) if isinstance(out, (list, tuple)) else [out]


def test_outputs_are_the_streams():
    torch, moe, calls, _keep = _setup()
    want = {n: [t.clone() for t in _tensors(f(None))] for n, f in calls.items()}
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for name, f in calls.items():
        for given in (st, torch.cuda.ExternalStream(st.cuda_stream)):
            outs = _tensors(f(given))
            st.synchronize()
            for t, w in zip(outs, want[name]):
                if t.numel() == 0:
                    continue
                home = [seg["stream"] for seg in torch.cuda.memory_snapshot()
                        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]]
                assert home == [st.cuda_stream], name
                assert torch.equal(t.view(torch.uint8), w.view(torch.uint8)), name
            del outs
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert moe.moe_nvfp4_device_status() == 0


def test_outputs_dropped_while_the_stream_runs():
    """An output read on its stream and dropped at once: what the current stream allocates then is other memory."""
    torch, moe, calls, _keep = _setup()
    f = calls["route_scored"]
    want = sum(float(t.double().sum()) for t in f(None))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        total = torch.zeros((), dtype=torch.float64, device="cuda")
    for _ in range(200):
        outs = f(st)
        sizes = [(t.numel(), t.dtype) for t in outs]
        with torch.cuda.stream(st):
            for t in outs:
                total += t.double().sum()
        del outs, t
        for n, dtype in sizes:
            torch.full((n,), 99, dtype=dtype, device="cuda")
    st.synchronize()
    assert np.isclose(float(total), 200 * want, rtol=1e-12)


def test_a_refused_call_leaves_the_current_stream():
    torch, moe, calls, _keep = _setup()
    st, home = torch.cuda.Stream(), torch.cuda.Stream()
    lg = torch.zeros(2, E, device="cuda")
    with torch.cuda.stream(home):
        with pytest.raises(ValueError):
            moe.moe_nvfp4_route_scored(lg, moe.make_router(), 40, stream=st)
        with pytest.raises(moe.MoeError):
            moe.moe_nvfp4_route(lg, 40, stream=st)
        assert torch.cuda.current_stream() == home
        calls["route"](st)
        assert torch.cuda.current_stream() == home
    torch.cuda.synchronize()


def test_given_outputs_are_written_on_the_stream():
    """Outputs of the caller's: the call is the stream's, in order behind the work that is on it."""
    torch, moe, _calls, _keep = _setup()
    st = torch.cuda.Stream()
    x = torch.zeros(64, 1024, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(64, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(64, 8, device="cuda")
    y = torch.empty(64, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for v in (1.0, 2.0, 3.0):
            torch.cuda._sleep(2_000_000)
            x.fill_(v)
    moe.moe_nvfp4_fp8_quantize(x, q=q, scales=s, stream=st)
    with torch.cuda.stream(st):
        y.copy_(q)
    st.synchronize()
    assert (s == torch.tensor(3.0) / 448).all() and (y.float() == 448).all()
