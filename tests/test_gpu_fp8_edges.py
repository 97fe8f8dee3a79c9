"""Edges of the block-scaled E4M3 operators on the GPU: inputs at the ends of their ranges, neighbours of the operands
in memory, streams, empty calls."""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    import nvfp4_weight_only_top_b200 as moe
    return torch, moe


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------------------ SwiGLU

FAR = [-60.0, -61.0, -75.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -100.0, -130.0, -177.0]
UPS = [1.0, 1e3, -1e3, 2.0 ** 40, 2.0 ** 99, 1e30, -2.0 ** 106, 3e38]


def _swiglu_against_64_bits(gu):
    """Codes from 2^-6 on are the nearest to the 64-bit products, but for products within 2^-44 of a step of a border
    between two codes (two computations in 64 bits differ by less); smaller codes are within one subnormal step of
    2^-9; scales within five steps and two roundings of 32 bits, 6 x 2^-23."""
    torch, moe = _torch()
    q, s = moe.moe_nvfp4_fp8_swiglu_quantize(gu)
    R, I = q.shape
    h = np.pad(fp8.swiglu(_np(gu)), ((0, 0), (0, -I % 128)))
    most = np.maximum(np.abs(h).reshape(R, -1, 128).max(2), 2.0 ** -100)
    p = (h * (448 / most).repeat(128, 1))[:, :I]
    got, want = _np(q), fp8.e4m3(p)
    _, e = np.frexp(np.abs(p))
    steps = np.abs(p) / np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    sure = (np.abs(p) >= 2.0 ** -6) & (np.abs(steps - np.floor(steps) - 0.5) > 2.0 ** -44)
    assert np.array_equal(got[sure], want[sure])
    assert (np.abs(got - want)[np.abs(p) < 2.0 ** -6] <= 2.0 ** -9).all()
    assert (np.abs(_np(s) - most / 448) <= 6 * 2.0 ** -23 * most / 448).all()


@pytest.mark.parametrize("I", [128, 144])
def test_swiglu_far_gates_alone(I):
    """Blocks of one gate so far below zero that 1 + e^-gate is at the end of f32 or past it, and one up."""
    torch, _ = _torch()
    gu = torch.tensor([[g] * I + [u] * I for g in FAR for u in UPS], device="cuda").to(torch.bfloat16)
    _swiglu_against_64_bits(gu)


@pytest.mark.parametrize("size", [1.0, 1e-12, 1e-25])
def test_swiglu_far_gates_among_ordinary_values(size):
    """One such value at every place of a block of ordinary ones (small ups make the block small)."""
    torch, _ = _torch()
    rng = np.random.default_rng(31)
    rows, I = len(FAR) * len(UPS), 272
    g = rng.standard_normal((rows, I)).astype(np.float32)
    u = (size * rng.standard_normal((rows, I))).astype(np.float32)
    for r in range(rows):
        at = (37 * r) % I
        g[r, at], u[r, at] = FAR[r // len(UPS)], UPS[r % len(UPS)]
    _swiglu_against_64_bits(torch.from_numpy(np.concatenate([g, u], 1)).cuda().to(torch.bfloat16))


def test_swiglu_zero_blocks_beside_far_gates():
    """Zero gates or zero ups give zero codes and the least scale; a far gate that cannot matter changes nothing."""
    torch, moe = _torch()
    gu = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    gu[1, 128:] = 1e30
    gu[2, :128] = -88.0
    gu[3, :128] = -300.0
    gu[3, 128:] = 1e3
    q, s = moe.moe_nvfp4_fp8_swiglu_quantize(gu)
    assert (_np(q) == 0).all() and (s == float(np.float32(2.0 ** -100) / np.float32(448))).all()
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    wq, ws = moe.moe_nvfp4_fp8_swiglu_quantize(x)
    x[:, 5] = -88.0
    q, s = moe.moe_nvfp4_fp8_swiglu_quantize(x)
    keep = [i for i in range(128) if i != 5]
    top = (_np(wq)[:, 5] != 448) & (_np(wq)[:, 5] != -448)      # (where the value replaced was not the largest)
    assert np.array_equal(_np(q)[top][:, keep], _np(wq)[top][:, keep]) and np.array_equal(_np(s)[top], _np(ws)[top])


# ------------------------------------------------------------------------------------------ no rows

def test_an_e4m3_layer_of_no_tokens():
    torch, moe = _torch()
    E, k, H, I = 8, 4, 256, 128
    bf = torch.bfloat16
    bgu, sgu = moe.moe_nvfp4_fp8_quantize_weights(torch.ones(E, 2 * I, H, dtype=bf, device="cuda"))
    bd, sd = moe.moe_nvfp4_fp8_quantize_weights(torch.ones(E, H, I, dtype=bf, device="cuda"))
    r = moe.moe_nvfp4_route_scored(torch.empty(0, E, device="cuda"), moe.make_router(), k)
    q, s = moe.moe_nvfp4_fp8_quantize(torch.empty(0, H, dtype=bf, device="cuda"), inv=r["inv"], k=k)
    gu = moe.moe_nvfp4_fp8_matmul(q, s, bgu, sgu, r["offsets"])
    h, hs = moe.moe_nvfp4_fp8_swiglu_quantize(gu)
    y = moe.moe_nvfp4_fp8_matmul(h, hs, bd, sd, r["offsets"], out_dtype=torch.float32)
    out = moe.moe_nvfp4_combine(y, r["w"], r["inv"], k)
    torch.cuda.synchronize()
    assert q.shape == (0, H) and s.shape == (0, 2) and gu.shape == (0, 2 * I) and out.shape == (0, H)
    assert moe.moe_nvfp4_device_status() == 0


# ------------------------------------------------------------------------------------------ products

def _codes(rng, *shape):
    """Every finite E4M3 encoding."""
    torch, _ = _torch()
    c = rng.integers(0, 256, shape, dtype=np.uint8)
    c[(c & 0x7F) == 0x7F] ^= 1
    return torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)


def _scales(rng, *shape):
    torch, _ = _torch()
    return torch.from_numpy(np.exp2(rng.uniform(-9, 3, shape)).astype(np.float32)).cuda()


def _before_nan(t):
    """The same values in a buffer that goes on with NaNs (codes 0x7F, or f32)."""
    torch, _ = _torch()
    flat = t.reshape(-1)
    if t.dtype == torch.float32:
        buf = torch.cat([flat, torch.full((1 << 14,), float("nan"), device="cuda")])
        return buf[:flat.numel()].view(t.shape)
    buf = torch.cat([flat.view(torch.uint8), torch.full((1 << 16,), 0x7F, dtype=torch.uint8, device="cuda")])
    return buf[:flat.numel()].view(t.dtype).view(t.shape)


def _check_product(a, sa, b, sb, off, out):
    """Against f64 products; f32 sums of 128 products (an addition loses at most 2^-23 of the magnitudes) and one
    multiply-add a block."""
    E, N, K = b.shape
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.start == r.stop:
            continue
        d = a[r].double() * sa[r].double().repeat_interleave(128, 1)[:, :K]
        w = b[e].double() * sb[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        tol = d.abs() @ w.abs().T * (132 + -(-K // 128)) * 2.0 ** -23
        assert ((out[r].double() - d @ w.T).abs() <= tol).all(), e


@pytest.mark.parametrize("tile", ["", "64", "128", "256", "64x2", "128x2"])
@pytest.mark.parametrize("M", [13, 33, 129, 257])
@pytest.mark.parametrize("N,K", [(40, 144), (264, 144), (264, 1296)])
def test_nothing_behind_the_operands_enters(M, N, K, tile, monkeypatch):
    """Codes and scales behind every operand are NaN, and so is what the call before left on the SMs: the row boxes past
    the last row, the weight boxes past the last expert's outputs and the inputs past K reach no output."""
    torch, moe = _torch()
    monkeypatch.setenv("MOE_NVFP4_FP8_TILE", tile)
    rng = np.random.default_rng(M + N + K)
    E = 2
    a, sa, b, sb = _codes(rng, M, K), _scales(rng, M, -(-K // 128)), _codes(rng, E, N, K), _scales(rng, E, -(-N // 128), -(-K // 128))
    for cut in (0, M // 3, M - 1):
        off = torch.tensor([0, cut, M], dtype=torch.int32, device="cuda")
        nan = [torch.full_like(t.view(torch.uint8), 0x7F).view(t.dtype) for t in (a, b)]
        left = moe.moe_nvfp4_fp8_matmul(nan[0], sa, nan[1], sb, off, out_dtype=torch.float32)
        assert torch.isnan(left).all()
        out = moe.moe_nvfp4_fp8_matmul(_before_nan(a), _before_nan(sa), _before_nan(b), _before_nan(sb), off,
                                       out_dtype=torch.float32)
        _check_product(a, sa, b, sb, off.tolist(), out)
    assert moe.moe_nvfp4_device_status() == 0


@pytest.mark.parametrize("M", [1, 8, 16, 200, 1500])
@pytest.mark.parametrize("E", [33, 256, 1024])
def test_products_over_many_experts(M, E):
    """Rows of a few of up to 1024 experts, the last one among them, and of all of them."""
    torch, moe = _torch()
    rng = np.random.default_rng(M + E)
    N, K = 136, 272
    a, sa, b, sb = _codes(rng, M, K), _scales(rng, M, 3), _codes(rng, E, N, K), _scales(rng, E, 2, 3)
    few = np.bincount(rng.choice([0, E // 2, E - 2, E - 1], M), minlength=E)
    last = np.bincount(np.full(M, E - 1), minlength=E)
    spread = np.bincount(rng.integers(0, E, M), minlength=E)
    for counts in (few, last, spread):
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        out = torch.full((M, N), float("nan"), device="cuda")
        moe.moe_nvfp4_fp8_matmul(a, sa, b, sb, torch.from_numpy(off).cuda(), out=out)
        _check_product(a, sa, b, sb, off, out)
    assert moe.moe_nvfp4_device_status() == 0
