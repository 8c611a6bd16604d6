"""Activations in 8 bits: every step but the rounding to e4m3 is exact, so codes and scale bytes are
compared bit for bit with the definition in 64 bits, and what comes back with code * scale."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def code_values():
    """The 256 e4m3 values in 64 bits (0x7f and 0xff: NaN)."""
    c = torch.arange(256)
    e, m = c >> 3 & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    v = torch.where(c > 127, -v, v)
    v[[127, 255]] = float("nan")
    return v


def reference(x):
    """(codes, scales) of x [M, K], by search: the nearest of the e4m3 values, ties to the even code."""
    M, K = x.shape
    G = -(-K // 16)
    p = torch.zeros(M, G * 16, dtype=torch.float64)
    p[:, :K] = x.double().cpu()
    p = p.view(M, G, 16)
    bad = ~torch.isfinite(p).all(2)
    top = torch.where(bad.unsqueeze(2), 0.0, p).abs().amax(2)
    byte = torch.ones(M, G, dtype=torch.int64)
    scales = torch.exp2(torch.arange(256).double() - 127)
    byte = torch.clamp(torch.searchsorted(scales * 448, top.contiguous()), min=1)  # the first scale with 448 * scale >= top
    v = torch.where(bad.unsqueeze(2), 0.0, p) / scales[byte].unsqueeze(2)
    grid = code_values()[:127]  # 0 .. 448, ascending
    hi = torch.searchsorted(grid, v.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = v.abs() - grid[lo], grid[hi] - v.abs()
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(torch.signbit(p), code + 128, code)
    code = torch.where(bad.unsqueeze(2), 127, code)
    byte = torch.where(bad, 255, byte)
    return code.view(M, -1)[:, :K].to(torch.uint8), byte.to(torch.uint8), bad


def same_codes(got, want, bad):
    K = got.shape[1]
    nan = torch.repeat_interleave(bad, 16, dim=1)[:, :K]
    got = got.cpu()
    assert ((got & 127)[nan] == 127).all()
    assert torch.equal(got[~nan], want[~nan])


def check(x):
    codes, scales = moe.moe_checkpoint_pack(x)
    wc, ws, bad = reference(x)
    assert torch.equal(scales.cpu(), ws)
    same_codes(codes, wc, bad)
    return codes, scales


def spread(M, K, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=g) * 10.0 ** (6 * torch.rand(M, 1, device="cuda", generator=g) - 3)
    x[torch.rand(M, K, device="cuda", generator=g) < 0.1] = 0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 15), (5, 17), (2, 31), (1, 2048), (257, 64), (33, 1111), (300, 48), (7, 1000),
                                 (1, 100_003), (1000, 8), (129, 24)])
def test_pack_and_unpack(M, K, dtype):
    x = spread(M, K, dtype, seed=M + K)
    codes, scales = check(x)
    for back in TYPES:
        y = moe.moe_checkpoint_unpack(codes, scales, back)
        v = code_values()[codes.cpu().long()] * torch.exp2(torch.repeat_interleave(scales.cpu().double(), 16, dim=1)[:, :K] - 127)
        top = torch.finfo(back).max
        assert torch.equal(y.cpu(), v.clamp(-top, top).to(back))
    # half a step of e4m3, relative, or of its smallest step under the scale
    y = moe.moe_checkpoint_unpack(codes, scales, torch.float32)
    step = torch.exp2(torch.repeat_interleave(scales.double(), 16, dim=1)[:, :K] - 127 - 10)
    assert ((y.double() - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, step)).all()
    again = moe.moe_checkpoint_pack(moe.moe_checkpoint_unpack(codes, scales, torch.float32))
    assert torch.equal(moe.moe_checkpoint_unpack(*again, torch.float32), y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [1, 16])
def test_every_16_bit_value(dtype, K):
    """Alone in its group, and with smaller ones beside it (subnormals, infinities and NaN among them)."""
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype).view(-1, 1)
    if K > 1:
        x = torch.cat([x] + [(x.float() * 2.0 ** -i * 0.77).to(dtype) for i in range(1, K)], 1).contiguous()
    codes, scales = check(x)
    y = moe.moe_checkpoint_unpack(codes, scales, dtype)
    bad = ~torch.isfinite(x.float()).all(1)
    assert y[bad].isnan().all() and torch.isfinite(y[~bad]).all()


def test_fp32_extremes():
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[big] * 16, [-big, 1e30] + [0.0] * 14, [1e-45] * 16, [2.0 ** -126, 2.0 ** -149] + [0.0] * 14, [448.0 * 2.0 ** -126] * 16,
                      [449.0 * 2.0 ** -126] * 16, [float("inf")] + [1.0] * 15, [1.0] * 15 + [-float("inf")], [float("nan")] + [big] * 15,
                      [-0.0] * 16, [448.0] * 16, [448.0 + 2 ** -15] * 16], device="cuda")
    codes, scales = check(x)
    y = moe.moe_checkpoint_unpack(codes, scales, torch.float32)
    assert torch.equal(y[0], x[0]) and y[1, 0] == -big       # 1.75 * 2^127 < big < 2^128: rounds up, comes back as the largest
    assert y[6:9].isnan().all() and torch.signbit(y[9]).all() and not y[9].any()


def test_ties_go_to_the_even_code():
    v = code_values()[:127]
    mid = ((v[1:] + v[:-1]) / 2).float()
    x = torch.cat([mid, -mid]).view(-1, 1).repeat(1, 16)
    x[:, 15] = 448.0  # the scale is 1
    check(x.cuda())


def test_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(1, 256).repeat(256, 1).contiguous()
    scales = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(256, 1).repeat(1, 16).contiguous()
    v = code_values()[None, :] * torch.exp2(torch.arange(256).double() - 127)[:, None]
    v[255] = float("nan")
    for dtype in TYPES:
        top = torch.finfo(dtype).max
        want = torch.where(v.isnan(), v, v.clamp(-top, top)).to(torch.float32).to(dtype)
        for c, s in ((codes, scales), (codes[:, :250].contiguous(), scales)):
            got = moe.moe_checkpoint_unpack(c, s, dtype).cpu()
            w = want[:, :c.shape[1]]
            assert torch.equal(got.isnan(), w.isnan())
            assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(w.float()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [64, 37])
def test_any_alignment_and_nothing_beside(dtype, K):
    M = 19
    x = spread(M, K, dtype, seed=K)
    want = moe.moe_checkpoint_pack(x)
    back = moe.moe_checkpoint_unpack(*want, dtype)
    G = want[1].shape[1]
    for shift in (1, 3, 8):
        flat = torch.full((M * K + 64,), 7.0, device="cuda").to(dtype)
        xs = flat[shift:shift + M * K].view(M, K)
        xs.copy_(x)
        cf = torch.full((M * K + 64,), 7, dtype=torch.uint8, device="cuda")
        sf = torch.full((M * G + 64,), 7, dtype=torch.uint8, device="cuda")
        c, s = cf[shift:shift + M * K].view(M, K), sf[shift:shift + M * G].view(M, G)
        moe.moe_checkpoint_pack(xs, codes=c, scales=s)
        assert torch.equal(c, want[0]) and torch.equal(s, want[1])
        flat.fill_(7.0)
        moe.moe_checkpoint_unpack(c, s, dtype, out=xs)
        assert torch.equal(xs, back)
        for buf, n in ((cf, M * K), (sf, M * G), (flat, M * K)):
            assert (buf[:shift] == 7).all() and (buf[shift + n:] == 7).all()


def test_empty_and_large():
    codes, scales = moe.moe_checkpoint_pack(torch.empty(0, 40, device="cuda"))
    assert codes.shape == (0, 40) and scales.shape == (0, 3)
    assert moe.moe_checkpoint_unpack(codes, scales, torch.float32).shape == (0, 40)
    for K in (4096, 4095):  # elements past 2^31
        M = (1 << 31) // K + 3
        x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
        x[-2:] = spread(2, K, torch.float16)
        codes, scales = moe.moe_checkpoint_pack(x)
        want = moe.moe_checkpoint_pack(x[-2:].clone())
        assert torch.equal(codes[-2:], want[0]) and torch.equal(scales[-2:], want[1]) and not codes[:-2].any()
        y = moe.moe_checkpoint_unpack(codes, scales, torch.float16)
        assert torch.equal(y[-2:], moe.moe_checkpoint_unpack(*want, torch.float16)) and not y[:-2].any()
        del x, y, codes, scales


def test_captured_and_on_another_stream():
    x = spread(50, 80, torch.bfloat16)
    want = [t.clone() for t in moe.moe_checkpoint_pack(x)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        codes, scales = moe.moe_checkpoint_pack(x)
        y = moe.moe_checkpoint_unpack(codes, scales, torch.bfloat16)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    z = moe.moe_checkpoint_unpack(codes, scales, torch.bfloat16, stream=s)
    s.synchronize()
    assert torch.equal(y, z)
