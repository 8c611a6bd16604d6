"""Argument checks of the gated feed-forward product, the 8-bit activations and the weighted sum's backward
pass: each documented error is returned before any launch, and the binding refuses tensors of the wrong
type, shape or place. No GPU needed; made-up addresses are not tried where a kernel could be launched on them."""
import ctypes

import pytest
import torch

from test_train_abi import BF, FP, HF, INVALID, L, at  # noqa: F401
from test_train_abi_memory import ACCEPTED, no_gpu, off

NONE, BITS16, E4M3 = 0, 1, 2


def gated(L, x=at(1), R=64, w=at(2), El=4, N=64, K=64, offsets=at(3), counts=at(4), act=0, dt=BF, h=at(5), keep=NONE,  # noqa: F811
          pre=None, scale=None):
    return L.moe_grouped_gated(x, R, w, El, N, K, offsets, counts, act, dt, h, keep, pre, scale, None)


def backward(L, dy=at(1), R=64, w=at(2), El=4, N=64, K=64, offsets=at(3), counts=at(4), act=0, dt=BF, keep=BITS16, pre=at(6),  # noqa: F811
             scale=None, d=at(8), h=at(5)):
    return L.moe_grouped_gated_backward(dy, R, w, El, N, K, offsets, counts, act, dt, keep, pre, scale, d, h, None)


KEPT = dict(keep=BITS16, pre=at(6))
EIGHT = dict(keep=E4M3, pre=at(6), scale=at(7))


def test_gated_refusals(L):  # noqa: F811
    for fn in (gated, backward):
        assert fn(L, R=0) == 0
        for bad in (dict(El=0), dict(El=1025), dict(N=60), dict(N=0), dict(N=1 << 30), dict(K=4), dict(K=12), dict(R=-1), dict(R=1 << 31),
                    dict(dt=FP), dict(dt=7), dict(act=2), dict(act=-1), dict(offsets=None), dict(w=None),
                    dict(w=off(2, 8)), dict(h=off(5, 8)), dict(offsets=off(3, 2)), dict(counts=off(4, 1)),
                    dict(R=(1 << 31) - 1, N=1 << 24), dict(El=1024, N=(1 << 30) - 8, K=(1 << 31) - 8), dict(keep=3), dict(keep=-1),
                    {**EIGHT, "N": 24}, {**EIGHT, "scale": None}, {**EIGHT, "pre": off(6, 8)}, {**KEPT, "pre": None}, {**KEPT, "scale": at(7)}):
            assert fn(L, **bad) == INVALID, (fn, bad)
    for bad in (dict(x=None), dict(h=None), dict(x=off(1, 8)), dict(pre=at(6)), dict(scale=at(7))):
        assert gated(L, **bad) == INVALID, bad
    for bad in (dict(dy=None), dict(d=None), dict(pre=None), dict(keep=NONE), dict(keep=NONE, pre=None), dict(dy=off(1, 8)), dict(d=off(8, 8))):
        assert backward(L, **bad) == INVALID, bad


@no_gpu
def test_gated_overlaps(L):  # noqa: F811
    for more in ({}, KEPT, EIGHT):
        assert gated(L, **more) in ACCEPTED and gated(L, counts=None, **more) in ACCEPTED
        for mib in (1, 2, 3, 4):
            assert gated(L, **{**more, "h": at(mib)}) == INVALID
    for more in (KEPT, EIGHT):
        for mib in (1, 2, 3, 4, 5):
            assert gated(L, **{**more, "pre": at(mib)}) == INVALID
    for mib in (1, 2, 3, 4, 5, 6):
        assert gated(L, **{**EIGHT, "scale": at(mib)}) == INVALID
    assert gated(L, **{**EIGHT, "scale": off(7, 3)}) in ACCEPTED       # bytes: aligned to nothing
    assert gated(L, **{**KEPT, "pre": off(5, 64 * 64 * 2)}) in ACCEPTED  # right behind h
    assert backward(L) in ACCEPTED and backward(L, h=None) in ACCEPTED and backward(L, **EIGHT) in ACCEPTED
    assert backward(L, d=at(6)) in ACCEPTED                            # the 16-bit values themselves
    for bad in (dict(d=off(6, 16)), {**EIGHT, "d": at(6)}, {**EIGHT, "d": at(7)}, dict(d=at(5)), dict(h=at(6)), dict(h=at(6), d=at(6)),
                {**EIGHT, "h": at(7)}):
        assert backward(L, **bad) == INVALID, bad
    for mib in (1, 2, 3, 4):
        assert backward(L, d=at(mib)) == INVALID and backward(L, h=at(mib)) == INVALID


def test_checkpoint_refusals(L):  # noqa: F811
    def pack(x=at(1), M=4, K=64, dt=BF, c=at(2), s=at(3)):
        return L.moe_checkpoint_pack(x, M, K, dt, c, s, None)

    def unpack(x=at(1), M=4, K=64, dt=BF, c=at(2), s=at(3)):
        return L.moe_checkpoint_unpack(c, s, M, K, dt, x, None)
    for fn in (pack, unpack):
        assert fn(M=0) == 0 and fn(M=0, x=None, c=None, s=None) == 0
        for bad in (dict(M=-1), dict(K=0), dict(K=(1 << 30) + 1), dict(dt=3), dict(dt=-1), dict(x=None), dict(c=None), dict(s=None),
                    dict(M=1 << 60), dict(M=1 << 40, K=1 << 8), dict(x=off(1, 1)), dict(x=off(1, 2), dt=FP), dict(c=off(1, 64)), dict(s=off(1, 64))):
            assert fn(**bad) == INVALID, bad
    assert pack(s=off(2, 64)) == INVALID


@no_gpu
def test_checkpoint_calls_that_are_taken(L):  # noqa: F811
    for dt, z in ((BF, 2), (HF, 2), (FP, 4)):
        for x in (at(1), off(1, z)):
            assert L.moe_checkpoint_pack(x, 4, 63, dt, off(2, 1), off(3, 1), None) in ACCEPTED
            assert L.moe_checkpoint_unpack(off(2, 1), off(2, 1), 4, 63, dt, x, None) in ACCEPTED  # both are only read


def combine(L, dout=at(1), y=at(2), rows=64, s=at(3), w=at(4), M=16, topk=4, K=128, unit=0, d=at(5), dw=at(6)):  # noqa: F811
    return L.moe_gather_weight_reduce_backward(dout, y, rows, s, w, M, topk, K, unit, d, dw, None)


def test_gather_backward_refusals(L):  # noqa: F811
    assert combine(L, M=0) == 0
    for bad in (dict(M=-1), dict(topk=0), dict(topk=33), dict(K=0), dict(K=64), dict(K=130), dict(K=(1 << 30) + 128), dict(rows=-1), dict(rows=1 << 31),
                dict(M=1 << 30), dict(dout=None), dict(y=None), dict(s=None), dict(w=None), dict(d=None), dict(unit=1),
                dict(dout=off(1, 8)), dict(y=off(2, 8)), dict(d=off(5, 8)), dict(s=off(3, 2)), dict(w=off(4, 2)), dict(dw=off(6, 2)),
                dict(d=at(1)), dict(d=at(2)), dict(d=at(3)), dict(d=at(4)), dict(dw=at(1)), dict(dw=at(2)), dict(dw=at(3)), dict(dw=at(4)),
                dict(dw=at(5))):
        assert combine(L, **bad) == INVALID, bad


@no_gpu
def test_gather_backward_calls_that_are_taken(L):  # noqa: F811
    for good in ({}, dict(dw=None), dict(dw=None, y=None), dict(unit=1, dw=None), dict(unit=1, dw=None, w=None), dict(rows=0, y=None, d=None)):
        assert combine(L, **good) in ACCEPTED, good


def test_binding_refusals(L):  # noqa: F811
    import moe_expert_layer_count_gb300 as moe
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    z = lambda *s, d=bf: torch.zeros(*s, dtype=d)  # noqa: E731
    o = z(3, d=i32)
    x, w13, w2, pre = z(4, 16), z(2, 32, 16), z(2, 16, 16), z(4, 32)
    codes, scale = z(4, 32, d=u8), z(4, 2, d=u8)
    fw, bw = moe.moe_grouped_gated, moe.moe_grouped_gated_backward
    for call in (lambda: fw(x, w13, o), lambda: bw(x, w2, pre, o),                       # host tensors
                 lambda: fw(z(4, 8), w13, o), lambda: fw(x, z(2, 31, 16), o), lambda: fw(x, w13, z(2, d=i32)),
                 lambda: fw(x.half(), w13, o), lambda: fw(x, w13, o, pre=pre), lambda: fw(x, w13, o, pre_scale=scale),
                 lambda: fw(x, w13, o, keep=moe.MOE_KEEP_16BIT, pre=codes), lambda: fw(x, w13, o, keep=moe.MOE_KEEP_E4M3, pre=pre),
                 lambda: fw(x, w13, o, keep=moe.MOE_KEEP_16BIT, pre=pre, pre_scale=scale),
                 lambda: fw(x, w13, o, out=z(4, 32)), lambda: bw(z(4, 8), w2, pre, o), lambda: bw(x, w2, codes, o),
                 lambda: bw(x, w2, pre, o, pre_scale=scale), lambda: bw(x, w2, codes, o, pre_scale=z(4, 4, d=u8)),
                 lambda: bw(x, w2, pre, o, h=z(4, 16), want_h=False), lambda: bw(x, w2, pre, o, d_pre=z(4, 16)),
                 lambda: bw(x, w2, pre, o, z(3, d=i32)),
                 lambda: moe.moe_checkpoint_pack(x), lambda: moe.moe_checkpoint_pack(x, codes=z(4, 16)),
                 lambda: moe.moe_checkpoint_pack(x, scales=z(4, 2, d=u8)),
                 lambda: moe.moe_checkpoint_unpack(codes, z(4, 1, d=u8), bf), lambda: moe.moe_checkpoint_unpack(codes, scale, bf, out=x),
                 lambda: moe.moe_checkpoint_unpack(codes, scale, bf)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fw(x.float(), w13.float(), o), lambda: bw(x.float(), w2.float(), pre.float(), o),
                 lambda: moe.moe_checkpoint_pack(x.double())):
        with pytest.raises(TypeError):
            call()
    g = moe.moe_gather_weight_reduce_backward
    d, y, s, w = z(4, 128), z(8, 128), z(4, 2, d=i32), z(4, 2, d=f32)
    for call in (lambda: g(d, y, s, w), lambda: g(z(5, 128), y, s, w), lambda: g(d, y, s.long(), w), lambda: g(d, y, s, z(4, 3, d=f32)),
                 lambda: g(d, y, s, w, d_y=z(7, 128)), lambda: g(d, y, s, w, True, d_topk_weights=w),
                 lambda: g(d, y, s, w, d_topk_weights=w, want_weights=False), lambda: g(d, y.half(), s, w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        g(d.float(), y, s, w)


def test_tensors_of_another_device_are_refused(L, monkeypatch):  # noqa: F811
    import types

    import moe_expert_layer_count_gb300 as moe

    def fake(i):
        return types.SimpleNamespace(get_device=lambda: i, device=f"cuda:{i}", shape=(4,), dtype=torch.int32, is_contiguous=lambda: True,
                                     data_ptr=lambda: 64 + i)
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    assert moe._here(fake(0)) == 0 and moe._take(fake(0), (4,), torch.int32, 0, "t") == 64
    for bad in (fake(1), fake(-1)):
        with pytest.raises(ValueError):
            moe._here(bad)
        with pytest.raises(ValueError):
            moe._take(bad, (4,), torch.int32, 0, "t")
