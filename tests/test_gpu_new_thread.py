"""Each entry point as the first CUDA call of a new thread, which has no context yet (autograd's threads among them):
it makes the device's own current and gives what the main thread gets."""
import threading

import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu


def calls():
    """Name -> (call, its outputs), every tensor made beforehand."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def bf(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()

    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    R, N, K, E = 60, 64, 128, 2
    off = torch.tensor([0, 20, R], dtype=torch.int32, device="cuda")
    x, dy, w13, w2, w, pre = bf(R, K), bf(R, K), bf(E, 2 * N, K), bf(E, K, N), bf(E, N, K), bf(R, 2 * N)
    h, dn = bf(R, N), bf(R, N)
    codes, scale = new(R, K, dtype=torch.uint8), new(R, K // 16, dtype=torch.uint8)
    c2, s2 = moe.moe_checkpoint_pack(x)
    o = {"fwd": new(R, N), "dgrad": new(R, K), "wgrad": new(E, N, K), "h": new(R, N), "d": new(R, 2 * N), "again": new(R, N), "back": new(R, K)}
    dout, src = bf(20, K), torch.arange(R, dtype=torch.int32, device="cuda").view(20, 3).contiguous()
    weights, d_y, d_w = torch.rand(20, 3, device="cuda", generator=g), new(R, K), new(20, 3, dtype=torch.float32)
    a8, b8 = (torch.randint(0, 100, s, device="cuda", generator=g, dtype=torch.uint8) for s in ((128, 128), (1, 128, 128)))
    sa, sb = torch.rand(128, 1, device="cuda", generator=g), torch.rand(1, 1, 1, device="cuda", generator=g)
    block = torch.tensor([0, 128], dtype=torch.int32, device="cuda")
    gemm = new(128, 128)
    return {
        "grouped_matmul": (lambda: moe.moe_grouped_matmul(x, w, off, out=o["fwd"]), [o["fwd"]]),
        "grouped_matmul_dgrad": (lambda: moe.moe_grouped_matmul_dgrad(dn, w, off, out=o["dgrad"]), [o["dgrad"]]),
        "grouped_matmul_wgrad": (lambda: moe.moe_grouped_matmul_wgrad(h, x, off, out=o["wgrad"]), [o["wgrad"]]),
        "grouped_gated": (lambda: moe.moe_grouped_gated(x, w13, off, out=o["h"]), [o["h"]]),
        "grouped_gated_backward": (lambda: moe.moe_grouped_gated_backward(dy, w2, pre, off, d_pre=o["d"], h=o["again"]), [o["d"], o["again"]]),
        "checkpoint_pack": (lambda: moe.moe_checkpoint_pack(x, codes, scale), [codes, scale]),
        "checkpoint_unpack": (lambda: moe.moe_checkpoint_unpack(c2, s2, torch.bfloat16, o["back"]), [o["back"]]),
        "gather_weight_reduce_backward": (lambda: moe.moe_gather_weight_reduce_backward(dout, x, src, weights, d_y=d_y, d_topk_weights=d_w),
                                          [d_y, d_w]),
        "grouped_gemm_fp8": (lambda: moe.moe_grouped_gemm_fp8(a8, sa, b8, sb, block, moe.MOE_EPI_BF16, out=gemm), [gemm]),
    }


@pytest.mark.parametrize("name", ["grouped_matmul", "grouped_matmul_dgrad", "grouped_matmul_wgrad", "grouped_gated", "grouped_gated_backward",
                                  "checkpoint_pack", "checkpoint_unpack", "gather_weight_reduce_backward", "grouped_gemm_fp8"])
def test_first_call_of_a_thread(name):
    call, outs = calls()[name]
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    got = [v.clone() for v in outs]
    for v in outs:
        v.zero_()
    call()
    assert any(v.any() for v in got) and all(torch.equal(a, b) for a, b in zip(got, outs))
