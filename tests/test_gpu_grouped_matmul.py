"""The ragged grouped products and their gradients against 64-bit products.

Bound of an element: the products of two 16-bit values are exact in fp32; a sum of n of
them in fp32, in any order and even with truncated additions, is off by at most
n * 2^-23 * sum |a||b|; storing rounds by u (2^-8 bf16, 2^-11 fp16, relative; fp16 also
2^-25 absolute where it is subnormal). Differences: the loss is linear in each operand, so
central differences of the 64-bit loss are exact up to its own rounding."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def offsets_of(counts, gap=0, first=0):
    off = [first]
    for c in counts:
        off.append(off[-1] + c + gap)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def make(counts, N, K, dtype, gap=0, first=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = first + sum(counts) + gap * len(counts)
    x = torch.randn(R, K, device="cuda", generator=g).to(dtype)
    dy = torch.randn(R, N, device="cuda", generator=g).to(dtype)
    w = (torch.randn(len(counts), N, K, device="cuda", generator=g) / 8).to(dtype)
    return x, dy, w, offsets_of(counts, gap, first)


def close(got, a, b, n):
    """|got - a @ b| within the bound, a and b 64-bit operands, n the sum's length."""
    ref, mag = a @ b, a.abs() @ b.abs()
    tol = U[got.dtype] * ref.abs() + (n * 2.0 ** -23) * mag + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), f"worst excess {(err - tol).max().item():.3g}"


def check(x, dy, w, off, counts, out_dtype, use_counts=False):
    N, K = w.shape[1:]
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda") if use_counts else None
    y = moe.moe_grouped_matmul(x, w, off, cnt, out_dtype=out_dtype)
    dx = moe.moe_grouped_matmul_dgrad(dy, w, off, cnt, out_dtype=out_dtype)
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off, cnt, out_dtype=out_dtype)
    torch.cuda.synchronize()
    for l, c in enumerate(counts):
        s = slice(int(off[l]), int(off[l]) + c)
        if c:
            close(y[s], x[s].double(), w[l].double().T, K)
            close(dx[s], dy[s].double(), w[l].double(), N)
            close(dw[l], dy[s].double().T, x[s].double(), c)
        else:
            assert not dw[l].any()
    return y, dx, dw


SHAPES = [
    ([1], 8, 8), ([3, 0, 1], 16, 24), ([64, 128, 256], 128, 64), ([0, 0, 5, 0], 136, 72),
    ([127, 129, 1, 255, 257, 16, 17, 15], 264, 200), ([700, 33], 256, 512), ([300], 520, 1000), ([1] * 20, 1400, 200),
    ([2048, 1], 384, 128), ([0], 64, 64), ([511, 513], 248, 2056),
]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("wide", [False, True])
def test_products_and_gradients(counts, N, K, dtype, wide):
    x, dy, w, off = make(counts, N, K, dtype, seed=N + K)
    check(x, dy, w, off, counts, torch.float32 if wide else None)


@pytest.mark.parametrize("gap,first", [(0, 5), (7, 0), (128, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_of_no_group_are_not_read_as_data_and_not_written(gap, first, dtype):
    counts = [3, 0, 130, 64, 257, 1]
    x, dy, w, off = make(counts, 72, 136, dtype, gap, first)
    inside = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    for l, c in enumerate(counts):
        inside[int(off[l]):int(off[l]) + c] = True
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(dtype)
    n = int((~inside).sum())
    x[~inside] = bad[torch.arange(n, device="cuda") % 3][:, None]
    dy[~inside] = bad[torch.arange(n, device="cuda") % 3][:, None]
    check(x, dy, w, off, counts, None, use_counts=True)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    y = torch.full((x.shape[0], 72), 7.0, dtype=dtype, device="cuda")
    dx = torch.full((x.shape[0], 136), 7.0, dtype=dtype, device="cuda")
    moe.moe_grouped_matmul(x, w, off, cnt, out=y)
    moe.moe_grouped_matmul_dgrad(dy, w, off, cnt, out=dx)
    assert (y[~inside] == 7).all() and (dx[~inside] == 7).all()


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_neighbouring_group_holds_nan(out_dtype):
    """A group's results do not see the rows of its neighbours, whose values may be anything."""
    counts = [37, 90, 41]
    x, dy, w, off = make(counts, 200, 136, torch.bfloat16, seed=3)
    s = slice(37, 127)
    x[s], dy[s], w[1] = float("nan"), float("inf"), float("nan")
    y = moe.moe_grouped_matmul(x, w, off, out_dtype=out_dtype)
    dx = moe.moe_grouped_matmul_dgrad(dy, w, off, out_dtype=out_dtype)
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off, out_dtype=out_dtype)
    for l, rows in ((0, slice(0, 37)), (2, slice(127, 168))):
        close(y[rows], x[rows].double(), w[l].double().T, 136)
        close(dx[rows], dy[rows].double(), w[l].double(), 200)
        close(dw[l], dy[rows].double().T, x[rows].double(), rows.stop - rows.start)


@pytest.mark.parametrize("counts,N,K", [([8192], 128, 264), ([3000, 5, 0, 4099], 256, 256), ([1025], 8, 8),
                                        ([0, 5001, 0], 136, 520), ([20000], 256, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("wide", [False, True])
def test_few_weights_and_many_rows(counts, N, K, dtype, wide):
    """The sums over rows are split into parts here, whatever the single groups' lengths."""
    assert moe.moe_grouped_matmul_wgrad_workspace_size(sum(counts), len(counts), N, K) > 0
    x, dy, w, off = make(counts, N, K, dtype, seed=N)
    check(x, dy, w, off, counts, torch.float32 if wide else None)


def test_offsets_past_the_rows_touch_nothing():
    x, dy, w, _ = make([40, 24], 64, 64, torch.bfloat16)
    guard = torch.full((64 + 64, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([-5, 30, 1 << 30], dtype=torch.int32, device="cuda")
    moe.moe_grouped_matmul(x, w, off, out=guard[:64])
    moe.moe_grouped_matmul_dgrad(dy, w, off, out=guard[:64])
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off)
    assert (guard[64:] == 3).all()
    close(dw[0], dy[:30].double().T, x[:30].double(), 30)
    close(dw[1], dy[30:].double().T, x[30:].double(), 34)


def test_no_rows():
    w = torch.ones(3, 64, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert moe.moe_grouped_matmul(x, w, off).shape == (0, 64)
    assert moe.moe_grouped_matmul_dgrad(x, w, off).shape == (0, 64)
    dw = torch.full((3, 64, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    assert not moe.moe_grouped_matmul_wgrad(x, x, off, out=dw).any()


def test_many_experts_skewed():
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 6, (1024,), generator=g)
    counts[17], counts[900] = 700, 333
    counts = counts.tolist()
    x, dy, w, off = make(counts, 64, 128, torch.bfloat16, seed=9)
    check(x, dy, w, off, counts, None)


def test_offsets_past_2_31_values():
    """Rows and weights whose element offsets do not fit 32 bits."""
    R, K, N = (1 << 31) // 2048 + 777, 2048, 16
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    x[-300:].normal_()
    dy[-300:].normal_()
    w = torch.randn(2, N, K, device="cuda").bfloat16()
    off = torch.tensor([0, R - 300, R], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_matmul(x, w, off)
    close(y[-300:], x[-300:].double(), w[1].double().T, K)
    dx = moe.moe_grouped_matmul_dgrad(dy, w, off)
    close(dx[-300:], dy[-300:].double(), w[1].double(), N)
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off)
    close(dw[1], dy[-300:].double().T, x[-300:].double(), 300)
    assert not dw[0].any()
    del x, dx, y
    E, N, K = 800, 1400, 2048                       # 2.3e9 weights
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[-1].normal_()
    x, dy = torch.randn(5, K, device="cuda").bfloat16(), torch.randn(5, N, device="cuda").bfloat16()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 5
    close(moe.moe_grouped_matmul(x, w, off), x.double(), w[-1].double().T, K)
    close(moe.moe_grouped_matmul_dgrad(dy, w, off), dy.double(), w[-1].double(), N)
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off, out=w)
    close(dw[-1], dy.double().T, x.double(), 5)
    assert not dw[-2].any()


def test_gradients_against_differences():
    counts = [5, 0, 9]
    x, dy, w, off = make(counts, 24, 40, torch.bfloat16, seed=11)
    dx = moe.moe_grouped_matmul_dgrad(dy, w, off, out_dtype=torch.float32)
    dw = moe.moe_grouped_matmul_wgrad(dy, x, off, out_dtype=torch.float32)

    def loss(x, w):
        return sum((dy[off[l]:off[l + 1]].double() * (x[off[l]:off[l + 1]] @ w[l].T)).sum() for l in range(3))
    xd, wd = x.double(), w.double()
    ux, uw = torch.randn_like(xd), torch.randn_like(wd)
    h = 1e-3
    num_x = (loss(xd + h * ux, wd) - loss(xd - h * ux, wd)) / (2 * h)
    num_w = (loss(xd, wd + h * uw) - loss(xd, wd - h * uw)) / (2 * h)
    assert abs(num_x - (dx.double() * ux).sum()) <= 40 * 2.0 ** -23 * (dx.double() * ux).abs().sum() + 1e-6
    assert abs(num_w - (dw.double() * uw).sum()) <= 40 * 2.0 ** -23 * (dw.double() * uw).abs().sum() + 1e-6


def test_same_result_every_call_and_on_another_stream():
    x, dy, w, off = make([100, 3, 400], 264, 520, torch.bfloat16, seed=2)
    first = [f(*a) for f, a in ((moe.moe_grouped_matmul, (x, w, off)), (moe.moe_grouped_matmul_dgrad, (dy, w, off)),
                                (moe.moe_grouped_matmul_wgrad, (dy, x, off)))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = [moe.moe_grouped_matmul(x, w, off, stream=s), moe.moe_grouped_matmul_dgrad(dy, w, off, stream=s),
             moe.moe_grouped_matmul_wgrad(dy, x, off, stream=s)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert moe.moe_device_error() == 0
