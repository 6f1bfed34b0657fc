"""Block-scaled e4m3 quantisation, grouped product and expert FFN on the GPU
against 64-bit references (fp8_reference.py)."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import mixture_experts_layer_53_b200 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_layer_53_b200 import build
    build.build()
    M.library()
    assert torch.cuda.is_available()


def np64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def offsets_of(lengths, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


def checked(got, want, bound):
    """got within bound of want, element by element (NaN never is)."""
    bad = ~(np.abs(np64(got) - want) <= bound + 1e-300)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.max(np.abs(np64(got) - want) / np.maximum(bound, 1e-300))))


# --------------------------------------------------------------- quantisers


def _rows_input(rows, cols, dtype, seed):
    x = torch.randn((rows, cols), generator=gen(seed), device=DEV)
    x *= torch.exp(8 * torch.randn((rows, 1), generator=gen(seed + 1), device=DEV))
    if rows > 2:
        x[1] = 0                                  # a row of zeros
        x[2, ::3] *= 1e-30                        # values far below the block's largest
    if rows > 4:
        x[3] = 448.0                              # exactly at the largest value
        x[4] = torch.nextafter(torch.tensor(448.0, device=DEV), torch.tensor(1e9, device=DEV))
    return x.to(dtype)


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (7, 112), (8, 1024), (9, 1040), (65, 2064), (33, 7168)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_rows(rows, cols, dtype):
    x = _rows_input(rows, cols, dtype, rows + cols)
    q, s = M.moe_quantize_rows(x)
    wq, ws = R.quantize_rows(np64(x))
    assert q.dtype == E4 and q.shape == x.shape and s.shape == (-(-cols // 128), rows)
    assert np.array_equal(np64(s), ws)
    assert np.array_equal(np64(q), wq)


@pytest.mark.parametrize("E,rows,cols", [(1, 16, 16), (2, 128, 128), (3, 144, 400), (2, 1040, 272), (5, 96, 1152)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_weights(E, rows, cols, transpose, dtype):
    W = torch.randn((E, rows, cols), generator=gen(E + rows), device=DEV)
    W *= torch.exp(3 * torch.randn((E, rows, 1), generator=gen(5), device=DEV))
    W[0, :16] = 0
    W = W.to(dtype)
    q, s = M.moe_quantize_weights(W, transpose=transpose)
    wq, ws = R.quantize_weights(np64(W), transpose)
    assert np.array_equal(np64(s), ws)
    assert np.array_equal(np64(q), wq)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_blocks_that_are_not_finite(bad, dtype):
    x = torch.randn((5, 400), generator=gen(1), device=DEV).to(dtype)
    want, ws = M.moe_quantize_rows(x)
    x[2, 130] = bad
    q, s = M.moe_quantize_rows(x)
    hit = torch.zeros((5, 400), dtype=torch.bool, device=DEV)
    hit[2, 128:256] = True
    assert torch.isnan(q.float()[hit]).all() and torch.isnan(s[1, 2])
    assert torch.equal(q.float()[~hit], want.float()[~hit])
    s[1, 2] = ws[1, 2]
    assert torch.equal(s, ws)
    W = torch.randn((2, 256, 272), generator=gen(2), device=DEV).to(dtype)
    W[1, 200, 271] = bad
    for t in (False, True):
        q, s = M.moe_quantize_weights(W, transpose=t)
        v = q.float().transpose(1, 2) if t else q.float()
        v, s = v.cpu(), (s.transpose(1, 2) if t else s).cpu()
        assert torch.isnan(v[1, 128:, 256:]).all() and torch.isnan(s[1, 1, 2])
        assert not torch.isnan(v[0]).any() and not torch.isnan(v[1, :128]).any() and not torch.isnan(v[1, :, :256]).any()


def test_largest_and_smallest_values():
    for dtype in (BF, F32):
        top = torch.finfo(dtype).max
        tiny = 2.0 ** -133 if dtype == BF else 2.0 ** -149
        x = torch.tensor([[top] * 16, [tiny] * 16, [0.0] * 16, [-top, tiny] * 8], dtype=dtype, device=DEV)
        q, s = M.moe_quantize_rows(x)
        wq, ws = R.quantize_rows(np64(x))
        assert np.array_equal(np64(q), wq) and np.array_equal(np64(s), ws)


def test_empty_rows():
    q, s = M.moe_quantize_rows(torch.empty((0, 256), dtype=BF, device=DEV))
    assert q.shape == (0, 256) and s.shape == (2, 0)


# ------------------------------------------------------------------ product


def _operands(lengths, n, k, seed, first=0, behind=0, free_scales=False):
    rows, E = first + sum(lengths) + behind, len(lengths)
    a = M.moe_quantize_rows(torch.randn((rows, k), generator=gen(seed), device=DEV).to(BF))
    w = M.moe_quantize_weights(torch.randn((E, n, k), generator=gen(seed + 1), device=DEV).mul_(0.05).to(BF))
    if free_scales:  # a checkpoint's: any fp32 numbers
        a = a[0], a[1] * torch.exp(torch.randn(a[1].shape, generator=gen(seed + 2), device=DEV))
        w = w[0], w[1] * torch.exp(torch.randn(w[1].shape, generator=gen(seed + 3), device=DEV))
    return a, w, offsets_of(lengths, first)


def _values(a, w):
    return R.row_values(np64(a[0]), np64(a[1])), R.weight_values(np64(w[0]), np64(w[1]))


PRODUCTS = {
    "one_row": ([1], 16, 16),
    "one_row_each": ([1] * 8, 272, 400),
    "short_k": ([5, 0, 130], 256, 48),
    "tile_edges": ([128, 129, 127, 0, 256], 384, 256),
    "odd": ([3, 77, 0, 0, 201, 1], 1040, 720),
    "long_k": ([2, 0, 40], 144, 4112),
    "one_expert": ([700], 528, 640),
    "many_experts": ([i % 5 for i in range(256)], 128, 272),
    "long_slices": ([256, 255, 257, 1000], 1040, 720),
    "wide": ([500, 241, 479, 700], 2560, 400),
    "tiny": ([2, 0, 5, 1, 1, 16, 17, 33], 2576, 272),
    "tiny_but_one": ([100] + [0] * 14 + [1], 528, 400),
    "split2": ([1, 0, 3, 0, 33, 1], 272, 2064),
    "split8": ([3], 160, 8208),
    "few": ([16, 112, 113, 0, 47], 272, 656),
    "many_tiles": ([300, 4, 500, 0, 900, 129, 10, 250], 1552, 384),
}


@pytest.mark.parametrize("name", sorted(PRODUCTS))
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("free_scales", [False, True])
def test_product(name, out, free_scales):
    lengths, n, k = PRODUCTS[name]
    a, w, off = _operands(lengths, n, k, seed=len(name), free_scales=free_scales)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = M.moe_expert_matmul_fp8(a, off, w, out_dtype=out, any_scales=free_scales, status=status)
    want, bound = R.product(*_values(a, w), off.cpu().numpy())
    checked(y, want, bound + (R.UBF * (np.abs(want) + bound) if out == BF else 0))
    assert int(status) == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("free_scales", [False, True])
def test_rows_outside_every_slice_are_left(out, free_scales):
    a, w, off = _operands([10, 0, 150], 144, 272, seed=3, first=7, behind=40)
    y = torch.full((207, 144), 7.0, dtype=out, device=DEV)
    M.moe_expert_matmul_fp8(a, off, w, out_dtype=out, out=y, any_scales=free_scales)
    assert (y[:7] == 7).all() and (y[167:] == 7).all()
    want, bound = R.product(*_values(a, w), off.cpu().numpy())
    checked(y[7:167], want[7:167], (bound + (R.UBF * (np.abs(want) + bound) if out == BF else 0))[7:167])


def test_scales_of_many_sizes():
    """Powers of two over 2^-100 .. 2^20 that differ from block to block and row to row, products near 1."""
    a, w, off = _operands([200, 9, 330], 400, 1168, seed=21)
    e = torch.randint(-100, 20, (1, a[1].shape[1]), generator=gen(1), device=DEV)
    f = torch.randint(-6, 6, a[1].shape, generator=gen(2), device=DEV)
    a = a[0], a[1] * torch.exp2((e + f).float())
    w = w[0], w[1] * torch.exp2(torch.randint(-8, 8, w[1].shape, generator=gen(3), device=DEV).float())
    want, bound = R.product(*_values(a, w), off.cpu().numpy())
    for free in (False, True):
        checked(M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32, any_scales=free), want, bound)


# (power of two of a's scales, of w's; q's values of a in units of 2^-9, or None: as quantised)
BEYOND = {"underflow": (-112, -10, None), "far_underflow": (-112, -18, None), "overflow": (80, 50, 3), "zero_blocks": (100, 60, 0)}


@pytest.mark.parametrize("name", sorted(BEYOND))
@pytest.mark.parametrize("free_scales", [False, True])
def test_scales_whose_product_leaves_fp32(name, free_scales):
    """Two scales' product below fp32's normal numbers or above its largest, the result inside: the result counts."""
    ea, ew, small = BEYOND[name]
    a, w, off = _operands([70, 0, 200], 272, 400, seed=31, free_scales=free_scales)
    if small is not None:  # few bits, far below the scale: the sum of a block times its scales is finite
        q = torch.randint(-small, small + 1, a[0].shape, generator=gen(4), device=DEV).float() * 2.0 ** -9
        a = q.to(E4), torch.ones_like(a[1]) * (1.37 if free_scales else 1.0)
        v = torch.randint(-3, 4, w[0].shape, generator=gen(5), device=DEV).float() * 2.0 ** -9
        w = v.to(E4), torch.ones_like(w[1]) * (1.71 if free_scales else 1.0)
    a, w = (a[0], a[1] * 2.0 ** ea), (w[0], w[1] * 2.0 ** ew)
    if small is not None:
        big = a[1].min().double() * w[1].min().double()
        assert big > torch.finfo(F32).max
    else:
        assert float(a[1].max().double() * w[1].max().double()) < torch.finfo(F32).tiny
    want, bound = R.product(*_values(a, w), off.cpu().numpy())
    assert np.abs(want).max() < torch.finfo(F32).max
    y = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32, any_scales=free_scales)
    checked(y, want, bound + 2.0 ** -149 * (128 + 8))  # a step of fp32's subnormal numbers for each addition


def test_a_block_scale_of_zero_is_a_block_of_zeros():
    """A checkpoint may hold 0 as the scale of a block without values; beside a large scale it stays 0."""
    a, w, off = _operands([40, 100], 272, 400, seed=33, free_scales=True)
    a = a[0], a[1] * 2.0 ** 60
    a[0].view(torch.uint8)[7] = 0
    a[1][:, 7] = 2.0 ** -126   # a row of zeros, as the quantiser leaves it
    w[1][:, 1, 2] = 0.0
    want, bound = R.product(*_values(a, w), off.cpu().numpy())
    checked(M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32, any_scales=True), want, bound)


def test_an_infinite_scale_is_not_passed_over():
    """Values times infinity are infinite or NaN, zeros NaN: never an ordinary number."""
    a, w, off = _operands([40, 100], 272, 400, seed=34, free_scales=True)
    clean = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32, any_scales=True)
    a[0].view(torch.uint8)[7] = 0                      # rows of zeros, with an infinite scale and with the quantiser's
    a[0].view(torch.uint8)[9] = 0
    a[1][:, 9] = 2.0 ** -126
    a[1][1, 7], a[1][2, 50] = float("inf"), -float("inf")
    y = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32, any_scales=True)
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[50]).any() and not y[9].any()
    keep = torch.ones(140, dtype=torch.bool, device=DEV)
    keep[[7, 9, 50]] = False
    assert torch.equal(y[keep], clean[keep])


def test_scales_that_are_no_powers_of_two_are_reported():
    a, w, off = _operands([20, 30], 64, 272, seed=5)
    for scales, at in ((a[1], (1, 45)), (w[1], (1, 0, 2))):
        for bad in (1.5, 0.0, -1.0, 1e-40, float("inf")):
            keep = float(scales[at])
            scales[at] = bad
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            M.moe_expert_matmul_fp8(a, off, w, status=status)
            assert int(status) == 1
            M.moe_expert_matmul_fp8(a, off, w, any_scales=True, status=status.zero_())
            assert int(status) == 0
            scales[at] = keep
    short = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    a[1][0, 45] = 3.0  # a row of no slice
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_expert_matmul_fp8(a, short, w, status=status)
    assert int(status) == 0


@pytest.mark.parametrize("lengths,n,k", [([20, 30], 272, 272), ([200, 9, 330], 400, 272), ([3], 160, 8208)])
@pytest.mark.parametrize("bad", [1.5, 0.0, -1.0, 1e-40, float("inf"), -float("inf")])
def test_a_scale_that_is_no_power_of_two_shows_in_the_results(lengths, n, k, bad):
    """Without a status word too: the results that the scale enters are NaN, all others as they were."""
    a, w, off = _operands(lengths, n, k, seed=7)
    clean = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    keep = float(a[1][1, 1])
    a[1][1, 1] = bad
    hit[1] = True
    y = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32)
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])
    a[1][1, 1] = keep
    w[1][0, 1, 2] = bad                                    # columns 128 .. 255 of the first expert's rows
    hit[:] = False
    hit[:lengths[0], 128:256] = True
    y = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32)
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])


def test_a_nan_scale_of_either_sign_is_a_nan():
    a, w, off = _operands([20, 30], 64, 272, seed=5)
    clean = M.moe_expert_matmul_fp8(a, off, w)
    for bits in (0x7FC00000, 0x7F800001, -0x400000, -0x7FFFFF):
        b = a[1].clone()
        b.view(torch.int32)[1, 45] = bits
        assert torch.isnan(b[1, 45])
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = M.moe_expert_matmul_fp8((a[0], b), off, w, status=status)
        assert int(status) == 0 and torch.isnan(y[45]).all()
        y[45] = clean[45]
        assert torch.equal(y, clean)


def test_offsets_are_held_inside_the_rows():
    a, w, off = _operands([10, 20, 30], 64, 64, seed=4)
    wild = torch.tensor([-5, 10, 30, 10 ** 9], dtype=torch.int32, device=DEV)
    assert torch.equal(M.moe_expert_matmul_fp8(a, wild, w), M.moe_expert_matmul_fp8(a, off, w))
    back = torch.tensor([60, 30, 10, 0], dtype=torch.int32, device=DEV)  # every slice empty
    y = torch.full((60, 64), 3.0, dtype=BF, device=DEV)
    M.moe_expert_matmul_fp8(a, back, w, out=y)
    assert (y == 3).all()


# (rows, experts, offsets' period): few rows, whose tiles clusters share, with more slices on paper than rows; many
@pytest.mark.parametrize("rows, E, ups", [(2, 256, (0, 2)), (128, 8, (0, 128)), (9, 24, (3, 9, 1, 5)), (900, 12, (900, 100, 500))])
@pytest.mark.parametrize("free_scales", [False, True])
def test_offsets_that_decrease_make_no_row_twice(rows, E, ups, free_scales):
    """A slice begins no earlier than the end of those before it."""
    n, k = 144, 2192
    a, w, _ = _operands([rows] + [0] * (E - 1), n, k, seed=6, free_scales=free_scales)
    wild = torch.tensor([ups[i % len(ups)] for i in range(E + 1)], dtype=torch.int32, device=DEV)
    held = torch.cummax(wild, 0).values.to(torch.int32)
    got, want = (M.moe_expert_matmul_fp8(a, o, w, out=torch.full((rows, n), 5.0, dtype=F32, device=DEV),
                                         out_dtype=F32, any_scales=free_scales) for o in (wild, held))
    assert torch.equal(got, want)


def test_no_rows_and_empty_slices():
    a, w, off = _operands([0, 0, 0], 64, 64, seed=5)
    assert M.moe_expert_matmul_fp8(a, off, w).shape == (0, 64)
    a, w, off = _operands([0, 0], 64, 64, seed=5, behind=9)
    y = torch.full((9, 64), 2.0, dtype=BF, device=DEV)
    assert (M.moe_expert_matmul_fp8(a, off, w, out=y) == 2).all()


def test_a_value_that_is_not_finite_stays_in_its_row():
    a, w, off = _operands([40, 100], 144, 272, seed=6)
    clean = M.moe_expert_matmul_fp8(a, off, w, out_dtype=F32)
    x = torch.randn((140, 272), generator=gen(6), device=DEV).to(BF)
    x[33, 200] = float("nan")
    y = M.moe_expert_matmul_fp8(M.moe_quantize_rows(x), off, w, out_dtype=F32)
    assert torch.isnan(y[33]).all()
    keep = torch.arange(140, device=DEV) != 33
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("lengths,n,k", [([5, 0, 130], 272, 144), ([64] * 4, 1040, 256)])
def test_input_gradient(lengths, n, k):
    """dx = dy W by the transposed weights: the formula in 64 bits, and <dy, P v> = <dx, v>: the product is linear in
    its rows, so this is the difference quotient of <dy, P> in direction v."""
    g = gen(9)
    W = torch.randn((len(lengths), n, k), generator=g, device=DEV).mul_(0.05).to(BF)
    w, wt = M.moe_quantize_weights(W), M.moe_quantize_weights(W, transpose=True)
    assert torch.equal(w[0].view(torch.uint8).transpose(1, 2), wt[0].view(torch.uint8))
    off = offsets_of(lengths)
    rows = sum(lengths)
    dy = M.moe_quantize_rows(torch.randn((rows, n), generator=g, device=DEV))
    v = M.moe_quantize_rows(torch.randn((rows, k), generator=g, device=DEV))
    dx = M.moe_expert_matmul_fp8(dy, off, wt, out_dtype=F32)
    dyv, Wv = R.row_values(np64(dy[0]), np64(dy[1])), R.weight_values(np64(w[0]), np64(w[1]))
    want, bound = R.product(dyv, Wv.transpose(0, 2, 1), off.cpu().numpy())
    checked(dx, want, bound)
    pv = M.moe_expert_matmul_fp8(v, off, w, out_dtype=F32)
    vv = R.row_values(np64(v[0]), np64(v[1]))
    _, pbound = R.product(vv, Wv, off.cpu().numpy())
    assert abs((dyv * np64(pv)).sum() - (np64(dx) * vv).sum()) <= (np.abs(dyv) * pbound).sum() + (bound * np.abs(vv)).sum()


@pytest.mark.parametrize("free_scales", [False, True])
def test_most_rows(free_scales):
    """The largest number of rows that is taken, in one slice: 2^31 - 1."""
    rows, n, k, seen = 2 ** 31 - 1, 16, 16, 500
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 * 2 ** 30:
        pytest.skip("needs 120 GiB")
    a, w, off = _operands([seen], n, k, seed=8, free_scales=free_scales)
    want = M.moe_expert_matmul_fp8(a, off, w, any_scales=free_scales)
    q = torch.zeros((rows, k), dtype=a[0].dtype, device=DEV)
    scales = torch.ones((1, rows), dtype=F32, device=DEV)
    for part in (slice(0, seen), slice(rows - seen, rows)):
        q[part], scales[:, part] = a[0], a[1]
    out = torch.full((rows, n), 7.0, dtype=BF, device=DEV)
    M.moe_expert_matmul_fp8((q, scales), offsets_of([rows]), w, out=out, any_scales=free_scales)
    assert torch.equal(out[:seen], want) and torch.equal(out[-seen:], want)
    assert not any(p.any() for p in out[seen:-seen].split(2 ** 26))
    del q, scales, out
    torch.cuda.empty_cache()


def test_offsets_beyond_32_bits():
    """Operands and results of more than 2^31 values: the last rows and experts are where they belong."""
    rows, cols = 300_000, 7168
    x = torch.zeros((rows, cols), dtype=BF, device=DEV)
    x[-3:] = torch.randn((3, cols), generator=gen(1), device=DEV)
    q, s = M.moe_quantize_rows(x)
    wq, ws = R.quantize_rows(np64(x[-3:]))
    assert np.array_equal(np64(q[-3:]), wq) and np.array_equal(np64(s[:, -3:]), ws)
    assert not q[:-3].view(torch.uint8).any()
    del x, q, s
    W = torch.zeros((256, 2048, 4112), dtype=BF, device=DEV)
    W[-1] = torch.randn((2048, 4112), generator=gen(2), device=DEV)
    for t in (False, True):
        q, s = M.moe_quantize_weights(W, transpose=t)
        wq, ws = R.quantize_weights(np64(W[-1:]), t)
        assert np.array_equal(np64(q[-1:]), wq) and np.array_equal(np64(s[-1:]), ws)
        assert not q[:-1].view(torch.uint8).any()
    a = M.moe_quantize_rows(torch.randn((5, 2048), generator=gen(3), device=DEV))
    off = torch.full((257,), 3, dtype=torch.int32, device=DEV)
    off[0], off[256] = 0, 5                       # three rows of the first expert, two of the last
    y = M.moe_expert_matmul_fp8(a, off, (q, s), out_dtype=F32)
    want, bound = R.product(R.row_values(np64(a[0]), np64(a[1]))[3:], R.weight_values(wq, ws), [0, 2])
    checked(y[3:], want, bound)
    assert not y[:3].any()
    del W, q, s
    rows = 1_100_000
    a = M.moe_quantize_rows(torch.randn((rows, 16), generator=gen(4), device=DEV))
    w = M.moe_quantize_weights(torch.randn((2, 2048, 16), generator=gen(5), device=DEV))
    off = torch.tensor([0, rows - 77, rows], dtype=torch.int32, device=DEV)
    for free in (False, True):
        y = M.moe_expert_matmul_fp8(a, off, w, any_scales=free)
        av, wv = R.row_values(np64(a[0][-300:]), np64(a[1][:, -300:])), R.weight_values(np64(w[0]), np64(w[1]))
        want, bound = R.product(av, wv, [0, 223, 300])
        checked(y[-300:], want, bound + R.UBF * (np.abs(want) + bound))
        del y


# ---------------------------------------------------------------------- FFN


def _weights(E, d, F, act, seed, biases):
    g = gen(seed)
    mk = lambda *s: torch.randn(s, generator=g, device=DEV).mul_(0.08).to(BF)  # noqa: E731
    W = {"W1": mk(E, F, d), "W2": mk(E, d, F), "W3": mk(E, F, d) if act == "swiglu" else None,
         "b1": mk(E, F) if act == "gelu" and biases else None, "b2": mk(E, d) if biases else None}
    q = {k: M.moe_quantize_weights(v) if k[0] == "W" and v is not None else v for k, v in W.items()}
    return W, q


def _ffn_reference(q, x, off, act):
    val = lambda k: R.weight_values(np64(q[k][0]), np64(q[k][1])) if q[k] is not None else None  # noqa: E731
    vec = lambda k: np64(q[k]) if q[k] is not None else None  # noqa: E731
    return R.ffn(np64(x), off.cpu().numpy(), val("W1"), val("W2"), act, val("W3"), vec("b1"), vec("b2"))


FFNS = {
    # lengths, d, F, act, biases
    "token": ([0, 1, 0, 1, 0, 0], 256, 384, "swiglu", False),
    "token_gelu": ([1], 64, 272, "gelu", True),
    "few": ([3, 0, 1, 17, 2, 9], 400, 208, "swiglu", True),
    "narrow": ([40, 33], 16, 16, "swiglu", False),
    "ragged": ([128, 0, 131, 1, 290], 272, 720, "swiglu", False),
    "ragged_gelu": ([128, 0, 131, 1, 290], 272, 720, "gelu", True),
    "gelu_plain": ([77, 200], 144, 144, "gelu", False),
    "many": ([i % 7 for i in range(200)], 144, 256, "swiglu", False),
    "wide": ([500, 300], 1040, 1152, "swiglu", True),
    "split": ([1, 0, 3], 4112, 272, "swiglu", False),
    "split_gelu": ([2], 2064, 2064, "gelu", True),
    "split_rows": ([0, 47, 0, 0], 2064, 144, "swiglu", False),
}


@pytest.mark.parametrize("name", sorted(FFNS))
def test_ffn(name):
    lengths, d, F, act, biases = FFNS[name]
    _, q = _weights(len(lengths), d, F, act, len(name), biases)
    rows, off = sum(lengths), offsets_of(lengths)
    x = torch.randn((rows, d), generator=gen(4), device=DEV).to(BF)
    cfg = M.make_config(rows, d, F, len(lengths), 1, act=act, dtype="bf16")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], b1=q["b1"], W3=q["W3"], b2=q["b2"], status=status)
    want, bound = _ffn_reference(q, x, off, act)
    checked(y, want, bound)
    checked(M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], b1=q["b1"], W3=q["W3"], b2=q["b2"], any_scales=True),
            want, bound)
    # The bound is a worst case, so its ratio to the result grows with the square root of the reduction (0.06 at 2064), but
    # a wrong row or column is off by the result's size, and one block of 17 with a scale of half or twice its value by
    # at least 0.5 / sqrt(17) = 0.12 of it: neither would pass a bound below 0.1.
    assert np.sqrt(np.mean(bound ** 2)) < 0.1 * np.sqrt(np.mean(want ** 2))
    assert int(status) == 0
    again = M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], b1=q["b1"], W3=q["W3"], b2=q["b2"])
    assert torch.equal(y, again)


# CTAs that process several tiles: what they carry from one to the next (barrier phases, stages, slots of scales, sets of
# accumulators) shows in results only with more tiles than SMs.
# name: (rows of an expert, experts, n, k, the tile's rows and columns)
SEVERAL_TILES = {
    "wide": ((200, 500), 24, 2000, 656, 240, 256),
    "tall": ((200, 480), 20, 2000, 656, 240, 128),
    "few": ((20, 130), 40, 2000, 656, 112, 256),
    "tiny": ((1, 28), 48, 2000, 656, 32, 256),
}


def _lengths(between, E, seed):
    """Uneven slices, one of them empty."""
    lengths = np.random.RandomState(seed).randint(between[0], between[1] + 1, E)
    lengths[E // 3] = 0
    return [int(v) for v in lengths]


def _several(lengths, n, tile_rows, tile_cols):
    tiles = sum(-(-v // tile_rows) for v in lengths) * -(-n // tile_cols)
    assert tiles > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    assert n % tile_cols


@pytest.mark.parametrize("name", sorted(SEVERAL_TILES))
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("free_scales", [False, True])
def test_product_of_several_tiles_a_cta(name, out, free_scales):
    between, E, n, k, tile_rows, tile_cols = SEVERAL_TILES[name]
    lengths = _lengths(between, E, E)
    _several(lengths, n, *((128, 256) if free_scales else (tile_rows, tile_cols)))
    a, w, off = _operands(lengths, n, k, seed=E, free_scales=free_scales, behind=5)
    y = torch.full((sum(lengths) + 5, n), 7.0, dtype=out, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_expert_matmul_fp8(a, off, w, out_dtype=out, out=y, any_scales=free_scales, status=status)
    assert (y[-5:] == 7).all() and int(status) == 0
    want, bound = R.product(*_values(a, w), off.cpu().numpy())
    checked(y[:-5], want[:-5], (bound + (R.UBF * (np.abs(want) + bound) if out == BF else 0))[:-5])


# name: (rows of an expert, experts, d, F, activation, biases, the first product's tile's rows; its columns are 128)
SEVERAL_TILES_FFN = {
    "wide": ((200, 500), 16, 656, 2000, "swiglu", True, 240),
    "few": ((20, 130), 24, 656, 2000, "swiglu", False, 112),
    "tiny": ((1, 28), 40, 656, 2000, "swiglu", False, 32),
    "gelu_tall": ((200, 500), 16, 656, 2000, "gelu", True, 240),
    "gelu_tiny": ((1, 28), 40, 656, 2000, "gelu", True, 32),
}


@pytest.mark.parametrize("name", sorted(SEVERAL_TILES_FFN))
def test_ffn_of_several_tiles_a_cta(name):
    between, E, d, F, act, biases, tile_rows = SEVERAL_TILES_FFN[name]
    lengths = _lengths(between, E, E)
    _several(lengths, F, tile_rows, 128)
    _, q = _weights(E, d, F, act, E, biases)
    rows, off = sum(lengths), offsets_of(lengths)
    x = torch.randn((rows, d), generator=gen(4), device=DEV).to(BF)
    cfg = M.make_config(rows, d, F, E, 1, act=act, dtype="bf16")
    want, bound = _ffn_reference(q, x, off, act)
    assert np.sqrt(np.mean(bound ** 2)) < 0.1 * np.sqrt(np.mean(want ** 2))   # as in test_ffn
    for free in (False, True):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], b1=q["b1"], W3=q["W3"], b2=q["b2"], any_scales=free, status=status)
        checked(y, want, bound)
        assert int(status) == 0


@pytest.mark.parametrize("tokens", [3, 700])
@pytest.mark.parametrize("free_scales", [False, True])
def test_ffn_on_weights_and_slices_written_just_before(tokens, free_scales):
    """The products of an FFN fetch weights and slices ahead of their rows, never ahead of the kernels that write them:
    quantisers and copies of some hundred MB straight before the call, on one stream."""
    E, d, F = 24, 2048, 1408
    sets = []
    for seed in (1, 2):
        W, _ = _weights(E, d, F, "swiglu", seed, False)
        lengths = np.random.RandomState(seed).multinomial(tokens, np.ones(E) / E)
        sets.append((W, offsets_of(lengths), torch.randn((tokens, d), generator=gen(seed), device=DEV).to(BF)))
    cfg = M.make_config(tokens, d, F, E, 1, act="swiglu", dtype="bf16")
    ffn = lambda q, off, x: M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], W3=q["W3"], any_scales=free_scales)  # noqa: E731
    names = ("W2", "W3", "W1")   # W1 last: the first product's weights are the newest
    want, qs = [], []
    for W, off, x in sets:
        qs.append({n: M.moe_quantize_weights(W[n]) for n in names})
        torch.cuda.synchronize()
        want.append(ffn(qs[-1], off, x))
        torch.cuda.synchronize()
    at = {n: (torch.empty_like(qs[0][n][0]), torch.empty_like(qs[0][n][1])) for n in names}
    off, x, got = torch.empty_like(sets[0][1]), torch.empty_like(sets[0][2]), []
    for i in range(6):
        W, o, v = sets[i % 2]
        got.append(ffn({n: M.moe_quantize_weights(W[n]) for n in names}, o, v))   # quantised just before
        x.copy_(v)
        off.copy_(o)
        for n in names:
            at[n][1].copy_(qs[i % 2][n][1])
            at[n][0].view(torch.uint8).copy_(qs[i % 2][n][0].view(torch.uint8))
        got.append(ffn(at, off, x))                                               # copied just before
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i // 2 % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_ffn_scales_whose_product_leaves_fp32(act):
    """The same inside an FFN: tiny rows (one of zeros) against small weight scales, brought back by large ones."""
    _, q = _weights(3, 400, 272, act, 8, False)
    g = gen(9)
    free = lambda w, e: (w[0], w[1] * torch.exp2(e + torch.rand(w[1].shape, generator=g, device=DEV)))  # noqa: E731
    off = offsets_of([40, 0, 150])
    x = (torch.randn((190, 400), generator=gen(4), device=DEV) * 2.0 ** -108).to(BF)
    x[3] = 0
    # gate: 2^-115 x 2^-24 = 2^-139 a block, about 2^-119 in all; swiglu's up: 2^-115 x 2^104
    q["W1"] = free(q["W1"], -13.0)
    if act == "swiglu":
        q["W3"] = free(q["W3"], 115.0)
    q["W2"] = free(q["W2"], 100.0)
    cfg = M.make_config(190, 400, 272, 3, 1, act=act, dtype="bf16")
    y = M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], W3=q["W3"], any_scales=True)
    want, bound = _ffn_reference(q, x, off, act)
    checked(y, want, bound)
    assert not y[3].any() and np.sqrt(np.mean(want ** 2)) > 2.0 ** -40


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_ffn_leaves_rows_outside_every_slice(act):
    _, q = _weights(3, 144, 272, act, 8, True)
    off = offsets_of([10, 0, 150], 7)
    x = torch.randn((207, 144), generator=gen(4), device=DEV).to(BF)
    x[190] = float("nan")  # a row of no slice holds anything
    cfg = M.make_config(207, 144, 272, 3, 1, act=act, dtype="bf16")
    y = torch.full((207, 144), 7.0, dtype=BF, device=DEV)
    M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], b1=q["b1"], W3=q["W3"], b2=q["b2"], out=y)
    assert (y[:7] == 7).all() and (y[167:] == 7).all()
    x[190] = 0
    want, bound = _ffn_reference(q, x, off, act)
    checked(y[7:167], want[7:167], bound[7:167])


def test_ffn_no_tokens():
    _, q = _weights(3, 144, 272, "swiglu", 8, False)
    cfg = M.make_config(0, 144, 272, 3, 2, act="swiglu", dtype="bf16")
    y = M.moe_expert_ffn_fp8(cfg, torch.empty((0, 144), dtype=BF, device=DEV), offsets_of([0, 0, 0]), q["W1"], q["W2"],
                             W3=q["W3"])
    assert y.shape == (0, 144)


def test_ffn_captured_and_replayed_beside_an_eager_call():
    """A captured call and an eager one on another stream, each with its workspace, replayed on new inputs."""
    lengths = [30, 0, 140, 6]
    _, q = _weights(4, 256, 384, "swiglu", 3, False)
    off, rows = offsets_of(lengths), 176
    cfg = M.make_config(rows, 256, 384, 4, 1, act="swiglu", dtype="bf16")
    xs = [torch.randn((rows, 256), generator=gen(i), device=DEV).to(BF) for i in range(3)]
    call = lambda x, **kw: M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], W3=q["W3"], **kw)  # noqa: E731
    want = [call(x) for x in xs]
    static, out, ws = xs[0].clone(), torch.empty((rows, 256), dtype=BF, device=DEV), M.moe_expert_ffn_fp8_workspace(cfg)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(static, ws=ws, out=out)
    side = torch.cuda.Stream()
    for i, x in enumerate(xs):
        static.copy_(x)
        side.wait_stream(torch.cuda.current_stream())
        other = call(xs[i - 1], stream=side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(other, want[i - 1])


@pytest.mark.parametrize("N,E,k,act,router", [(1, 8, 2, "swiglu", "softmax_topk"), (64, 40, 6, "swiglu", "sigmoid"),
                                              (333, 6, 2, "gelu", "softmax_topk")])
def test_layer_on_quantised_experts(N, E, k, act, router):
    """route -> dispatch -> FFN on 8-bit weights -> combine, as a serving program chains them: every step within its
    bound of the same chain in 64 bits, and near the bf16 layer."""
    d, F = 272, 208
    W, q = _weights(E, d, F, act, 11, False)
    g = gen(12)
    x, Wg = torch.randn((N, d), generator=g, device=DEV).to(BF), torch.randn((E, d), generator=g, device=DEV).mul_(0.1).to(BF)
    cfg = M.make_config(N, d, F, E, k, router=router, act=act, dtype="bf16")
    ids, w, _ = M.moe_route(cfg, x, Wg)
    dsp = M.moe_dispatch(cfg, ids, x)
    ys = M.moe_expert_ffn_fp8(cfg, dsp["x_sorted"], dsp["offsets"], q["W1"], q["W2"], W3=q["W3"])
    y = M.moe_combine(cfg, ys, w, dsp["inv_perm"])
    want, bound = _ffn_reference(q, dsp["x_sorted"], dsp["offsets"], act)
    checked(ys, want, bound)
    inv = dsp["inv_perm"].cpu().numpy().reshape(N, k)
    full = (np64(w)[:, :, None] * want[inv]).sum(1)
    off = (np64(w)[:, :, None] * bound[inv]).sum(1)
    size = (np64(w)[:, :, None] * (np.abs(want) + bound)[inv]).sum(1)
    checked(y, full, off + k * R.U32 * size + R.UBF * (np.abs(full) + off + k * R.U32 * size))
    # Against the bf16 layer: each operand of a product is off by at most 2^-4 of itself and, over a row, by about
    # 2^-4 / sqrt(3) at random; two operands twice give under 0.1 of the result's norm.
    ref = M.moe_forward(cfg, x, Wg, W["W1"], W["W2"], W3=W["W3"])["y"]
    rel = np.linalg.norm(np64(y) - np64(ref)) / np.linalg.norm(np64(ref))
    assert 1e-4 < rel < 0.1, rel


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_expert_parallel_phase_on_quantised_experts(act):
    """Two ranks' experts, driven phase by phase as one process: each rank's share on 8-bit weights is the layer's."""
    from mixture_experts_layer_53_b200 import ep as EP
    N, d, F, E, k, world = 150, 144, 272, 6, 2, 2
    _, q = _weights(E, d, F, act, 13, True)
    g = gen(14)
    cfg = M.make_config(N, d, F, E, k, act=act, dtype="bf16")
    x, Wg = torch.randn((N, d), generator=g, device=DEV).to(BF), torch.randn((E, d), generator=g, device=DEV).mul_(0.1).to(BF)
    ranks = [EP.ExpertParallelMoE(cfg, world=world, rank=r) for r in range(world)]
    st = ranks[0].dispatch_phase(x, Wg)
    counts, E_r = st.counts.cpu().numpy(), E // world
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
    want = M.moe_expert_ffn_fp8(cfg, st.x_sorted, off, q["W1"], q["W2"], W3=q["W3"], b1=q["b1"], b2=q["b2"])
    back = []
    for r in range(world):
        mine = slice(r * E_r, (r + 1) * E_r)
        # this rank receives rank 0's rows only: its own, or none of another's
        recv = np.zeros((world, E_r), np.int64)
        recv[0] = counts[mine]
        p = EP.plan(counts, recv, world)
        rows = st.x_sorted[int(counts[:r * E_r].sum()):int(counts[:(r + 1) * E_r].sum())]
        part = lambda v: None if v is None else (tuple(t[mine].contiguous() for t in v) if isinstance(v, tuple)  # noqa: E731
                                                 else v[mine].contiguous())
        back.append(ranks[r].expert_phase(rows, p, part(q["W1"]), part(q["W2"]), W3=part(q["W3"]), b1=part(q["b1"]),
                                          b2=part(q["b2"])))
    y_sorted = torch.cat(back)
    assert torch.equal(y_sorted, want)
    y, _ = ranks[0].combine_phase(st, y_sorted)
    assert torch.equal(y, M.moe_combine(cfg, want, st.w, st.inv_perm))


def test_expert_parallel_phase_with_a_checkpoints_scales():
    """Scales that are no powers of two through the expert-parallel phase: with any_scales the single process's result,
    without it a status (and NaN); the status of a layer on bf16 weights is wired too."""
    from mixture_experts_layer_53_b200 import ep as EP
    N, d, F, E = 70, 144, 272, 3
    W, q = _weights(E, d, F, "swiglu", 15, False)
    g = gen(16)
    free = lambda w: [w[0], w[1] * torch.exp(torch.randn(w[1].shape, generator=g, device=DEV))]  # noqa: E731
    f = {k: free(q[k]) for k in ("W1", "W2", "W3")}
    cfg = M.make_config(N, d, F, E, 1, act="swiglu", dtype="bf16")
    x = torch.randn((N, d), generator=g, device=DEV).to(BF)
    counts = np.array([20, 0, 50])
    off = offsets_of(counts)
    layer, p = EP.ExpertParallelMoE(cfg, world=1, rank=0), EP.plan(counts, counts[None], 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = layer.expert_phase(x, p, f["W1"], f["W2"], W3=f["W3"], any_scales=True, status=status)
    assert torch.equal(y, M.moe_expert_ffn_fp8(cfg, x, off, f["W1"], f["W2"], W3=f["W3"], any_scales=True)) and int(status) == 0
    want, bound = _ffn_reference({**q, **f}, x, off, "swiglu")
    checked(y, want, bound)
    y = layer.expert_phase(x, p, f["W1"], f["W2"], W3=f["W3"], status=status)
    assert int(status) == 1 and torch.isnan(y).all()
    plain = layer.expert_phase(x, p, W["W1"], W["W2"], W3=W["W3"], status=status.zero_())
    assert torch.equal(plain, M.moe_expert_ffn(cfg, x, off, W["W1"], W["W2"], W3=W["W3"])) and int(status) == 0


def test_workspaces_that_are_too_small_are_refused():
    _, q = _weights(2, 64, 64, "swiglu", 1, False)
    cfg = M.make_config(8, 64, 64, 2, 1, act="swiglu", dtype="bf16")
    x, off, ws = torch.zeros((8, 64), dtype=BF, device=DEV), offsets_of([4, 4]), M.moe_expert_ffn_fp8_workspace(cfg)
    call = lambda w: M.moe_expert_ffn_fp8(cfg, x, off, q["W1"], q["W2"], W3=q["W3"], ws=w)  # noqa: E731
    assert not call(ws).any()
    for bad in (ws[:-1], ws[64:]):
        with pytest.raises(M.MoeError, match="WORKSPACE"):
            call(bad)
    with pytest.raises(ValueError, match="ws"):
        call(ws.cpu())


def test_a_side_stream_owns_its_results():
    """A call given a stream allocates there: its temporaries are not handed to the current stream while it runs."""
    a, w, off = _operands([300, 200], 528, 640, seed=2)
    want = M.moe_expert_matmul_fp8(a, off, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [M.moe_expert_matmul_fp8(a, off, w, stream=side) for _ in range(8)]
    junk = [torch.full((500, 528), float(i), dtype=BF, device=DEV) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and len(junk) == 8


def test_refusals_of_the_binding():
    a, w, off = _operands([4, 4], 64, 64, seed=1)
    ok = dict(a=a, offsets=off, w=w)
    for bad, match in [
        (dict(a=(a[0].float(), a[1])), "a must be"), (dict(a=(a[0], a[1].t().contiguous())), "scales"),
        (dict(offsets=off.long()), "offsets"), (dict(offsets=off[:2]), "offsets"),
        (dict(w=(w[0][:, :48].contiguous(), w[1][:, :0].contiguous())), "scales"),
        (dict(w=(w[0].transpose(1, 2), w[1])), "contiguous"), (dict(out_dtype=torch.float16), "out_dtype"),
        (dict(out=torch.empty((8, 80), dtype=BF, device=DEV)), "out must be"),
        (dict(out=torch.empty((8, 64), dtype=F32, device=DEV)), "out must be"),
        (dict(offsets=off.cpu()), "is on cpu"),
    ]:
        with pytest.raises(ValueError, match=match):
            M.moe_expert_matmul_fp8(**{**ok, **bad})
    with pytest.raises(M.MoeError, match="UNSUPPORTED"):
        M.moe_quantize_rows(torch.zeros((4, 24), device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_quantize_rows(torch.zeros((64, 64), device=DEV).t()[:, :32])
