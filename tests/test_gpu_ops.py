"""GPU tests of wino_group_norm and wino_matmul against plain implementations in 64 bits.

Tolerances follow from the arithmetic, element by element, with u = 2^-24:
 - a sum of n fp32 terms in any order is off by at most n u (to first order) times the sum of the
   terms' magnitudes (2 n u on the tensor cores, whose partial sums may be truncated);
 - SiLU and GELU have slopes of magnitude at most 1.13 and are themselves evaluated to 2^-20 of their
   value for bf16 results (the hardware exponential and reciprocal) and 8 u for fp32 results; GELU's
   erfc(t) is off by a further 2 t^2 u of its value through the rounding of t, and t^2 = v^2 / 2;
 - the final rounding is off by at most eps / 2 of the result.
"""
import math

import pytest
import torch

from group_wise_int8_b200 import synth, wino

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
ACTS = {"none": wino.ACT_NONE, "silu": wino.ACT_SILU, "gelu": wino.ACT_GELU}


def randn(seed, *shape, dtype=F32, mean=0.0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * spread + mean).to(dtype)


def ref_act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    return v


def act_error(v, act, err, fast):
    """Bound on the error of act(v) when v is off by err."""
    if act == "none":
        return err
    own = (2.0 ** -20 if fast else 8 * U) + (2 * v * v * U if act == "gelu" else 0)
    return 1.13 * err + own * ref_act(v, act).abs() * (1 + v.abs() * U * 4)


def check(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol + torch.finfo(torch.float32).tiny)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d off; first at %s: got %r want %r tolerance %r"
                             % (what, int(bad.sum()), bad.numel(), i, got[i].item(), want[i].item(), tol[i].item()))


def ref_norm(x, groups, gamma, beta, eps, act, add, x2, out_dtype):
    """-> (reference in 64 bits, tolerance)."""
    v = x.double() if x2 is None else torch.cat([x.double(), x2.double()], -1)
    N, H, W, C = v.shape
    if add is not None:
        v = v + add.double().view(N, 1, 1, C)
    gam = torch.ones(C, device=v.device, dtype=torch.float64) if gamma is None else gamma.double()
    bet = torch.zeros(C, device=v.device, dtype=torch.float64) if beta is None else beta.double()
    g = v.view(N, H * W, groups, C // groups)
    mean = g.mean(dim=(1, 3), keepdim=True)
    var = (g - mean).square().mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    z = (g - mean) * rstd
    pre = (z.view_as(v) * gam + bet)
    want = ref_act(pre, act)
    # n: terms of the longest sum, a thread's pixels and then the joins; the statistics' sums run over
    # deviations from values of the group, at most `spread` wide, and var >= 0 from squares of them
    n = H * W + C // groups + 64
    top = g.abs().amax(dim=(1, 3), keepdim=True)
    spread = (g.amax(dim=(1, 3), keepdim=True) - g.amin(dim=(1, 3), keepdim=True))
    mean_err = 8 * U * top + n * U * spread
    var_err = 4 * n * U * (spread * spread) + 8 * U * top * spread
    rel = 0.5 * var_err * rstd * rstd + 4 * U                      # of rstd (to first order)
    z_err = (mean_err + 4 * U * top) * rstd + z.abs() * rel
    err = act_error(pre, act, z_err.expand_as(g).reshape(v.shape) * gam.abs() + 4 * U * (pre.abs() + bet.abs()),
                    out_dtype == BF16)
    tol = err + (want.abs() + err) * torch.finfo(out_dtype).eps / 2
    return want, tol


def run_norm(x, groups, gamma=None, beta=None, eps=1e-5, act="none", add=None, x2=None, out_dtype=None, **kw):
    y = wino.group_norm(x, groups, gamma, beta, eps=eps, act=ACTS[act], add=add, x2=x2, out_dtype=out_dtype, **kw)
    want, tol = ref_norm(x, groups, gamma, beta, eps, act, add, x2, y.dtype)
    check(y, want, tol, "group_norm")
    return y


NORMS = {
    # N, H, W, C, C2, groups, dtype, out, act, add, affine
    "one_pixel_one_channel_groups": (2, 1, 1, 64, 0, 64, BF16, BF16, "silu", True, True),
    "one_pixel": (3, 1, 1, 96, 0, 32, F32, F32, "gelu", False, True),
    "one_channel": (1, 5, 3, 1, 0, 1, F32, F32, "none", False, True),
    "one_channel_bf16": (2, 7, 5, 1, 0, 1, BF16, BF16, "silu", True, True),
    "odd_channels": (2, 9, 7, 33, 0, 3, BF16, BF16, "silu", False, True),
    "odd_channels_f32": (2, 9, 7, 35, 0, 7, F32, F32, "silu", True, True),
    "groups_of_ten": (2, 16, 16, 320, 0, 32, BF16, BF16, "silu", True, True),
    "groups_of_three": (1, 13, 11, 96, 0, 32, BF16, F32, "gelu", False, True),
    "groups_of_one": (1, 8, 8, 32, 0, 32, BF16, BF16, "none", True, True),
    "eight_groups": (2, 12, 10, 640, 0, 8, F32, BF16, "silu", False, False),
    "no_affine": (1, 8, 8, 1280, 0, 32, BF16, BF16, "none", False, False),
    "two_sources_straddled": (2, 17, 13, 640, 320, 32, BF16, BF16, "silu", True, True),
    "two_sources_scalar": (2, 6, 5, 20, 15, 5, BF16, F32, "none", True, True),
    "two_sources_f32": (1, 10, 9, 36, 60, 8, F32, F32, "silu", False, True),
    "two_sources_one_group": (1, 6, 6, 64, 32, 1, BF16, BF16, "silu", False, True),
    "layer_norm_wide": (2, 3, 3, 4096, 0, 1, BF16, BF16, "none", False, True),
    "wider_than_a_block": (1, 2, 3, 16384, 0, 1, BF16, BF16, "silu", False, True),
    "wider_than_a_block_odd": (1, 2, 2, 4097, 0, 17, F32, F32, "none", True, True),
    "many_groups": (1, 2, 2, 16384, 0, 16384, F32, F32, "none", False, True),
    "streamed": (1, 160, 150, 128, 0, 1, BF16, BF16, "silu", False, True),
    "streamed_f32": (1, 131, 97, 64, 64, 2, F32, F32, "silu", True, True),
    "many_images": (3000, 1, 2, 32, 0, 4, BF16, BF16, "silu", True, True),
    "level_64": (2, 64, 64, 320, 0, 32, BF16, BF16, "silu", True, True),
    "level_32_skip": (2, 32, 32, 1280, 640, 32, BF16, BF16, "silu", False, True),
    "level_8": (1, 8, 8, 1280, 0, 32, F32, BF16, "silu", True, True),
    "tall": (1, 999, 1, 48, 0, 6, F32, F32, "gelu", False, True),
}


@pytest.mark.parametrize("variant", ["release", "debug"])
@pytest.mark.parametrize("name", NORMS)
def test_group_norm_matches_64_bits(cuda_dev, name, variant):
    N, H, W, C, C2, groups, dtype, out, act, add, affine = NORMS[name]
    x = randn(1, N, H, W, C, dtype=dtype, mean=0.7, spread=1.5)
    x2 = randn(2, N, H, W, C2, dtype=dtype, mean=-0.5) if C2 else None
    run_norm(x, groups, randn(3, C + C2, mean=1.0, spread=0.3) if affine else None, randn(4, C + C2) if affine else None,
             act=act, add=randn(5, N, C + C2) if add else None, x2=x2, out_dtype=out, variant=variant)
    assert wino.check_device_error_ops(variant=variant) == wino.OK


NARROW = {
    # N, H, W, C, groups, dtype: much shared memory beside the kept rows, by hundreds of groups of one or two channels in a slab
    "one_channel_911": (2, 32, 32, 911, 911, F32),
    "one_channel_1061": (1, 16, 16, 1061, 1061, F32),
    "one_channel_2039": (1, 16, 16, 2039, 2039, BF16),
    "two_channels_907": (2, 32, 32, 1814, 907, BF16),
    "one_channel_2048": (1, 24, 20, 2048, 2048, BF16),
    "two_channels_1024": (1, 40, 40, 2048, 1024, F32),
    "one_channel_1021": (1, 160, 100, 1021, 1021, BF16),
    "one_channel_16381": (1, 9, 5, 16381, 16381, F32),
    # clusters of 16 CTAs with an SM each
    "two_channels_2018": (3, 8, 8, 4036, 2018, F32),
    "two_channels_523": (3, 16, 16, 1046, 523, BF16),
    "one_wide_group": (8, 15, 17, 15504, 1, F32),
}


@pytest.mark.parametrize("variant", ["release", "debug"])
@pytest.mark.parametrize("name", NARROW)
def test_group_norm_of_many_narrow_groups(cuda_dev, name, variant):
    N, H, W, C, groups, dtype = NARROW[name]
    run_norm(randn(1, N, H, W, C, dtype=dtype, mean=0.7), groups, randn(2, C, mean=1.0, spread=0.3), randn(3, C), act="silu",
             variant=variant)
    assert wino.check_device_error_ops(variant=variant) == wino.OK


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_group_norm_of_constants_and_far_means(cuda_dev, dtype):
    """A constant group has variance 0; a mean of 1000 spreads keeps its digits (the pivot)."""
    x = torch.full((1, 8, 8, 64), 3.0, device="cuda", dtype=dtype)
    beta = randn(1, 64)
    y = wino.group_norm(x, 8, None, beta, out_dtype=F32)
    assert torch.equal(y, beta.expand_as(y))
    far = randn(2, 2, 24, 20, 64, dtype=F32, mean=1000.0).to(dtype)
    run_norm(far, 8, out_dtype=F32)
    if dtype == F32:
        # the plain bound on such data is dominated by n u spread / std; held to a few roundings of 1000 / std too
        want, _ = ref_norm(far, 8, None, None, 1e-5, "none", None, None, F32)
        assert (wino.group_norm(far, 8).double() - want).abs().max() < 16 * U * 1005


def test_group_norm_first_pixel_is_an_outlier(cuda_dev):
    """The pivot is the first value a thread sees: an outlier there must not spoil the statistics."""
    x = randn(3, 1, 32, 32, 64, dtype=F32)
    x[:, 0, :8] = 50.0
    run_norm(x, 4, act="silu")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_group_norm_non_finite_stays_in_its_group(cuda_dev, bad):
    x = randn(4, 2, 16, 16, 64, dtype=BF16)
    clean = wino.group_norm(x, 8, act=wino.ACT_SILU)
    x[1, 5, 7, 19] = bad    # image 1, group 2
    y = wino.group_norm(x, 8, act=wino.ACT_SILU)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, :, :, 16:24] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lo,pad", [(0, 8), (8, 24), (3, 5), (1, 0)])
def test_group_norm_channel_ranges(cuda_dev, dtype, lo, pad):
    """Inputs and output are channel ranges of wider tensors; what lies around the output stays."""
    C, C2 = 48, 24
    wide = randn(5, 2, 7, 9, lo + C + pad, dtype=dtype)
    wide2 = randn(6, 2, 7, 9, lo + C2 + pad, dtype=dtype)
    outer = torch.full((2, 7, 9, lo + C + C2 + pad), 7.0, device="cuda", dtype=BF16)
    x, x2, out = wide[..., lo:lo + C], wide2[..., lo:lo + C2], outer[..., lo:lo + C + C2]
    gamma, beta = randn(7, C + C2 + 1)[1:], randn(8, C + C2 + 1)[1:]
    y = run_norm(x, 6, gamma, beta, act="silu", x2=x2, out=out)
    assert y.data_ptr() == out.data_ptr()
    rest = torch.ones_like(outer, dtype=torch.bool)
    rest[..., lo:lo + C + C2] = False
    assert (outer[rest] == 7.0).all()


def test_group_norm_ranges_of_one_buffer_and_in_place(cuda_dev):
    buf = randn(9, 2, 8, 8, 128, dtype=BF16)
    x, out = buf[..., :64], buf[..., 64:]
    want = wino.group_norm(x.clone(), 8, act=wino.ACT_SILU)
    wino.group_norm(x, 8, act=wino.ACT_SILU, out=out)
    assert torch.equal(out, want)
    for shape in ((2, 8, 8, 64), (1, 150, 160, 128)):   # kept whole, and read twice
        y = randn(10, *shape, dtype=BF16)
        want = wino.group_norm(y.clone(), 1, act=wino.ACT_SILU)
        wino.group_norm(y, 1, act=wino.ACT_SILU, out=y)
        assert torch.equal(y, want)


def test_group_norm_beyond_32_bit_offsets(cuda_dev):
    """2.2e9 values: the first, a middle and the last image against 64 bits.  (Not against a call on that image alone bit
    for bit: the split, and with it the order of the sums, goes by the number of images too.)"""
    N, S, C = 33, 256, 1024
    x = torch.empty(N, S, S, C, device="cuda", dtype=BF16)
    for n in range(N):
        x[n].normal_(mean=0.1 * n)
    y = wino.group_norm(x, 32, act=wino.ACT_SILU)
    for n in (0, N // 2, N - 1):
        want, tol = ref_norm(x[n:n + 1], 32, None, None, 1e-5, "silu", None, None, BF16)
        check(y[n:n + 1], want, tol, "image %d" % n)
        del want, tol


# ---------------------------------------------------------------- matmul
def ref_matmul(a, w, bias, act, residual, a2, out_dtype):
    A = a.double().reshape(-1, a.shape[-1])
    if a2 is not None:
        A = torch.cat([A, a2.double().reshape(-1, a2.shape[-1])], 1)
    Wd = w.double()
    v, mag = A @ Wd.t(), A.abs() @ Wd.abs().t()
    if bias is not None:
        v, mag = v + bias.double(), mag + bias.double().abs()
    want = ref_act(v, act)
    err = act_error(v, act, 2 * (A.shape[1] + 8) * U * mag, out_dtype == BF16)
    if residual is not None:
        want = want + residual.double().reshape(want.shape)
        err = err + U * (want.abs() + err)
    tol = err + (want.abs() + err) * torch.finfo(out_dtype).eps / 2
    shape = (*a.shape[:-1], w.shape[0])
    return want.view(shape), tol.view(shape)


def run_matmul(a, w, bias=None, act="none", residual=None, a2=None, out_dtype=None, **kw):
    kept = None if residual is None else residual.clone()
    y = wino.matmul(a, w, bias=bias, act=ACTS[act], residual=residual, a2=a2, out_dtype=out_dtype, **kw)
    want, tol = ref_matmul(a, w, bias, act, kept, a2, y.dtype)
    check(y, want, tol, "matmul")
    return y


PRODUCTS = {
    # M, K, K2, N, dtype, out, act, bias, residual
    "one": (1, 1, 0, 1, BF16, F32, "none", True, True),
    "one_row": (1, 1280, 0, 1280, BF16, BF16, "silu", True, False),
    "one_row_f32": (1, 320, 0, 1280, F32, F32, "silu", True, False),
    "one_row_odd": (1, 77, 0, 13, BF16, BF16, "gelu", True, True),
    "one_column": (300, 64, 0, 1, BF16, BF16, "none", True, True),
    "two_rows": (2, 200, 56, 33, F32, BF16, "none", False, True),
    "three_rows_long": (3, 2560, 0, 320, BF16, F32, "none", True, False),
    "eight_rows": (8, 1280, 0, 640, BF16, BF16, "silu", True, False),
    "eight_rows_f32": (8, 320, 0, 1280, F32, F32, "silu", True, True),
    "nine_rows": (9, 96, 32, 100, BF16, BF16, "gelu", True, True),
    "sixteen_rows": (16, 512, 0, 72, F32, F32, "gelu", True, False),
    "seventeen_rows": (17, 512, 0, 72, BF16, F32, "gelu", True, False),
    "classifier": (32, 512, 0, 1000, BF16, F32, "none", True, False),
    "ten_classes": (64, 512, 0, 10, BF16, F32, "none", True, False),
    "odd_everything": (131, 77, 0, 37, BF16, BF16, "silu", True, True),
    "odd_depth_two_sources": (45, 33, 31, 66, BF16, BF16, "none", True, True),
    "odd_columns": (200, 128, 0, 333, BF16, BF16, "gelu", True, True),
    "odd_columns_f32_out": (200, 128, 64, 333, BF16, F32, "silu", True, True),
    "short_depth": (500, 8, 0, 64, BF16, BF16, "none", True, False),
    "ragged_depth": (257, 200, 0, 160, BF16, BF16, "none", True, True),
    "ragged_two_sources": (129, 72, 40, 192, BF16, BF16, "silu", True, True),
    "tile": (128, 64, 0, 128, BF16, BF16, "none", False, False),
    "tile_and_a_row": (129, 128, 0, 256, BF16, BF16, "none", False, True),
    "f32_operands": (150, 96, 0, 130, F32, F32, "gelu", True, True),
    "f32_to_bf16": (70, 65, 0, 70, F32, BF16, "none", True, True),
    "skip_shortcut_8": (128, 1280, 1280, 1280, BF16, BF16, "none", True, True),
    "skip_shortcut_64": (4096, 640, 320, 320, BF16, BF16, "none", True, True),
    "ragged_images": (3219, 640, 0, 640, BF16, BF16, "none", True, True),
    "widening": (1024, 320, 0, 1280, BF16, BF16, "gelu", True, False),
    "more_tiles_than_sms": (9000, 128, 0, 640, BF16, BF16, "silu", True, True),
    "more_tiles_than_sms_f32_out": (9001, 64, 0, 520, BF16, F32, "none", True, True),
    "more_tiles_odd_columns": (9001, 64, 0, 517, BF16, BF16, "none", True, True),
    "narrow_and_tall": (20000, 320, 0, 21, BF16, BF16, "gelu", False, True),
    "deep_and_small": (40, 8192, 0, 24, BF16, BF16, "none", True, True),
}


@pytest.mark.parametrize("variant", ["release", "debug"])
@pytest.mark.parametrize("name", PRODUCTS)
def test_matmul_matches_64_bits(cuda_dev, name, variant):
    M, K, K2, N, dtype, out, act, bias, residual = PRODUCTS[name]
    run_matmul(randn(1, M, K, dtype=dtype, mean=0.1), randn(2, N, K + K2, dtype=dtype, spread=(K + K2) ** -0.5),
               randn(3, N) if bias else None, act, randn(4, M, N, dtype=out) if residual else None,
               randn(5, M, K2, dtype=dtype) if K2 else None, out_dtype=out, variant=variant)
    assert wino.check_device_error_ops(variant=variant) == wino.OK


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("lo,pad", [(0, 8), (8, 24), (3, 5), (1, 0)])
@pytest.mark.parametrize("M", [4, 150])
def test_matmul_ranges_of_wider_tensors(cuda_dev, dtype, out, lo, pad, M):
    """Operands, residual and output are column ranges of wider tensors whose other columns are NaN
    (never read into a result) or a mark (never written)."""
    K, K2, N = 72, 40, 48

    def part(seed, rows, cols, dt):
        t = torch.full((rows + 1, lo + cols + pad), float("nan"), device="cuda", dtype=dt)
        v = t[:rows, lo:lo + cols]
        v.copy_(randn(seed, rows, cols, dtype=dt))
        return v
    outer = torch.full((M + 1, lo + N + pad), 7.0, device="cuda", dtype=out)
    y = outer[:M, lo:lo + N]
    run_matmul(part(1, M, K, dtype), part(2, N, K + K2, dtype), randn(3, N + 1)[1:], "silu", part(4, M, N, out),
               part(5, M, K2, dtype), out=y)
    rest = torch.ones_like(outer, dtype=torch.bool)
    rest[:M, lo:lo + N] = False
    assert (outer[rest] == 7.0).all()


@pytest.mark.parametrize("M,K,N", [(3, 64, 40), (300, 128, 96), (9000, 64, 640), (130, 40, 33), (512, 2560, 1280)])
def test_matmul_adds_in_place(cuda_dev, M, K, N):
    a, w, res = randn(1, M, K, dtype=BF16), randn(2, N, K, dtype=BF16, spread=K ** -0.5), randn(3, M, N, dtype=BF16)
    want = wino.matmul(a, w, residual=res)
    y = wino.matmul(a, w, residual=res, out=res)
    assert y is res and torch.equal(y, want)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("out_lo,out_pad,res_lo,res_pad", [(1, 0, 0, 0), (0, 1, 5, 2), (7, 6, 2, 9), (4, 4, 1, 6), (0, 0, 3, 0)])
@pytest.mark.parametrize("M,N", [(17, 1), (33, 7), (129, 66), (300, 250), (65, 515)])
def test_matmul_rows_start_anywhere(cuda_dev, out, out_lo, out_pad, res_lo, res_pad, M, N):
    """Rows of the output and of the residual start at any offset within 16 bytes, each its own; beside them lie NaN
    (the residual, never read into a result) and marks (the output, never written)."""
    K = 96
    wide = torch.full((M, res_lo + N + res_pad), float("nan"), device="cuda", dtype=out)
    res = wide[:, res_lo:res_lo + N]
    res.copy_(randn(4, M, N, dtype=out))
    outer = torch.full((M + 1, out_lo + N + out_pad), 7.0, device="cuda", dtype=out)
    y = outer[:M, out_lo:out_lo + N]
    for variant in ("release", "debug"):
        run_matmul(randn(1, M, K, dtype=BF16), randn(2, N, K, dtype=BF16, spread=K ** -0.5), randn(3, N), "gelu", res, out=y,
                   variant=variant)
    rest = torch.ones_like(outer, dtype=torch.bool)
    rest[:M, out_lo:out_lo + N] = False
    assert (outer[rest] == 7.0).all() and wino.check_device_error_ops(variant="debug") == wino.OK


@pytest.mark.parametrize("M,K,N", [(9001, 64, 517), (9000, 320, 640), (9000, 192, 1280), (20001, 128, 333)])
@pytest.mark.parametrize("in_place", [False, True])
def test_matmul_many_tiles_of_few_blocks(cuda_dev, M, K, N, in_place):
    a, w, res = randn(1, M, K, dtype=BF16), randn(2, N, K, dtype=BF16, spread=K ** -0.5), randn(3, M, N, dtype=BF16)
    run_matmul(a, w, None, "silu", res, **({"out": res} if in_place else {}))


def test_given_outputs_count_as_changed(cuda_dev):
    """A backward pass that saved a tensor which a call then writes raises, as after any in-place change."""
    x = randn(1, 2, 4, 4, 32).requires_grad_()
    w, g = randn(2, 32, 32), randn(3, 2, 4, 4, 32)
    for call in (lambda t: wino.group_norm(g, 4, out=t), lambda t: wino.matmul(g, w, out=t)):
        h = x * 2.0
        z = (h * h).sum()
        with torch.no_grad():
            call(h)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()


def test_refused_calls_leave_the_output_unchanged(cuda_dev):
    """A refused call writes nothing, and a backward pass that saved its output tensor is not told of a change."""
    x = randn(1, 2, 4, 4, 32).requires_grad_()
    w, g = randn(2, 32, 32), randn(3, 2, 4, 4, 32)
    for call in (lambda t: wino.group_norm(g, 5, out=t), lambda t: wino.matmul(g, w, act=9, out=t)):
        h = x * 2.0
        kept, version = h.detach().clone(), h._version
        z = (h * h).sum()
        with torch.no_grad(), pytest.raises(wino.WinoError):
            call(h)
        assert h._version == version and torch.equal(h, kept)
        z.backward()
    with torch.inference_mode():
        frozen = torch.zeros_like(g)
        assert wino.matmul(g, w, out=frozen) is frozen
    kept = frozen.clone()
    for call in (lambda: wino.matmul(w, w, out=frozen[0].view(16, 32)[:4]), lambda: wino.group_norm(g, 4, out=frozen)):
        with pytest.raises((RuntimeError, ValueError)):
            call()
    assert torch.equal(frozen, kept)


@pytest.mark.parametrize("M,K,N", [(5, 200, 64), (200, 200, 96), (9000, 128, 640), (512, 2560, 320)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_matmul_non_finite_stays_in_its_row_and_column(cuda_dev, M, K, N, bad):
    a, w = randn(1, M, K, dtype=BF16), randn(2, N, K, dtype=BF16)
    clean = wino.matmul(a, w)
    a2, w2 = a.clone(), w.clone()
    a2[M // 2, K - 1] = bad
    y = wino.matmul(a2, w)
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[M // 2]).any()
    w2[N - 1, 0] = bad
    y = wino.matmul(a, w2)
    assert torch.equal(y[:, :N - 1], clean[:, :N - 1]) and not torch.isfinite(y[:, N - 1]).any()


@pytest.mark.parametrize("M,K,K2,N,out", [(300, 77, 0, 45, BF16), (300, 77, 0, 45, F32), (140, 40, 27, 333, BF16),
                                          (9001, 64, 0, 517, BF16), (40, 200, 8, 3, F32), (2000, 129, 0, 65, BF16)])
def test_matmul_odd_sizes_in_padded_rows(cuda_dev, M, K, K2, N, out):
    """Sizes that are no multiple of anything in rows padded to 16 bytes: the padding is neither read into a result
    (it holds NaN) nor written (it holds a mark)."""
    def padded(seed, rows, cols, dt):
        t = torch.full((rows, (cols + 7) // 8 * 8 + 8), float("nan"), device="cuda", dtype=dt)
        t[:, :cols] = randn(seed, rows, cols, dtype=dt)
        return t[:, :cols]
    outer = torch.full((M + 3, (N + 7) // 8 * 8 + 8), 7.0, device="cuda", dtype=out)
    run_matmul(padded(1, M, K, BF16), padded(2, N, K + K2, BF16), randn(3, N), "gelu", padded(4, M, N, out),
               padded(5, M, K2, BF16) if K2 else None, out=outer[:M, :N])
    assert (outer[M:] == 7.0).all() and (outer[:, N:] == 7.0).all()


@pytest.mark.parametrize("M,K,N", [(2200000, 1024, 40), (70000, 64, 32768), (33, 64, 40)])
def test_matmul_beyond_32_bit_offsets(cuda_dev, M, K, N):
    """More than 2^31 values in a, or in the output: a row's result does not depend on the rows before it."""
    a = torch.empty(M, K, device="cuda", dtype=BF16).normal_()
    w = randn(2, N, K, dtype=BF16)
    y = wino.matmul(a, w)
    for lo in (0, M // 2 // 256 * 256, max(0, M - 200) // 256 * 256):
        part = a[lo:lo + 256].clone()
        assert torch.equal(y[lo:lo + part.shape[0]], wino.matmul(part, w))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("variant", ["release", "debug"])
def test_matmul_rows_longer_than_2_gb(cuda_dev, out, variant):
    """Rows of the output and of the residual of more than 2^31 bytes (each row starts anywhere within 16): columns at both
    ends and on either side of where as many bytes are left, against 64 bits."""
    M, K = 9, 8
    N = (1 << 31) // out.itemsize + 1
    a, w = randn(1, M, K, dtype=BF16), torch.empty(N, K, device="cuda", dtype=BF16)
    res = torch.empty(M, N, device="cuda", dtype=out)
    for r in (*w.split(1 << 27), *res):
        r.normal_()
    ranges = [slice(lo, lo + 700) for lo in (0, N // 2 - 350, N - 700)]
    kept = [res[:, s].clone() for s in ranges]
    assert wino.matmul(a, w, residual=res, out=res, variant=variant) is res
    assert wino.check_device_error_ops(variant=variant) == wino.OK
    for s, r in zip(ranges, kept):
        check(res[:, s], *ref_matmul(a, w[s], None, "none", r, None, out), "columns from %d" % s.start)


def test_matmul_residual_of_infinities(cuda_dev):
    a, w = randn(1, 40, 64, dtype=BF16), randn(2, 48, 64, dtype=BF16)
    res = randn(3, 40, 48, dtype=BF16)
    res[3, 4], res[5, 6] = float("inf"), float("nan")
    y = run_free = wino.matmul(a, w, residual=res)
    assert y[3, 4] == float("inf") and torch.isnan(run_free[5, 6]) and int((~torch.isfinite(y)).sum()) == 2


def test_extreme_preactivations(cuda_dev):
    """SiLU and GELU at both ends: no overflow on the way, zeros on the left, identity on the right."""
    v = torch.tensor([-1e30, -1e4, -200.0, -90.0, -88.0, -20.0, 0.0, 20.0, 90.0, 1e4, 1e30], device="cuda")
    one = torch.ones(1, 8, device="cuda")
    w = torch.zeros(v.numel(), 8, device="cuda")
    w[:, 0] = v
    for act in ("silu", "gelu"):
        for dt in (F32, BF16):
            y = wino.matmul(one.to(dt), w.to(dt), act=ACTS[act], out_dtype=F32)[0]
            want = ref_act(w.to(dt)[:, 0].double(), act)
            assert ((y.double() - want).abs() <= 1e-5 * want.abs() + 1e-30).all(), (act, dt, y, want)
            yb = wino.matmul(one.to(dt), w.to(dt), act=ACTS[act], out_dtype=BF16)[0]
            assert ((yb.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all(), (act, dt, yb, want)


# ---------------------------------------------------------------- both
def _block(x, skip, emb, p):
    """A residual block of an image network as the library runs it: norm + SiLU, int8 convolution, norm
    (with the time embedding's projection added) + SiLU, int8 convolution, 1x1 shortcut + residual."""
    t = wino.matmul(emb, p["w_emb"], bias=p["b_emb"], out_dtype=F32)
    h = wino.group_norm(x, 32, p["g1"], p["b1"], act=wino.ACT_SILU, x2=skip)
    h = p["plan"].conv2d(h, p["wt1"], p["cout"])
    h = wino.group_norm(h, 32, p["g2"], p["b2"], act=wino.ACT_SILU, add=t)
    h = p["plan"].conv2d(h, p["wt2"], p["cout"])
    return t, wino.matmul(x, p["w_sc"], bias=p["b_sc"], residual=h, a2=skip, out=h)


def test_residual_block(cuda_dev):
    """The operators with the convolution between them: the block's projection, norms and shortcut each
    match 64 bits on the tensors that the run itself produced, and the whole run repeats bit for bit."""
    N, H, W, c0, c1, cout, E = 2, 16, 13, 128, 64, 128, 256
    plan = wino.Plan(6, synth.POINTS_F6, group=64)
    p = dict(plan=plan, cout=cout, w_emb=randn(1, cout, E, dtype=BF16, spread=E ** -0.5), b_emb=randn(2, cout),
             g1=randn(3, c0 + c1, mean=1.0, spread=0.1), b1=randn(4, c0 + c1, spread=0.1),
             g2=randn(5, cout, mean=1.0, spread=0.1), b2=randn(6, cout, spread=0.1),
             w_sc=randn(7, cout, c0 + c1, dtype=BF16, spread=(c0 + c1) ** -0.5), b_sc=randn(8, cout, spread=0.1),
             wt1=plan.transform_weights(randn(9, cout, 3, 3, c0 + c1, spread=0.03)),
             wt2=plan.transform_weights(randn(10, cout, 3, 3, cout, spread=0.03)))
    x, skip = randn(11, N, H, W, c0, dtype=BF16), randn(12, N, H, W, c1, dtype=BF16)
    emb = randn(13, N, E, dtype=BF16)
    t, y = _block(x, skip, emb, p)
    # step by step
    want, tol = ref_matmul(emb, p["w_emb"], p["b_emb"], "none", None, None, F32)
    check(t, want, tol, "embedding")
    h = run_norm(x, 32, p["g1"], p["b1"], act="silu", x2=skip)
    h = plan.conv2d(h, p["wt1"], cout)
    h = run_norm(h, 32, p["g2"], p["b2"], act="silu", add=t)
    h = plan.conv2d(h, p["wt2"], cout)
    want, tol = ref_matmul(x, p["w_sc"], p["b_sc"], "none", h, skip, BF16)
    check(y, want, tol, "shortcut")
    t2, y2 = _block(x, skip, emb, p)
    assert torch.equal(t, t2) and torch.equal(y, y2)
    assert wino.check_device_error_ops() == wino.OK


CALLS = {
    "norm": lambda s: wino.group_norm(s["x"], 32, s["gamma"], s["beta"], act=wino.ACT_SILU, add=s["add"], x2=s["x2"], out=s["y"]),
    "one_row": lambda s: wino.matmul(s["e"], s["we"], bias=s["be"], act=wino.ACT_SILU, out=s["t"]),
    "deep": lambda s: wino.matmul(s["d"], s["wd"], residual=s["rd"], out=s["od"]),
    "tall": lambda s: wino.matmul(s["p"], s["wp"], bias=s["bp"], act=wino.ACT_GELU, out=s["op"]),
}


def _state(seed):
    return dict(x=randn(seed, 2, 20, 20, 96, dtype=BF16), x2=randn(seed + 1, 2, 20, 20, 32, dtype=BF16),
                gamma=randn(seed + 2, 128), beta=randn(seed + 3, 128), add=randn(seed + 4, 2, 128),
                y=torch.empty(2, 20, 20, 128, device="cuda", dtype=BF16),
                e=randn(seed + 5, 2, 256, dtype=BF16), we=randn(seed + 6, 128, 256, dtype=BF16), be=randn(seed + 7, 128),
                t=torch.empty(2, 128, device="cuda", dtype=BF16),
                d=randn(seed + 8, 256, 2048, dtype=BF16), wd=randn(seed + 9, 256, 2048, dtype=BF16),
                rd=randn(seed + 10, 256, 256, dtype=BF16), od=torch.empty(256, 256, device="cuda", dtype=BF16),
                p=randn(seed + 11, 9000, 96, dtype=BF16), wp=randn(seed + 12, 640, 96, dtype=BF16), bp=randn(seed + 13, 640),
                op=torch.empty(9000, 640, device="cuda", dtype=BF16))


@pytest.mark.parametrize("name", CALLS)
def test_repeats_bit_for_bit(cuda_dev, name):
    s = _state(100)
    first = CALLS[name](s).clone()
    for _ in range(5):
        assert torch.equal(CALLS[name](s), first)


@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(cuda_dev, name):
    s = _state(200)
    CALLS[name](s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        CALLS[name](s)
        out = CALLS[name](s)
    for seed in (300, 400):
        other = _state(seed)
        for k, v in s.items():
            v.copy_(other[k])
        want = CALLS[name](other).clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_streams_at_once(cuda_dev):
    """Calls of all kinds on two streams at the same time give what they give alone."""
    states = [_state(500), _state(600)]
    want = [{n: f(s).clone() for n, f in CALLS.items()} for s in states]
    for s in states:
        for k in ("y", "t", "od", "op"):
            s[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(20):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                for f in CALLS.values():
                    f(s)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        for n, k in (("norm", "y"), ("one_row", "t"), ("deep", "od"), ("tall", "op")):
            assert torch.equal(s[k], w[n]), n


def test_explicit_stream(cuda_dev):
    st = torch.cuda.Stream()
    x = randn(1, 1, 16, 16, 64, dtype=BF16)
    a, w = randn(2, 300, 64, dtype=BF16), randn(3, 80, 64, dtype=BF16)
    want = wino.group_norm(x, 8), wino.matmul(a, w)
    torch.cuda.synchronize()
    got = wino.group_norm(x, 8, stream=st), wino.matmul(a, w, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


FIRST_CALL_IN_CAPTURE = """
import torch
from group_wise_int8_b200 import wino
x = torch.randn(2, 16, 16, 64, device="cuda", dtype=torch.bfloat16)
a, w = torch.randn(700, 64, device="cuda", dtype=torch.bfloat16), torch.randn(96, 64, device="cuda", dtype=torch.bfloat16)
f, v = torch.randn(700, 64, device="cuda"), torch.randn(96, 64, device="cuda")
wino.load_torch_ops()
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    y = wino.group_norm(x, 8, act=wino.ACT_SILU)
    z = wino.matmul(a, w), wino.matmul(f, v), wino.matmul(a[:2], w)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, wino.group_norm(x, 8, act=wino.ACT_SILU))
assert torch.equal(z[0], wino.matmul(a, w)) and torch.equal(z[1], wino.matmul(f, v)) and torch.equal(z[2], wino.matmul(a[:2], w))
print("captured")
"""


def test_first_call_in_a_capture(cuda_dev):
    """A process whose very first calls are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_two_host_threads(cuda_dev):
    """Calls from two threads, each on a stream of its own."""
    import threading
    states = [_state(700), _state(800)]
    want = [{n: f(s).clone() for n, f in CALLS.items()} for s in states]
    torch.cuda.synchronize()
    failed = []

    def work(s, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                for n, f in CALLS.items():
                    if not torch.equal(f(s), w[n]):
                        failed.append(n)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=p) for p in zip(states, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("M,K,N,out", [(129, 128, 256, BF16), (512, 2560, 1280, BF16), (9000, 320, 640, BF16), (9001, 64, 517, BF16),
                                       (20000, 1280, 320, F32)])
@pytest.mark.parametrize("residual", [False, True])
def test_bounded_wait_expiry_is_reported_and_recoverable(cuda_dev, M, K, N, out, residual):
    """A wait of the tensor-core kernel that runs out after 1 ms, before each pair's last tile: the kernel returns at once
    (both CTAs of a pair leave, with loads and products under way), the error is reported once, and the next call is right."""
    a, w, res = randn(1, M, K, dtype=BF16), randn(2, N, K, dtype=BF16, spread=K ** -0.5), randn(3, M, N, dtype=out)
    y = torch.empty(M, N, device="cuda", dtype=out)
    lib = wino.load_library()
    want = run_matmul(a, w, residual=res if residual else None, out_dtype=out)
    assert wino.check_device_error_ops() == wino.OK
    for _ in range(3):
        args = wino._MATMUL_ARGS.pack(a.data_ptr(), 0, w.data_ptr(), 0, res.data_ptr() if residual else 0, y.data_ptr(), K, 0, K, N, N,
                                      wino.BF16, wino.BF16 if out == BF16 else wino.F32, M, N, K, 0, wino.ACT_NONE,
                                      wino.DEBUG_FORCE_TIMEOUT)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        assert lib.wino_matmul(args, torch.cuda.current_stream().cuda_stream) == wino.OK
        end.record()
        assert wino.check_device_error_ops() == wino.ERR_DEVICE_TIMEOUT
        assert wino.check_device_error_ops() == wino.OK
        assert start.elapsed_time(end) < 500
        assert torch.equal(wino.matmul(a, w, residual=res if residual else None, out_dtype=out), want)
    assert wino.check_device_error_ops() == wino.OK


@pytest.mark.parametrize("N,hw,C,groups,dtype", [(65536, 1, 32, 4, BF16), (70001, 2, 33, 3, F32), (131072, 1, 8, 8, F32)])
def test_group_norm_of_more_images_than_a_grid_dimension(cuda_dev, N, hw, C, groups, dtype):
    run_norm(randn(1, N, hw, 1, C, dtype=dtype, mean=0.3), groups, randn(2, C), randn(3, C), act="silu", add=randn(4, N, C))


@pytest.mark.parametrize("M", [524279, 524280, 524281])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matmul_of_many_rows_and_one_column(cuda_dev, M, dtype):
    """Around the most rows that the row kernel's grid holds (fp32 takes it for one column of a long K)."""
    run_matmul(randn(1, M, 700, dtype=dtype), randn(2, 1, 700, dtype=dtype, spread=0.04), randn(3, 1), "silu", randn(4, M, 1, dtype=dtype))


def test_the_same_tensor_in_two_places(cuda_dev):
    x, a = randn(1, 2, 9, 7, 48, dtype=BF16), randn(2, 300, 64, dtype=BF16)
    run_norm(x, 6, x2=x, act="silu")
    p = randn(3, 48)
    run_norm(x, 6, p, p, add=torch.stack([p, p]))
    run_matmul(a, a)
    run_matmul(a, torch.cat([a[:80], a[:80]], 1), a2=a, residual=None)
    sq = randn(4, 64, 64, dtype=BF16)
    run_matmul(sq, sq, None, "gelu", sq, None)


def test_single_rows_of_any_pitch(cuda_dev):
    """One pixel or row: its pitch is read by nothing, through the C ABI too."""
    lib, st = wino.load_library(), torch.cuda.current_stream().cuda_stream
    x, y = randn(1, 1, 1, 1, 64, dtype=BF16), torch.full((80,), 7.0, device="cuda", dtype=BF16)
    want = wino.group_norm(x, 8).flatten()
    a, w = randn(2, 1, 64, dtype=BF16), randn(3, 40, 64, dtype=BF16)
    product = wino.matmul(a, w).flatten()
    for pitch in (0, 3, 64, 1000):
        y.fill_(7.0)
        args = wino._GROUP_NORM_ARGS.pack(x.data_ptr(), 0, 0, 0, 0, y.data_ptr(), pitch, 0, pitch, wino.BF16, wino.BF16, 1, 1, 1, 64, 0, 8, 0,
                                          1e-5)
        assert lib.wino_group_norm(args, st) == wino.OK and torch.equal(y[:64], want) and (y[64:] == 7.0).all()
        y.fill_(7.0)
        args = wino._MATMUL_ARGS.pack(a.data_ptr(), 0, w.data_ptr(), 0, 0, y.data_ptr(), pitch, 0, 64, 0, pitch, wino.BF16, wino.BF16,
                                      1, 40, 64, 0, 0, 0)
        assert lib.wino_matmul(args, st) == wino.OK and torch.equal(y[:40], product) and (y[40:] == 7.0).all()


def test_forward_mode_tangents_are_refused(cuda_dev):
    import torch.autograd.forward_ad as fwd
    x, g, a, w = randn(1, 1, 4, 4, 32), randn(2, 32), randn(3, 4, 32), randn(4, 8, 32)
    with fwd.dual_level():
        dual = {k: fwd.make_dual(t, torch.ones_like(t)) for k, t in dict(x=x, g=g, a=a, w=w).items()}
        for call in (lambda: wino.group_norm(dual["x"], 8), lambda: wino.group_norm(x, 8, gamma=dual["g"]),
                     lambda: wino.group_norm(x, 8, x2=dual["x"]), lambda: wino.group_norm(x, 8, out=dual["x"]),
                     lambda: wino.matmul(dual["a"], w), lambda: wino.matmul(a, dual["w"]),
                     lambda: wino.matmul(a, w, residual=dual["a"][:, :8].contiguous())):
            for mode in (torch.enable_grad, torch.no_grad):   # (which stops the recording of backward passes only)
                with mode(), pytest.raises(ValueError, match="tangent"):
                    call()
        # their primals, and plain tensors beside them, are fine
        assert torch.equal(wino.matmul(fwd.unpack_dual(dual["a"]).primal, w), wino.matmul(a, w))
        with fwd._set_fwd_grad_enabled(False):
            assert torch.equal(wino.matmul(dual["a"], w), wino.matmul(a, w))
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.jvp(lambda t: wino.matmul(t, w), (a,), (a,))
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.grad(lambda t: wino.matmul(t, w).sum())(a)
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.vmap(lambda t: wino.matmul(t, w))(a[None])


def test_negated_views_are_refused(cuda_dev):
    x, g, a, w = randn(1, 1, 4, 4, 32), randn(2, 32), randn(3, 4, 32), randn(4, 8, 32)
    neg = torch._neg_view
    for call in (lambda: wino.group_norm(neg(x), 8), lambda: wino.group_norm(x, 8, gamma=neg(g)), lambda: wino.group_norm(x, 8, x2=neg(x)),
                 lambda: wino.group_norm(x, 8, out=neg(x)), lambda: wino.matmul(neg(a), w), lambda: wino.matmul(a, neg(w)),
                 lambda: wino.matmul(a, w, bias=neg(g)[:8]), lambda: wino.matmul(a, w, a2=neg(a))):
        with pytest.raises(ValueError, match="negated"):
            call()
    c = torch.complex(randn(5, 8, 1), randn(6, 8, 1)).conj().imag   # one column: any distance between rows will do
    with pytest.raises(ValueError, match="negated"):
        wino.matmul(c, w[:, :1])
    assert torch.equal(wino.matmul(neg(a).resolve_neg(), w), -wino.matmul(a, w))


def test_no_memory_for_the_output(cuda_dev):
    """An output of 2 TB: torch's own error, and the next call works."""
    a, w = randn(1, 1 << 20, 8, dtype=BF16), randn(2, 1 << 20, 8, dtype=BF16)
    with pytest.raises(torch.OutOfMemoryError, match="out of memory"):
        wino.matmul(a, w)
    run_matmul(a[:300], w[:40])


def test_binding_refusals(cuda_dev):
    x, a, w = randn(1, 1, 4, 4, 32, dtype=BF16), randn(2, 4, 32, dtype=BF16), randn(3, 8, 32, dtype=BF16)
    for bad in (lambda: wino.group_norm(x[0], 8), lambda: wino.group_norm(x.half(), 8),
                lambda: wino.group_norm(x, 8, gamma=torch.ones(31, device="cuda")),
                lambda: wino.group_norm(x, 8, gamma=torch.ones(32, device="cuda", dtype=BF16)),
                lambda: wino.group_norm(x, 8, gamma=torch.ones(32)),
                lambda: wino.group_norm(x, 8, beta=torch.ones(64, device="cuda")[::2]),
                lambda: wino.group_norm(x, 8, add=torch.ones(2, 32, device="cuda")),
                lambda: wino.group_norm(x, 8, x2=x.float()), lambda: wino.group_norm(x, 8, x2=x[:, :2]),
                lambda: wino.group_norm(x, 8, out=torch.empty(1, 4, 4, 64, device="cuda", dtype=BF16)),
                lambda: wino.group_norm(x.permute(0, 3, 1, 2), 4), lambda: wino.group_norm(x, 8, out_dtype=torch.float16),
                lambda: wino.group_norm(x, 8, gamma=torch.ones(32, device="cuda", requires_grad=True)),
                lambda: wino.matmul(a, w[:, :16]), lambda: wino.matmul(a, w.float()), lambda: wino.matmul(a, w.cpu()),
                lambda: wino.matmul(a, w, bias=torch.ones(9, device="cuda")), lambda: wino.matmul(a.half(), w.half()),
                lambda: wino.matmul(a, w, residual=torch.ones(4, 9, device="cuda", dtype=BF16)),
                lambda: wino.matmul(a, w, residual=torch.ones(4, 8, device="cuda"), out_dtype=BF16),
                lambda: wino.matmul(a, w, a2=a[:2]), lambda: wino.matmul(a.t(), w),
                lambda: wino.matmul(a, w.float().requires_grad_().to(BF16))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: wino.group_norm(x, 5), lambda: wino.group_norm(x, 8, eps=-1.0), lambda: wino.group_norm(x, 8, act=9),
                lambda: wino.group_norm(x[:, :0], 8), lambda: wino.matmul(a[:0], w), lambda: wino.matmul(a[:, :0], w[:, :0]),
                lambda: wino.matmul(a, w, act=9), lambda: wino.matmul(a[:1].expand(4, 32), w),
                lambda: wino.matmul(a, a, out=a[:, :4])):
        with pytest.raises(wino.WinoError) as e:
            bad()
        assert e.value.status == wino.ERR_INVALID_ARG
    # parameters that require grad are fine where no gradient is recorded
    with torch.no_grad():
        wino.group_norm(x, 8, gamma=torch.ones(32, device="cuda", requires_grad=True))
