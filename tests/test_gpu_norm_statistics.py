"""GPU tests of wino_group_norm's statistics with bounds that follow the sums the kernel makes, for images of many pixels.

With u = 2^-24: a thread sums squares around a pivot in blocks of at most BLOCK rows, then adds the blocks with two more
roundings each, and the joins of row offsets, channels and CTAs add a few dozen terms more (JOINS).  Each sum of n terms
is off by at most n u of its terms' magnitudes, so the variance is off by
  (BLOCK + JOINS + 2 rows of a thread / BLOCK) u  times  (the squares that were summed) / (pixels x channels of the group).
Around a pivot that is the mean of the rows so far, the squares summed are those of the deviations from the mean, within
a factor of SQUARES; a first block around an outlier adds BLOCK times the outlier's square.
"""
import pytest
import torch

from group_wise_int8_b200 import wino
from tests.test_gpu_ops import BF16, F32, U, act_error, check, randn, ref_act

pytestmark = pytest.mark.gpu

BLOCK, JOINS, SQUARES = 64, 64, 8
CTAS = 16          # of a cluster, at most: a thread has at least pixels / CTAS / 256 rows, at most pixels / CTAS


def ref_norm(x, groups, act, out_dtype, outliers=0, outlier=0.0, rows=None):
    """-> (reference in 64 bits, tolerance); `outliers` pixels lie `outlier` from the others; `rows`: of a thread."""
    N, H, W, C = x.shape
    g = x.double().view(N, H * W, groups, C // groups)
    mean, var = g.mean(dim=(1, 3), keepdim=True), g.var(dim=(1, 3), correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + 1e-5)
    z = (g - mean) * rstd
    pre = z.view_as(x)
    want = ref_act(pre, act)
    terms = BLOCK + JOINS + (H * W // CTAS if rows is None else rows) * 2 / BLOCK
    summed = SQUARES * var + outliers * BLOCK * outlier ** 2 / (H * W)
    rel = 0.5 * terms * U * summed * rstd * rstd + 4 * U                    # of rstd
    top = g.abs().amax(dim=(1, 3), keepdim=True) if not outliers else outlier
    mean_err = terms * U * torch.sqrt(summed) + 8 * U * top
    err = act_error(pre, act, ((mean_err + 4 * U * g.abs()) * rstd + z.abs() * rel).view_as(x), out_dtype == BF16)
    return want, err + (want.abs() + err) * torch.finfo(out_dtype).eps / 2


@pytest.mark.parametrize("H,W,C,groups,dtype,rows", [
    (2048, 2048, 32, 8, F32, 8192), (2048, 2048, 32, 1, BF16, 8192), (1500, 1401, 33, 33, F32, 20000),
    (512, 500, 512, 2, BF16, 4000), (400, 400, 2048, 1, BF16, 10000)])
def test_outliers_at_the_first_pixels(cuda_dev, H, W, C, groups, dtype, rows):
    """Large images, zero at most pixels, whose first pixels lie far from all others: around those, which are the first
    CTA's first values, thousands of equal squares would be summed, and their roundings with them."""
    outliers, outlier = 4, 1000.1
    x = randn(1, 1, H, W, C, dtype=dtype)
    x *= torch.arange(H * W, device="cuda").view(1, H, W, 1) % 16 == 0
    x.view(H * W, C)[:outliers] = outlier
    y = wino.group_norm(x, groups, out_dtype=F32)
    want, tol = ref_norm(x, groups, "none", F32, outliers, outlier, rows)
    assert (tol < 0.01 * (1 + want.abs())).all()
    check(y, want, tol)


def banded(seed, N, H, W, C, dtype):
    """Every channel and every band of rows has a mean and a spread of its own, so that statistics of a subset differ."""
    x = randn(seed, N, H, W, C)
    bands = torch.arange(H, device="cuda") * 24 // max(H, 24)
    x *= torch.exp(0.5 * randn(seed + 1, 24, C)[bands]).view(1, H, 1, C)
    x += randn(seed + 2, 24, C)[bands].view(1, H, 1, C) + 0.5 * randn(seed + 3, N, 1, 1, C)
    return x.to(dtype)


IMAGES = {
    # N, H, W, C, groups, dtype, out, act, rows of a thread at most
    "level_64": (2, 64, 64, 320, 32, BF16, BF16, "silu", 256),
    "level_64_f32": (2, 64, 64, 320, 32, F32, F32, "silu", 256),
    "streamed": (1, 160, 150, 128, 1, BF16, BF16, "silu", 1500),
    "streamed_f32": (1, 131, 97, 128, 2, F32, F32, "none", 800),
    "decoder": (1, 256, 256, 128, 32, BF16, BF16, "silu", 4096),
    "decoder_f32": (1, 256, 240, 128, 32, F32, F32, "none", 4096),
    "odd": (2, 131, 120, 33, 3, BF16, F32, "none", 1000),
    "wide_images": (3, 256, 256, 1024, 32, BF16, BF16, "silu", 4096),
}


@pytest.mark.parametrize("name", IMAGES)
def test_statistics_of_many_pixels(cuda_dev, name):
    N, H, W, C, groups, dtype, out, act, rows = IMAGES[name]
    x = banded(1, N, H, W, C, dtype)
    y = wino.group_norm(x, groups, act={"none": wino.ACT_NONE, "silu": wino.ACT_SILU}[act], out_dtype=out)
    for n in range(N):
        want, tol = ref_norm(x[n:n + 1], groups, act, out, rows=rows)
        check(y[n:n + 1], want, tol, "image %d" % n)


def test_the_bound_rejects_statistics_of_a_subset(cuda_dev):
    """The same bound against 64-bit results (on the CPU) whose statistics leave out one CTA's rows, a 64th of the image (where
    the output is fp32), or whose variance is off by 1 %: each is off at many elements."""
    for N, H, W, C, groups, dtype, out, act, rows in (IMAGES["level_64"], IMAGES["streamed"], IMAGES["streamed_f32"], IMAGES["odd"]):
        x = banded(1, N, H, W, C, dtype)[:1].cpu()
        want, tol = ref_norm(x, groups, act, out, rows=rows)
        g = x.double().view(1, H * W, groups, C // groups)
        for lost in (slice(0, H * W // CTAS), slice(H * W // 2, H * W // 2 + H * W // CTAS), slice(H * W - H * W // 64, H * W), None):
            kept = g
            # A 64th is lost in bf16's rounding where a group has many channels: the missing rows' mean over 128 channels lies
            # 128^-1/2 = 0.09 spreads from the group's, which moves the mean by 0.09 / 64 = 0.0014 of them, against a rounding of
            # up to 2^-8 = 0.004 of the value; their squares, averaged alike, move the variance by as little.
            if out == BF16 and lost is not None and lost.start == H * W - H * W // 64:
                continue
            if lost is not None:
                keep = torch.ones(H * W, dtype=torch.bool)
                keep[lost] = False
                kept = g[:, keep]
            mean, var = kept.mean(dim=(1, 3), keepdim=True), kept.var(dim=(1, 3), correction=0, keepdim=True)
            if lost is None:
                var = var * 1.01
            wrong = ref_act(((g - mean) / torch.sqrt(var + 1e-5)).view_as(x), act).to(out)
            off = ((wrong.double() - want).abs() > tol).double().mean().item()
            assert off > 0.02, (H, W, lost, off)
