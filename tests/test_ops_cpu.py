"""Host-side checks of wino_group_norm and wino_matmul that need no GPU: every refusal comes before
anything is launched, and the binding's argument packing matches the header's structs."""
import os
import subprocess

import pytest
import torch

from group_wise_int8_b200 import build, wino

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NORM_FIELDS = ["x", "x2", "add", "gamma", "beta", "y", "x_pitch", "x2_pitch", "y_pitch", "x_dtype", "y_dtype",
               "N", "H", "W", "C", "C2", "groups", "act", "eps"]
MATMUL_FIELDS = ["a", "a2", "w", "bias", "residual", "out", "a_pitch", "a2_pitch", "w_pitch", "residual_pitch",
                 "out_pitch", "dtype", "out_dtype", "M", "N", "K", "K2", "act", "reserved"]
# addresses for calls that are refused before anything reads them
P = [0x10000000 * (i + 1) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wino.load_library()


def norm(lib, **kw):
    v = dict(x=P[0], x2=0, add=P[2], gamma=P[3], beta=P[4], y=P[5], x_pitch=64, x2_pitch=0, y_pitch=64, x_dtype=wino.BF16,
             y_dtype=wino.BF16, N=2, H=4, W=4, C=64, C2=0, groups=32, act=0, eps=1e-5)
    assert set(kw) <= set(v)
    v.update(kw)
    return lib.wino_group_norm(wino._GROUP_NORM_ARGS.pack(*[v[f] for f in NORM_FIELDS]), None)


def product(lib, **kw):
    v = dict(a=P[0], a2=0, w=P[2], bias=P[3], residual=P[4], out=P[5], a_pitch=64, a2_pitch=0, w_pitch=64,
             residual_pitch=48, out_pitch=48, dtype=wino.BF16, out_dtype=wino.BF16, M=16, N=48, K=64, K2=0, act=0, reserved=0)
    assert set(kw) <= set(v)
    v.update(kw)
    return lib.wino_matmul(wino._MATMUL_ARGS.pack(*[v[f] for f in MATMUL_FIELDS]), None)


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(y=0), dict(N=0), dict(H=0), dict(W=-1), dict(C=0), dict(C2=-1), dict(groups=0), dict(groups=-32),
    dict(groups=48), dict(groups=128), dict(x_dtype=2), dict(y_dtype=-1), dict(act=3), dict(act=-1), dict(eps=-1e-5),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x_pitch=63), dict(y_pitch=32), dict(x_pitch=(1 << 31) + 1),
    dict(x2=P[1]),                                              # a second source of no channels
    dict(C2=64, x2_pitch=64, y_pitch=128),                      # channels of no second source
    dict(x2=P[1], C2=64, x2_pitch=32, y_pitch=128), dict(x2=P[1], C2=64, x2_pitch=64, y_pitch=64),
    dict(x=P[0] + 1), dict(y=P[5] + 1), dict(add=P[2] + 2), dict(gamma=P[3] + 1), dict(beta=P[4] + 3),
    dict(x=P[0] + 2, x_dtype=wino.F32),
    dict(H=1 << 16, W=1 << 16), dict(N=1 << 20, H=1 << 14, W=1 << 14),
    dict(y=P[0] + 64), dict(y=P[0], y_pitch=128), dict(y=P[0], y_dtype=wino.F32),   # overlaps, not in place
    dict(y=P[2]), dict(y=P[3]), dict(y=P[4] - 2),
    dict(x2=P[5], C2=64, x2_pitch=64, y_pitch=128),
    dict(x2=P[1], C2=64, x2_pitch=64, y=P[0], x_pitch=128, y_pitch=128),            # in place needs one source
], ids=str)
def test_group_norm_refuses(lib, kw):
    assert norm(lib, **kw) == wino.ERR_INVALID_ARG


def test_group_norm_refuses_too_many_channels(lib):
    C = wino.GROUP_NORM_MAX_CHANNELS + 32
    assert norm(lib, C=C, x_pitch=C, y_pitch=C) == wino.ERR_UNSUPPORTED
    assert norm(lib, N=wino.GROUP_NORM_MAX_IMAGES + 1, H=1, W=1, C=32, x_pitch=32, y_pitch=32, x=P[0], y=1 << 50) == wino.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(a=0), dict(w=0), dict(out=0), dict(M=0), dict(M=-1), dict(N=0), dict(K=0), dict(K2=-64), dict(dtype=2),
    dict(out_dtype=7), dict(act=3), dict(a_pitch=63), dict(w_pitch=0), dict(residual_pitch=47), dict(out_pitch=47),
    dict(out_pitch=(1 << 31) + 1), dict(a2=P[1]), dict(K2=64, w_pitch=128), dict(a2=P[1], K2=64, a2_pitch=63, w_pitch=128),
    dict(a2=P[1], K2=64, a2_pitch=64, w_pitch=64), dict(a=P[0] + 1), dict(w=P[2] + 1), dict(out=P[5] + 1),
    dict(residual=P[4] + 1), dict(bias=P[3] + 2), dict(a=P[0] + 2, dtype=wino.F32), dict(out=P[5] + 2, out_dtype=wino.F32),
    dict(M=(1 << 31) - 1, K=1, a_pitch=1, w_pitch=1), dict(M=1 << 30, K=1 << 20, a_pitch=1 << 20, w_pitch=1 << 20),
    dict(out=P[0]), dict(out=P[2] + 64), dict(out=P[3]), dict(residual=P[5] + 16), dict(residual=P[5], residual_pitch=64),
    dict(a2=P[5], K2=64, a2_pitch=64, w_pitch=128),
], ids=str)
def test_matmul_refuses(lib, kw):
    assert product(lib, **kw) == wino.ERR_INVALID_ARG


def test_pitches_of_single_rows(lib):
    """A single row's pitch is read by nothing: 0 and any other count as the row's length in the overlap check."""
    one = dict(N=1, H=1, W=1)
    for pitch in (0, 1, 64, 128, 200):
        for at in (2, 126, -126):
            assert norm(lib, x_pitch=pitch, y_pitch=pitch, y=P[0] + at, **one) == wino.ERR_INVALID_ARG
        assert product(lib, M=1, N=1, a_pitch=pitch, out_pitch=pitch, residual_pitch=pitch, residual=0, out=P[0] + 2) == wino.ERR_INVALID_ARG
        assert product(lib, M=1, N=48, out_pitch=pitch, residual_pitch=pitch, residual=P[5] + 2) == wino.ERR_INVALID_ARG
    # side by side, and the same row: past the overlap check, refused for the channels after it
    C = wino.GROUP_NORM_MAX_CHANNELS + 32
    for pitch in (0, 7, C):
        for y in (P[0] + 2 * C, P[0] - 2 * C, P[0]):
            assert norm(lib, C=C, x_pitch=pitch, y_pitch=pitch, x=P[0], y=y, add=0, gamma=0, beta=0, **one) == wino.ERR_UNSUPPORTED
    # a single row between the columns that the output writes, and one that reaches into them
    wide = dict(C=C, x_pitch=C, y_pitch=4 * C, add=0, beta=0)
    assert norm(lib, gamma=P[5] + 2 * C, **wide) == norm(lib, gamma=P[5] + 4 * C, **wide) == wino.ERR_UNSUPPORTED
    assert norm(lib, gamma=P[5] + 2 * C - 4, **wide) == norm(lib, gamma=P[5] + 4 * C + 4, **wide) == wino.ERR_INVALID_ARG


SPLITS = r"""
#include <cstdio>
#include "group_norm_split.h"
using namespace wino;
using namespace wino::group_norm;
int main() {
    long calls = 0;
    auto fail = [&](const char* what, const GroupNormShape& a, int vec, const GroupNormSplit& s) {
        std::printf("%s: N %d, HW %ld, C %d, groups %d, %d bytes, vec %d -> %d groups, %d CTAs\n", what, a.N, a.HW, a.C, a.groups,
                    a.es, vec, s.gps, s.cluster);
        return 1;
    };
    const long pixels[] = {1, 2, 7, 64, 255, 256, 1024, 5000, 65536, 1l << 22, 1l << 30};
    const int images[] = {1, 2, 3, 8, 40, 3000};
    for (int groups = 1; groups <= 16384; groups += groups < 40 ? 1 : (groups < 2100 ? 23 : 389))
        for (int cg = 1; (long)groups * cg <= 16384; cg += cg < 5 ? 1 : cg / 3)
            for (long HW : pixels)
                for (int N : images) {
                    if ((HW + N + groups) % 3 != 0) continue;   // a third of them
                    for (int form = 0; form < 4; ++form) {
                        const GroupNormShape a = {HW, N, groups * cg, groups, form & 1 ? 2 : 4};
                        const int vec = form & 2 ? 16 / a.es : 1;
                        if (a.C % vec != 0) continue;
                        ++calls;
                        const GroupNormSplit s = choose(a, vec, 148);
                        Split k;
                        if (make_split(a, vec, s, &k) > kMaxSmem) return fail("too much shared memory", a, vec, s);
                        if (s.gps * k.slabs != groups || k.nv * vec != s.gps * cg) return fail("no whole slabs", a, vec, s);
                        if (s.cluster > HW || (s.cluster & (s.cluster - 1)) || s.cluster > kMaxCluster) return fail("no cluster", a, vec, s);
                        if ((long)k.share * s.cluster + k.extra != HW || k.extra >= s.cluster) return fail("rows lost", a, vec, s);
                        if (k.res_rows * (long)k.nch * a.es > k.keep_bytes) return fail("kept rows overlap", a, vec, s);
                        for (int tid = 0; tid < kThreads; ++tid)
                            if ((int)((uint32_t)tid * k.inv_tv >> 20) != tid / k.TV) return fail("row offsets", a, vec, s);
                        if (k.inv_cg)
                            for (int c = k.nch - 1; c >= 0; c -= 1 + k.nch / 7)
                                if ((int)(((uint64_t)c * k.inv_cg) >> 32) != c / cg) return fail("groups of channels", a, vec, s);
                    }
                }
    std::printf("ok %ld\n", calls);
    return 0;
}
"""


def test_every_split_fits(tmp_path):
    """The group norm's split rule over its whole range (up to 16384 channels in groups of any width): the chosen split's
    shared memory fits, its slabs and rows are whole."""
    src, exe = tmp_path / "splits.cpp", tmp_path / "splits"
    src.write_text(SPLITS)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "group_wise_int8_b200", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
    assert int(r.stdout.split()[1]) > 100000


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: needs a machine on which no launch can follow")
@pytest.mark.parametrize("N,hw,C,groups", [(2, 1024, 911, 911), (1, 256, 1061, 1061), (1, 256, 2039, 2039), (2, 1024, 1814, 907)])
def test_narrow_groups_reach_the_launch(lib, N, hw, C, groups):
    """Their exchange areas outgrow shared memory in the cheapest split; the call takes another one (and then finds no device)."""
    assert norm(lib, N=N, H=hw, W=1, C=C, groups=groups, x_pitch=C, y_pitch=C, y=1 << 40) == wino.ERR_CUDA
    assert lib.wino_last_cuda_error(None) != 9   # cudaErrorInvalidConfiguration


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: needs a machine on which no launch can follow")
def test_refusals_name_no_earlier_cuda_error(lib):
    assert norm(lib) == wino.ERR_CUDA and lib.wino_last_cuda_error(None) != 0   # no device here
    assert "cudaError" in str(wino._failed(wino.ERR_CUDA, "wino_group_norm", "release"))
    assert norm(lib, groups=5) == wino.ERR_INVALID_ARG
    assert "cudaError" not in str(wino._failed(wino.ERR_INVALID_ARG, "wino_group_norm", "release"))


def test_null_arguments_are_refused(lib):
    assert lib.wino_group_norm(None, None) == wino.ERR_INVALID_ARG
    assert lib.wino_matmul(None, None) == wino.ERR_INVALID_ARG


def test_channel_ranges_of_one_buffer_are_no_overlap(lib):
    """Two column ranges of one wider buffer with the same pitch share no byte, although their
    address ranges overlap: the call passes its checks (and then finds no device here, or a GPU
    box's first launch is never reached because the sizes are refused for their channels)."""
    C = wino.GROUP_NORM_MAX_CHANNELS + 32   # refused after the overlap check, before any launch
    wide = dict(C=C, x_pitch=2 * C, y_pitch=2 * C)
    assert norm(lib, y=P[0] + 2 * C, **wide) == wino.ERR_UNSUPPORTED
    assert norm(lib, y=P[0] + 2 * C - 2, **wide) == wino.ERR_INVALID_ARG
    assert norm(lib, x=P[0] + 2 * C, y=P[0], **wide) == wino.ERR_UNSUPPORTED
    assert norm(lib, x=P[0] + 2 * C - 2, y=P[0], **wide) == wino.ERR_INVALID_ARG
    assert norm(lib, y=P[0], **wide) == wino.ERR_UNSUPPORTED          # in place


@pytest.mark.parametrize("struct,name,fields", [(wino._GROUP_NORM_ARGS, "wino_group_norm_args", NORM_FIELDS),
                                                (wino._MATMUL_ARGS, "wino_matmul_args", MATMUL_FIELDS)])
def test_packing_matches_the_header(tmp_path, struct, name, fields):
    """Size and field offsets of the C struct against the binding's format."""
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "wino.h"\nint main(void) {\nprintf("%zu", sizeof(' + name + "));\n" +
                   "".join('printf(" %%zu", offsetof(%s, %s));\n' % (name, f) for f in fields) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got[0] == struct.size
    codes = []
    rest = struct.format.lstrip("@")
    while rest:
        digits = ""
        while rest[0].isdigit():
            digits, rest = digits + rest[0], rest[1:]
        codes += [rest[0]] * int(digits or 1)
        rest = rest[1:]
    sizes = {"P": 8, "q": 8, "i": 4, "f": 4}
    offsets, at = [], 0
    for c in codes:
        offsets.append(at)
        at += sizes[c]
    assert got[1:] == offsets


def test_binding_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "wino.h")).read()
    for name, value in (("WINO_ACT_NONE", wino.ACT_NONE), ("WINO_ACT_SILU", wino.ACT_SILU), ("WINO_ACT_GELU", wino.ACT_GELU),
                        ("WINO_GROUP_NORM_MAX_CHANNELS", wino.GROUP_NORM_MAX_CHANNELS),
                        ("WINO_GROUP_NORM_MAX_IMAGES", wino.GROUP_NORM_MAX_IMAGES)):
        assert "#define %s %d" % (name, value) in src


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(ValueError, match="CUDA"):
        wino.group_norm(torch.zeros(1, 4, 4, 32), 32)
    with pytest.raises(ValueError, match="CUDA"):
        wino.matmul(torch.zeros(4, 32), torch.zeros(8, 32))


def test_row_pitch_of_views(lib):
    pitch = wino.load_torch_ops()[0].pitch
    t = torch.zeros(2, 3, 4, 40)
    assert pitch(t) == 40
    assert pitch(t[..., 8:24]) == 40
    assert pitch(t[:1, :1, :1]) == 40                       # one row: its own length
    assert pitch(t[:, :, ::2]) == 80
    with pytest.raises(ValueError, match="evenly"):
        pitch(t[:, :, :3])
    with pytest.raises(ValueError, match="contiguous"):
        pitch(t.transpose(2, 3))
    assert pitch(torch.zeros(5, 1)[:, :1]) == 1
    assert pitch(torch.zeros(7)) == 7
