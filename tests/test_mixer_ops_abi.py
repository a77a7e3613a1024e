"""The C ABI of sliding-window attention and the RMS norm on the CPU: every
argument check with fake device addresses (rejected before any HIP call; not
run where a GPU is visible), and the host code under the sanitizers."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

import mamba_chunked_ssd_amd as ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GiB = 1 << 30
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        from mamba_chunked_ssd_amd import build
        build.build()
    return ssd.load_library()


no_gpu = pytest.mark.skipif(
    __import__("torch").cuda.is_available(),
    reason="fake device addresses are only passed where no GPU can be reached")


def addresses(names):
    return {n: (1 << 44) + 64 * GiB * i for i, n in enumerate(names.split())}


def attn_shape(**kw):
    d = dict(batch=2, seqlen=50, nheads=4, nkvheads=2, headdim=64, window=20, sinks=3, scale=0.125, dtype=BF16)
    d.update(kw)
    s = ssd.AttnShape(*[d.pop(k) for k in ("batch", "seqlen", "nheads", "nkvheads", "headdim", "window", "sinks", "scale",
                                           "dtype")])
    for k, v in d.items():
        if k == "reserved":
            s.reserved[0] = v
        else:
            setattr(s, k, ssd.HeadStride(*v))
    return s


def norm_shape(**kw):
    d = dict(batch=2, seqlen=50, channels=24, eps=1e-5, dtype=BF16, res_dtype=F32, y_dtype=BF16, scale_block=0)
    d.update(kw)
    s = ssd.NormShape(*[d.pop(k) for k in ("batch", "seqlen", "channels", "eps", "dtype", "res_dtype", "y_dtype",
                                           "scale_block")])
    for k, v in d.items():
        setattr(s, k, ssd.Stride(*v) if isinstance(v, tuple) else v)
    return s


def codes(**kw):
    return norm_shape(**{"y_dtype": E4M3, **kw})


CALLS = {
    "ssd_window_attn_fwd": ("q k v positions lengths kc vc y lse", attn_shape, None),
    "ssd_window_attn_bwd": ("q k v y lse dy lengths dq dk dv ws", attn_shape, "ssd_window_attn_bwd_workspace_size"),
    "ssd_window_attn_step": ("q k v positions kc vc y ws", lambda **k: attn_shape(**{"seqlen": 1, "window": 3000, **k}),
                             "ssd_window_attn_step_workspace_size"),
    "ssd_rms_norm_fwd": ("x residual weight lengths y scales residual_out", codes, None),
    "ssd_rms_norm_bwd": ("dy u weight dres lengths dx dresidual dweight ws", norm_shape, "ssd_rms_norm_bwd_workspace_size"),
}
OPTIONAL = {"ssd_window_attn_fwd": "positions lengths lse", "ssd_window_attn_bwd": "lengths", "ssd_window_attn_step": "",
            "ssd_rms_norm_fwd": "residual weight lengths residual_out",
            "ssd_rms_norm_bwd": "weight dres lengths dresidual dweight"}
OUTPUTS = {"ssd_window_attn_fwd": "kc vc y lse", "ssd_window_attn_bwd": "dq dk dv", "ssd_window_attn_step": "kc vc y",
           "ssd_rms_norm_fwd": "y scales residual_out", "ssd_rms_norm_bwd": "dx dresidual dweight"}
IN_PLACE = {("residual_out", "residual"), ("dresidual", "dres")}


def call(lib, name, shape=None, size=None, **over):
    names, make, query = CALLS[name]
    p = addresses(names)
    p.update(over)
    s = make() if shape is None else shape
    args = [ctypes.byref(s)] + [p[n] for n in names.split()]
    if query is not None:
        args.append(getattr(lib, query)(ctypes.byref(s)) if size is None else size)
    return getattr(lib, name)(*args, None)


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_required_pointers(lib, name):
    for n in CALLS[name][0].split():
        if n not in OPTIONAL[name].split() and n != "ws":
            assert call(lib, name, **{n: None}) == INVALID, n


@no_gpu
def test_arguments_that_belong_together(lib):
    # a past needs the cache it lies in; scales belong to 8 bits
    assert call(lib, "ssd_window_attn_fwd", kc=None, vc=None) == INVALID
    assert call(lib, "ssd_rms_norm_fwd", norm_shape()) == INVALID
    assert call(lib, "ssd_rms_norm_fwd", codes(), scales=None) == INVALID


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_alignment(lib, name):
    shape = norm_shape() if name == "ssd_rms_norm_fwd" else None
    for n, a in addresses(CALLS[name][0]).items():
        if n == "ws":
            assert call(lib, name, ws=a + 128) == MISALIGNED
        elif n != "scales":
            assert call(lib, name, shape, **{"scales": None, n: a + 1} if shape else {n: a + 1}) == MISALIGNED, n
    if name == "ssd_rms_norm_fwd":
        assert call(lib, name, scales=addresses(CALLS[name][0])["scales"] + 2) == MISALIGNED
    if "attn" in name:
        for n in "q k v y".split():
            if n in addresses(CALLS[name][0]):
                assert call(lib, name, **{n: addresses(CALLS[name][0])[n] + 8}) == MISALIGNED, n


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_no_output_may_meet_another_buffer(lib, name):
    p = addresses(CALLS[name][0])
    for o in OUTPUTS[name].split():
        for other in p:
            if other != o and other != "ws" and (o, other) not in IN_PLACE:
                assert call(lib, name, **{o: p[other]}) == INVALID, (o, other)
    for o, i in IN_PLACE:
        if o in p:  # the very buffer, if it is dense, and not halfway
            assert call(lib, name, **{o: p[i] + 64}) == INVALID
            strided = CALLS[name][1](**{"residual" if i == "residual" else "dres": (0, 30)})
            assert call(lib, name, strided, **{o: p[i]}) == INVALID


@no_gpu
@pytest.mark.parametrize("name", [n for n in CALLS if CALLS[n][2]])
def test_workspace(lib, name):
    s = CALLS[name][1]()
    need = getattr(lib, CALLS[name][2])(ctypes.byref(s))
    assert need > 0 and need % 256 == 0
    assert call(lib, name, s, size=need - 1) == WORKSPACE
    assert call(lib, name, s, size=need, ws=None) == WORKSPACE
    assert call(lib, name, s, ws=addresses(CALLS[name][0])[OUTPUTS[name].split()[0]]) == INVALID


@no_gpu
@pytest.mark.parametrize("name", [n for n in CALLS if "attn" in n])
def test_bad_attention_shapes(lib, name):
    make = CALLS[name][1]
    bad = [dict(batch=-1), dict(seqlen=-1), dict(nheads=0), dict(nkvheads=0), dict(nheads=3), dict(headdim=0), dict(window=0),
           dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
           dict(dtype=E4M3), dict(dtype=3), dict(reserved=1), dict(q=(-8, 256, 64)), dict(k=(0, 128, -64))]
    beyond = [dict(headdim=16), dict(headdim=96), dict(headdim=256), dict(batch=65536), dict(nheads=1 << 17)]
    crooked = [dict(q=(4, 256, 64)), dict(v=(12800, 128, 68))]
    if name.endswith("step"):
        bad.append(dict(seqlen=2))
    else:
        bad.append(dict(k=(0, 32, 64)))  # a token's row within the one before
        beyond += [dict(seqlen=(1 << 30) + 1), dict(q=(0, 1 << 22, 64))]
        crooked.append(dict(k=(12800, 132, 64)))
    if not name.endswith("bwd"):
        beyond += [dict(window=1 << 31), dict(sinks=1 << 40)]  # slots of a cache
    for kw in bad:
        assert call(lib, name, make(**kw), size=1 << 60) == INVALID, kw
    for kw in beyond:
        assert call(lib, name, make(**kw), size=1 << 60) == UNSUPPORTED, kw
    for kw in crooked:
        assert call(lib, name, make(**kw), size=1 << 60) == MISALIGNED, kw


@no_gpu
@pytest.mark.parametrize("name", [n for n in CALLS if "norm" in n])
def test_bad_norm_shapes(lib, name):
    make = CALLS[name][1]
    bad = [dict(batch=-1), dict(seqlen=-1), dict(channels=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
           dict(dtype=E4M3), dict(res_dtype=E4M3), dict(y_dtype=3), dict(reserved=1), dict(scale_block=16),
           dict(residual=(0, 23))]
    bad += [dict(y_dtype=E4M3), dict(scale_block=32)] if name.endswith("bwd") else [dict(y_dtype=F32, scale_block=32)]
    beyond = [dict(batch=65536), dict(seqlen=(1 << 30) + 1), dict(channels=1 << 24), dict(residual=(0, 1 << 24)),
              dict(batch=4, seqlen=1 << 29)]
    for kw in bad:
        assert call(lib, name, make(**kw), size=1 << 60) == INVALID, kw
    for kw in beyond:
        assert call(lib, name, make(**kw), size=1 << 60) == UNSUPPORTED, kw


@no_gpu
def test_null_shapes(lib):
    for name in CALLS:
        n = len(getattr(lib, name).argtypes)
        assert getattr(lib, name)(*([None] * (n - 2)), 0, None) == INVALID if CALLS[name][2] else \
            getattr(lib, name)(*([None] * n)) == INVALID
    for name in ("ssd_window_attn_bwd", "ssd_window_attn_step", "ssd_rms_norm_bwd"):
        assert getattr(lib, name + "_workspace_size")(None) == 0


@no_gpu
def test_empty_calls_launch_nothing(lib):
    for name in CALLS:
        if name != "ssd_rms_norm_bwd":
            assert call(lib, name, CALLS[name][1](batch=0)) == OK
    for name in ("ssd_window_attn_fwd", "ssd_window_attn_bwd", "ssd_rms_norm_fwd"):
        assert call(lib, name, CALLS[name][1](seqlen=0)) == OK
    assert call(lib, "ssd_rms_norm_bwd", norm_shape(batch=0), dweight=None) == OK


def test_struct_sizes_match_the_header(lib, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "s.c"
    src.write_text('#include "ssd.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %zu %zu %d\\n", '
                   "sizeof(ssd_attn_shape), offsetof(ssd_attn_shape, dtype), offsetof(ssd_attn_shape, dy), "
                   "sizeof(ssd_norm_shape), offsetof(ssd_norm_shape, scale_block), "
                   "offsetof(ssd_norm_shape, dres), (int)SSD_DTYPE_E4M3); return 0; }\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    a, n = ssd.AttnShape, ssd.NormShape
    assert got == [ctypes.sizeof(a), a.dtype.offset, a.dy.offset, ctypes.sizeof(n), n.scale_block.offset, n.dres.offset,
                   ssd.SSD_DTYPE_E4M3]


SOURCES = [os.path.join(ROOT, *p.split("/")) for p in (
    "mamba_chunked_ssd_amd/csrc/ssd_api.cpp", "mamba_chunked_ssd_amd/csrc/ssd_bwd.cpp",
    "mamba_chunked_ssd_amd/csrc/ssd_mixer_ops.cpp", "tests/host/stub_launch.cpp", "tests/host/stub_mixer_launch.cpp",
    "tests/host/mixer_driver.cpp")]
ROCM_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE),
                    reason="needs g++ and the ROCm headers")
@pytest.mark.parametrize("sanitize", ["address,undefined", "thread"])
def test_host_code_under_sanitizers(tmp_path, sanitize):
    exe = str(tmp_path / "mixer_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INCLUDE,
           "-Wno-attributes", "-fsanitize=" + sanitize, "-fno-sanitize-recover=all", "-pthread"] + SOURCES + ["-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout[-2000:], r.stderr[-4000:])


def test_status_strings_name_these_calls_limits(lib):
    assert b"window attention: headdim 32/64/128" in lib.ssd_status_string(UNSUPPORTED)
    text = lib.ssd_status_string(MISALIGNED)
    assert b"window attention: 16 B" in text and b"RMS norm: the element size" in text
