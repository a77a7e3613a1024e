"""The C ABI of the convolution and the selective scan on the CPU: every
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


def conv_shape(**kw):
    d = dict(batch=2, seqlen=50, channels=24, width=4, activation=1, dtype=1, y_dtype=0, dx_dtype=1)
    d.update(kw)
    s = ssd.ConvShape(*[d.pop(k) for k in ("batch", "seqlen", "channels", "width", "activation", "dtype", "y_dtype",
                                           "dx_dtype")])
    for k, v in d.items():
        setattr(s, k, ssd.Stride(*v) if isinstance(v, tuple) else v)
    return s


def scan_shape(**kw):
    d = dict(batch=2, seqlen=50, channels=24, dstate=16, ngroups=2, dtype=1, y_dtype=0, flags=1)
    d.update(kw)
    s = ssd.SelectiveShape(*[d.pop(k) for k in ("batch", "seqlen", "channels", "dstate", "ngroups", "dtype", "y_dtype",
                                                "flags")])
    for k, v in d.items():
        setattr(s, k, ssd.Stride(*v) if isinstance(v, tuple) else v)
    return s


CALLS = {
    "ssd_causal_conv_fwd": ("x weight bias init lengths y final", conv_shape, None),
    "ssd_causal_conv_bwd": ("x weight bias init lengths dy dfinal dx dweight dbias dinit ws", conv_shape,
                            "ssd_causal_conv_bwd_workspace_size"),
    "ssd_causal_conv_step": ("x weight bias state y", lambda **k: conv_shape(**{"seqlen": 1, **k}), None),
    "ssd_selective_scan_fwd": ("x dt A B C D z dt_bias init lengths y final ws", scan_shape,
                               "ssd_selective_scan_fwd_workspace_size"),
    "ssd_selective_scan_bwd": ("x dt A B C D z dt_bias init lengths dy dfinal dx ddt dA dB dC dD dz ddt_bias dinit ws",
                               scan_shape, "ssd_selective_scan_bwd_workspace_size"),
    "ssd_selective_scan_step": ("x dt A B C D z dt_bias state y", lambda **k: scan_shape(**{"seqlen": 1, **k}), None),
}
OPTIONAL = "bias init lengths final dfinal dbias dinit D z dt_bias dD dz ddt_bias".split()
OUTPUTS = "y final dx dweight dbias dinit ddt dA dB dC dD dz ddt_bias state ws".split()


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
        if n not in OPTIONAL and n != "ws":
            assert call(lib, name, **{n: None}) == INVALID, n
    # a gate needs its gradient, and only then is there one
    if name == "ssd_selective_scan_bwd":
        assert call(lib, name, z=None) == INVALID and call(lib, name, dz=None) == INVALID


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_alignment(lib, name):
    for n, a in addresses(CALLS[name][0]).items():
        if n == "ws":
            if getattr(lib, CALLS[name][2])(ctypes.byref(CALLS[name][1]())) > 0:
                assert call(lib, name, ws=a + 128) == MISALIGNED
        else:
            assert call(lib, name, **{n: a + 1}) == MISALIGNED, n


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_no_output_may_meet_another_buffer(lib, name):
    p = addresses(CALLS[name][0])
    for o in p:
        if o not in OUTPUTS or o == "ws":
            continue
        for other in p:
            if other == o or (o, other) in (("final", "init"), ("ws", "final")) or other == "ws":
                continue
            if (other, o) == ("final", "init"):
                continue
            assert call(lib, name, **{o: p[other]}) == INVALID, (o, other)
    # the final state may be the initial one, but not meet it halfway
    if "final" in p:
        assert call(lib, name, final=p["init"] + 64) == INVALID


@no_gpu
@pytest.mark.parametrize("name", [n for n in CALLS if CALLS[n][2]])
def test_workspace(lib, name):
    s = CALLS[name][1](seqlen=3000)
    need = getattr(lib, CALLS[name][2])(ctypes.byref(s))
    assert need > 0 and need % 256 == 0
    assert call(lib, name, s, size=need - 1) == WORKSPACE
    assert call(lib, name, s, size=need, ws=None) == WORKSPACE
    out = "y" if name.endswith("fwd") else "dx"
    assert call(lib, name, s, ws=addresses(CALLS[name][0])[out]) == INVALID


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_bad_shapes(lib, name):
    make = CALLS[name][1]
    bad = [dict(batch=-1), dict(seqlen=-1), dict(channels=0), dict(dtype=2), dict(dtype=0, y_dtype=1), dict(reserved=1),
           dict(x=(-1, 24)), dict(x=(5, -1))]
    if "conv" in name:
        bad += [dict(activation=2), dict(width=0), dict(dtype=0, dx_dtype=1)]
        beyond = [dict(width=1), dict(width=5)]
    else:
        bad += [dict(ngroups=5), dict(ngroups=0), dict(dstate=0), dict(flags=2)]
        beyond = [dict(dstate=65)]
    if "step" in name:
        bad.append(dict(seqlen=2))
    else:
        bad.append(dict(x=(0, 23)))  # rows of different tokens overlap
        beyond += [dict(x=(0, 1 << 24)), dict(seqlen=(1 << 30) + 1)]
    beyond += [dict(batch=65536), dict(channels=1 << 40)]
    for kw in bad:
        assert call(lib, name, make(**kw), size=1 << 60) == INVALID, kw
    for kw in beyond:
        assert call(lib, name, make(**kw), size=1 << 60) == UNSUPPORTED, kw
    assert getattr(lib, name)(*([None] * (len(getattr(lib, name).argtypes) - 2)), 0, None) == INVALID \
        if CALLS[name][2] else getattr(lib, name)(*([None] * len(getattr(lib, name).argtypes))) == INVALID


@no_gpu
def test_empty_batches_launch_nothing(lib):
    for name in ("ssd_causal_conv_fwd", "ssd_causal_conv_step", "ssd_selective_scan_fwd", "ssd_selective_scan_step"):
        assert call(lib, name, CALLS[name][1](batch=0)) == OK


def test_invalid_shapes_need_no_workspace(lib):
    assert lib.ssd_causal_conv_bwd_workspace_size(ctypes.byref(conv_shape(width=7))) == 0
    assert lib.ssd_selective_scan_bwd_workspace_size(ctypes.byref(scan_shape(dstate=65))) == 0
    assert lib.ssd_selective_scan_fwd_workspace_size(None) == 0
    # enough channels to fill the GPU: one segment, no workspace
    assert lib.ssd_selective_scan_fwd_workspace_size(ctypes.byref(scan_shape(batch=64, channels=5120))) == 0


def test_struct_sizes_match_the_header(lib, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "s.c"
    src.write_text('#include "ssd.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", '
                   "sizeof(ssd_conv_shape), offsetof(ssd_conv_shape, width), offsetof(ssd_conv_shape, x), "
                   "sizeof(ssd_selective_shape), offsetof(ssd_selective_shape, flags), "
                   "offsetof(ssd_selective_shape, dy)); return 0; }\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    c, s = ssd.ConvShape, ssd.SelectiveShape
    assert got == [ctypes.sizeof(c), c.width.offset, c.x.offset, ctypes.sizeof(s), s.flags.offset, s.dy.offset]


SOURCES = [os.path.join(ROOT, *p.split("/")) for p in (
    "mamba_chunked_ssd_amd/csrc/ssd_api.cpp", "mamba_chunked_ssd_amd/csrc/ssd_bwd.cpp",
    "mamba_chunked_ssd_amd/csrc/ssd_ops.cpp", "tests/host/stub_launch.cpp", "tests/host/stub_ops_launch.cpp",
    "tests/host/ops_driver.cpp")]
ROCM_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE),
                    reason="needs g++ and the ROCm headers")
@pytest.mark.parametrize("sanitize", ["address,undefined", "thread"])
def test_host_code_under_sanitizers(tmp_path, sanitize):
    exe = str(tmp_path / "ops_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INCLUDE,
           "-Wno-attributes", "-fsanitize=" + sanitize, "-fno-sanitize-recover=all", "-pthread"] + SOURCES + ["-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout[-2000:], r.stderr[-4000:])


def test_status_strings_name_every_calls_limits(lib):
    text = lib.ssd_status_string(MISALIGNED)
    assert b"16 B for x/B/C/y/states" in text and b"element size" in text and b"256 B for workspace" in text
    assert b"ssd_chunk_scan_fwd_workspace_size()" in lib.ssd_status_string(WORKSPACE)
