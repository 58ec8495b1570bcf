"""Prompt attention and rotations of several axes on the host: sizes, refusals, the axis of each frequency (CPU only)."""

import ctypes
import os
import shutil
import subprocess

import pytest

from quantized_kv_cache_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def prompt(**kw):
    a = _lib.kvq_prompt_args()
    base = dict(dtype=_lib.F16, n_seq=2, n_rows=100, max_q=60, n_q_heads=8, n_kv_heads=2, head_dim=128, softmax_scale=0.0, q=1 << 50,
                k=1 << 51, v=1 << 52, cu=4096, out=4096, q_stride=1024, k_stride=256, v_stride=256)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(dtype=_lib.Q8_0), dict(dtype=100), dict(n_seq=-1), dict(n_rows=-1), dict(max_q=-1), dict(n_q_heads=0),
                                dict(n_kv_heads=0), dict(n_kv_heads=3), dict(n_q_heads=34, q_stride=8192), dict(head_dim=96), dict(head_dim=512),
                                dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")), dict(q=None), dict(k=None), dict(v=None),
                                dict(cu=None), dict(out=None), dict(q=4104), dict(k=8200), dict(v=16388), dict(out=32770), dict(cu=4098),
                                dict(q=4096), dict(k=4096 + 2 * 100 * 1024 - 16), dict(v=4096 - 16), dict(out=(1 << 50) + 2 * (99 * 1024 + 1024) - 16),
                                dict(q_stride=1000), dict(k_stride=248), dict(v_stride=257)])
def test_prompt_refusals(kw):
    """Refused on the host: the pointers here are never followed."""
    with pytest.raises(_lib.KVQError) as e:
        _lib.kv_prompt_attn(ctypes.byref(prompt(**kw)), None, 4096, 1 << 40)
    assert e.value.code == 1


@pytest.mark.parametrize("opts", [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e-38), dict(softcap=3e38), dict(window=-1),
                                  dict(slopes=2), dict(prefix=2), dict(lse=2)])
def test_prompt_options_refused(opts):
    o = _lib.kvq_attn_opts(**opts)
    with pytest.raises(_lib.KVQError) as e:
        _lib.kv_prompt_attn(ctypes.byref(prompt()), ctypes.byref(o), 4096, 1 << 40)
    assert e.value.code == 1


def test_prompt_workspaces_and_sizes_refused(lib):
    a = ctypes.byref(prompt())
    need = _lib.kv_prompt_required_bytes(100, 8, 128)
    for ws, n in ((None, 1 << 40), (4100, 1 << 40), (4096, need - 1)):
        assert lib.kv_prompt_attn(a, None, ws, n, None) == 1
    assert lib.kv_prompt_attn(None, None, 4096, 1 << 40, None) == 1
    assert lib.kv_prompt_get_status(None, None) == 1 and lib.kv_prompt_get_status(4100, None) == 1
    for bad in ((-1, 8, 128), (1 << 31, 8, 128), (10, 0, 128), (10, 8, 96)):
        with pytest.raises(_lib.KVQError):
            _lib.kv_prompt_required_bytes(*bad)
    for kw in (dict(n_seq=65536), dict(n_rows=1 << 27), dict(n_rows=(1 << 27) - 1), dict(k_stride=1 << 38), dict(v_stride=1 << 40)):
        assert lib.kv_prompt_attn(ctypes.byref(prompt(**kw)), None, 4096, 1 << 60, None) == 3, kw
    for kw in (dict(n_seq=0), dict(n_rows=0), dict(max_q=0)):
        assert lib.kv_prompt_attn(ctypes.byref(prompt(**kw)), None, None, 0, None) == 0


def rope(**kw):
    a = _lib.kvq_norm_rope_args()
    base = dict(dtype=_lib.F16, n_tok=4, n_q_heads=8, n_k_heads=2, head_dim=128, rot_dim=128, max_pos=100, eps=1e-6, q=4096, k=8192,
                cos_sin=4096, positions=4096, q_out=16384, k_out=32768, q_stride=1024, k_stride=256, q_out_stride=1024, k_out_stride=256)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("sections", [(), (20, 20, 20), (65, -1), (16, 16, 16, 8, 8), (1 << 30, 1 << 30, 1 << 30), (128,), (0,)])
def test_sections_refused(sections):
    with pytest.raises(_lib.KVQError) as e:
        _lib.kv_qk_norm_rope_axes(ctypes.byref(rope()), sections, 0)
    assert e.value.code == 1


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=24), dict(head_dim=96), dict(positions=None), dict(q=4104), dict(eps=-1.0),
                                dict(n_tok=-1), dict(cos_sin=None), dict(k_stride=250)])
def test_rope_axes_refusals(kw):
    with pytest.raises(_lib.KVQError) as e:
        _lib.kv_qk_norm_rope_axes(ctypes.byref(rope(**kw)), (kw.get("rot_dim", 128) // 2,), 0)
    assert e.value.code == 1


def test_rope_axes_null_and_no_tokens(lib):
    assert lib.kv_qk_norm_rope_axes(None, 1, (ctypes.c_int32 * 1)(64), 0, None) == 1
    assert lib.kv_qk_norm_rope_axes(ctypes.byref(rope()), 1, None, 0, None) == 1
    assert lib.kv_qk_norm_rope_axes(ctypes.byref(rope(n_tok=0)), 1, (ctypes.c_int32 * 1)(64), 0, None) == 0


PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "paged_internal.h"
using namespace kvq;
int main(int n, char** v) {
    int32_t s[4];
    for (int i = 2; i < n; ++i) s[i - 2] = std::atoi(v[i]);
    RopeAxes x;
    rope_axes(n - 2, s, v[1][0] == '1', &x);
    std::printf("%u", x.used);
    for (int f = 0; f < 256; ++f) std::printf(" %d", (x.of8[f / 8] >> 2 * (f % 8)) & 3);
    // the row tiles that a grid holds cover every prompt, whatever the lengths
    long bad = 0;
    for (int D = 64; D <= 256; D *= 2)
        for (int G = 1; G <= 16; ++G)
            for (int a = 0; a < 600; a += 7)
                for (int b = 0; b < 600; b += 13) {
                    const int t = D == 256 ? 128 : 256;
                    bad += (a * G + t - 1) / t + (b * G + t - 1) / t > prompt_tiles(a + b, 2, G, D);
                }
    std::printf("\n%ld\n", bad);
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cc = shutil.which("g++")
    if not cc:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("axes")
    src, exe = at / "axes.cpp", at / "axes"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-I", os.path.join(ROOT, "quantized_kv_cache_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    return exe


@pytest.mark.parametrize("sections", [(64,), (16, 24, 24), (24, 20, 20), (1, 0, 45, 2), (0, 3, 5), (64, 64, 64, 64), (100, 156)])
def test_axis_of_each_frequency(program, sections):
    for cyclic in (0, 1):
        r = subprocess.run([str(program), str(cyclic)] + list(map(str, sections)), check=True, capture_output=True, text=True).stdout.split("\n")
        got = list(map(int, r[0].split()))
        want = [a for a, n in enumerate(sections) for _ in range(n)]
        if cyclic:
            want = [a for k in range(max(sections)) for a, n in enumerate(sections) if k < n]
        assert got[0] == sum(1 << a for a, n in enumerate(sections) if n) and got[1:1 + sum(sections)] == want
        assert r[1] == "0"
