"""Host-side checks of the expert products on a machine without a GPU: sizes,
refusals, the binding's parameter blocks.  No call here reaches a kernel."""

import ctypes
import os
import subprocess

import pytest

import decode_expert_routing_gb300 as mr
from decode_expert_routing_gb300 import build as mrbuild

P = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    mrbuild.build()
    return mr.load_library()


def test_packed_scale_bytes(lib):
    f = lib.mr_mx_packed_scale_bytes
    assert f(1, 128, 128, 1, 0) == 512
    assert f(1, 129, 128, 1, 0) == 1024
    assert f(1, 128, 160, 1, 0) == 1024
    assert f(1, 128, 256, 2, 0) == 1024        # E2M1: 256 elements a stage, two words a row
    assert f(8, 1536, 6144, 1, 1) == 8 * 12 * 48 * 512
    assert f(1, 64, 128, 1, 1) == 512          # 32 features: one tile
    for bad in ((0, 128, 128, 1, 0), (1, 0, 128, 1, 0), (1, 128, 100, 1, 0), (1, 128, 128, 0, 0), (1, 128, 128, 3, 0),
                (1025, 128, 128, 1, 0), (1, 96, 128, 1, 1)):
        assert f(*bad) == 0, bad


def test_expert_scratch_bytes(lib):
    f = lib.mr_expert_scratch_bytes
    assert f(1, 8, 6144) >= 8 * 6144 * 2
    assert f(4096, 8, 6144) >= 32768 * 6144 * 2
    for m in (1, 7, 100, 2047):  # grows with the rows
        assert f(m, 1, 6144) <= f(m + 1, 1, 6144)
    for bad in ((0, 8, 64), (1, 0, 64), (1, 33, 64), (1, 8, 0), (1 << 28, 32, 64)):
        assert f(*bad) == 0, bad


def fill(p, **kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


GEMM = dict(q=P, ldq=256, scale=P, lds=8, w=P, w_scale=P, M=4, R=100, K=256, format=1, out=P, ldo=100, out_fp32=0)
UP = dict(q=P, ldq=256, scale=P, lds=8, sorted_rows=0, w13=P, w13_scale=P, E=8, I=64, K=256, format=1,
          sorted_token_ids=P, expert_ids=P, n_blocks=8, block=16, M=4, topk=2, out_format=0, act=P, act_scale=P)
DOWN = dict(q=P, ldq=64, scale=P, lds=2, w2=P, w2_scale=P, E=8, R=100, I=64, format=1, sorted_token_ids=P,
            expert_ids=P, n_blocks=8, block=16, M=4, topk=2, topk_ids=P, topk_weights=P, add=None, out=P, scratch=P,
            scratch_bytes=1 << 30)

INVALID = [
    ("gemm", dict(q=None)), ("gemm", dict(q=P + 8)), ("gemm", dict(ldq=240)), ("gemm", dict(ldq=264)),
    ("gemm", dict(lds=7)), ("gemm", dict(scale=None)), ("gemm", dict(w=P + 4)), ("gemm", dict(w_scale=None)),
    ("gemm", dict(M=0)), ("gemm", dict(R=0)), ("gemm", dict(K=0)), ("gemm", dict(format=0)), ("gemm", dict(format=7)),
    ("gemm", dict(out=None)), ("gemm", dict(out=P + 1)), ("gemm", dict(out=P + 2, out_fp32=1)), ("gemm", dict(ldo=99)),
    ("up", dict(I=0)), ("up", dict(E=0)), ("up", dict(M=0)), ("up", dict(topk=0)), ("up", dict(block=0)),
    ("up", dict(n_blocks=0)), ("up", dict(sorted_token_ids=None)), ("up", dict(expert_ids=P + 2)),
    ("up", dict(w13=None)), ("up", dict(act=None)), ("up", dict(act=P + 8)), ("up", dict(out_format=3)),
    ("up", dict(out_format=1, act_scale=None)),
    ("down", dict(w2=P + 8)), ("down", dict(topk_ids=None)), ("down", dict(topk_weights=P + 2)),
    ("down", dict(out=None)), ("down", dict(add=P + 1)), ("down", dict(R=0)), ("down", dict(scratch=None)),
    ("down", dict(scratch=P + 16)),
]
UNSUPPORTED = [
    ("gemm", dict(K=272, ldq=272, lds=9)), ("gemm", dict(R=(1 << 24) + 1, ldo=1 << 25)),
    ("gemm", dict(M=1 << 30)),
    ("up", dict(I=48)), ("up", dict(E=1025)), ("up", dict(topk=33)), ("up", dict(block=1025)),
    ("up", dict(M=1 << 27, topk=8)), ("up", dict(n_blocks=1 << 28)),
    ("down", dict(E=2000)), ("down", dict(I=80, ldq=80, lds=3)),
]


def call(lib, op, change):
    base, cls, fn = {"gemm": (GEMM, mr.MxGemmParams, lib.mr_mx_gemm), "up": (UP, mr.GateUpParams, lib.mr_moe_gate_up),
                     "down": (DOWN, mr.DownParams, lib.mr_moe_down)}[op]
    return fn(fill(cls(), **{**base, **change}), None)


@pytest.mark.parametrize("op,change", INVALID)
def test_invalid_arguments(lib, op, change):
    assert call(lib, op, change) == mr.MR_ERR_INVALID_ARG


@pytest.mark.parametrize("op,change", UNSUPPORTED)
def test_unsupported_shapes(lib, op, change):
    assert call(lib, op, change) == mr.MR_ERR_UNSUPPORTED


def test_short_scratch(lib):
    need = lib.mr_expert_scratch_bytes(DOWN["M"], DOWN["topk"], DOWN["R"])
    assert call(lib, "down", dict(scratch_bytes=need - 1)) == mr.MR_ERR_SCRATCH_TOO_SMALL


def test_null_parameter_blocks(lib):
    for fn in (lib.mr_mx_gemm, lib.mr_moe_gate_up, lib.mr_moe_down):
        assert fn(None, None) == mr.MR_ERR_INVALID_ARG
    assert lib.mr_mx_pack_scales(None, 1, 128, 128, 1, 0, P, None) == mr.MR_ERR_INVALID_ARG
    assert lib.mr_mx_pack_scales(P, 1, 128, 128, 1, 0, P + 8, None) == mr.MR_ERR_INVALID_ARG
    assert lib.mr_mx_pack_scales(P, 1, 128, 100, 1, 0, P, None) == mr.MR_ERR_UNSUPPORTED


# ------------------------------------------------------------------ the launch's shape

PROBE = r'''
#include <cstdio>
#include "expert_plan.h"
static unsigned seed = 1;
static int rnd(int n) { seed = seed * 1664525u + 1013904223u; return (int)((seed >> 8) % (unsigned)n); }
int main() {
    long split = 0, bad = 0;
    for (int i = 0; i < 400000; ++i) {
        const bool fp4 = rnd(2), gate_up = rnd(3) == 0;
        const int R = gate_up ? 64 * (1 + rnd(40)) : 1 + rnd(rnd(2) ? 300 : 6144), K = 32 * (1 + rnd(600));
        const int ctas = rnd(3) ? 152 : 16 + rnd(140);
        const mr::ExpertShape s = mr::expert_shape(R, K, fp4, gate_up);
        const bool gemm = !gate_up && rnd(2);
        const int E = gemm ? 1 : 1 + rnd(rnd(2) ? 8 : 200), mk = 1 + rnd(rnd(2) ? 64 : 3000);
        int len = 0;
        const int n = mr::expert_slices(mk, E, s, ctas, &len);
        const bool pair = n == 1 && mr::expert_pair(mk, E);
        if (n > 1) {
            ++split;
            const int group = 4 / s.W;
            if ((n != 2 && n != 4 && n != 8) || len % group != 0 || (long)len * (n - 1) >= s.KI || (long)len * n < s.KI) ++bad;
        } else if (len != s.KI) ++bad;
        long tiles = 0;
        if (gemm) {
            const int per = mr::expert_gemm_rows(mk, s.RT, pair, n, ctas);
            if (per < 16 || per > 256 || per % (pair ? 32 : 16)) ++bad;
            tiles = ((long)mk + per - 1) / per * s.RT;
        } else {  // any distribution of the assignments over the experts; a run has up to 15 rows more
            int left = mk;
            for (int e = 0; e < E && left > 0; ++e) {
                int rows = e + 1 == E ? left : rnd(3) == 0 ? 1 + rnd(left) : 1 + rnd(left < 300 ? left : 300);
                if (rows > left) rows = left;
                left -= rows;
                tiles += ((rows + 15) / 16 * 16 + 255) / 256;
            }
            tiles *= s.RT;
        }
        if (n > 1 && tiles > ctas / n) {
            if (++bad < 5) printf("E %d mk %d R %d K %d fp4 %d ctas %d: %ld tiles, %d slices\n", E, mk, R, K, fp4, ctas, tiles, n);
        }
    }
    printf("%ld %ld\n", split, bad);
}
'''


def test_every_tile_of_a_split_has_a_cluster(tmp_path):
    """A cluster whose CTAs share a tile's K range takes one tile: the host's rule leaves none over."""
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(PROBE)
    csrc = os.path.join(os.path.dirname(os.path.abspath(mr.__file__)), "csrc")
    cuda = os.path.join(os.path.dirname(os.path.dirname(mrbuild.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, "-I", cuda, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    split, bad = map(int, out.split("\n")[-2].split())
    assert split > 1000 and bad == 0, out
