"""The residual norm, the FP8 product and the rows to the experts and back on
a machine without a GPU: parameter blocks, refusals, and the product's plan."""

import ctypes
import os
import subprocess

import pytest

import decode_expert_routing_gb300 as mr
from decode_expert_routing_gb300 import build as mrbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BLOCKS = [("mr_add_rms_norm_params", "AddNormParams"), ("mr_fp8_gemm_params", "Fp8GemmParams"),
          ("mr_moe_permute_params", "PermuteParams"), ("mr_moe_combine_params", "CombineParams"),
          ("mr_moe_combine_grad_params", "CombineGradParams")]
A = 1 << 20  # an address that is never read: validation fails first
BAD, NO = mr.MR_ERR_INVALID_ARG, mr.MR_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    mrbuild.build()
    return mr.load_library()


@pytest.mark.parametrize("name,cls", BLOCKS)
def test_parameter_blocks_match_the_header(tmp_path, name, cls):
    cls = getattr(mr, cls)
    fields = [f for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_route.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields)
                   + f'  printf("%zu\\n", sizeof({name}));\n  return 0;\n}}\n')
    subprocess.run(["gcc", "-std=c11", "-I", mrbuild.INCLUDE, "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]


NORM = dict(x=A, ldx=256, residual=A, ldr=256, norm_weight=A, norm_kind=1, eps=1e-6, M=3, K=256, quant_format=3,
            sres=A, lds=256, rstd=A, xn=A, q=A, scale=A)
GEMM = dict(q=A, ldq=256, x_scale=A, ldxs=2, w=A, ldw=256, w_scale=A, ldws=2, M=3, R=200, K=256, out=A, ldo=200,
            out_fp32=0)
PERMUTE = dict(x=A, ldx=100, row_type=0, M=3, K=100, topk=2, E=8, topk_ids=A, sorted_token_ids=A,
               num_tokens_post_padded=A, capacity=96, rows=A, positions=A)
COMBINE = dict(y=A, ldy=100, row_type=0, capacity=96, M=3, K=100, topk=2, positions=A, topk_weights=A, add=A,
               ldadd=100, out=A)
GRAD = dict(grad_out=A, ldg=100, y=A, ldy=100, row_type=0, capacity=96, M=3, K=100, topk=2, positions=A,
            topk_weights=A, sorted_token_ids=A, num_tokens_post_padded=A, grad_y=A, grad_weights=A)

REFUSED = [
    ("mr_add_rms_norm", "AddNormParams", NORM, [
        (BAD, dict(x=None)), (BAD, dict(x=A + 2)), (BAD, dict(ldx=255)), (BAD, dict(ldx=260)), (BAD, dict(M=0)),
        (BAD, dict(residual=A + 8)), (BAD, dict(ldr=248)), (BAD, dict(ldr=257)), (BAD, dict(norm_weight=None)),
        (BAD, dict(norm_weight=A + 2)), (BAD, dict(norm_kind=2)), (BAD, dict(eps=-1e-6)),
        (BAD, dict(eps=float("nan"))), (BAD, dict(eps=float("inf"))), (BAD, dict(quant_format=4)),
        (BAD, dict(quant_format=-1)), (BAD, dict(quant_format=0)), (BAD, dict(q=None)), (BAD, dict(scale=None)),
        (BAD, dict(q=A + 4)), (BAD, dict(scale=A + 2)), (BAD, dict(sres=A + 2)), (BAD, dict(lds=255)),
        (BAD, dict(lds=260)), (BAD, dict(rstd=A + 2)), (BAD, dict(xn=A + 8)),
        (BAD, dict(quant_format=0, q=None, scale=None, sres=None, rstd=None, xn=None)),
        (NO, dict(K=248, quant_format=3)), (NO, dict(K=240, quant_format=1)), (NO, dict(K=208, quant_format=2)),
        (NO, dict(K=252, quant_format=0, q=None, scale=None)),
        (NO, dict(K=65552, ldx=65552, ldr=65552, lds=65552))]),
    ("mr_fp8_gemm", "Fp8GemmParams", GEMM, [
        (BAD, dict(q=None)), (BAD, dict(q=A + 8)), (BAD, dict(ldq=240)), (BAD, dict(ldq=264)), (BAD, dict(w=None)),
        (BAD, dict(w=A + 4)), (BAD, dict(ldw=255)), (BAD, dict(ldw=260)), (BAD, dict(x_scale=None)),
        (BAD, dict(x_scale=A + 2)), (BAD, dict(ldxs=1)), (BAD, dict(w_scale=None)), (BAD, dict(w_scale=A + 1)),
        (BAD, dict(ldws=1)), (BAD, dict(M=0)), (BAD, dict(R=0)), (BAD, dict(K=0)), (BAD, dict(M=-1)),
        (BAD, dict(out=None)), (BAD, dict(out=A + 1)), (BAD, dict(out=A + 2, out_fp32=1)), (BAD, dict(ldo=199)),
        (NO, dict(R=(1 << 24) + 1, ldo=1 << 25)), (NO, dict(M=(1 << 30) + 1)), (NO, dict(ldq=1 << 40)),
        (NO, dict(ldw=1 << 40)), (NO, dict(K=(1 << 24) + 1, ldq=1 << 25, ldw=1 << 25, ldxs=1 << 18, ldws=1 << 18))]),
    ("mr_moe_permute", "PermuteParams", PERMUTE, [
        (BAD, dict(x=None)), (BAD, dict(x=A + 1)), (BAD, dict(x=A + 2, row_type=2)), (BAD, dict(ldx=99)),
        (BAD, dict(row_type=4)), (BAD, dict(row_type=-1)), (BAD, dict(M=0)), (BAD, dict(K=0)), (BAD, dict(topk=0)),
        (BAD, dict(E=0)), (BAD, dict(capacity=0)), (BAD, dict(topk_ids=None)), (BAD, dict(sorted_token_ids=A + 2)),
        (BAD, dict(num_tokens_post_padded=None)), (BAD, dict(rows=None)), (BAD, dict(rows=A + 1)),
        (BAD, dict(positions=None)), (NO, dict(topk=33)), (NO, dict(capacity=1 << 31)), (NO, dict(M=1 << 29)),
        (NO, dict(K=(1 << 24) + 1, ldx=1 << 25))]),
    ("mr_moe_combine", "CombineParams", COMBINE, [
        (BAD, dict(y=None)), (BAD, dict(y=A + 1)), (BAD, dict(ldy=99)), (BAD, dict(row_type=3)), (BAD, dict(M=0)),
        (BAD, dict(topk=0)), (BAD, dict(capacity=0)), (BAD, dict(positions=None)), (BAD, dict(positions=A + 2)),
        (BAD, dict(topk_weights=A + 2)), (BAD, dict(add=A + 1)), (BAD, dict(ldadd=99)), (BAD, dict(out=None)),
        (BAD, dict(out=A + 2, row_type=2)), (NO, dict(topk=33)), (NO, dict(capacity=1 << 31))]),
    ("mr_moe_combine_grad", "CombineGradParams", GRAD, [
        (BAD, dict(grad_out=None)), (BAD, dict(ldg=99)), (BAD, dict(y=None)), (BAD, dict(ldy=99)),
        (BAD, dict(row_type=3)), (BAD, dict(positions=None)), (BAD, dict(topk_weights=A + 1)),
        (BAD, dict(sorted_token_ids=None)), (BAD, dict(num_tokens_post_padded=A + 2)), (BAD, dict(grad_y=None)),
        (BAD, dict(grad_weights=None)), (BAD, dict(grad_weights=A + 2)), (NO, dict(topk=33)),
        (NO, dict(capacity=1 << 31))]),
]


@pytest.mark.parametrize("name,cls,good,bad", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(lib, name, cls, good, bad):
    fn = getattr(lib, name)
    assert fn(None, None) == BAD
    for want, change in bad:
        p = getattr(mr, cls)(**{**good, **change})
        assert fn(ctypes.byref(p), None) == want, change


def test_fp8_quant_refusals(lib):
    P = ctypes.c_void_p
    fn = lib.mr_fp8_quant
    assert fn(None, 64, 2, 64, P(A), P(A), None) == BAD
    assert fn(P(A + 2), 64, 2, 64, P(A), P(A), None) == BAD
    assert fn(P(A), 60, 2, 64, P(A), P(A), None) == BAD
    assert fn(P(A), 64, 0, 64, P(A), P(A), None) == BAD
    assert fn(P(A), 64, 2, 64, P(A + 4), P(A), None) == BAD
    assert fn(P(A), 64, 2, 64, P(A), P(A + 2), None) == BAD
    assert fn(P(A), 64, 2, 64, P(A), None, None) == BAD
    assert fn(P(A), 64, 2, 56, P(A), P(A), None) == NO


def test_the_bindings_refuse_tensors_of_the_host():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: mr.add_rms_norm(x, None, x[0]), lambda: mr.fp8_quant(x), lambda: mr.moe_permute(x, i, 4, i, i),
                 lambda: mr.moe_combine(x, i), lambda: mr.moe_permute_grad(x, i),
                 lambda: mr.moe_combine_grad(x, x, i, None, i, i), lambda: mr.fp8_gemm(x, x, x, x)):
        with pytest.raises(ValueError):
            call()


PLAN = r'''
#include <cstdio>
#include "fp8_plan.h"
int main() {
    const int Ms[] = {1, 7, 8, 9, 16, 33, 64, 100, 127, 128, 129, 200, 255, 256, 257, 300, 500, 1001, 4096, 70000};
    const int Rs[] = {1, 15, 16, 17, 33, 100, 128, 129, 255, 256, 500, 1536, 2000, 6144, 9000, 100000};
    const int Ks[] = {1, 16, 100, 128, 129, 768, 2976, 6144, 20000};
    const int sms[] = {1, 2, 100, 148, 152};
    for (int M : Ms) for (int R : Rs) for (int K : Ks) for (int s : sms) {
        const mr::Fp8Plan p = mr::fp8_plan(M, R, K, s);
        printf("%d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d\n", M, R, K, s, p.pair, p.n, p.xrows, p.RT, p.CT, p.D, p.mc, p.nst,
               p.nbuf, p.grid, p.slices, p.slice_len);
    }
}
'''


def test_plans_keep_what_the_kernel_relies_on(tmp_path):
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(PLAN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "decode_expert_routing_gb300", "csrc"),
                    "-I", "/usr/local/cuda/include", "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(out) == 20 * 16 * 9 * 5
    for line in out:
        M, R, K, sms, pair, n, xrows, RT, CT, D, mc, nst, nbuf, grid, slices, len_ = map(int, line.split())
        of = 2 if pair else 1
        assert n % (16 * of) == 0 and 16 * of <= n <= 224 and (D, n <= {1: 224, 2: 128, 4: 64}[D]) in {(1, True), (2, True), (4, True)}
        # copies: whole groups of 8 rows, no more than the operand's 128, and every row of x has one
        assert xrows % 8 == 0 and 8 <= xrows <= 128 and (xrows == 128 or (M <= xrows and not pair))
        assert RT == -(-M // (128 * of)) and (CT - 1) * n < R <= CT * n
        # two groups of mc chunks of 16 columns cover the tile, and none is wider than it
        assert mc <= n // 16 <= 2 * mc and (pair, D, mc) in {
            (0, 4, 1), (0, 4, 2), (0, 2, 1), (0, 2, 2), (0, 2, 3), (0, 2, 4), (0, 1, 4), (0, 1, 6), (0, 1, 7), (1, 1, 6),
            (1, 1, 7)}
        # accumulators and stages (the product reads 128 rows of x whatever was copied)
        assert 2 <= nbuf and nbuf * D <= 8 and nbuf * D * n <= 512
        assert 3 <= nst <= 24 and nst * D * (xrows + n // of) * 128 + (128 - xrows) * 128 + 1024 <= 208 * 1024
        KI = -(-K // 128)
        if slices == 1:
            assert grid % of == 0 and grid >= of and grid // of <= RT * CT
            assert grid <= sms or (pair == 0 and grid == 1)
        else:  # one tile a cluster, blocks for every slice in whole stages, and room for the sums where the stages were
            assert not pair and slices in (2, 4, 8) and grid == RT * CT * slices <= sms
            assert len_ % D == 0 and len_ * (slices - 1) < KI <= len_ * slices
            assert slices * -(-(n // 16) // slices) * 16 * 128 * 4 + 1024 <= 208 * 1024


SIZES = r'''
#include <cstdio>
#include <cstdlib>
#include "fp8_plan.h"
int main(int n, char** v) {
    for (int i = 1; i + 2 < n; i += 3) {
        const int M = atoi(v[i]), R = atoi(v[i + 1]), K = atoi(v[i + 2]);
        if (mr::fp8_few(M)) {
            const mr::Fp8FewPlan p = mr::fp8_few_plan(M, R, K, 152);
            printf("few %d %d\n", p.A, p.B);
        } else {
            const mr::Fp8Plan p = mr::fp8_plan(M, R, K, 152);
            printf("%d %d %d %d\n", p.pair, p.D, p.mc, p.slices > 1);
        }
    }
}
'''


def test_the_sizes_run_on_the_gpu_take_every_variant(tmp_path):
    from tests.test_gpu_operators_together import VARIANTS
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(SIZES)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "decode_expert_routing_gb300", "csrc"),
                    "-I", "/usr/local/cuda/include", "-o", str(exe), str(src)], check=True)
    args = [str(x) for v in VARIANTS for x in v]
    taken = set(subprocess.run([str(exe), *args], check=True, capture_output=True, text=True).stdout.split("\n")) - {""}
    single = [(4, 1), (4, 2), (2, 1), (2, 2), (2, 3), (2, 4), (1, 4), (1, 6), (1, 7)]
    assert taken == {f"few {a} {b}" for a in (1, 2) for b in (1, 2)} | {"1 1 6 0", "1 1 7 0"} | {
        f"0 {d} {mc} {s}" for d, mc in single for s in (0, 1)}
