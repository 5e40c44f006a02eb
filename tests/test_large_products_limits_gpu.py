"""The large segmented products at the limits of their values, lengths and sizes (GPU), against 64-bit implementations."""
import pytest
import torch

import segmented_gather_gemm_expand_b200 as sg
from test_large_products_gpu import _clean, gen, ints, run_lora  # noqa: F401

pytestmark = pytest.mark.gpu

INT64_MAX = 2 ** 63 - 1


# ---------------------------------------------------------------- lengths

@pytest.mark.parametrize("rows", [300, 20])
def test_lengths_to_the_end_of_64_bits(rows):
    """A length so large that start + length has no 64-bit value: every part of every call takes the rows to the end."""
    g = gen(91)
    K, N, A = 128, 200, 3
    m = [torch.tensor(v, dtype=torch.int64).cuda() for v in ([1, 0, INT64_MAX, -7], [INT64_MAX, 1, INT64_MAX, INT64_MAX], [1, 2, 0, 0])]
    cut = [(0, 1, 2), (1, rows, 1)]
    x, w = ints(g, (rows, K), "bf16", 1), ints(g, (N, K), "bf16", 1)
    a, b, out = ints(g, (A, 16, K), "bf16", 1), ints(g, (A, N, 16), "bf16", 1), torch.zeros(rows, N, device="cuda")
    ref = x.double() @ w.double().T
    for lo, hi, i in cut:
        ref[lo:hi] += (x[lo:hi].double() @ a[i].double().T) @ b[i].double().T
    for variant in (sg.VARIANT_AUTO, sg.VARIANT_SIMT):
        sg.set_variant(variant)
        run_lora(x, w, a, b, out, m, 4, rows)
        assert torch.equal(out, ref.float()), variant
    e, t, dw, y = ints(g, (A, N, K), "bf16", 1), torch.zeros(rows, 16).cuda(), torch.zeros(A, N, K).cuda(), torch.zeros(rows, N).cuda()
    dy = ints(g, (rows, N), "bf16", 1)
    rt, ry, rw = torch.zeros_like(t, dtype=torch.float64), torch.zeros_like(y, dtype=torch.float64), torch.zeros_like(dw, dtype=torch.float64)
    for lo, hi, i in cut:
        rt[lo:hi], ry[lo:hi] = x[lo:hi].double() @ a[i].double().T, x[lo:hi].double() @ e[i].double().T
        rw[i] += dy[lo:hi].double().T @ x[lo:hi].double()
    for variant in (sg.VARIANT_AUTO, sg.VARIANT_SIMT):
        sg.set_variant(variant)
        for v in (t, y, dw):
            v.zero_()
        sg.sgmv_shrink(x, a, t, *m, 4, rows)
        sg.sgmv_grouped_gemm(x, e, y, *m, 4, rows)
        sg.sgmv_grouped_wgrad(dy, x, dw, *m, 4, rows)
        assert torch.equal(t, rt.float()) and torch.equal(y, ry.float()) and torch.equal(dw, rw.float()), variant
        z = torch.zeros(rows, N).cuda()
        sg.sgmv_expand(t.bfloat16(), b, z, *m, 4, rows)
        rz = torch.zeros_like(ry)
        for lo, hi, i in cut:
            rz[lo:hi] = t[lo:hi].bfloat16().double() @ b[i].double().T
        assert torch.equal(z, rz.float()), variant


def test_metadata_check_at_the_end_of_64_bits():
    m = [torch.tensor(v, dtype=torch.int64).cuda() for v in ([1, 50], [INT64_MAX, 10], [0, 0])]
    assert sg.validate_metadata(*m, 2, 1, 100) == 4 | 8
    m[0], m[1] = torch.tensor([50, 1]).cuda(), torch.tensor([10, INT64_MAX]).cuda()
    assert sg.validate_metadata(*m, 2, 1, 100) == 4 | 8 | 16
    m[1] = torch.tensor([INT64_MAX, 49]).cuda()
    assert sg.validate_metadata(*m, 2, 1, INT64_MAX) == 4 | 16
