"""The large segmented products at the limits of their values, lengths and sizes (GPU), against 64-bit implementations."""
import pytest
import torch

import segmented_gather_gemm_expand_b200 as sg
from test_large_products_gpu import DT, _clean, gen, ints, lora_ref, meta, run_lora  # noqa: F401

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

# ---------------------------------------------------------------- the low-rank input t

def one_entry_rows(T, K, scale, dt, g):
    """Rows of x with one entry, a power of two: t = x A^T is then that entry times a column of A, without any rounding."""
    k = torch.randint(0, K, (T,), generator=g)
    x = torch.zeros(T, K, dtype=DT[dt])
    x[torch.arange(T), k] = torch.as_tensor(scale, dtype=torch.float64).expand(T).to(DT[dt])
    return x.cuda()


# power of two in x, size of A, size of B: t about 1e6, 2e5, 1e-3, 1e-5, 1e-6 and 1e-8
T_RANGE = {"1e6": (2.0 ** 10, 1000.0, 2.0 ** -10), "2e5": (2.0 ** 8, 800.0, 2.0 ** -7), "1e-3": (2.0 ** -4, 0.016, 4.0),
           "1e-5": (2.0 ** -8, 0.0026, 500.0), "1e-6": (2.0 ** -12, 0.004, 5000.0), "1e-8": (2.0 ** -14, 0.00016, 30000.0)}


@pytest.mark.parametrize("variant", [sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE])
@pytest.mark.parametrize("size", [*T_RANGE, "mixed"])
@pytest.mark.parametrize("R", [8, 16, 24, 40])
@pytest.mark.parametrize("dt,out_dt", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_lora_t_over_its_range(variant, size, R, dt, out_dt):
    """The low-rank part alone (the shared weight is zero) for t of any size, on the tensor cores and beside single tokens.

    t is exact here, so what is left is the split of t (none for fp32 out: three bf16 parts hold 24 bits; for two parts, t in
    [1, 2): the first leaves at most 2^-8, whose own bf16 steps are 2^-16 at most below 2^-8, half of that is 2^-17), at most
    6 R + K / 16 additions of the accumulator with 2^-23 of the sum of |products| each, and the rounding of out: half a step
    of its type, at least half of its smallest one."""
    g = gen(101 + R)
    lens = [90, 1, 70, 33, 1, 60]
    m, T = meta(lens, [0, 1, 2, 1, 0, 2])
    K, N, A = 64, 136, 3
    if size == "mixed":
        scale, sa, sb = 2.0 ** torch.randint(-14, 11, (T,), generator=g).double(), 30.0, 2.0 ** -6
    else:
        scale, sa, sb = T_RANGE[size]
    x = one_entry_rows(T, K, scale, dt, g)
    a = (torch.rand(A, R, K, generator=g) * 2 * sa - sa).to(DT[dt]).cuda()
    b = (torch.rand(A, N, R, generator=g) * 2 * sb - sb).to(DT[dt]).cuda()
    w, out = torch.zeros(N, K, dtype=DT[dt], device="cuda"), torch.full((T, N), float("nan"), dtype=DT[out_dt], device="cuda")
    sg.set_variant(variant)
    assert sg.lora_linear_plan(x, w, a, b, out, *m, len(lens), max(lens))[0] == sg.VARIANT_TC
    run_lora(x, w, a, b, out, m, len(lens), max(lens))
    ref, sums = lora_ref(x, w, a, b, m, None, T), lora_ref(x.abs(), w, a.abs(), b.abs(), m, None, T)
    f = torch.finfo(DT[out_dt])
    bound = ((0 if out_dt == "f32" else 2 ** -17) + (6 * R + K // 16) * 2 ** -23) * sums
    bound = bound + torch.clamp(ref.abs() + bound, min=f.tiny) * (f.eps / 2)
    bad = (out.double() - ref).abs() > bound
    assert not bad.any(), ((out.double() - ref).abs() / sums.clamp(min=1e-30))[bad].max()
    assert (ref.abs() < f.max).all() and (sums > 0).any()


@pytest.mark.parametrize("variant", [sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE])
@pytest.mark.parametrize("dt,out_dt", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_lora_infinite_t(variant, dt, out_dt):
    """One infinity in an adapter's A makes t infinite in one rank: outputs are the infinities that the formula has, signs too."""
    g = gen(111)
    lens = [90, 1, 70, 33, 1, 60]
    m, T = meta(lens, [0, 1, 2, 1, 0, 2])
    x, w = torch.ones(T, 64, dtype=DT[dt], device="cuda"), ints(g, (136, 64), dt, 1)
    a, b = ints(g, (3, 16, 64), dt, 1), ints(g, (3, 136, 16), dt, 1)
    a[1, 5, 7] = float("inf")
    b[1, :, 5] = torch.where(torch.arange(136) % 2 == 0, 1.0, -2.0).to(DT[dt]).cuda()
    out = torch.zeros(T, 136, dtype=DT[out_dt], device="cuda")
    sg.set_variant(variant)
    run_lora(x, w, a, b, out, m, len(lens), max(lens))
    assert torch.equal(out, lora_ref(x, w, a, b, m, None, T).to(DT[out_dt]))
    assert torch.isinf(out[90:91]).all() and torch.isinf(out[161:194]).all() and torch.isfinite(out[:90]).all()


@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
def test_lora_t_above_bf16s_largest_number(out_dt):
    """fp32 goes a little further than bf16: such a t is finite, and so is its product with a small B."""
    m, T = meta([60, 40], [0, 1])
    x, a = torch.zeros(T, 64, device="cuda").bfloat16(), torch.zeros(2, 16, 64, device="cuda").bfloat16()
    x[:, 0], x[:, 1] = 255 / 128 * 2.0 ** 64, 1.5 * 2.0 ** 60
    a[:, :, 0], a[:, :, 1] = 255 / 128 * 2.0 ** 62, 2.0 ** 60
    w, b = torch.zeros(136, 64, device="cuda").bfloat16(), torch.full((2, 136, 16), 2.0 ** -100, device="cuda").bfloat16()
    t = x[0].double() @ a[0, 0].double()
    assert torch.finfo(torch.bfloat16).max < t < torch.finfo(torch.float32).max
    out = torch.zeros(T, 136, dtype=DT[out_dt], device="cuda")
    run_lora(x, w, a, b, out, m, 2, 60)
    assert torch.equal(out, lora_ref(x, w, a, b, m, None, T).float().to(DT[out_dt]))


# ---------------------------------------------------------------- many segments, many rows

@pytest.mark.parametrize("rows,segs,K,N,R,dt", [(16384, 4096, 128, 512, 16, "bf16"), (16000, 4000, 256, 136, 8, "f16"), (20480, 4096, 64, 136, 16, "f16"),
                                                (32768, 4096, 64, 264, 32, "bf16"), (2200000, 5, 64, 72, 16, "bf16")])
def test_lora_counts_at_the_tables_limits(rows, segs, K, N, R, dt):
    """As many segments as the tensor-core forms take, four to eight rows each, and more rows than a table of runs holds."""
    g = gen(121)
    x, w = ints(g, (rows, K), dt, 1), ints(g, (N, K), dt, 1)
    a, b = ints(g, (7, R, K), dt, 1), ints(g, (7, N, R), dt, 1)
    n = rows // segs
    m = [(torch.arange(segs) * n).int().cuda(), torch.full((segs,), n).int().cuda(), (torch.arange(segs) % 8 - 1).int().cuda()]
    out = torch.zeros(rows, N, device="cuda")
    assert sg.lora_linear_plan(x, w, a, b, out, *m, segs, n)[0] == sg.VARIANT_TC
    run_lora(x, w, a, b, out, m, segs, n)
    ids = (torch.arange(rows, device="cuda") // n).clamp(max=segs - 1) % 8 - 1
    ref = x.float() @ w.float().T          # whole numbers below 2^24: exact
    for i in range(7):
        at = (ids == i).nonzero()[:, 0]
        ref[at] += (x[at].float() @ a[i].float().T) @ b[i].float().T
    assert torch.equal(out, ref)


@pytest.mark.parametrize("adapters", [3, 40, 90])
@pytest.mark.parametrize("R", [4, 16])
def test_lora_turned_b_of_fewer_adapters_than_segments(adapters, R):
    """A B that has to be laid out anew takes the space of the adapters or of the segments' copies, whichever is less."""
    g = gen(131)
    K, N, segs = 64, 264, 60
    m, T = meta([5 + i % 4 for i in range(segs)], [(7 * i) % (min(adapters, 30) + 2) - 1 for i in range(segs)], gaps=[i % 2 for i in range(segs)])
    x, w, a = ints(g, (T, K), "bf16", 1), ints(g, (N, K), "bf16", 1), ints(g, (adapters, R, K), "bf16", 1)
    b, out = ints(g, (adapters, R, N), "bf16", 1).transpose(1, 2), torch.zeros(T, N, device="cuda")
    _, need, pref = sg.lora_linear_plan(x, w, a, b, out, *m, segs, 8)
    # what the sums of t take beside it: nothing at ranks that are no multiple of 16
    straight = sg.lora_linear_plan(x, w, a, b.contiguous(), out, *m, segs, 8)[2] if R == 16 else need
    assert need < pref <= straight + min(adapters, segs) * N * ((R + 7) // 8 * 8) * 2 + 256
    for spare in (True, False):
        out.fill_(float("nan"))
        run_lora(x, w, a, b, out, m, segs, 8, spare=spare)
        assert torch.equal(out, lora_ref(x, w, a, b, m, None, T).float())


# ---------------------------------------------------------------- values that are no numbers

@pytest.mark.parametrize("variant", [sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE])
@pytest.mark.parametrize("T,K,N,turned", [(700, 28672, 136, False), (700, 28672, 136, True), (60, 4100 * 2, 40, False), (2100, 1004, 777, False)])
@pytest.mark.parametrize("dt,out_dt", [("f16", "f16"), ("bf16", "f32")])
def test_lora_one_adapter_full_of_nan(variant, T, K, N, turned, dt, out_dt):
    """A long prompt whose adapter's B is NaN from end to end, beside others in the same token tiles: the others come out
    right, bias included, however long K is, and soon (the kernels' waits are limited to two seconds)."""
    g = gen(141)
    lens = [T // 7, T // 5, 1, T // 9, T // 3]
    m, rows = meta(lens, [0, 1, 2, 1, 0], gaps=[1, 0, 3, 0, 2])
    x = torch.zeros(rows + 5, (K + 7) // 8 * 8, dtype=DT[dt], device="cuda")[:, :K]
    x.copy_(ints(g, (rows + 5, K), dt, 1))
    w = ints(g, (K, (N + 7) // 8 * 8), dt, 1).t()[:N] if turned else torch.zeros(N, (K + 7) // 8 * 8, dtype=DT[dt], device="cuda")[:, :K]
    if not turned:
        w.copy_(ints(g, (N, K), dt, 1))
    a, b, bias = ints(g, (3, 16, K), dt, 1) * (torch.rand(3, 16, K, generator=g) < 0.02).cuda(), ints(g, (3, N, 16), dt, 1), ints(g, (N,), dt, 9)
    ref = lora_ref(x, w, a, b, m, bias, rows + 5).to(DT[out_dt])
    b[1] = float("nan")
    out = torch.zeros(rows + 5, N, dtype=DT[out_dt], device="cuda")
    sg.set_variant(variant)
    assert sg.lora_linear_plan(x, w, a, b, out, *m, 5, max(lens), bias=bias)[0] == sg.VARIANT_TC
    run_lora(x, w, a, b, out, m, 5, max(lens), bias)
    own = torch.zeros(rows + 5, dtype=torch.bool, device="cuda")
    for s, n, e in zip(*[v.tolist() for v in m]):
        own[s:s + n] |= e == 1
    assert torch.equal(out[~own], ref[~own]) and torch.isnan(out[own]).all()


# ---------------------------------------------------------------- what the two CTAs of a pair write for each other

def test_ragged_ends_and_short_runs_many_times():
    """Rows zeroed, and t written, by the pair's second CTA for the first one's MMAs: the same bits every time."""
    g = gen(151)
    lens = [1 + (37 * i) % 61 for i in range(64)]
    m, T = meta(lens, [i % 5 for i in range(64)])
    x, dy = ints(g, (T, 520), "bf16", 1), ints(g, (T, 264), "bf16", 1)
    w, a, b = ints(g, (264, 520), "bf16", 1), ints(g, (5, 16, 520), "bf16", 1), ints(g, (5, 264, 16), "bf16", 1)
    ref, rw = lora_ref(x, w, a, b, m, None, T).float(), torch.zeros(5, 264, 520, dtype=torch.float64, device="cuda")
    for s, n, e in zip(*[v.tolist() for v in m]):
        rw[e] += dy[s:s + n].double().T @ x[s:s + n].double()
    out, dw = torch.zeros(T, 264, device="cuda"), torch.zeros(5, 264, 520, device="cuda")
    sg.set_variant(sg.VARIANT_TC_WIDE)
    for _ in range(100):
        run_lora(x, w, a, b, out, m, 64, 61)
        sg.sgmv_grouped_wgrad(dy, x, dw, *m, 64, 61)
        assert torch.equal(out, ref) and torch.equal(dw, rw.float())


def test_lora_when_the_shrink_takes_longer_than_the_waits_limit():
    """Single tokens in random order, so many that finding their adapters takes seconds: the projection's roles that start
    before that is done wait for it, and their limits of two seconds count from then on."""
    T, g = 800_000, gen(161)
    x, w, a, b = ints(g, (T, 64), "bf16", 1), ints(g, (64, 64), "bf16", 1), ints(g, (7, 8, 64), "bf16", 1), ints(g, (7, 64, 8), "bf16", 1)
    start, ids = torch.randperm(T, generator=g), torch.randint(-1, 7, (T,), generator=g)
    m = [start.int().cuda(), torch.ones(T).int().cuda(), ids.int().cuda()]
    out = torch.zeros(T, 64, device="cuda")
    assert sg.lora_linear_plan(x, w, a, b, out, *m, T, 1)[0] == sg.VARIANT_TC
    run_lora(x, w, a, b, out, m, T, 1)
    row = torch.empty_like(ids)
    row[start] = ids
    ref = x.float() @ w.float().T          # whole numbers below 2^24: exact
    for i in range(7):
        at = (row == i).nonzero()[:, 0].cuda()
        ref[at] += (x[at].float() @ a[i].float().T) @ b[i].float().T
    assert torch.equal(out, ref)


# ---------------------------------------------------------------- gradients of adapters from half t

@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R,K,N", [(16, 264, 136), (64, 136, 200), (8, 128, 96)])
@pytest.mark.parametrize("out_dt,add", [("f32", True), (None, False)])
def test_adapters_gradients_from_half_t(dt, R, K, N, out_dt, add):
    """dA and dB with t and dt as sgmv_shrink writes them in the weights' type: the tensor-core form, both short sides."""
    g = gen(171 + R)
    lens, A = [90, 40, 0, 33, 130, 1, 1, 17], 5
    m, T = meta(lens, [1, 0, 2, 1, 3, -1, 0, 2], gaps=[i % 3 for i in range(8)])
    sparse = lambda v: v * (torch.rand(v.shape, generator=g) < 0.2).to(v.device)   # sums below 128: whole in bf16
    x, dy = sparse(ints(g, (T, K), dt, 1)), sparse(ints(g, (T, N), dt, 1))
    a, b = ints(g, (A, R, K), dt, 1), ints(g, (A, N, R), dt, 1)
    t, s = torch.zeros(T, R, device="cuda", dtype=DT[dt]), torch.zeros(T, R, device="cuda", dtype=DT[dt])   # x A^T, dY B
    sg.sgmv_shrink(x, a, t, *m, 8, 130)
    sg.sgmv_shrink(dy, b.transpose(1, 2), s, *m, 8, 130)
    od = DT[out_dt or dt]
    da, db = ints(g, (A, R, K), "f32", 9).to(od), ints(g, (A, N, R), "f32", 9).to(od)
    ra, rb = (da.double(), db.double()) if add else (torch.zeros_like(da).double(), torch.zeros_like(db).double())
    for lo, n, i in zip(*[v.tolist() for v in m]):
        if i < 0:
            continue
        xd, yd = x[lo:lo + n].double(), dy[lo:lo + n].double()
        ra[i] += (yd @ b[i].double()).T @ xd
        rb[i] += yd.T @ (xd @ a[i].double().T)
    for y, z, grad in ((s, x, da), (dy, t, db)):
        assert sg.grouped_wgrad_plan(y, z, grad, *m, 8, 130, add) == sg.VARIANT_TC
        sg.sgmv_grouped_wgrad(y, z, grad, *m, 8, 130, add)
    assert t.abs().max() < 256 and s.abs().max() < 256      # whole numbers in bf16
    assert torch.equal(da, ra.to(od)) and torch.equal(db, rb.to(od))
