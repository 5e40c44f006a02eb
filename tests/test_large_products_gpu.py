"""The large segmented products on the GPU against plain 64-bit implementations.

Most cases draw small whole numbers, for which every partial sum is a whole
number below 2^24: fp32 arithmetic in any order is then exact, and the kernels
must return the 64-bit result rounded once to the output type, bit for bit.
The cases with normal inputs bound the error by the rounding of the result
(eps / 2 of it; half of the smallest step where the result is subnormal) plus K * 2^-23 * sum |products|, the bound of K truncated or
rounded fp32 additions.
"""
import pytest
import torch

import segmented_gather_gemm_expand_b200 as sg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _clean():
    sg.set_variant(sg.VARIANT_AUTO)
    yield
    sg.set_variant(sg.VARIANT_AUTO)
    assert sg.device_error() == 0


def within(got, ref, sums):
    """|got - ref| <= half a step of got's type at ref (one part in 2^7 for ref's own distance from the fp32 sum that was
    rounded) + sums.  Below the type's smallest normal number `tiny` the steps no longer shrink with the value: they are
    tiny * eps (fp16: 2^-14 * 2^-10 = 2^-24), so half a step is tiny * eps / 2 there."""
    f = torch.finfo(got.dtype)
    half = torch.clamp(ref.abs() * (1 + 2 ** -7), min=f.tiny) * (f.eps / 2)
    over = (got.double() - ref).abs() - half - sums
    return bool((over <= 0).all())


def ints(g, shape, dt, top=2):
    return torch.randint(-top, top + 1, shape, generator=g, dtype=torch.int32).to(DT[dt]).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def meta(lens, ids, gaps=None, dtype=torch.int32):
    """Starts (with optional gaps before each segment), lengths and indexes on the GPU; rows covered in all."""
    starts, at = [], 0
    for i, n in enumerate(lens):
        at += gaps[i] if gaps else 0
        starts.append(at)
        at += max(n, 0)
    return [torch.tensor(v, dtype=dtype).cuda() for v in (starts, lens, ids)], at


def rows_of(m, lim, num):
    for s, n, e in zip(*[v.tolist() for v in m]):
        if 0 <= e < num and s >= 0 and n > 0 and min(s + n, lim) > s:
            yield s, min(s + n, lim), e


def rounded(v, dt):
    return v.float().to(DT[dt])


# ---------------------------------------------------------------- grouped products

def grouped_ref(x, w, out, m, add):
    ref = out.double()
    lim = min(x.shape[0], out.shape[0])
    for a, b, e in rows_of(m, lim, w.shape[0]):
        prod = x[a:b].double() @ w[e].double().T
        ref[a:b] = ref[a:b] + prod if add else prod
    return ref


SEGS = {
    "one": [1], "sixteen": [16], "ragged": [1, 0, 17, 130, 5, 64, 33], "long": [700, 3, 257], "many": [2] * 90 + [31],
    "prefill": [1100, 900],
}


@pytest.mark.parametrize("segs", SEGS)
@pytest.mark.parametrize("K,N", [(64, 128), (8, 7), (520, 777), (2048, 256), (136, 1000)])
@pytest.mark.parametrize("turned", [False, True])
def test_grouped_exact(segs, K, N, turned):
    if turned and N % 8:
        N += 8 - N % 8
    lens = SEGS[segs]
    g = gen(K + N)
    E = 6
    ids = torch.randint(-1, E + 1, (len(lens),), generator=g).tolist()
    ids[0] = 3
    m, T = meta(lens, ids)
    T += 9
    dt = "bf16" if K % 16 else "f16"
    x = ints(g, (T, K), dt)
    w = ints(g, (E, K, N), dt).transpose(1, 2) if turned else ints(g, (E, N, K), dt)
    for out_dt, add in (("f32", False), (dt, False), ("f32", True)):
        out = ints(g, (T, N), out_dt, 40)
        ref = rounded(grouped_ref(x, w, out, m, add), out_dt)
        assert sg.grouped_gemm_plan(x, w, out, *m, len(lens), max(lens), add) == sg.VARIANT_TC
        for variant in (sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE):
            got = out.clone()
            sg.set_variant(variant)
            sg.sgmv_grouped_gemm(x, w, got, *m, len(lens), max(lens), add)
            assert torch.equal(got, ref), (out_dt, add, variant, (got.float() - ref.float()).abs().max())


@pytest.mark.parametrize("K,N,T,layout", [(33, 50, 40, "odd"), (64, 96, 70, "strided"), (24, 40, 0, "odd"), (0, 24, 30, "odd")])
def test_grouped_generic(K, N, T, layout):
    g = gen(7)
    lens, ids = ([T - 20, 20], [1, 0]) if T else ([0, 0], [1, 0])
    m, _ = meta(lens, ids, dtype=torch.int64)
    x = ints(g, (T, 2 * K), "bf16")[:, ::2] if layout == "strided" else ints(g, (T, K), "bf16")
    w = ints(g, (3, N, K), "bf16")
    out = ints(g, (T, N), "f32")
    ref = grouped_ref(x, w, out, m, False).float()
    if T:
        assert sg.grouped_gemm_plan(x, w, out, *m, 2, 40) == sg.VARIANT_SIMT
    sg.sgmv_grouped_gemm(x, w, out, *m, 2, 40)
    assert torch.equal(out, ref)


def test_grouped_output_rows_of_a_wider_tensor():
    g = gen(3)
    m, T = meta([100, 37], [0, 1], gaps=[4, 11])
    x, w = ints(g, (T + 3, 256), "bf16"), ints(g, (2, 192, 256), "bf16")
    wide = ints(g, (T + 3, 500), "bf16")
    before = wide.clone()
    out = wide[:, 101:293]
    ref = rounded(grouped_ref(x, w, out, m, False), "bf16")
    sg.sgmv_grouped_gemm(x, w, out, *m, 2, 100)
    assert torch.equal(out, ref)
    keep = torch.ones(500, dtype=torch.bool)
    keep[101:293] = False
    assert torch.equal(wide[:, keep], before[:, keep])


@pytest.mark.parametrize("variant", [sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE, sg.VARIANT_SIMT])
def test_grouped_bad_metadata_and_foreign_rows(variant):
    """Negative starts and lengths, indexes out of range, segments past the end, NaN in rows of nobody."""
    g = gen(5)
    T, K, N, E = 300, 128, 200, 4
    m = [torch.tensor(v).cuda() for v in ([0, -3, 40, 120, 290, 200, 260], [37, 9, 50, -4, 1000, 60, 20], [2, 1, 0, 1, 3, 4, -1])]
    x, w = ints(g, (T, K), "f16"), ints(g, (E, N, K), "f16")
    x[37:40] = float("nan")
    x[90:290] = float("inf")
    out = ints(g, (T, N), "f32")
    ref = grouped_ref(x, w, out, m, False).float()
    sg.set_variant(variant)
    sg.sgmv_grouped_gemm(x, w, out, *m, 7, 1000)
    assert torch.equal(out, ref) and torch.isfinite(out).all()


def test_grouped_same_expert_twice_and_int64_metadata():
    g = gen(6)
    m, T = meta([90, 40, 90], [2, 1, 2], dtype=torch.int64)
    x, w, out = ints(g, (T, 320), "bf16"), ints(g, (3, 1, 264, 320), "bf16"), torch.zeros(T, 264).cuda()
    sg.sgmv_grouped_gemm(x, w, out, *m, 3, 90)
    assert torch.equal(out, grouped_ref(x, w[:, 0], out, m, False).float())


@pytest.mark.parametrize("T,B,K,N", [(96, 64, 2048, 1408), (6, 3, 4096, 512), (2500, 8, 1024, 1536)])
def test_grouped_normal_inputs(T, B, K, N):
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [T // B + (1 if i < T % B else 0) for i in range(B)]
    m, _ = meta(lens, list(range(B)))
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    w = (torch.randn(B, N, K, device="cuda", generator=g) * 0.02).bfloat16()
    out = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    sg.sgmv_grouped_gemm(x, w, out, *m, B, max(lens))
    for a, b, e in rows_of(m, T, B):
        ref, size = x[a:b].double() @ w[e].double().T, x[a:b].double().abs() @ w[e].double().abs().T
        assert within(out[a:b], ref, K * 2 ** -23 * size)


# ---------------------------------------------------------------- weight gradients

def wgrad_ref(dy, x, dw, m, add):
    ref = dw.double() if add else torch.zeros_like(dw, dtype=torch.float64)
    for a, b, e in rows_of(m, min(dy.shape[0], x.shape[0]), dw.shape[0]):
        ref[e] += dy[a:b].double().T @ x[a:b].double()
    return ref


@pytest.mark.parametrize("segs", SEGS)
@pytest.mark.parametrize("N,K", [(128, 64), (16, 520), (520, 16), (264, 1000), (8, 8)])
def test_wgrad_exact(segs, N, K):
    lens = SEGS[segs]
    g = gen(N + K)
    E = 5
    ids = torch.randint(-1, E, (len(lens),), generator=g).tolist()
    ids[0] = 3
    m, T = meta(lens, ids, gaps=[i % 3 for i in range(len(lens))])
    T += 4
    dt = "bf16" if N % 16 else "f16"
    dy, x = ints(g, (T, N), dt, 1), ints(g, (T, K), dt)
    owned = torch.zeros(T, dtype=torch.bool)
    for a, b, _ in rows_of(m, T, E):
        owned[a:b] = True
    dy[~owned.cuda()] = float("nan")   # rows of no segment never reach the sums
    x[~owned.cuda()] = float("inf")
    for out_dt, add in (("f32", False), (dt, False), ("f32", True)):
        dw = ints(g, (E, N, K), out_dt, 30)
        ref = rounded(wgrad_ref(dy, x, dw, m, add), out_dt)
        assert sg.grouped_wgrad_plan(dy, x, dw, *m, len(lens), max(lens), add) == sg.VARIANT_TC
        sg.sgmv_grouped_wgrad(dy, x, dw, *m, len(lens), max(lens), add)
        assert torch.equal(dw, ref), (out_dt, add, (dw.float() - ref.float()).abs().max())


@pytest.mark.parametrize("N,K,T,B", [(31, 45, 50, 2), (16, 24, 0, 1), (16, 24, 30, 0)])
@pytest.mark.parametrize("add", [False, True])
def test_wgrad_generic(N, K, T, B, add):
    g = gen(2)
    m, _ = meta([T - 9, 9][:B] if T else [0] * B, [1, 1][:B])
    dy, x, dw = ints(g, (T, N), "bf16"), ints(g, (T, K), "bf16"), ints(g, (3, N, K), "f32")
    ref = wgrad_ref(dy, x, dw, m, add).float()
    sg.sgmv_grouped_wgrad(dy, x, dw, *m, B, T, add)
    assert torch.equal(dw, ref)


def test_wgrad_normal_inputs_and_experts_without_rows():
    g = torch.Generator(device="cuda").manual_seed(1)
    lens, ids = [700, 1, 333, 64], [4, 0, 2, 4]
    m, T = meta(lens, ids)
    dy = torch.randn(T, 400, device="cuda", generator=g).half()
    x = torch.randn(T, 776, device="cuda", generator=g).half()
    dw = torch.full((6, 400, 776), float("nan"), device="cuda", dtype=torch.float16)
    sg.sgmv_grouped_wgrad(dy, x, dw, *m, 4, 700)
    ref, size = torch.zeros(6, 400, 776, device="cuda", dtype=torch.float64), torch.zeros(6, 400, 776, device="cuda", dtype=torch.float64)
    for a, b, e in rows_of(m, T, 6):
        ref[e] += dy[a:b].double().T @ x[a:b].double()
        size[e] += dy[a:b].double().T.abs() @ x[a:b].double().abs()
    assert within(dw, ref, 764 * 2 ** -23 * size)
    assert (dw[[1, 3, 5]] == 0).all()


# ---------------------------------------------------------------- shared projection with adapters

def lora_ref(x, w, a, b, m, bias, T):
    ref = x[:T].double() @ w.double().T
    if bias is not None:
        ref += bias.double()
    for s, e, i in rows_of(m, T, a.shape[0]):
        ref[s:e] += (x[s:e].double() @ a[i].double().T) @ b[i].double().T
    return ref


def run_lora(x, w, a, b, out, m, n, longest, bias=None, spare=True):
    _, need, pref = sg.lora_linear_plan(x, w, a, b, out, *m, n, longest, bias=bias)
    ws = torch.full((max(pref if spare else need, 16),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere
    return sg.sgmv_lora_linear(x, w, a, b, out, *m, n, longest, bias=bias, workspace=ws)


LORA_SEGS = {"one": [1], "decode": [1] * 40, "decode_300": [1] * 300, "mixed": [1, 200, 1, 0, 57, 1, 90], "prefill": [500, 700, 3]}


@pytest.mark.parametrize("segs", LORA_SEGS)
@pytest.mark.parametrize("R", [8, 16, 24, 64])
@pytest.mark.parametrize("K,N", [(256, 384), (1032, 777), (4096, 264)])
def test_lora_exact(segs, R, K, N):
    lens = LORA_SEGS[segs]
    g = gen(R + K)
    A = 7
    ids = torch.randint(-1, A + 1, (len(lens),), generator=g).tolist()
    ids[0] = 5
    m, T = meta(lens, ids, gaps=[3] * len(lens) if segs == "mixed" else None)
    T += 5
    dt = "f16" if R % 16 else "bf16"
    x, w = ints(g, (T, K), dt, 1), ints(g, (N, K), dt)
    a, b, bias = ints(g, (A, R, K), dt, 1), ints(g, (A, N, R), dt, 1), ints(g, (N,), dt, 9)
    for out_dt, bi, spare in (("f32", bias, True), (dt, None, False)):
        out = torch.full((T + 2, N), 77.0, device="cuda", dtype=DT[out_dt])
        ref = rounded(lora_ref(x, w, a, b, m, bi, T), out_dt)
        for variant in (sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE):
            sg.set_variant(variant)
            assert sg.lora_linear_plan(x, w, a, b, out, *m, len(lens), max(lens), bias=bi)[0] == sg.VARIANT_TC
            run_lora(x, w, a, b, out, m, len(lens), max(lens), bi, spare)
            assert torch.equal(out[:T], ref), (out_dt, variant, (out[:T].float() - ref.float()).abs().max())
            assert (out[T:] == 77).all()


@pytest.mark.parametrize("case", ["odd", "f32_x", "strided", "no_adapters", "no_k", "forced"])
def test_lora_generic_and_edges(case):
    g = gen(11)
    K, N, R, T, A = (0 if case == "no_k" else 45 if case == "odd" else 64), 50, 5, 300, (0 if case == "no_adapters" else 3)
    m, _ = meta([100, 1, 60], [0, -1, 2], gaps=[2, 0, 5])
    x = ints(g, (T, K), "f32" if case == "f32_x" else "bf16", 1)
    if case == "strided":
        x = ints(g, (T, 2 * K), "bf16", 1)[:, ::2]
    w, a, b = ints(g, (N, K), "bf16"), ints(g, (A, R, K), "bf16", 1), ints(g, (A, N, R), "bf16", 1)
    if case == "strided":
        b = ints(g, (A, R, N), "bf16", 1).transpose(1, 2)
    bias = ints(g, (2 * N,), "bf16", 5)[::2]
    out = torch.zeros(T, N, device="cuda")
    if case == "forced":
        sg.set_variant(sg.VARIANT_SIMT)
    run_lora(x, w, a, b, out, m, 3, 100, bias)
    assert torch.equal(out, lora_ref(x, w, a, b, m, bias, T).float())
    if case == "no_adapters":
        sg.sgmv_lora_linear(x, w, a, b, out, *m, 3, 100, bias=bias)   # needs no workspace


def test_lora_infinite_rows_stay_their_own():
    """An infinity in one request's row reaches that row alone."""
    g = gen(12)
    m, T = meta([1] * 20, [i % 4 for i in range(20)])
    x, w, a, b = ints(g, (T, 512), "bf16", 1), ints(g, (256, 512), "bf16"), ints(g, (4, 16, 512), "bf16", 1), ints(g, (4, 256, 16), "bf16", 1)
    ref = lora_ref(x, w, a, b, m, None, T).float()
    x[7, 3] = float("inf")
    out = torch.zeros(T, 256, device="cuda")
    run_lora(x, w, a, b, out, m, 20, 1)
    rest = [i for i in range(T) if i != 7]
    assert torch.equal(out[rest], ref[rest]) and not torch.isfinite(out[7]).any()


@pytest.mark.parametrize("T,K,N,R,dt", [(48, 4096, 768, 16, "f16"), (256, 5120, 640, 32, "bf16"), (900, 1024, 2777, 24, "bf16")])
def test_lora_normal_inputs(T, K, N, R, dt):
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [1] * T if T <= 256 else [300, 1, 599]
    n = len(lens)
    m, _ = meta(lens, [i % 50 for i in range(n)])
    def normal(*s, std=1.0):
        return (torch.randn(*s, device="cuda", generator=g) * std).to(DT[dt])
    x, w, a, b = normal(T, K), normal(N, K, std=0.02), normal(50, R, K, std=0.02), normal(50, N, R, std=0.1)
    out = torch.empty(T, N, device="cuda", dtype=DT[dt])
    run_lora(x, w, a, b, out, m, n, max(lens))
    ref = lora_ref(x, w, a, b, m, None, T)
    # t's own sum has the bound of K additions, and enters with |B|; R more additions follow
    size = lora_ref(x.abs(), w.abs(), a.abs(), b.abs(), m, None, T)
    assert within(out, ref, (2 * K + R) * 2 ** -23 * size)


# ---------------------------------------------------------------- together, and in a program

def chain(dt, seed=4):
    """A projection with adapters, two expert products on top, and the gradients back to x and both experts' weights."""
    g = gen(seed)
    lens, ids = [70, 1, 1, 130, 44], [2, -1, 0, 1, 2]
    m, T = meta(lens, ids)
    em, _ = meta([100, 0, 91, 55], [0, 1, 2, 3])
    K, N, R = 192, 256, 16
    v = dict(x=ints(g, (T, K), dt, 1), w=ints(g, (N, K), dt, 1), a=ints(g, (3, R, K), dt, 1), b=ints(g, (3, N, R), dt, 1),
             up=ints(g, (4, 320, N), dt, 1), dy=ints(g, (T, 320), dt, 1), h=torch.zeros(T, N, device="cuda", dtype=DT[dt]),
             y=torch.zeros(T, 320, device="cuda"), dh=torch.zeros(T, N, device="cuda"), dup=torch.zeros(4, 320, N, device="cuda"))
    _, _, pref = sg.lora_linear_plan(v["x"], v["w"], v["a"], v["b"], v["h"], *m, 5, 130)
    v["ws"] = torch.empty(pref, dtype=torch.uint8, device="cuda")

    def go():
        sg.sgmv_lora_linear(v["x"], v["w"], v["a"], v["b"], v["h"], *m, 5, 130, workspace=v["ws"])
        sg.sgmv_grouped_gemm(v["h"], v["up"], v["y"], *em, 4, 100)
        sg.sgmv_grouped_gemm(v["dy"], v["up"].transpose(1, 2), v["dh"], *em, 4, 100)
        sg.sgmv_grouped_wgrad(v["dy"], v["h"], v["dup"], *em, 4, 100)

    def check():
        h = rounded(lora_ref(v["x"], v["w"], v["a"], v["b"], m, None, T), dt)
        assert torch.equal(v["h"], h)
        y, dh = torch.zeros(T, 320, dtype=torch.float64, device="cuda"), torch.zeros(T, N, dtype=torch.float64, device="cuda")
        y = grouped_ref(h, v["up"], y, em, False)
        dh = grouped_ref(v["dy"], v["up"].transpose(1, 2), dh, em, False)
        dup = wgrad_ref(v["dy"], h, v["dup"], em, False)
        assert torch.equal(v["y"], y.float()) and torch.equal(v["dh"], dh.float()) and torch.equal(v["dup"], dup.float())
    return v, go, check


def test_chain_eager_then_graph():
    v, go, check = chain("bf16")
    go()
    check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go()
    for seed in (9, 10):
        other, _, _ = chain("bf16", seed)
        for k in ("x", "w", "a", "b", "up", "dy"):
            v[k].copy_(other[k])
        for k in ("h", "y", "dh", "dup"):
            v[k].fill_(float("nan"))
        graph.replay()
        check()


def test_chains_on_two_streams_at_once():
    chains = [chain("f16", s) for s in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(20):
        for (v, go, _), s in zip(chains, streams):
            with torch.cuda.stream(s):
                go()
    torch.cuda.synchronize()
    for _, _, check in chains:
        check()


def test_gradient_against_differences():
    """Whole numbers make a central difference of the (linear) forward pass exact."""
    g = gen(8)
    m, T = meta([30, 21], [1, 0])
    x, w, dy = ints(g, (T, 64), "bf16", 1), ints(g, (2, 72, 64), "bf16", 1), ints(g, (T, 72), "bf16", 1)
    dw, dx = torch.zeros(2, 72, 64, device="cuda"), torch.zeros(T, 64, device="cuda")
    sg.sgmv_grouped_wgrad(dy, x, dw, *m, 2, 30)
    sg.sgmv_grouped_gemm(dy, w.transpose(1, 2), dx, *m, 2, 30)

    def loss(x_, w_):
        y = torch.zeros(T, 72, device="cuda")
        sg.sgmv_grouped_gemm(x_, w_, y, *m, 2, 30)
        return (y.double() * dy.double()).sum().item()

    for e, n, k in ((0, 0, 0), (1, 71, 63), (1, 5, 33)):
        d = torch.zeros_like(w)
        d[e, n, k] = 1
        assert (loss(x, w + d) - loss(x, w - d)) / 2 == dw[e, n, k].item()
    for r, k in ((0, 0), (T - 1, 63), (30, 7)):
        d = torch.zeros_like(x)
        d[r, k] = 1
        assert (loss(x + d, w) - loss(x - d, w)) / 2 == dx[r, k].item()


def test_repeated_calls_give_the_same_bits():
    g = torch.Generator(device="cuda").manual_seed(3)
    m, T = meta([1] * 9, list(range(9)))
    x = torch.randn(T, 4096, device="cuda", generator=g).bfloat16()
    w = torch.randn(9, 640, 4096, device="cuda", generator=g).bfloat16()
    outs = [torch.empty(T, 640, device="cuda", dtype=torch.float32) for _ in range(3)]
    for o in outs:
        sg.sgmv_grouped_gemm(x, w, o, *m, 9, 1)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------- layouts, limits and values at the edges

@pytest.mark.parametrize("lens", ["decode", "decode_many", "long"])
@pytest.mark.parametrize("layout", ["rank5", "rank72", "turned", "pitched"])
def test_lora_b_layouts(lens, layout):
    """Ranks and B layouts that the copies of whole rows do not take, beside inputs that the tensor cores do."""
    g = gen(21)
    lens = {"decode": [1] * 33, "decode_many": [1] * 300, "long": [150, 300, 7]}[lens]
    n, K, N, A = len(lens), 128, 200, 9
    R = {"rank5": 5, "rank72": 72, "turned": 16, "pitched": 16}[layout]
    m, T = meta(lens, [(5 * i) % (A + 1) - 1 for i in range(n)])
    x, w, a = ints(g, (T, K), "bf16", 1), ints(g, (N, K), "bf16"), ints(g, (A, R, K), "bf16", 1)
    b = {"turned": lambda: ints(g, (A, R, N), "bf16", 1).transpose(1, 2), "pitched": lambda: ints(g, (A, N, R + 8), "bf16", 1)[:, :, :R]}.get(
        layout, lambda: ints(g, (A, N, R), "bf16", 1))()
    for out_dt in ("bf16", "f32"):
        out = torch.zeros(T, N, device="cuda", dtype=DT[out_dt])
        assert sg.lora_linear_plan(x, w, a, b, out, *m, n, max(lens))[0] == sg.VARIANT_TC
        run_lora(x, w, a, b, out, m, n, max(lens))
        assert torch.equal(out, rounded(lora_ref(x, w, a, b, m, None, T), out_dt))


def test_lora_weight_read_along_its_other_axis():
    g = gen(22)
    m, T = meta([90, 1, 60], [1, 0, 1])
    x, w = ints(g, (T, 200), "f16", 1), ints(g, (200, 328), "f16").t()
    a, b, out = ints(g, (2, 16, 200), "f16", 1), ints(g, (2, 328, 16), "f16", 1), torch.zeros(T, 328, device="cuda")
    assert sg.lora_linear_plan(x, w, a, b, out, *m, 3, 90)[0] == sg.VARIANT_TC
    run_lora(x, w, a, b, out, m, 3, 90)
    assert torch.equal(out, lora_ref(x, w, a, b, m, None, T).float())


@pytest.mark.parametrize("variant", [sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE])
@pytest.mark.parametrize("K,bad", [(256, float("inf")), (4096, float("nan"))])
def test_one_requests_broken_adapter_or_row_stays_its_own(variant, K, bad):
    """An adapter whose B holds infinities or NaN, and a row of x that does, reach their own rows only, also in a batch whose
    runs share token tiles."""
    g = gen(23)
    m, T = meta([70, 33, 50, 20, 90], [0, 1, 2, 1, 0])
    x, w, a, b = ints(g, (T, K), "bf16", 1), ints(g, (264, K), "bf16", 1), ints(g, (3, 16, K), "bf16", 1), ints(g, (3, 264, 16), "bf16", 1)
    ref = lora_ref(x, w, a, b, m, None, T).float()
    b[1, 5:200, 3] = bad
    x[160, 7] = bad
    out = torch.zeros(T, 264, device="cuda")
    sg.set_variant(variant)
    run_lora(x, w, a, b, out, m, 5, 90)
    keep = torch.ones(T, dtype=torch.bool)
    keep[70:103] = keep[153:173] = False
    assert torch.equal(out[keep], ref[keep])
    assert torch.equal(out[70:103, 200:], ref[70:103, 200:])   # the adapter's finite columns too
    assert not torch.isfinite(out[160]).any()


def test_lora_t_beyond_fp16():
    """t is held in fp32: values past fp16's largest number enter the product whole."""
    g = gen(24)
    m, T = meta([40, 25], [0, 1])
    x = torch.full((T, 512), 16.0, device="cuda", dtype=torch.float16)
    a = torch.full((2, 16, 512), 16.0, device="cuda", dtype=torch.float16)   # t = 131072
    w, b = ints(g, (264, 512), "f16", 1), ints(g, (2, 264, 16), "f16", 1)
    out = torch.zeros(T, 264, device="cuda")
    run_lora(x, w, a, b, out, m, 2, 40)
    assert torch.equal(out, lora_ref(x, w, a, b, m, None, T).float())


@pytest.mark.parametrize("count,length", [(4000, 2), (5000, 1)])
def test_many_segments(count, length):
    g = gen(25)
    E = 50
    m, T = meta([length] * count, [i % E for i in range(count)])
    x, w, out = ints(g, (T, 64), "bf16"), ints(g, (E, 72, 64), "bf16"), torch.zeros(T, 72, device="cuda")
    sg.sgmv_grouped_gemm(x, w, out, *m, count, length)
    e = (torch.arange(T) // length % E).cuda()
    assert torch.equal(out, torch.bmm(w.float()[e], x.float()[:, :, None])[:, :, 0])
    dy, dw = ints(g, (T, 72), "bf16", 1), torch.zeros(E, 72, 64, device="cuda")
    sg.sgmv_grouped_wgrad(dy, x, dw, *m, count, length)
    ref = torch.zeros(E, 72, 64, device="cuda").index_add_(0, e, dy.float()[:, :, None] * x.float()[:, None, :])
    assert torch.equal(dw, ref)
    base, a, b = ints(g, (72, 64), "bf16"), ints(g, (E, 8, 64), "bf16", 1), ints(g, (E, 72, 8), "bf16", 1)
    run_lora(x, base, a, b, out, m, count, length)
    t = torch.bmm(a.float()[e], x.float()[:, :, None])
    assert torch.equal(out, x.float() @ base.float().T + torch.bmm(b.float()[e], t)[:, :, 0])


def test_outputs_and_weights_past_32_bit_offsets():
    """Elements of the output and of the experts' weights at offsets beyond 2^31."""
    g = gen(26)
    T, N, K = 66000, 33000, 64      # 2.18e9 outputs
    out = torch.zeros(T, N, device="cuda", dtype=torch.bfloat16)
    m = [torch.tensor(v).cuda() for v in ([0, 65900], [70, 100], [0, 1])]
    x, w = torch.zeros(T, K, device="cuda", dtype=torch.bfloat16), ints(g, (2, N, K), "bf16")
    x[:70], x[65900:] = ints(g, (70, K), "bf16"), ints(g, (100, K), "bf16")
    sg.sgmv_grouped_gemm(x, w, out, *m, 2, 100)
    for a, b, e in ((0, 70, 0), (65900, 66000, 1)):
        assert torch.equal(out[a:b], rounded(x[a:b].double() @ w[e].double().T, "bf16"))
    assert not out[70:65900].any()
    del out, w
    E, N, K = 540, 1000, 4096       # 2.2e9 weights
    w = torch.zeros(E, N, K, device="cuda", dtype=torch.bfloat16)
    w[E - 1] = ints(g, (N, K), "bf16")
    x, out = ints(g, (20, K), "bf16"), torch.zeros(20, N, device="cuda")
    m, _ = meta([20], [E - 1])
    sg.sgmv_grouped_gemm(x, w, out, *m, 1, 20)
    assert torch.equal(out, (x.double() @ w[E - 1].double().T).float())
    dy = ints(g, (20, N), "bf16", 1)
    sg.sgmv_grouped_wgrad(dy, x, w, *m, 1, 20)
    assert torch.equal(w[E - 1], rounded(dy.double().T @ x.double(), "bf16")) and not w[: E - 1].any()


def test_inputs_and_output_of_different_row_counts():
    g = gen(27)
    m, _ = meta([64, 64], [0, 1])
    x, w, out = ints(g, (100, 64), "bf16"), ints(g, (2, 40, 64), "bf16"), ints(g, (90, 40), "f32")
    ref = grouped_ref(x, w, out, m, False).float()
    sg.sgmv_grouped_gemm(x, w, out, *m, 2, 64)
    assert torch.equal(out, ref)
    a, b, base = ints(g, (2, 8, 64), "bf16", 1), ints(g, (2, 40, 8), "bf16", 1), ints(g, (40, 64), "bf16")
    out = torch.full((130, 40), 5.0, device="cuda")
    run_lora(x, base, a, b, out, m, 2, 64)
    assert torch.equal(out[:100], lora_ref(x, base, a, b, m, None, 100).float()) and (out[100:] == 5).all()


def test_empty_calls_and_workspace_refusals():
    g = gen(28)
    m, T = meta([3], [0])
    x, w, a, b = ints(g, (T, 64), "bf16"), ints(g, (40, 64), "bf16"), ints(g, (1, 16, 64), "bf16"), ints(g, (1, 40, 16), "bf16")
    out = torch.full((T, 40), 3.0, device="cuda")
    _, need, pref = sg.lora_linear_plan(x, w, a, b, out, *m, 1, 3)
    assert 0 < need <= pref
    ws = torch.empty(pref + 16, dtype=torch.uint8, device="cuda")
    for bad in (None, ws[: need - 1], ws[8:]):
        with pytest.raises(sg.SgmvError) as e:
            sg.sgmv_lora_linear(x, w, a, b, out, *m, 1, 3, workspace=bad)
        assert e.value.code == -17
    sg.sgmv_lora_linear(x[:0], w, a, b, out[:0], *m, 1, 3)
    sg.sgmv_lora_linear(x, w[:0], a, b[:, :0], out[:, :0], *m, 1, 3)
    sg.sgmv_grouped_gemm(x, w[None], out, *m, 0, 3)
    assert (out == 3).all()
    with pytest.raises(ValueError):
        sg.sgmv_grouped_gemm(x, w[None].cpu(), out, *m, 1, 3)
    with pytest.raises(TypeError):
        sg.sgmv_grouped_gemm(x.double(), w[None], out, *m, 1, 3)
    sg.set_variant(sg.VARIANT_DECODE)
    for call in (lambda: sg.sgmv_grouped_gemm(x, w[None], out, *m, 1, 3), lambda: sg.sgmv_grouped_wgrad(x, x, torch.zeros(1, 64, 64).cuda(), *m, 1, 3),
                 lambda: sg.sgmv_lora_linear(x, w, a, b, out, *m, 1, 3, workspace=ws)):
        with pytest.raises(sg.SgmvError) as e:
            call()
        assert e.value.code == -13


def test_call_reads_what_the_preceding_kernels_wrote():
    """x, weights, adapters and metadata rewritten on the device right before each call."""
    g = gen(29)
    m, T = meta([30, 1, 40], [1, 0, 1])
    x, w, a, b = ints(g, (T, 512), "bf16", 1), ints(g, (264, 512), "bf16", 1), ints(g, (2, 16, 512), "bf16", 1), ints(g, (2, 264, 16), "bf16", 1)
    out = torch.zeros(T, 264, device="cuda")
    _, _, pref = sg.lora_linear_plan(x, w, a, b, out, *m, 3, 40)
    ws = torch.empty(pref, dtype=torch.uint8, device="cuda")
    outs, refs = [], []
    for i in range(6):
        for t in (x, w, a, b):
            t.mul_(-1 if i % 2 else 1).add_(1 if i % 3 else -1)
        m[2].copy_(torch.tensor([i % 2, 1, -1 if i == 3 else (i + 1) % 2], dtype=torch.int32), non_blocking=True)
        sg.sgmv_lora_linear(x, w, a, b, out, *m, 3, 40, workspace=ws)
        outs.append(out.clone())
        refs.append(lora_ref(x, w, a, b, m, None, T).float())
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


def test_python_calls_on_another_device_than_the_current_one():
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    g = gen(30)
    with torch.cuda.device(1):
        m, T = meta([9], [0])
        x, w, out = ints(g, (T, 64), "bf16"), ints(g, (1, 40, 64), "bf16"), torch.zeros(T, 40, device="cuda")
    sg.sgmv_grouped_gemm(x, w, out, *m, 1, 9)
    torch.cuda.synchronize(1)
    assert torch.equal(out, (x.double() @ w[0].double().T).float())


def test_values_that_are_no_numbers_in_shared_inputs():
    """NaN rows of x and infinite rows of the shared weight come out as the formula has them, at no other place."""
    g = gen(31)
    m, T = meta([140, 160], [0, 1])
    x, w, a, b = ints(g, (T, 4096), "bf16", 1), ints(g, (264, 4096), "bf16", 1), ints(g, (2, 16, 4096), "bf16", 1), ints(g, (2, 264, 16), "bf16", 1)
    ref = lora_ref(x, w, a, b, m, None, T).float()
    x[::3] = float("nan")
    w[7, 5] = float("inf")
    out = torch.zeros(T, 264, device="cuda")
    run_lora(x, w, a, b, out, m, 2, 160)
    rows = torch.arange(T) % 3 != 0
    cols = torch.arange(264) != 7
    assert torch.isnan(out[::3]).all() and not torch.isfinite(out[:, 7]).any()
    assert torch.equal(out[rows][:, cols], ref[rows][:, cols])


# ---------------------------------------------------------------- backward pass of a projection with adapters

@pytest.mark.parametrize("lens", [[90, 40, 0, 33, 130], [1] * 7])
@pytest.mark.parametrize("R,K,N", [(16, 264, 136), (4, 136, 200), (13, 128, 96)])
def test_lora_backward_from_views(lens, R, K, N):
    """dX from transposed views, dA and dB from the weight gradient, against the formulas."""
    g = gen(31 + R)
    A, n = 3, len(lens)
    m, T = meta(lens, [(2 * i) % (A + 1) - 1 for i in range(n)])
    x, w, dy = ints(g, (T, K), "bf16", 1), ints(g, (N, K), "bf16", 1), ints(g, (T, N), "bf16", 1)
    a, b = ints(g, (A, R, K), "bf16", 1), ints(g, (A, N, R), "bf16", 1)
    wt, at, bt = w.t(), a.transpose(1, 2), b.transpose(1, 2)
    for dt in ("bf16", "f32"):
        for spare in (True, False):
            dx = torch.full((T, K), float("nan"), device="cuda", dtype=DT[dt])
            run_lora(dy, wt, bt, at, dx, m, n, max(lens), spare=spare)
            assert torch.equal(dx, rounded(lora_ref(dy, wt, bt, at, m, None, T), dt))
    da, db = torch.zeros(A, R, K, device="cuda"), torch.zeros(A, N, R, device="cuda")
    t, s = torch.zeros(T, R, device="cuda"), torch.zeros(T, R, device="cuda")   # x A^T, dY B
    sg.sgmv_shrink(x, a, t, *m, n, max(lens))
    sg.sgmv_shrink(dy, bt, s, *m, n, max(lens))
    sg.sgmv_grouped_wgrad(s, x, da, *m, n, max(lens))
    sg.sgmv_grouped_wgrad(dy, t, db, *m, n, max(lens))
    ra, rb = torch.zeros(A, R, K, device="cuda", dtype=torch.float64), torch.zeros(A, N, R, device="cuda", dtype=torch.float64)
    for lo, hi, i in rows_of(m, T, A):
        xd, yd = x[lo:hi].double(), dy[lo:hi].double()
        ra[i] += (yd @ b[i].double()).T @ xd
        rb[i] += yd.T @ (xd @ a[i].double().T)
    assert torch.equal(da, ra.float()) and torch.equal(db, rb.float())


def test_plans_follow_the_tensors():
    """Calls of the same shapes on other tensors, at other alignments too."""
    g = gen(41)
    m, T = meta([70, 1, 60], [0, 1, 0])
    K, N = 128, 256
    for shift in (0, 0, 8, 1, 0):
        x, w, dw, out = ints(g, (T * K + 8,), "bf16", 1)[shift:shift + T * K].view(T, K), ints(g, (2, N, K), "bf16", 1), torch.zeros(
            2, N, K, device="cuda"), torch.zeros(T, N, device="cuda", dtype=torch.bfloat16)
        sg.sgmv_grouped_gemm(x, w, out, *m, 3, 70)
        assert torch.equal(out, rounded(grouped_ref(x, w, torch.zeros_like(out), m, False), "bf16"))
        dy = ints(g, (T, N), "bf16", 1)
        sg.sgmv_grouped_wgrad(dy, x, dw, *m, 3, 70)
        ref = torch.zeros(2, N, K, device="cuda", dtype=torch.float64)
        for lo, hi, e in rows_of(m, T, 2):
            ref[e] += dy[lo:hi].double().T @ x[lo:hi].double()
        assert torch.equal(dw, ref.float())


@pytest.mark.parametrize("T,seg,R", [(600, 1, 16), (4096, 1, 8), (515, 2, 16), (1000, 3, 16), (250, 50, 64), (4097, 2, 8)])
def test_lora_many_short_segments_in_any_order(T, seg, R):
    """Segments against the rows' order, and the same adapter in neighbouring ones: a row's segment has to be searched for."""
    g = gen(51)
    n, A, K, N = T // seg, 6, 96, 72
    ids = torch.randint(-1, A + 1, (n,), generator=g).int().cuda()
    m = [(torch.arange(n - 1, -1, -1) * seg).int().cuda(), torch.full((n,), seg, dtype=torch.int32).cuda(), ids]
    x, w = ints(g, (T, K), "bf16", 1), ints(g, (N, K), "bf16", 1)
    a, b = ints(g, (A, R, K), "bf16", 1), ints(g, (A, N, R), "bf16", 1)
    out = torch.zeros(T, N, device="cuda")
    run_lora(x, w, a, b, out, m, n, seg)
    assert torch.equal(out, lora_ref(x, w, a, b, m, None, T).float())


@pytest.mark.parametrize("R", [4, 8, 13, 16, 17, 40])
@pytest.mark.parametrize("lens", [[60, 70, 55], [20] * 30, [17, 200, 33, 40, 64, 31]])
def test_lora_runs_that_share_steps(R, lens):
    """Odd and even numbers of runs in a token tile of a CTA pair, some without an adapter, gaps between them."""
    g = gen(61 + R)
    n, A, K, N = len(lens), 5, 128, 300
    m, T = meta(lens, [(3 * i) % (A + 1) - 1 for i in range(n)], gaps=[(5 * i) % 7 for i in range(n)])
    T += 9
    x, w = ints(g, (T, K), "f16", 1), ints(g, (N, K), "f16", 1)
    a, b = ints(g, (A, R, K), "f16", 1), ints(g, (A, N, R), "f16", 1)
    for variant in (sg.VARIANT_AUTO, sg.VARIANT_TC_WIDE):
        sg.set_variant(variant)
        for dt in ("f16", "f32"):
            out = torch.full((T, N), float("nan"), device="cuda", dtype=DT[dt])
            run_lora(x, w, a, b, out, m, n, max(lens))
            assert torch.equal(out, rounded(lora_ref(x, w, a, b, m, None, T), dt))


@pytest.mark.parametrize("cols,rows_dy", [(264, 40), (136, 300), (520, 776), (300, 48)])
@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
def test_wgrad_zeros_stay_inside_their_index(cols, rows_dy, out_dt):
    """Indexes without rows between those with some, in a dW whose rows and indexes have gaps: the gaps keep their bits."""
    g = gen(71)
    m, T = meta([3, 70, 1], [4, 1, 1])
    dy, x = ints(g, (T, rows_dy), "bf16", 1), ints(g, (T, cols + 4 if cols % 8 else cols), "bf16", 1)[:, :cols]
    full = torch.full((6, rows_dy + 1, cols + 8), 7.0, device="cuda", dtype=DT[out_dt])
    dw = full[:, :rows_dy, :cols]
    sg.sgmv_grouped_wgrad(dy, x, dw, *m, 3, 70)
    ref = torch.full_like(full, 7.0, dtype=torch.float64)
    ref[:, :rows_dy, :cols] = 0
    for lo, hi, e in rows_of(m, T, 6):
        ref[e, :rows_dy, :cols] += dy[lo:hi].double().T @ x[lo:hi].double()
    assert torch.equal(full, ref.to(DT[out_dt]))


def test_lora_lengths_beyond_any_number_of_rows():
    """64-bit metadata at its limits: every part of a call takes the same rows for a segment."""
    g = gen(81)
    m = [torch.tensor([0, 100, -5, 2 ** 62, 260], dtype=torch.int64).cuda(), torch.tensor([100, 60, 50, 5, 2 ** 62], dtype=torch.int64).cuda(),
         torch.tensor([0, 1, 2, 1, 0], dtype=torch.int64).cuda()]
    T, K, N, A = 300, 128, 200, 3
    x, w = ints(g, (T, K), "bf16", 1), ints(g, (N, K), "bf16", 1)
    a, b, out = ints(g, (A, 16, K), "bf16", 1), ints(g, (A, N, 16), "bf16", 1), torch.zeros(T, N, device="cuda")
    run_lora(x, w, a, b, out, m, 5, 300)
    ref = x.double() @ w.double().T
    for lo, hi, i in ((0, 100, 0), (100, 160, 1), (260, 300, 0)):
        ref[lo:hi] += (x[lo:hi].double() @ a[i].double().T) @ b[i].double().T
    assert torch.equal(out, ref.float())
