"""Cases that measure the library's large segmented products.

Three operators, each in its plain form (elementary torch operations in 32 bits) and through the library:

  lora_linear    out[r] = x[r] W^T + bias + (x[r] A[a]^T) B[a]^T     a: adapter of the sequence that holds row r
  grouped_gemm   out[r] = x[r] W[e]^T                                e: expert of the segment that holds row r
  grouped_wgrad  dW[e]  = sum over the rows r of expert e of dY[r]^T X[r]

A case fixes the sizes, the ragged lengths and the adapter or expert of every segment (all drawn from the
case's own "lens" number), the seed fixes the values.
"""
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one request's next token through an attention projection with its adapter: the call whose latency counts
        {"name": "linear_one_token", "op": "lora_linear", "segments": 1, "rows": 1, "tail": 0, "K": 4096, "N": 4096, "rank": 16, "adapters": 32,
         "idle": 0, "bias": False, "dtype": "bf16", "lens": 1},
        # a decode step of 48 requests, each with an adapter of its own, some with none; fp16, with bias
        {"name": "linear_decode_48", "op": "lora_linear", "segments": 48, "rows": 48, "tail": 0, "K": 4096, "N": 12288, "rank": 16, "adapters": 64,
         "idle": 5, "bias": True, "dtype": "f16", "lens": 2},
        # the decode batch of 256 adapters: adapters and weights weigh alike
        {"name": "linear_decode_256", "op": "lora_linear", "segments": 256, "rows": 256, "tail": 0, "K": 5120, "N": 5120, "rank": 32, "adapters": 256,
         "idle": 26, "bias": False, "dtype": "bf16", "lens": 3},
        # a prefill of 16 ragged prompts through the fused query/key/value projection
        {"name": "linear_prefill_qkv", "op": "lora_linear", "segments": 16, "rows": 8764, "tail": 8, "K": 4096, "N": 12288, "rank": 16, "adapters": 32,
         "idle": 2, "bias": False, "dtype": "bf16", "lens": 4},
        # chunks and single tokens together, odd sizes, a rank that is no power of two, rows behind the last sequence
        {"name": "linear_mixed_odd", "op": "lora_linear", "segments": 37, "rows": 1531, "tail": 6, "K": 1032, "N": 2777, "rank": 24, "adapters": 19,
         "idle": 4, "bias": True, "dtype": "f16", "lens": 5},
        # a decode step of 48 tokens, two experts each of 64: every used expert's weights are read for one or two rows
        {"name": "experts_decode", "op": "grouped_gemm", "segments": 64, "rows": 96, "tail": 0, "K": 2048, "N": 1408, "experts": 64,
         "turned": False, "dtype": "bf16", "lens": 6},
        # a prefill through the up projection of 8 experts
        {"name": "experts_prefill", "op": "grouped_gemm", "segments": 8, "rows": 16384, "tail": 0, "K": 4096, "N": 11008, "experts": 8,
         "turned": False, "dtype": "bf16", "lens": 7},
        # the input gradient of 16 experts: weights read along their other axis
        {"name": "experts_dgrad", "op": "grouped_gemm", "segments": 16, "rows": 8192, "tail": 0, "K": 2816, "N": 2048, "experts": 16,
         "turned": True, "dtype": "bf16", "lens": 8},
        # few rows, odd sizes, fp16, more experts than segments
        {"name": "experts_odd", "op": "grouped_gemm", "segments": 5, "rows": 611, "tail": 3, "K": 520, "N": 777, "experts": 9,
         "turned": False, "dtype": "f16", "lens": 9},
        # the weight gradient of 16 experts
        {"name": "wgrad_experts", "op": "grouped_wgrad", "segments": 16, "rows": 8192, "tail": 0, "K": 2048, "N": 2816, "experts": 16,
         "dtype": "bf16", "out": "bf16", "lens": 8},
        # the largest: the weight gradient of the prefill's experts
        {"name": "wgrad_large", "op": "grouped_wgrad", "segments": 8, "rows": 16384, "tail": 0, "K": 4096, "N": 11008, "experts": 8,
         "dtype": "bf16", "out": "bf16", "lens": 7},
        # the gradient of adapters' A weights: a short side of 16, several sequences of one adapter, adapters without rows
        {"name": "wgrad_adapters", "op": "grouped_wgrad", "segments": 24, "rows": 4099, "tail": 5, "K": 4096, "N": 16, "experts": 32,
         "dtype": "f16", "out": "f16", "lens": 11},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["lora_linear", "lora_linear", "grouped_gemm", "grouped_gemm", "grouped_wgrad"])
    K, N = 8 * _spread(rng, 64, 640), _spread(rng, 256, 12288)
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "lens": rng.randrange(1 << 20), "tail": rng.choice([0, 0, 7])}
    if op == "lora_linear":
        segments = _spread(rng, 1, 256)
        rows = segments if rng.random() < 0.4 else max(segments, _spread(rng, 16, 8192))
        adapters = _spread(rng, 1, 256)
        case.update(K=K, N=N, segments=segments, rows=rows, rank=rng.choice([8, 16, 16, 24, 32, 64]), adapters=adapters,
                    idle=rng.randrange(segments // 4 + 1), bias=rng.random() < 0.5)
    elif op == "grouped_gemm":
        experts = _spread(rng, 2, 64)
        segments = rng.randint(1, experts)
        case.update(K=K, N=min(N, 4096) // 8 * 8 if rng.random() < 0.5 else min(N, 4096), segments=segments, experts=experts,
                    rows=max(segments, _spread(rng, 16, 8192)), turned=False)
        case["turned"] = case["N"] % 8 == 0 and rng.random() < 0.5
    else:
        experts = _spread(rng, 2, 32)
        segments = rng.randint(1, 2 * experts)
        N = rng.choice([16, 64]) if rng.random() < 0.3 else 8 * _spread(rng, 32, 512)
        case.update(K=min(K, 4096), N=N, segments=segments, experts=experts, rows=max(segments, _spread(rng, 16, 8192)), out=case["dtype"])
    return case


def _segments(case):
    """Lengths, and the adapter or expert (-1: none) of each segment, as lists; every segment has a row."""
    rng = random.Random(case["lens"])
    n, rows = case["segments"], case["rows"]
    share = [rng.expovariate(1.0) + 0.15 for _ in range(n)]
    spare = rows - n
    lens = [1 + int(spare * s / sum(share)) for s in share]
    for i in rng.choices(range(n), weights=share, k=rows - sum(lens)):
        lens[i] += 1
    if case["op"] == "lora_linear":
        ids = [i % case["adapters"] for i in range(n)]
        rng.shuffle(ids)
        for i in rng.sample(range(n), case["idle"]):
            ids[i] = -1
    elif case["op"] == "grouped_gemm":
        ids = sorted(rng.sample(range(case["experts"]), n))
    else:
        ids = [rng.randrange(case["experts"]) for _ in range(n)] if n > case["experts"] or case["N"] < 256 else sorted(rng.sample(range(case["experts"]), n))
    return lens, ids


def work(case):
    lens, ids = _segments(case)
    active = sum(l for l, a in zip(lens, ids) if a >= 0)
    used = len({a for a in ids if a >= 0})
    K, N = case["K"], case["N"]
    meta = 12 * len(lens)
    if case["op"] == "lora_linear":
        T, R = case["rows"] + case["tail"], case["rank"]
        return {"bytes": 2 * (T * K + N * K + T * N + used * R * (K + N) + (N if case["bias"] else 0)) + meta,
                "flops": 2 * T * N * K + 2 * active * R * (K + N)}
    if case["op"] == "grouped_gemm":
        return {"bytes": 2 * (active * (K + N) + used * N * K) + meta, "flops": 2 * active * N * K}
    return {"bytes": 2 * active * (K + N) + _DT[case["out"]].itemsize * case["experts"] * N * K + meta, "flops": 2 * active * N * K}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, T, K, N = _DT[case["dtype"]], case["rows"] + case["tail"], case["K"], case["N"]

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, std, generator=g)

    lens, ids = _segments(case)
    length = torch.tensor(lens, dtype=torch.int32)
    start = torch.cumsum(length, 0, dtype=torch.int32) - length
    s = {"op": case["op"], "x": normal(T, K), "start": start.cuda(), "len": length.cuda(), "idx": torch.tensor(ids, dtype=torch.int32).cuda(),
         "batches": len(lens), "longest": max(lens)}
    if case["op"] == "lora_linear":
        s["w"] = normal(N, K, std=0.02)
        s["bias"] = normal(N, std=0.5) if case["bias"] else None
        s["a"] = normal(case["adapters"], case["rank"], K, std=0.02)
        s["b"] = normal(case["adapters"], N, case["rank"], std=0.1)
        s["out"] = torch.zeros(T, N, dtype=dt, device="cuda")
        # the scratch memory that a program keeps for its largest call
        s["workspace"] = torch.empty(T * case["rank"] * 4 * 9 + T * 4 + 4096, dtype=torch.uint8, device="cuda")
    elif case["op"] == "grouped_gemm":
        if case["turned"]:  # the forward weights (E, out, in), seen as the (E, in, out) that the input gradient multiplies by
            s["w"] = normal(case["experts"], K, N, std=0.02).transpose(1, 2)
        else:
            s["w"] = normal(case["experts"], N, K, std=0.02)
        s["out"] = normal(T, N)  # rows behind the last segment keep these
        s["old_tail"] = s["out"][case["rows"]:].clone()
    else:
        s["dy"] = normal(T, N)
        s["dw"] = torch.empty(case["experts"], N, K, dtype=_DT[case["out"]], device="cuda")
    return s


def _padded(v, s):
    """(segments, longest, columns) of v's rows in 32 bits, zero behind each segment's end, and which places are filled."""
    at = torch.arange(s["longest"], device=v.device)
    here = at[None, :] < s["len"][:, None]
    rows = (s["start"][:, None] + at[None, :]) * here
    return v.float()[rows] * here[:, :, None], rows, here


def run(state):
    s = state
    if own:
        import segmented_gather_gemm_expand_b200 as sg
        meta = (s["start"], s["len"], s["idx"], s["batches"], s["longest"])
        if s["op"] == "lora_linear":
            return sg.sgmv_lora_linear(s["x"], s["w"], s["a"], s["b"], s["out"], *meta, bias=s["bias"], workspace=s["workspace"])
        if s["op"] == "grouped_gemm":
            return sg.sgmv_grouped_gemm(s["x"], s["w"], s["out"], *meta)
        return sg.sgmv_grouped_wgrad(s["dy"], s["x"], s["dw"], *meta)
    if s["op"] == "lora_linear":
        x = s["x"].float()
        A, R, K = s["a"].shape
        # the adapter of every row: the last segment that starts at or before it, if it reaches that far
        r = torch.arange(x.shape[0], device=x.device)
        inside = (r[:, None] >= s["start"][None, :]) & (r[:, None] < (s["start"] + s["len"])[None, :])
        adapter = torch.where(inside, s["idx"][None, :].long(), -1).amax(1)
        hot = adapter[:, None] == torch.arange(A, device=x.device)[None, :]
        t = (x @ s["a"].float().reshape(A * R, K).T).reshape(-1, A, R) * hot[:, :, None]
        y = x @ s["w"].float().T + t.reshape(-1, A * R) @ s["b"].float().transpose(1, 2).reshape(A * R, -1)
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y.to(s["x"].dtype)
    xp, rows, here = _padded(s["x"], s)
    if s["op"] == "grouped_gemm":
        y = torch.bmm(xp, s["w"][s["idx"].long()].float().transpose(1, 2))
        out = torch.empty_like(s["out"])
        out[out.shape[0] - s["old_tail"].shape[0]:] = s["old_tail"]
        out[rows[here]] = y[here].to(out.dtype)
        return out
    dyp = _padded(s["dy"], s)[0]
    dw = torch.bmm(dyp.transpose(1, 2), xp)
    total = torch.zeros(s["dw"].shape, dtype=torch.float32, device=dw.device)
    return total.index_add_(0, s["idx"].long(), dw).to(s["dw"].dtype)


def exact(case, seed):
    s = prepare(case, seed)
    lens, ids = _segments(case)
    x = s["x"].double()
    if case["op"] == "lora_linear":
        out = x @ s["w"].double().T
        if s["bias"] is not None:
            out += s["bias"].double()
        at = 0
        for n, a in zip(lens, ids):
            if a >= 0:
                out[at:at + n] += (x[at:at + n] @ s["a"][a].double().T) @ s["b"][a].double().T
            at += n
        return out
    if case["op"] == "grouped_gemm":
        out, at = s["out"].double(), 0
        for n, e in zip(lens, ids):
            out[at:at + n] = x[at:at + n] @ s["w"][e].double().T
            at += n
        return out
    dw, at = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda"), 0
    for n, e in zip(lens, ids):
        dw[e] += s["dy"][at:at + n].double().T @ x[at:at + n]
        at += n
    return dw
