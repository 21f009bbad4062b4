"""Cases for measuring the operators that train a mixture-of-experts block's weights and run it
in 16 bits.

Each operator has a plain form here (elementary torch operations in 32 bits, rounded once at the
end), a call of the library's own kernel, and an evaluation in 64 bits from its definition:

* mm: rows packed by expert times each expert's matrix, in bf16 or fp16: the forward product
  (out = x . w^T) and, with the same weights read the other way, the product of the backward
  pass (dx = dy . w);
* weight_grad: the gradient of each expert's matrix, dw = dy^T . x over the expert's rows, onto
  what was accumulated before where there is some;
* grad_norm: the norm of all gradients of a model taken together;
* clip: the gradients scaled so that this norm does not exceed a bound.

``own`` selects the library's kernels; a case is a dict of plain values.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
MIXED = ("bf16", "fp32", "bf16", "fp16")
CLIP_EPS = 1e-6
MAX_FLOPS = 2 * 32768 * 4096 * 7168     # of a product: those of the largest listed one


def _mm(**more):
    return {"spare": 0, "pad": 0, "transposed": False, **more}


def listed():
    """4 to 12 cases over the real range: hidden size 7168 with experts of width 2048 (gate and
    up side by side: 4096), 32 experts on the device, 8 per token."""
    return [
        # one token of a decode step: eight experts' gate/up matrices are read for a row each
        _mm(name="mm_decode_1", op="mm", tokens=1, top_k=8, experts=32, n=4096, k=7168,
            dtype="bf16"),
        # a decode batch: the down matrices of nearly all experts, a few rows each
        _mm(name="mm_decode_45", op="mm", tokens=45, top_k=8, experts=32, n=7168, k=2048,
            dtype="fp16"),
        # odd sizes all round, rows that are slices of wider ones, rows past the last expert's
        _mm(name="mm_odd_333", op="mm", tokens=333, top_k=2, experts=7, n=1000, k=1001,
            dtype="bf16", spare=37, pad=6),
        # a training micro-batch through the gate/up matrices
        _mm(name="mm_forward_4096", op="mm", tokens=4096, top_k=8, experts=32, n=4096, k=7168,
            dtype="bf16"),
        # its gradient back through the same matrices
        _mm(name="mm_input_grad_4096", op="mm", tokens=4096, top_k=8, experts=32, n=7168,
            k=4096, dtype="bf16", transposed=True),
        # a small model's step: few tokens, small matrices
        _mm(name="mm_input_grad_64", op="mm", tokens=64, top_k=4, experts=16, n=1024, k=512,
            dtype="fp16", transposed=True),
        # the weights' gradient of the micro-batch, fp32 for the optimizer
        _mm(name="weight_grad_4096", op="weight_grad", tokens=4096, top_k=8, experts=32,
            n=4096, k=7168, dtype="bf16", grad="fp32", add=False),
        # a short last micro-batch added to the gradient accumulated so far
        _mm(name="weight_grad_add_75", op="weight_grad", tokens=75, top_k=8, experts=32,
            n=7168, k=2048, dtype="bf16", grad="bf16", add=True),
        # norms, biases and a router: little data, latency counts
        {"name": "grad_norm_small", "op": "grad_norm", "count": 12, "smallest": 32,
         "largest": 7168, "dtype": "bf16", "align": 64, "inf": False},
        # every gradient of a model shard
        {"name": "grad_norm_model", "op": "grad_norm", "count": 160, "smallest": 7168,
         "largest": 58720256, "dtype": "bf16", "align": 64, "inf": False},
        # the same kind of list clipped, of several types
        {"name": "clip_model", "op": "clip", "count": 100, "smallest": 7168,
         "largest": 58720256, "dtype": "mixed", "align": 64, "inf": False, "max_norm": 1.0},
        # a small model's list, odd sizes end to end in one buffer
        {"name": "clip_small_odd", "op": "clip", "count": 37, "smallest": 1, "largest": 65537,
         "dtype": "fp32", "align": 1, "inf": False, "max_norm": 0.5},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case: sizes over their whole range (tokens from one up, odd and ragged sizes
    among them), every type, form and direction."""
    op = rng.choice(["mm", "mm", "mm", "weight_grad", "weight_grad", "grad_norm", "clip"])
    if op in ("mm", "weight_grad"):
        experts = rng.choice([1, 2, 5, 8, 16, 32, 60, 128])
        sizes = [64, 200, 256, 1000, 1024, 1408, 2048, 2816, 4096, 5120, 7168]
        n, k = rng.choice(sizes), rng.choice(sizes)
        if rng.random() < 0.2:
            n, k = rng.choice([(333, 1000), (1001, 250), (1536, 77), (515, 1027)])
        while experts * n * k > 32 * 4096 * 7168:
            experts = max(1, experts // 2)
        top_k = rng.randint(1, min(8, experts))
        most = min(65536, MAX_FLOPS // (2 * n * k), 1_500_000_000 // (n + k)) // top_k
        case = _mm(op=op, tokens=_log_uniform(rng, 1, most), top_k=top_k, experts=experts, n=n,
                   k=k, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                   spare=rng.choice([0, 0, 19]), pad=rng.choice([0, 0, 0, 8, 3]))
        if op == "mm":
            case["transposed"] = rng.random() < 0.5
        else:
            case["grad"] = rng.choice(["fp32", "fp32", case["dtype"]])
            case["add"] = rng.random() < 0.4
        return case
    largest = _log_uniform(rng, 100, 50_000_000)
    dtype = rng.choice(["bf16", "fp16", "fp32", "mixed"])
    case = {"op": op, "count": _log_uniform(rng, 1, 400 if largest < 1_000_000 else 60),
            "smallest": rng.randint(1, 100), "largest": largest, "dtype": dtype,
            "align": rng.choice([64, 64, 8, 1]), "inf": rng.random() < 0.25}
    if op == "clip":
        case["max_norm"] = rng.choice([1.0, 0.01, 1000.0])
    return case


def _kinds(case):
    """The type of each tensor of a list of gradients."""
    if case["dtype"] != "mixed":
        return [case["dtype"]] * case["count"]
    return [MIXED[i % len(MIXED)] for i in range(case["count"])]


def _sizes(case):
    """The sizes of a list of gradients, spread over their logarithm; the first is the
    largest."""
    lo, hi = case["smallest"], case["largest"]
    return [hi if i == 0 else max(1, round(lo * (hi / lo) ** (i * 0.6180339887498949 % 1)))
            for i in range(case["count"])]


def work(case):
    """Bytes that one pass has to read and write (each input and output once) and its
    floating-point operations."""
    op = case["op"]
    if op in ("grad_norm", "clip"):
        sizes, kinds = _sizes(case), _kinds(case)
        read = sum(n * SIZE[t] for n, t in zip(sizes, kinds))
        return {"bytes": read * (2 if op == "clip" else 1) + 4,
                "flops": sum(sizes) * (3 if op == "clip" else 2)}
    rows, e, n, k = case["tokens"] * case["top_k"], case["experts"], case["n"], case["k"]
    size = SIZE[case["dtype"]]
    flops = 2 * rows * n * k
    if op == "weight_grad":
        return {"bytes": rows * (n + k) * size
                + e * n * k * SIZE[case["grad"]] * (1 + case["add"]), "flops": flops}
    # experts with a row, on average over even choices
    active = e * (1.0 - (1.0 - case["top_k"] / e) ** case["tokens"])
    return {"bytes": rows * (n + k) * size + active * n * k * size, "flops": flops}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _row_counts(case, gen):
    """[experts] int64 rows per expert: top_k distinct choices of each token, popularity
    Zipf(1.1) as in the MoE workloads."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    rank = torch.arange(1, e + 1, device="cuda", dtype=torch.float32)
    gumbel = -torch.log(-torch.log(torch.rand((t, e), generator=gen, device="cuda")
                                   .clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(gumbel - 1.1 * torch.log(rank), k, dim=1).indices
    counts = torch.zeros(e, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, ids.reshape(-1), torch.ones_like(ids).reshape(-1))
    return counts[torch.randperm(e, generator=gen, device="cuda")]


def _rows(gen, rows, width, pad, dt):
    """Rows of different sizes; with pad, the first columns of wider rows."""
    x = _randn(gen, rows, width + pad).mul_(torch.exp(0.5 * _randn(gen, rows, 1)))
    return x.to(dt)[:, :width]


def _flat(case, make):
    """The gradients as views of one buffer per type, as a program keeps them: (buffers by type,
    views in the list's order)."""
    sizes, kinds = _sizes(case), _kinds(case)
    places, ends = [], {}
    for n, t in zip(sizes, kinds):
        at = -(-ends.get(t, 0) // case["align"]) * case["align"]
        places.append(at)
        ends[t] = at + n
    flat = {t: make(t, ends[t]) for t in sorted(ends)}
    return flat, [flat[t][at:at + n] for n, t, at in zip(sizes, kinds, places)]


def prepare(case, seed):
    """Inputs and output buffers on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case), "op": op}
    if op in ("grad_norm", "clip"):
        def zeros(t, n):
            return torch.zeros(n, dtype=DTYPES[t], device="cuda")
        s["flat"], s["grads"] = _flat(case, zeros)
        for g in s["grads"]:
            g.copy_(_randn(gen, *g.shape).mul_(0.01 * torch.exp(_randn(gen, 1))))
        norm = torch.zeros((), device="cuda")
        if op == "grad_norm":
            s["out"] = norm
        else:
            s["flat_out"], views = _flat(case, zeros)
            s["out"] = (norm, views)
        return s
    dt, e, n, k = DTYPES[case["dtype"]], case["experts"], case["n"], case["k"]
    s["m_sizes"] = _row_counts(case, gen)
    s["counts"] = s["m_sizes"].tolist()
    rows = case["tokens"] * case["top_k"] + case["spare"]
    s["x"] = _rows(gen, rows, k, case["pad"], dt)
    if op == "mm":
        shape = (e, k, n) if case["transposed"] else (e, n, k)
        s["w"] = _randn(gen, *shape).mul_(k ** -0.5).to(dt)
        s["out"] = torch.zeros((rows, n), dtype=dt, device="cuda")
    else:
        s["dy"] = _rows(gen, rows, n, case["pad"], dt)
        grad = DTYPES[case["grad"]]
        s["add"] = _randn(gen, e, n, k).to(grad) if case["add"] else None
        s["out"] = torch.zeros((e, n, k), dtype=grad, device="cuda")
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _plain_mm(s, case):
    """Expert by expert: a product of the rows that it has."""
    out, at = torch.zeros_like(s["out"]), 0
    for g, m in enumerate(s["counts"]):
        if m:
            w = s["w"][g].float()
            x = s["x"][at:at + m].float()
            out[at:at + m] = x @ (w if case["transposed"] else w.t())
        at += m
    return out


def _plain_weight_grad(s, case):
    out, at = torch.empty_like(s["out"]), 0
    for g, m in enumerate(s["counts"]):
        dw = s["dy"][at:at + m].float().t() @ s["x"][at:at + m].float()
        out[g] = dw if s["add"] is None else dw + s["add"][g].float()
        at += m
    return out


def _plain_norm(s, case):
    """The padding between the views is zero, so whole buffers do."""
    flat = s["flat"].values()
    if case["inf"]:
        return torch.stack([v.abs().amax().float() for v in flat]).amax()
    return torch.stack([v.float().square().sum(dtype=torch.float64) for v in flat]).sum() \
        .sqrt().float()


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "mm":
        return _plain_mm(s, case)
    if op == "weight_grad":
        return _plain_weight_grad(s, case)
    norm = _plain_norm(s, case)
    if op == "grad_norm":
        return norm
    scale = (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return {"norm": norm, "grads": {t: (v.float() * scale).to(v.dtype)
                                    for t, v in s["flat"].items()}}


# ---------------------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------------------
def _own(s):
    import fp8_rowwise_scaled_gb300 as fx
    case, op, out = s["case"], s["op"], s["out"]
    if op == "mm":
        return fx.grouped_mm(s["x"], s["w"], s["m_sizes"], transposed=case["transposed"],
                             out=out)
    if op == "weight_grad":
        return fx.grouped_mm_weight_grad(s["dy"], s["x"], s["m_sizes"], add=s["add"], out=out)
    norm_type = float("inf") if case["inf"] else 2.0
    if op == "grad_norm":
        return fx.grad_norm(s["grads"], norm_type=norm_type, out=out)
    norm, _ = fx.clip_grad_norm(s["grads"], case["max_norm"], norm_type=norm_type,
                                eps=CLIP_EPS, out=out)
    return {"norm": norm, "grads": s["flat_out"]}


def run(state):
    """One pass through the operator, and its outputs."""
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _experts_rows(s):
    """[rows] the expert of each row, -1 past the last expert's."""
    last = torch.cumsum(s["m_sizes"], 0)
    row = torch.arange(s["x"].shape[0], device="cuda")
    expert = torch.searchsorted(last, row, right=True)
    return torch.where(expert < len(last), expert, -1)


def _exact_mm(s, case):
    expert = _experts_rows(s)
    out = torch.zeros((len(expert), case["n"]), dtype=torch.float64, device="cuda")
    spec = "rk,kn->rn" if case["transposed"] else "rk,nk->rn"
    for e in torch.unique(expert[expert >= 0]):
        r = torch.nonzero(expert == e)[:, 0]
        out[r] = torch.einsum(spec, s["x"][r].double(), s["w"][e].double())
    return out


def _exact_weight_grad(s, case):
    expert = _experts_rows(s)
    if case["add"]:
        out = s["add"].double()
    else:
        out = torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64,
                          device="cuda")
    for e in torch.unique(expert[expert >= 0]):
        r = torch.nonzero(expert == e)[:, 0]
        out[e] += torch.einsum("rn,rk->nk", s["dy"][r].double(), s["x"][r].double())
    return out


def _exact_lists(s, case):
    each = torch.stack([torch.linalg.vector_norm(g.double(), float("inf") if case["inf"] else 2)
                        for g in s["grads"]])
    norm = torch.linalg.vector_norm(each, float("inf") if case["inf"] else 2)
    if case["op"] == "grad_norm":
        return norm
    factor = min(1.0, case["max_norm"] / (norm.item() + CLIP_EPS))
    return {"norm": norm, "grads": {t: v.double() * factor for t, v in s["flat"].items()}}


def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits, before the rounding
    to the type of the result."""
    s = prepare(case, seed)
    if case["op"] == "mm":
        return _exact_mm(s, case)
    return (_exact_weight_grad if case["op"] == "weight_grad" else _exact_lists)(s, case)
