"""The 8-bit integer products and the quantisers that feed them as measured work:
plain forms in elementary torch operations, and (``own``) the library's calls a
user's program makes.

Operators: rows_quant (rows to 8-bit codes and a scale each: weights by channel,
activations by token), norm_quant (the residual's addition, RMSNorm, codes and
scales), silu_quant (silu(gate) * up, codes and scales), i8_matmul (the product of
two such matrices). Codes are returned as the values they stand for.
"""
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4.0, "f16": 2.0, "bf16": 2.0, "q8_0": 34 / 32}
GGUF = {"f32": 0, "f16": 1, "bf16": 30, "q8_0": 8}
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # four beams' attention outputs on the 135M heads before their output projection: latency
        dict(name="rows_step_135m", op="rows", type="f32", rows=4, k=576),
        # the 7B gate and up matrices of a Q8_0 file turned into channel-scaled codes when a model is loaded
        dict(name="rows_weights_7b", op="rows", type="q8_0", rows=28672, k=4096),
        # one token of the 135M model
        dict(name="norm_step_135m", op="norm", type="f32", rows=1, k=576, delta=True),
        # prompts of several sequences together through a 7B layer
        dict(name="norm_prompts_7b", op="norm", type="f32", rows=8195, k=4096, delta=True),
        # an odd width in 16 bits, first layer (nothing to add yet)
        dict(name="norm_odd", op="norm", type="bf16", rows=333, k=1001, delta=False),
        # eight sequences' MLP on the 135M model
        dict(name="silu_step_135m", op="silu", type="f32", rows=8, k=1536),
        # a long prompt's MLP on the 7B model, activations in 16 bits
        dict(name="silu_prompt_7b", op="silu", type="bf16", rows=2048, k=14336),
        # one token through the 135M Q/K/V projections: latency
        dict(name="matmul_step_135m", op="matmul", type="f32", m=1, n=960, k=576),
        # one token through the 7B gate and up matrices: the weights' bytes
        dict(name="matmul_step_7b", op="matmul", type="f32", m=1, n=28672, k=4096),
        # a served batch through the 7B down projection
        dict(name="matmul_batch_7b", op="matmul", type="f32", m=48, n=4096, k=14336),
        # the 512-token prompt through the 7B gate and up matrices
        dict(name="matmul_prompt_7b", op="matmul", type="f32", m=512, n=28672, k=4096),
        # a full context through the 7B down projection, 16-bit outputs
        dict(name="matmul_context_7b", op="matmul", type="bf16", m=4096, n=4096, k=14336),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["rows", "norm", "silu", "matmul", "matmul", "matmul"])
    cost = "flops" if op == "matmul" else "bytes"
    most = max(work(c)[cost] for c in listed() if c["op"] == op)
    while True:
        kind = rng.choice(sorted(TYPES))
        if op == "matmul":
            c = dict(op=op, type=kind, m=_log(rng, 1, 4096), n=_log(rng, 1, 49152), k=_log(rng, 1, 14336))
            if rng.random() < 0.5:  # the sizes of most models
                c["n"], c["k"] = -(-c["n"] // 64) * 64, -(-c["k"] // 64) * 64
        else:
            c = dict(op=op, type=kind, rows=_log(rng, 1, 28672), k=_log(rng, 1, 14336))
            if rng.random() < 0.5:
                c["k"] = -(-c["k"] // 64) * 64
            if op == "rows" and rng.random() < 0.3:
                c["type"], c["k"] = "q8_0", -(-c["k"] // 32) * 32
            if op == "norm":
                c["delta"] = rng.random() < 0.7
        if work(c)[cost] <= most:
            return c


def _row_bytes(k):
    return -(-k // 16) * 16


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k + m * k + 4 * (m + n) + m * n * SIZES[case["type"]], "flops": 2 * m * n * k}
    size, cells = SIZES[case["type"]], case["rows"] * case["k"]
    arrays = {"rows": 1, "norm": 3 if case.get("delta") else 1, "silu": 2}[case["op"]]
    return {"bytes": cells * (arrays * size + 4) + 4 * case["rows"] + (4 * case["k"] if case["op"] == "norm" else 0),
            "flops": cells * {"rows": 3, "norm": 7, "silu": 10}[case["op"]]}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _hidden(g, rows, k, scale=1.0):
    """Hidden states: normal, with the few channels that are much larger in every row."""
    x = _normal(g, rows, k) * scale
    x[:, torch.randint(0, k, (max(1, k // 500),), generator=g, device="cuda")] *= 8.0
    return x


def _coded(x):
    """Codes of the rows of x, in rows of a multiple of 16 bytes, and their scales: what the quantiser left."""
    d = (x.abs().amax(1) / 127.0).clamp(min=1e-30)
    codes = torch.zeros((x.shape[0], _row_bytes(x.shape[1])), dtype=torch.int8, device="cuda")
    codes[:, :x.shape[1]] = torch.round(x / d[:, None]).clamp(-127, 127).to(torch.int8)
    return codes, d


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "matmul":
        st["a"], st["sa"] = _coded(_hidden(g, case["m"], case["k"]))
        st["w"], st["sw"] = _coded(_normal(g, case["n"], case["k"]) * 0.02)
        st["y"] = torch.empty((case["m"], case["n"]), dtype=TYPES[case["type"]], device="cuda")
    else:
        rows, k = case["rows"], case["k"]
        st["codes"] = torch.zeros((rows, _row_bytes(k)), dtype=torch.int8, device="cuda")
        st["scale"] = torch.zeros(rows, device="cuda")
        if case["type"] == "q8_0":
            # blocks of 32: an fp16 scale and 32 codes
            blocks = torch.empty((rows, k // 32, 34), dtype=torch.int8, device="cuda")
            blocks[..., 2:] = torch.randint(-127, 128, (rows, k // 32, 32), generator=g, device="cuda", dtype=torch.int8)
            d = (0.0003 + 0.0002 * torch.rand((rows, k // 32, 1), generator=g, device="cuda")).half()
            blocks[..., :2] = d.view(torch.int8)
            st["x"] = blocks.view(torch.uint8).reshape(rows, k // 32 * 34)
        elif case["op"] == "silu":
            st["both"] = (_hidden(g, rows, 2 * k) * 1.5).to(TYPES[case["type"]])  # gate | up
        else:
            st["x"] = _hidden(g, rows, k, 2.0).to(TYPES[case["type"]])
        if case["op"] == "norm":
            st["g"] = 1.0 + 0.1 * _normal(g, k)
            st["delta"] = (_normal(g, rows, k) * 0.5).to(TYPES[case["type"]]) if case["delta"] else None
            st["h"] = torch.empty_like(st["x"]) if case["delta"] else None
    if own and case["op"] == "matmul":
        _keep(st)
    return st


# ------------------------------------------------------------------ the library's calls

def _keep(st):
    """What a program that uses the library keeps: the weights in its layout, a workspace."""
    from q8_quantized_llama_gb300 import binding as B
    m, n, k = (st["case"][x] for x in "mnk")
    st["packed"] = torch.empty(B.llama_q8_i8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
    B.llama_q8_i8_pack(st["w"], st["sw"], n, k, st["packed"])
    st["ws_bytes"] = B.llama_q8_i8_matmul_workspace_bytes(n, k, m)
    st["ws"] = torch.zeros(max(16, st["ws_bytes"]), dtype=torch.uint8, device="cuda")
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _run_own(st):
    from q8_quantized_llama_gb300 import binding as B
    case = st["case"]
    kind = GGUF[case["type"]]
    if case["op"] == "matmul":
        B.llama_q8_i8_matmul(st["packed"], case["n"], case["k"], st["a"], st["sa"], case["m"], kind, st["y"],
                             case["n"], st["ws"], st["ws_bytes"], st["err"])
        return {"y": st["y"]}
    rows, k, codes, scale = case["rows"], case["k"], st["codes"], st["scale"]
    if case["op"] == "rows":
        B.llama_q8_rows_quant(kind, st["x"], k, rows, k, codes, scale)
    elif case["op"] == "norm":
        B.llama_q8_norm_quant(kind, st["x"], k, st["delta"], k, st["h"], k, st["g"], EPS, rows, k, codes, scale)
    else:
        B.llama_q8_silu_quant(kind, st["both"], st["both"][:, k:], 2 * k, rows, k, codes, scale)
    out = {"values": codes[:, :k] * scale[:, None], "scale": scale}
    if case["op"] == "norm" and case["delta"]:
        out["x"] = st["h"]
    return out


# ------------------------------------------------------------------ the plain forms

def run(st):
    if own:
        return _run_own(st)
    return {"rows": _rows, "norm": _norm, "silu": _silu, "matmul": _matmul}[st["case"]["op"]](st)


def _levels(v, factor):
    """Codes and scales of the rows of v: a code lies next to a border between two, so v is in 64 bits."""
    top = v.abs().amax(1, keepdim=True)
    a = 127.0 * v.abs() / torch.where(top == 0, 1.0, top)
    q = torch.floor(a)
    q = torch.where(a - q >= 0.5, q + 1.0, q) * torch.sign(v)
    scale = (top * factor / 127.0).float()
    return {"values": q.float() * scale, "scale": scale[:, 0]}


def _rows(st):
    case = st["case"]
    if case["type"] != "q8_0":
        return _levels(st["x"].double(), 1.0)
    blocks = st["x"].view(case["rows"], -1, 34)
    d, q = blocks[..., :2].contiguous().view(torch.float16), blocks[..., 2:].view(torch.int8)
    return _levels((d.double() * q.double()).view(case["rows"], -1), 1.0)


def _norm(st):
    h = st["x"]
    if st["delta"] is not None:
        h = (h.float() + st["delta"].float()).to(h.dtype)
    x = h.double()
    out = _levels(x * st["g"].double(), 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS))
    return out | ({"x": h} if st["delta"] is not None else {})


def _silu(st):
    k = st["case"]["k"]
    gate, up = st["both"][:, :k].double(), st["both"][:, k:].double()
    return _levels(gate / (1.0 + torch.exp(-gate)) * up, 1.0)


def _matmul(st):
    k = st["case"]["k"]
    y = st["a"][:, :k].float() @ st["w"][:, :k].float().T
    return {"y": (y * st["sa"][:, None] * st["sw"][None, :]).to(st["y"].dtype)}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rows": _exact_rows, "norm": _exact_norm, "silu": _exact_silu, "matmul": _exact_matmul}[case["op"]](case, st)


def _nearest(v):
    """The multiple of a 127th of each row's largest magnitude that is nearest to v, ties away from zero."""
    unit = torch.linalg.vector_norm(v, float("inf"), dim=1, keepdim=True)
    twice = 2.0 * unit
    steps = torch.div(254.0 * v.abs() + unit, torch.where(unit == 0, 1.0, twice), rounding_mode="floor")
    return torch.copysign(steps, v) * (unit / 127.0), unit[:, 0] / 127.0


def _exact_rows(case, st):
    if case["type"] == "q8_0":
        raw = st["x"].view(case["rows"], case["k"] // 32, 34)
        scale = (raw[..., 0].to(torch.int32) + 256 * raw[..., 1].to(torch.int32)).to(torch.int16).view(torch.float16)
        x = (raw[..., 2:].view(torch.int8) * scale.double()[..., None]).reshape(case["rows"], case["k"])
    else:
        x = st["x"].to(torch.float64)
    values, scale = _nearest(x)
    return {"values": values, "scale": scale}


def _exact_norm(case, st):
    h = st["x"]
    if case["delta"]:
        # the stored sum: added in f32, kept in the type
        h = torch.add(h.double(), st["delta"].double()).to(torch.float32).to(h.dtype)
    values, scale = _nearest(torch.mul(h.double(), st["g"].double()))
    rms = torch.linalg.vector_norm(h.double(), dim=1).square().div(case["k"]).add(EPS).rsqrt()
    out = {"values": values * rms[:, None], "scale": scale * rms}
    return out | ({"x": h.double()} if case["delta"] else {})


def _exact_silu(case, st):
    gate, up = st["both"].double().split(case["k"], dim=1)
    values, scale = _nearest(gate * torch.sigmoid(gate) * up)
    return {"values": values, "scale": scale}


def _exact_matmul(case, st):
    # the scales first, row by row and channel by channel, then the products in 64 bits
    a = st["a"][:, :case["k"]].double().mul_(st["sa"].double()[:, None])
    w = st["w"][:, :case["k"]].double().mul_(st["sw"].double()[:, None])
    return {"y": torch.einsum("mk,nk->mn", a, w)}


if __name__ == "__main__":
    rng = random.Random(0)
    for c in listed() + [draw(rng) for _ in range(4)]:
        print(c, work(c))
