"""Performance cases of the four-bit head and of the log probabilities read from its logits:
quantisation to block-scaled 4-bit floating point and back (fp4_quantize, fp4_dequantize), the
product of two such matrices (fp4_linear), and the log probabilities of given tokens with the
entropy and the most likely alternatives of each row (token_logprobs).

listed() gives the cases, draw() more of the same ranges, prepare() the inputs a serving loop has
in hand, run() one pass: through the library where `own` is true, else in a plain form of
elementary torch operations in 32 bits.  exact() restates the definitions in 64 bits.
"""
import math

import torch

own = False  # run() calls the library instead of the plain form

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = {"mx": 32, "nv": 16}  # elements that share a scale
# The second-level scale of a matrix: 1 in the mx format.  In the nv format the block scales are
# themselves 8-bit numbers, and the tensor's scale moves them into their range.
FEATURE_SCALE = {"mx": 1.0, "nv": 2.0 ** -4}
WEIGHT_SCALE = {"mx": 1.0, "nv": 2.0 ** -10}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _quantize_case(name, R, K, fmt="mx", dtype="bf16", std=1.0):
    return {"name": name, "op": "quantize", "R": R, "K": K, "format": fmt, "dtype": dtype, "std": std}


def _linear_case(name, R, V, K, fmt="mx", dtype="bf16"):
    return {"name": name, "op": "linear", "R": R, "V": V, "K": K, "format": fmt, "dtype": dtype}


def _logprob_case(name, n, V, dtype="bf16", given=1, k=5, T=1.0, trees=0, depth=0):
    """n rows of logits; trees > 0: only the rows on the accepted paths of that many trees."""
    return {"name": name, "op": "logprobs", "n": n, "V": V, "dtype": dtype, "given": given, "k": k,
            "T": T, "trees": trees, "depth": depth}


def listed():
    return [
        # the features of the next token of one request: latency
        _quantize_case("quantize one row", 1, 4096),
        # the head's weight, once when a model is loaded
        _quantize_case("quantize a head", 128256, 4096, "mx", "bf16", 0.02),
        # features of a small fp32 model, ragged rows that end inside a block
        _quantize_case("quantize ragged f32 rows", 1920, 2207, "nv", "f32"),
        # the next token of one request through the head: latency and the weight's bytes
        _linear_case("head, one row", 1, 128256, 4096, "nv"),
        # one request's draft layer: 10 expanded nodes, odd vocabulary, fp32 logits
        _linear_case("head, 10 nodes, f32 logits", 10, 32001, 4096, "mx", "f32"),
        # the draft model's projection of two concatenated feature rows, a 60-node tree
        _linear_case("layer, 60 nodes", 60, 4096, 8192, "nv"),
        # the expanded nodes of 64 draft trees through the draft head
        _linear_case("head, 640 draft nodes", 640, 128256, 4096, "mx"),
        # the target head of the 64 x 60-node verify step
        _linear_case("head, 3840 tree nodes", 3840, 128256, 4096, "nv"),
        # the next token of one request, with the five best alternatives: latency
        _logprob_case("log probabilities, one row", 1, 128256),
        # the tokens that a verify step emitted, by their rows among the 64 x 60 nodes'
        _logprob_case("log probabilities, emitted", 3840, 128256, trees=64, depth=7),
        # every node of 256 26-node trees, fp32 logits, two candidate tokens each
        _logprob_case("log probabilities, f32 nodes", 1664, 152064, "f32", 2, 20, 0.7),
        # chain drafts over a toy vocabulary: many short rows
        _logprob_case("log probabilities, V = 32", 40000, 32, "f32", 1, 1),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "linear", "linear", "logprobs", "logprobs"])
    fmt, dtype = rng.choice(["mx", "nv"]), rng.choice(["bf16", "bf16", "f32"])
    if op == "quantize":
        K = rng.choice([log(16, 8192), 32 * log(1, 256)])
        R = log(1, min(128256, max(1, 300_000_000 // K)))
        return _without_name(_quantize_case("", R, K, fmt, dtype, rng.choice([1.0, 0.02])))
    if op == "linear":
        K = rng.choice([log(32, 8192), 64 * log(1, 128), 4096])
        V = rng.choice([log(64, 152064), 32000, 128256])
        V = min(V, 500_000_000 // K)
        R = log(1, min(3840, max(1, 1_000_000_000_000 // (V * K))))
        return _without_name(_linear_case("", R, V, K, fmt, dtype))
    V = rng.choice([log(2, 152064), 32000, 128256, 152064])
    n = log(1, min(40000, max(1, 400_000_000 // V)))
    trees = rng.choice([0, 0, log(1, 64)])
    if trees and n >= 2 * trees:
        n = n // trees * trees
    else:
        trees = 0
    return _without_name(_logprob_case("", n, V, dtype, rng.choice([1, 1, 3]),
                                       min(V, rng.choice([1, 1, 5, 10, 20])),
                                       rng.choice([1.0, 1.0, 0.7]), trees, 5 if trees else 0))


def _without_name(case):
    return {k: v for k, v in case.items() if k != "name"}


def _accepted(c):
    """Accepted lengths belong to the case, not to the seed: work() counts them."""
    return [b % min(c["depth"], c["n"] // c["trees"]) for b in range(c["trees"])]


def work(case):
    c = case
    if c["op"] == "logprobs":
        es = 4 if c["dtype"] == "f32" else 2
        rows = sum(a + 1 for a in _accepted(c)) if c["trees"] else c["n"]
        return {"bytes": float(rows) * (c["V"] * es + 8 * c["given"] + 8 * c["k"] + 8),
                "flops": 5.0 * rows * c["V"]}
    packed = 0.5 + 1.0 / BLOCK[c["format"]]  # bytes of an element and of its share of a scale
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "quantize":  # values in, codes out and in again, values out
        return {"bytes": float(c["R"]) * c["K"] * (2 * es + 2 * packed), "flops": 0}
    return {"bytes": c["R"] * c["K"] * 2.0 + c["V"] * c["K"] * packed + float(c["R"]) * c["V"] * es,
            "flops": 2.0 * c["R"] * c["V"] * c["K"]}


# ---------------------------------------------------------------------------------------
# the format, in plain operations
# ---------------------------------------------------------------------------------------
def _encode(x, fmt, tensor_scale):
    """Element codes [R, K32] (sign << 3 | index into 0, 0.5, 1, 1.5, 2, 3, 4, 6; K padded with
    zeros to a multiple of 32) and the scales' bytes [R, blocks] of a matrix [R, K]."""
    R, K = x.shape
    n = BLOCK[fmt]
    x = torch.nn.functional.pad(x.float(), (0, -K % 32)).view(R, -1, n)
    top = x.abs().amax(-1)
    if fmt == "mx":  # 2 ** (floor(log2 top) - 2)
        e = (torch.frexp(top)[1] - 3).clamp(-127, 127).masked_fill(top == 0, -127)
        byte = (e + 127).to(torch.uint8)
        scale = torch.pow(2.0, e.double()).float()
    else:  # top / 6, in the tensor's scale, rounded to 4 + 3 bits
        v = top.double() / (6.0 * tensor_scale)
        step = torch.pow(2.0, (torch.frexp(v)[1] - 1).clamp(min=-6).double() - 3)
        r = (torch.round(v / step) * step).clamp(max=448.0).float()
        byte = r.to(torch.float8_e4m3fn).view(torch.uint8)
        scale = r * tensor_scale
    y = torch.where(scale[..., None] > 0, x.abs() / scale[..., None], torch.zeros_like(x))
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    half = (torch.round(y / step) * step * 2).clamp(max=12).int()  # twice the rounded value
    index = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], dtype=torch.uint8, device=x.device)
    code = index[half] | ((x < 0).to(torch.uint8) << 3)
    # blocks that only pad K to a multiple of 32 have no scale
    return code.view(R, -1), byte[:, :-(-K // n)]


def _pack(code, byte):
    """Two codes to a byte, the even element in the low half; scales in tiles of 128 rows by 4."""
    R, n = byte.shape
    tiles, groups = -(-R // 128), -(-n // 4)
    full = torch.nn.functional.pad(byte, (0, 4 * groups - n, 0, 128 * tiles - R))
    scales = full.view(tiles, 4, 32, groups, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def _decode(codes, scales, R, K, fmt, tensor_scale):
    """The fp32 values of packed codes and tiled scales."""
    n = BLOCK[fmt]
    tiles, groups = -(-R // 128), -(-(-(-K // n)) // 4)
    byte = scales.view(tiles, groups, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles * 128, groups * 4)
    byte = byte[:R, :-(-K // n)]
    if fmt == "mx":
        scale = torch.pow(2.0, byte.double() - 127).float()
    else:
        scale = byte.contiguous().view(torch.float8_e4m3fn).float() * tensor_scale
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    both = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1)
    x = torch.nn.functional.pad(both.view(R, -1)[:, :K], (0, -K % n))
    return (x.view(R, -1, n) * scale[..., None]).view(R, -1)[:, :K]


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _rows(R, V, dtype, g, std):
    """[R, V] whose rows start on 16-byte boundaries."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    x = torch.randn((R, -(-V // per) * per), generator=g, device=DEV, dtype=dtype) * std
    return x[:, :V]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"op": c["op"]}
    if c["op"] == "quantize":
        s.update(x=_rows(c["R"], c["K"], TYPES[c["dtype"]], g, c["std"]), format=c["format"],
                 scale=(FEATURE_SCALE if c["std"] == 1.0 else WEIGHT_SCALE)[c["format"]])
        return s
    if c["op"] == "linear":
        # a head's weight is kept in four bits, the features come from the model in bf16
        w = torch.randn((c["V"], c["K"]), generator=g, device=DEV, dtype=torch.bfloat16) * 0.02
        codes, scales = _pack(*_encode(w, c["format"], WEIGHT_SCALE[c["format"]]))
        s.update(x=_rows(c["R"], c["K"], torch.bfloat16, g, 1.0), codes=codes, scales=scales,
                 V=c["V"], K=c["K"], format=c["format"], out=TYPES[c["dtype"]])
        return s
    s.update(logits=_rows(c["n"], c["V"], TYPES[c["dtype"]], g, 3.0), k=c["k"], T=c["T"], rows=None)
    many = c["n"]
    if c["trees"]:  # row numbers of the accepted nodes, -1 behind a path's end
        nodes = c["n"] // c["trees"]
        width = min(c["depth"], nodes)
        path = torch.rand((c["trees"], nodes - 1), generator=g, device=DEV).argsort(1)[:, :width - 1] + 1
        path = torch.cat([torch.zeros_like(path[:, :1]) if width > 1 else
                          torch.zeros((c["trees"], 1), dtype=torch.int64, device=DEV),
                          path.sort(1)[0]], 1)
        last = torch.tensor(_accepted(c), device=DEV)[:, None]
        rows = torch.arange(c["trees"], device=DEV)[:, None] * nodes + path
        rows = torch.where(torch.arange(width, device=DEV)[None] <= last, rows, -1)
        s["rows"] = rows.reshape(-1).to(torch.int32)
        many = c["trees"] * width
    # given tokens as a sampler emits them: likely ones, by the largest of a few random candidates
    cand = torch.randint(0, c["V"], (many, c["given"], 64), generator=g, device=DEV)
    at = torch.arange(many, device=DEV) if s["rows"] is None else s["rows"].long().clamp(min=0)
    best = s["logits"][at[:, None, None], cand].float().argmax(-1, keepdim=True)
    s["tokens"] = cand.gather(-1, best)[..., 0].to(torch.int32)
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        from speculative_decoding_tree_spec_gb300 import binding
        if s["op"] == "quantize":
            q = binding.fp4_quantize(s["x"], s["format"], s["scale"])
            return binding.fp4_dequantize(q, s["x"].dtype)
        if s["op"] == "linear":
            a = binding.fp4_quantize(s["x"], s["format"], FEATURE_SCALE[s["format"]])
            w = binding.Fp4Matrix(s["codes"], s["scales"], s["V"], s["K"], s["format"],
                                  WEIGHT_SCALE[s["format"]])
            return binding.fp4_linear(a, w, s["out"])
        r = binding.token_logprobs(s["logits"], s["tokens"], s["k"], s["T"], rows=s["rows"])
        return {n: r[n] for n in ("logprobs", "entropy", "top_tokens", "top_logprobs")}
    return {"quantize": _plain_quantize, "linear": _plain_linear, "logprobs": _plain_logprobs}[s["op"]](s)


def _plain_quantize(s):
    codes, scales = _pack(*_encode(s["x"], s["format"], s["scale"]))
    R, K = s["x"].shape
    return _decode(codes, scales, R, K, s["format"], s["scale"]).to(s["x"].dtype)


def _plain_linear(s):
    fmt = s["format"]
    R, K = s["x"].shape
    codes, scales = _pack(*_encode(s["x"], fmt, FEATURE_SCALE[fmt]))
    a = _decode(codes, scales, R, K, fmt, FEATURE_SCALE[fmt])
    w = _decode(s["codes"], s["scales"], s["V"], K, fmt, WEIGHT_SCALE[fmt])
    return (a @ w.T).to(s["out"])


def _plain_logprobs(s):
    none = None
    z = s["logits"]
    if s["rows"] is not None:
        none = s["rows"] < 0
        z = z[s["rows"].long().clamp(min=0)]
    z = z.float()
    V, k = z.shape[1], s["k"]
    m = z.amax(-1, keepdim=True)
    x = (z - m) / s["T"]
    w = x.exp()
    total = w.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = (log_total - (w * x).nan_to_num(0.0).sum(-1, keepdim=True) / total)[:, 0]
    del w
    given = x.gather(1, s["tokens"].long()) - log_total
    # the largest logits, ties to the lower index: both in one 64-bit key
    bits = (z + 0.0).view(torch.int32).long() & 0xFFFFFFFF
    bits = torch.where(bits >= 1 << 31, (1 << 32) - 1 - bits, bits + (1 << 31)) - (1 << 31)
    key = bits * (1 << 31) + ((1 << 31) - 1 - torch.arange(V, device=DEV))
    index = (1 << 31) - 1 - key.topk(k, -1)[0] % (1 << 31)
    top = x.gather(1, index) - log_total
    if none is not None:  # no row: nothing is likely there
        given = given.masked_fill(none[:, None], -math.inf)
        top = top.masked_fill(none[:, None], -math.inf)
        index = index.masked_fill(none[:, None], -1)
        entropy = entropy.masked_fill(none, 0.0)
    return {"logprobs": given, "entropy": entropy, "top_tokens": index.to(torch.int32),
            "top_logprobs": top}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, some rows at a time
# ---------------------------------------------------------------------------------------
def _nearest(v, grid, even):
    """Index of the nearest of grid's ascending values; halfway, the one that `even` allows."""
    mid = (grid[1:] + grid[:-1]) / 2
    low = torch.bucketize(v, mid)  # v <= mid: the lower one
    tie = (low < len(mid)) & (v == mid[low.clamp(max=len(mid) - 1)])
    return torch.where(tie & ~even[low], low + 1, low)


def _exact_values(x, fmt, tensor_scale):
    """What quantised rows stand for: each block's elements are the nearest multiples of its scale
    by 0, 0.5, 1, 1.5, 2, 3, 4 and 6, halves to the even code."""
    R, K = x.shape
    n = BLOCK[fmt]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    even = torch.arange(8, device=x.device) % 2 == 0
    x = torch.nn.functional.pad(x.double(), (0, -K % n)).view(R, -1, n)
    top = x.abs().amax(-1)
    if fmt == "mx":
        powers = torch.pow(2.0, torch.arange(-127, 128, dtype=torch.float64, device=x.device))
        # the largest power of two at or below the block's largest element, and a quarter of it
        scale = powers[(torch.bucketize(top / 4, powers, right=True) - 1).clamp(0, 254)]
    else:
        e4m3 = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
        scale = e4m3[_nearest(top / tensor_scale / 6, e4m3, torch.arange(127, device=x.device) % 2 == 0)]
        scale = scale * tensor_scale
    some = (scale > 0)[..., None]
    i = _nearest(x.abs() / torch.where(some, scale[..., None], 1.0), grid, even)
    v = torch.where(some, grid[i] * scale[..., None], 0.0) * x.sign()
    return v.view(R, -1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    some = max(1, (1 << 25) // (case["V"] if case["op"] == "logprobs" else case["K"]))
    if s["op"] == "quantize":
        return torch.cat([_exact_values(x, s["format"], s["scale"]) for x in s["x"].split(some)])
    if s["op"] == "linear":
        if case["R"] * case["V"] * case["K"] > 3e12:  # 64-bit products take long here
            return None
        fmt, V, K = s["format"], s["V"], s["K"]
        a = _exact_values(s["x"], fmt, FEATURE_SCALE[fmt])
        w = _decode(s["codes"], s["scales"], V, K, fmt, WEIGHT_SCALE[fmt])  # exact in 32 bits
        return torch.cat([a @ part.double().T for part in w.split(some)], 1)
    out = {"logprobs": [], "entropy": [], "top_logprobs": []}
    rows = torch.arange(case["n"], device=DEV) if s["rows"] is None else s["rows"].long()
    for r, t in zip(rows.split(some), s["tokens"].long().split(some)):
        logp = torch.log_softmax(s["logits"][r.clamp(min=0)].double() / s["T"], -1)
        gone = (r < 0)[:, None]
        out["logprobs"].append(logp.gather(1, t).masked_fill(gone, -math.inf))
        out["entropy"].append(-(logp.exp() * logp).sum(-1).masked_fill(gone[:, 0], 0.0))
        out["top_logprobs"].append(logp.sort(-1, descending=True)[0][:, :s["k"]].masked_fill(gone, -math.inf)
                                   if case["n"] * case["V"] < 1 << 22 else
                                   logp.topk(s["k"], -1)[0].masked_fill(gone, -math.inf))
    return {**{n: torch.cat(v) for n, v in out.items()}, "top_tokens": None}
