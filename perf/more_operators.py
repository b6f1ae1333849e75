"""Operators for drafted tokens and for experts: the cases they are measured on, and their plain forms.

What a transformer layer served in MX formats needs beside the operators of operators.py and the grouped product:

* append    the position rotation of queries and keys, and keys and values into the paged MX cache, in one call;
* tree      attention over that cache for a tree of drafted tokens per sequence, each seeing its ancestors;
* dispatch  tokens sorted by expert into the grouped product's A operand (E4M3 codes and E8M0 scales, or BF16);
* combine   the experts' rows back to their tokens, with the router's weights, and the gradients of that.

`own` False computes them in elementary torch operations, True with the library's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32                      # values that share one E8M0 scale
EMAX = {"fp8": 8, "fp4": 2}     # exponent of the largest E4M3 / E2M1 value
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step: a token of each of 64 sequences, into small pages
        dict(op="append", name="append_step", tokens=64, step=True, q_heads=32, heads=8, dim=128, rot=128, inter=False,
             page=16, pages=4096, fmt="fp8"),
        # a prompt's queries, keys and values, into larger pages
        dict(op="append", name="append_prompt", tokens=8191, step=False, q_heads=32, heads=8, dim=128, rot=128, inter=False,
             page=64, pages=1024, fmt="fp8"),
        # half of each 64-wide head rotated, in adjacent pairs, into the 4-bit cache, and the chunk read back
        dict(op="append", name="append_part_fp4", tokens=1000, step=False, q_heads=20, heads=4, dim=64, rot=32, inter=True,
             page=32, pages=512, fmt="fp4"),
        # one sequence, a small tree of drafted tokens, a short context: latency
        dict(op="tree", name="tree_one", seqs=1, nodes=27, nodes_lo=27, branch=3, kv=1051, kv_lo=1051, q_heads=32, heads=8,
             dim=128, page=16, fmt="fp8", window=0),
        # a batch of sequences of ragged lengths, trees of the same budget
        dict(op="tree", name="tree_batch", seqs=32, nodes=16, nodes_lo=16, branch=2, kv=16000, kv_lo=100, q_heads=32, heads=8,
             dim=128, page=64, fmt="fp8", window=0),
        # long contexts in the 4-bit cache, with the wider head group of a large model
        dict(op="tree", name="tree_long_fp4", seqs=2, nodes=61, nodes_lo=40, branch=4, kv=131072, kv_lo=60000, q_heads=64,
             heads=8, dim=128, page=256, fmt="fp4", window=0),
        # large trees of many sizes, a sliding window, 64-wide heads
        dict(op="tree", name="tree_wide", seqs=24, nodes=200, nodes_lo=1, branch=2, kv=5000, kv_lo=700, q_heads=16, heads=4,
             dim=64, page=16, fmt="fp8", window=1024),
        # a decode step's tokens to the experts of a fine-grained layer: latency
        dict(op="dispatch", name="dispatch_step", tokens=64, k=8, experts=128, first=0, held=128, K=2048, out="fp8"),
        # a prompt to the experts that this worker holds, half of them
        dict(op="dispatch", name="dispatch_prompt", tokens=8191, k=4, experts=64, first=16, held=32, K=4096, out="fp8"),
        # the decode step's rows back
        dict(op="combine", name="combine_step", tokens=64, k=8, experts=128, first=0, held=128, K=2048, grad=False, weights=True),
        # a prompt's rows back
        dict(op="combine", name="combine_prompt", tokens=8191, k=4, experts=64, first=0, held=64, K=4096, grad=False, weights=True),
        # the backward pass of a training step
        dict(op="combine", name="combine_grad", tokens=4095, k=2, experts=8, first=0, held=8, K=4096, grad=True, weights=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "dispatch", "dispatch", "combine", "combine"])
    heads = rng.choice([1, 2, 4, 8])
    if op == "append":
        dim, page = rng.choice([64, 96, 128]), rng.choice([16, 32, 64, 128, 256])
        tokens = _log(rng, 1, 8192)
        step = tokens <= 128 and rng.random() < 0.5
        return dict(op=op, tokens=tokens, step=step, q_heads=heads * rng.choice([1, 2, 4, 5, 7]), heads=heads, dim=dim,
                    rot=rng.choice([dim, dim, dim, dim // 2]), inter=rng.random() < 0.3, page=page,
                    pages=(tokens if step else -(-tokens // page)) + rng.randint(1, 500), fmt=rng.choice(["fp8", "fp8", "fp4"]))
    if op == "tree":
        d = dict(op=op, branch=rng.choice([1, 2, 3, 4, 8]), q_heads=heads * rng.choice([1, 2, 4, 5, 7, 8]), heads=heads,
                 dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]), fmt=rng.choice(["fp8", "fp8", "fp4"]),
                 window=rng.choice([0, 0, 0, 512, 1000]))
        kind = rng.choice(["one", "batch", "wide"])
        if kind == "one":
            nodes = _log(rng, 1, 256)
            kv = nodes + _log(rng, 16, 100000)
            return dict(d, seqs=1, nodes=nodes, nodes_lo=nodes, kv=kv, kv_lo=kv)
        nodes = _log(rng, 2, 64) if kind == "batch" else rng.randint(65, 256)
        lo = nodes + _log(rng, 16, 2000)
        return dict(d, seqs=_log(rng, 2, 40 if kind == "batch" else 12), nodes=nodes, nodes_lo=rng.choice([nodes, 1 + nodes // 3]),
                    kv=_log(rng, lo + 1, 8000), kv_lo=lo)
    experts = rng.choice([8, 16, 60, 64, 128, 256])
    k = rng.choice([1, 2, 2, 4, 6, 8])
    held = rng.choice([experts, experts, experts // 4])
    grad = op == "combine" and rng.random() < 0.5
    d = dict(op=op, tokens=_log(rng, 1, min(8192, (16384 if grad else 32768) // k)), k=k, experts=experts,
             first=rng.randint(0, experts - held), held=held, K=BLOCK * rng.randint(16, 128))
    if op == "dispatch":
        return dict(d, out=rng.choice(["fp8", "fp8", "bf16"]))
    return dict(d, grad=grad, weights=grad or rng.random() < 0.7)


def _spread(lo, hi, n, turn):
    """n lengths between lo and hi, spread over their logarithm in no order; the first is hi."""
    return [int(round(hi * (lo / hi) ** ((i * 0.6180339887 * turn) % 1.0))) for i in range(n)]


def _lens(case):
    """(drafted tokens, keys) of each sequence: by the case alone."""
    kv = _spread(case["kv_lo"], case["kv"], case["seqs"], 1)
    return [min(n, k) for n, k in zip(_spread(case["nodes_lo"], case["nodes"], case["seqs"], 3), kv)], kv


def _ancestors(n, branch):
    """bool [n][n]: the nodes that each node sees, itself and its ancestors: node i > 0 is a child of (i - 1) // branch,
    so that the first nodes of a tree are a smaller one."""
    sees = torch.eye(n, dtype=torch.bool)
    for i in range(1, n):
        sees[i] |= sees[(i - 1) // branch]
    return sees


def _kept(case):
    """Assignments that go to the experts held here, on average."""
    return case["tokens"] * case["k"] * case["held"] / case["experts"]


def work(case):
    """Bytes that have to be read and written once, and operations, of one pass."""
    T = case.get("tokens")
    if case["op"] == "append":
        size = {"fp8": 1, "fp4": 0.5}[case["fmt"]] + 1 / BLOCK
        kv = 2 * case["heads"] * case["dim"]
        back = kv * (size + 2) + 8 if case["fmt"] == "fp4" else 0
        return {"bytes": T * (4 * case["q_heads"] * case["dim"] + kv * (2 + size) + 16 + 4 * case["rot"] + back),
                "flops": 3 * T * (case["q_heads"] + case["heads"]) * case["rot"]}
    if case["op"] == "tree":
        size = {"fp8": 1, "fp4": 0.5}[case["fmt"]] + 1 / BLOCK
        new, kv = _lens(case)
        sees = _ancestors(max(new), case["branch"]).sum(1)
        w = case["window"] or (1 << 40)
        # node i at depth sees[i] - 1 behind its context: that much of the window lies among the nodes
        pairs = sum(int((torch.clamp(w - sees[:n], max=k - n).clamp(min=0) + sees[:n]).sum()) for n, k in zip(new, kv))
        keys = sum(n + min(k - n, w - 1) for n, k in zip(new, kv))
        d = case["dim"]
        return {"bytes": keys * 2 * case["heads"] * d * size + sum(new) * (case["q_heads"] * (4 * d + 4) + 8 * -(-max(new) // 64)),
                "flops": 4 * pairs * case["q_heads"] * d}
    rows, K = _kept(case), case["K"]
    if case["op"] == "dispatch":
        out = 2 if case["out"] == "bf16" else 1 + 1 / BLOCK
        return {"bytes": T * K * 2 + rows * K * out + T * case["k"] * 12 + 4 * case["held"], "flops": 0}
    if case["grad"]:
        return {"bytes": T * K * 2 + rows * K * 4 + T * case["k"] * 12, "flops": 3 * rows * K}
    return {"bytes": T * K * 2 + rows * K * 2 + T * case["k"] * (8 if case["weights"] else 4), "flops": 2 * rows * K}


# ------------------------------------------------------------ the inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cache_of(g, case, pages):
    """Codes and scales of a cache that holds quantized N(0, 1) keys and values, heads of unequal size."""
    shape = (pages, case["heads"], case["page"], case["dim"])
    parts = []
    for _ in "kv":
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        x *= torch.exp2(torch.randint(-2, 3, (1, case["heads"], 1, 1), generator=g, device="cuda")).bfloat16()
        codes, scales = zip(*(_quantize(part, case["fmt"]) for part in x.split(max(1, (1 << 27) // x[0].numel()))))
        parts += [torch.cat(codes), torch.cat(scales)]
    return parts


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    {"append": _prepare_append, "tree": _prepare_tree, "dispatch": _prepare_experts, "combine": _prepare_experts}[case["op"]](g, case, s)
    if own and "parts" in s:     # the handle that a program keeps with its cache
        import block_scaled_precision_mm_amd as mx
        s["cache"] = mx.KVCache(*s["parts"], fmt=case["fmt"])
    return s


def _prepare_append(g, case, s):
    T, H, K, D, page = case["tokens"], case["q_heads"], case["heads"], case["dim"], case["page"]
    # queries, keys and values are parts of the rows that the QKV product wrote
    qkv = _normal(g, T, (H + 2 * K) * D).bfloat16()
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split((H * D, K * D, K * D), dim=1))
    s["q_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    s["parts"] = _cache_of(g, case, case["pages"])
    order = torch.randperm(case["pages"], generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    if case["step"]:    # a decode step: each token goes to a page of its own, at its sequence's position
        s["positions"] = torch.randint(0, 32768, (T,), generator=g, device="cuda")
        s["slots"] = order[:T] * page + s["positions"] % page
    else:               # consecutive tokens of a sequence, behind a context of some pages, in pages that lie anywhere
        s["positions"] = t + page * int(torch.randint(0, 16384 // page, (1,), generator=g, device="cuda"))
        s["slots"] = order[t // page] * page + t % page
    # cosines and sines by position, which a program keeps: [positions][rot / 2][2]
    angle = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / -case["rot"])
    s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float()
    s["back"] = [torch.empty((T, K, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"] if case["fmt"] == "fp4" else None


def _prepare_tree(g, case, s):
    new, kv = _lens(case)
    per = [-(-k // case["page"]) for k in kv]
    pages = sum(per) + 3
    s["parts"] = _cache_of(g, case, pages)
    table = torch.full((case["seqs"], max(per)), -1, dtype=torch.int32, device="cuda")
    filled = torch.arange(max(per), device="cuda")[None, :] < torch.tensor(per, device="cuda")[:, None]
    table[filled] = torch.randperm(pages, generator=g, device="cuda")[:sum(per)].int()
    s["table"] = table
    s["ends"] = torch.tensor(new, device="cuda").cumsum(0).int()
    s["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["max_new"] = max(new)
    # the nodes that a node sees, 64 to a word; a program keeps the words of its draft trees
    words = -(-max(new) // 64)
    sees = torch.nn.functional.pad(_ancestors(max(new), case["branch"]), (0, 64 * words - max(new))).view(-1, words, 64)
    bits = (sees.long() << torch.arange(64)).sum(-1)
    s["mask"] = torch.cat([bits[:n] for n in new]).cuda()
    T, H, D = sum(new), case["q_heads"], case["dim"]
    # queries are the first part of the rows that the QKV product wrote
    s["q"] = _normal(g, T, (H + 2 * case["heads"]) * D).bfloat16()[:, :H * D].view(T, H, D)
    s["out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")


def _prepare_experts(g, case, s):
    T, k, E, K = case["tokens"], case["k"], case["experts"], case["K"]
    # some experts are chosen more often than others
    logits = _normal(g, T, E) + 0.5 * _normal(g, E)
    chosen = logits.topk(k, dim=1)
    s["ids"] = chosen.indices - case["first"]       # those outside [0, held) are another worker's
    s["w"] = chosen.values.softmax(1) if case.get("weights", True) else None
    if case["op"] == "dispatch":
        s["x"] = _normal(g, T, K).bfloat16()
        # rows past the last expert's are not written
        s["y"] = torch.zeros((T * k, K), dtype=torch.uint8 if case["out"] == "fp8" else torch.bfloat16, device="cuda")
        s["ys"] = torch.zeros((T * k, K // BLOCK), dtype=torch.uint8, device="cuda") if case["out"] == "fp8" else None
        s["offs"] = torch.empty(case["held"], dtype=torch.int32, device="cuda")
        s["pos"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        return
    s["pos"] = _sorted(s["ids"], case["held"])[1].int()
    s["y"] = _normal(g, T * k, K).bfloat16()
    if case["grad"]:
        s["d_out"] = _normal(g, T, K).bfloat16()
        s["d_y"] = torch.zeros((T * k, K), dtype=torch.bfloat16, device="cuda")
        s["d_w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")


# ------------------------------------------------------------ one pass
def run(s):
    if own:
        return {"append": _append_own, "tree": _tree_own, "dispatch": _dispatch_own, "combine": _combine_own}[s["op"]](s)
    return {"append": _append, "tree": _tree, "dispatch": _dispatch, "combine": _combine}[s["op"]](s)


def _append_own(s):
    import block_scaled_precision_mm_amd as mx
    mx.mx_rope_cache_write(s["cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["q_out"],
                           interleaved=s["inter"])
    if s["back"] is not None:
        mx.mx_kv_cache_read(s["cache"], *s["back"], s["slots"])
    return _append_out(s, s["q_out"], s["back"])


def _tree_own(s):
    import block_scaled_precision_mm_amd as mx
    mx.mx_tree_attention(s["cache"], s["q"], s["ends"], s["lens"], s["table"], s["mask"], s["out"], lse=s["lse"],
                         window=s["window"], max_new=s["max_new"])
    return {"out": s["out"], "lse": s["lse"]}


def _dispatch_own(s):
    import block_scaled_precision_mm_amd as mx
    mx.mx_moe_dispatch(s["x"], s["ids"], s["y"], s["ys"], s["offs"], s["pos"])
    return _dispatch_out(s, s["y"], s["ys"], s["offs"], s["pos"])


def _combine_own(s):
    import block_scaled_precision_mm_amd as mx
    if s["grad"]:
        mx.mx_moe_combine_grad(s["d_out"], s["y"], s["pos"], s["w"], s["d_y"], None, s["d_w"])
        return {"d_y": s["d_y"], "d_w": s["d_w"]}
    mx.mx_moe_combine(s["y"], s["pos"], s["w"], s["out"])
    return {"out": s["out"]}


# ------------------------------------------------------------ plain forms
def _quantize(x, fmt):
    """MX blocks of BF16 values along the last axis: codes (E4M3, or E2M1 pairs in bytes) and E8M0 scales, as uint8."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1)
    bad = ~torch.isfinite(a)
    e = torch.frexp(torch.where(bad, 0.0, a)).exponent - 1
    s = torch.where(a == 0, 0, (e - EMAX[fmt] + 127).clamp(0, 254))
    v = torch.ldexp(b, (127 - s).unsqueeze(-1))
    if fmt == "fp8":
        codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        m = v.abs().clamp(max=6.0)
        # steps of 1/2 below 2, of 1 below 4, of 2 above; halves go to the even code
        code = torch.where(m < 2, (2 * m).round(), torch.where(m < 4, m.round() + 2, (m / 2).round() + 4))
        code = code.to(torch.uint8) + torch.signbit(v).to(torch.uint8) * 8
        codes = code[..., 0::2] + 16 * code[..., 1::2]
    codes = torch.where(bad.unsqueeze(-1), 0, codes).to(torch.uint8).flatten(-2)
    return codes, torch.where(bad, 255, s).to(torch.uint8)


def _values(codes, scales, fmt):
    """What codes and scales stand for, in 32 bits."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(FP4_VALUES + tuple(-f for f in FP4_VALUES), device=codes.device)
        v = table[torch.stack((codes & 15, codes >> 4), -1).int()].flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * scales.view(torch.float8_e8m0fnu).float().unsqueeze(-1)).flatten(-2)


def _rotated(s, x):
    """The first `rot` values of every head turned in pairs, (i, i + rot / 2) or (2 i, 2 i + 1).  A product of a BF16 and
    an FP32 value is exact in 64 bits, so that no value next to a border of BF16, and so of a block's code, depends on how
    the two products are rounded."""
    cos, sin = s["rope"][s["positions"]].double()[:, None].unbind(-1)
    r = s["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["inter"] else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a.double(), b.double()
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if s["inter"] else torch.cat((a, b), -1)
    return torch.cat((y.float().bfloat16(), x[..., r:]), -1)


def _append(s):
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    for x, codes, scales in ((_rotated(s, s["k"]), *s["parts"][:2]), (s["v"], *s["parts"][2:])):
        c, e = _quantize(x, s["fmt"])
        codes[page, :, at] = c
        scales[page, :, at] = e
    kc, ks, vc, vs = s["parts"]
    back = [_values(c[page, :, at], e[page, :, at], s["fmt"]).bfloat16() for c, e in ((kc, ks), (vc, vs))] if s["back"] else None
    return _append_out(s, _rotated(s, s["q"]), back)


def _append_out(s, q, back):
    """What a pass gives: the queries, and the tokens as the 4-bit cache holds them or the 8-bit cache that it wrote into."""
    if back is not None:
        return {"q": q, "k": back[0], "v": back[1]}
    kc, ks, vc, vs = s["parts"]
    return {"q": q, "k": kc.view(torch.float8_e4m3fn), "ks": ks.view(torch.float8_e8m0fnu),
            "v": vc.view(torch.float8_e4m3fn), "vs": vs.view(torch.float8_e8m0fnu)}


def _tree(s):
    """Every sequence padded to the longest: drafted tokens to N, keys to L."""
    S, H, G, D = s["seqs"], s["heads"], s["q_heads"] // s["heads"], s["dim"]
    ends, lens = s["ends"].long(), s["lens"].long()
    new = torch.diff(ends, prepend=ends.new_zeros(1))
    N, L = s["max_new"], s["table"].shape[1] * s["page"]
    i, p = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    mine = i < new[:, None]
    rows = torch.where(mine, (ends - new)[:, None] + i, 0)           # [S, N]: the row of a node
    q = s["q"][rows].float().view(S, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * N, D)
    # [S, N, nodes]: the nodes that a node sees; of the context, all or what its window leaves
    sees = (s["mask"][rows][..., None] >> torch.arange(64, device="cuda") & 1).flatten(-2).bool()
    node = p - (lens - new)[:, None]                                 # [S, L]: the node of a key, or < 0
    first = torch.zeros_like(rows)
    if s["window"]:
        nodes = sees & (torch.arange(sees.shape[-1], device="cuda") < new[:, None, None])
        first = (lens - new)[:, None] + (nodes.sum(-1) - 1).clamp(min=0) - s["window"] + 1
    at = node.clamp(0, sees.shape[-1] - 1)[:, None].expand(S, N, L)
    sees = torch.where((node < 0)[:, None], p >= first[..., None], torch.gather(sees, 2, at) & (node < new[:, None])[:, None])
    sees &= mine[..., None]                                          # [S, N, L]
    table = s["table"].long()
    held = (table >= 0).repeat_interleave(s["page"], 1) & (p < lens[:, None])   # [S, L]
    table = table.clamp(min=0)
    kc, ks, vc, vs = s["parts"]
    pages = lambda t: t[table].transpose(1, 2).flatten(2, 3)         # [S, H, L, ..]  # noqa: E731
    k = _values(pages(kc), pages(ks), s["fmt"]).transpose(2, 3).contiguous()
    x = (torch.matmul(q, k) / math.sqrt(D)).view(S, H, G, N, L)
    del k
    x = x.masked_fill_(~(sees & held[:, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)  # noqa: E741
    v = torch.where(held[:, None, :, None], _values(pages(vc), pages(vs), s["fmt"]), 0.0)
    o = torch.matmul(x.view(S, H, G * N, L), v).view(S, H, G, N, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 3, 1, 2, 4)
    lse = (m + l.log())[..., 0].permute(0, 3, 1, 2)
    return {"out": o[mine].reshape(-1, H * G, D).bfloat16(), "lse": lse[mine].reshape(-1, H * G)}


def _sorted(ids, held):
    """(ends of the experts' rows, row of each assignment or -1): by expert, then in the order of tokens and choices."""
    e = ids.flatten()
    e = torch.where((e >= 0) & (e < held), e, held)
    order = torch.argsort(e, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(len(order), device=order.device)
    ends = torch.zeros(held + 1, dtype=torch.int64, device=e.device).index_add_(0, e, torch.ones_like(e)).cumsum(0)
    return ends[:held].int(), torch.where(e < held, pos, -1).view(ids.shape)


def _dispatch(s):
    offs, pos = _sorted(s["ids"], s["held"])
    here = pos >= 0
    rows, token = pos[here], torch.nonzero(here)[:, 0]
    y, ys = _quantize(s["x"], "fp8") if s["out"] == "fp8" else (s["x"], None)
    s["y"][rows] = y[token]
    if ys is not None:
        s["ys"][rows] = ys[token]
    return _dispatch_out(s, s["y"], s["ys"], offs, pos.int())


def _dispatch_out(s, y, ys, offs, pos):
    if ys is None:
        return {"y": y, "offs": offs, "pos": pos}
    return {"codes": y.view(torch.float8_e4m3fn), "scales": ys.view(torch.float8_e8m0fnu), "offs": offs, "pos": pos}


def _combine(s):
    here = s["pos"] >= 0
    rows = s["pos"].long().clamp(min=0)
    if s["grad"]:
        d = s["d_out"].float()
        token = torch.nonzero(here)[:, 0]
        s["d_y"][rows[here]] = (d[token] * s["w"][here][:, None]).bfloat16()
        d_w = torch.where(here, (d[:, None] * s["y"][rows].float()).double().sum(-1), 0.0).float()
        return {"d_y": s["d_y"], "d_w": d_w}
    w = here.float() if s["w"] is None else torch.where(here, s["w"], 0.0)
    return {"out": (s["y"][rows].float() * w[..., None]).sum(1).bfloat16()}


# ------------------------------------------------------- the definitions in 64 bits
_E4M3 = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]


def _nearest(v, fmt):
    """The index of the value of a format's non-negative ones that is nearest to v >= 0; halves to the even one."""
    vals = torch.tensor(_E4M3 if fmt == "fp8" else FP4_VALUES, dtype=torch.float64, device=v.device)
    mid = (vals[1:] + vals[:-1]) / 2
    up = torch.bucketize(v, mid, right=True)          # at a half: the upper one
    down = torch.bucketize(v, mid, right=False)       # the lower one
    return torch.where(up % 2 == 0, up, down), vals


def _blocks64(x, fmt):
    """(values of the codes, values of the scales) of the MX blocks along the last axis of x, given in 64 bits."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().max(-1).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -126)))
    e = torch.where(top < 2.0 ** e, e - 1, torch.where(top >= 2.0 ** (e + 1), e + 1, e))
    s = torch.where(top < 2.0 ** -126, torch.full_like(e, -127.0), (e - EMAX[fmt]).clamp(min=-127))
    scale = torch.exp2(s)
    i, vals = _nearest((b / scale[..., None]).abs(), fmt)
    v = vals[i] * torch.where(torch.signbit(b), -1.0, 1.0)
    return v.reshape(x.shape), scale


def _decode64(codes, scales, fmt):
    if fmt == "fp8":
        vals = torch.tensor(_E4M3 + [math.nan] + [-f for f in _E4M3] + [math.nan], dtype=torch.float64, device=codes.device)
        v = vals[codes.long()]
    else:
        vals = torch.tensor(FP4_VALUES + tuple(-f for f in FP4_VALUES), dtype=torch.float64, device=codes.device)
        v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
        v[..., 0::2] = vals[(codes % 16).long()]
        v[..., 1::2] = vals[(codes // 16).long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def _turned64(s, x):
    """Pairs as complex numbers, times cos + i sin."""
    r = s["rot"]
    turn = torch.view_as_complex(s["rope"][s["positions"]].double())[:, None]
    pairs = x[..., :r].double().reshape(*x.shape[:-1], r // 2, 2) if s["inter"] else \
        x[..., :r].double().reshape(*x.shape[:-1], 2, r // 2).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z if s["inter"] else z.transpose(-1, -2)
    return torch.cat((z.reshape(*x.shape[:-1], r), x[..., r:].double()), -1)


def _ranks64(case, s):
    """(ends, rows) from the counts of each expert before each assignment."""
    e = s["ids"].reshape(-1)
    hot = (e[:, None] == torch.arange(case["held"], device=e.device)).int()
    ends = hot.sum(0).cumsum(0)
    rank = (hot.cumsum(0) - hot + (ends - hot.sum(0))) * hot
    return ends, torch.where(hot.any(1), rank.sum(1), -1).reshape(s["ids"].shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        fmt, page = case["fmt"], case["page"]
        at = (s["slots"] // page, s["slots"] % page)
        whole = []
        for x, codes, scales in ((_turned64(s, s["k"]).to(torch.bfloat16).double(), *s["parts"][:2]), (s["v"].double(), *s["parts"][2:])):
            v, e = _blocks64(x, fmt)
            if fmt == "fp4":
                whole.append(v * e.repeat_interleave(BLOCK, -1))
            else:
                one = _decode64(codes, torch.full_like(scales, 127), fmt)
                one[at[0], :, at[1]] = v
                exps = torch.exp2(scales.double() - 127)
                exps[at[0], :, at[1]] = e
                whole += [one, exps]
        q = _turned64(s, s["q"])
        return {"q": q, "k": whole[0], "v": whole[1]} if fmt == "fp4" else {"q": q, "k": whole[0], "ks": whole[1], "v": whole[2], "vs": whole[3]}
    if case["op"] == "dispatch":
        ends, pos = _ranks64(case, s)
        y = torch.zeros_like(s["y"], dtype=torch.float64)
        v, e = (s["x"].double(), None) if s["ys"] is None else _blocks64(s["x"].double(), "fp8")
        ys = None if e is None else torch.full_like(s["ys"], 2.0 ** -127, dtype=torch.float64)
        for j in range(case["k"]):
            here = pos[:, j] >= 0
            y[pos[here, j]] = v[here]
            if e is not None:
                ys[pos[here, j]] = e[here]
        return {"y": y, "offs": ends.int(), "pos": pos.int()} if e is None else {"codes": y, "scales": ys, "offs": ends.int(), "pos": pos.int()}
    if case["op"] == "combine":
        T, K = case["tokens"], case["K"]
        pos = s["pos"].long()
        if case["grad"]:
            d_y = torch.zeros_like(s["y"], dtype=torch.float64)
            d_w = torch.zeros_like(s["w"], dtype=torch.float64)
        else:
            out = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            row = pos[t, j]
            w = torch.ones(len(t), dtype=torch.float64, device="cuda") if s["w"] is None else s["w"][t, j].double()
            if case["grad"]:
                d = s["d_out"][t].double()
                d_y[row] = d * w[:, None]
                d_w[t, j] = (d * s["y"][row].double()).sum(1)
            else:
                out[t] += s["y"][row].double() * w[:, None]
        return {"d_y": d_y, "d_w": d_w} if case["grad"] else {"out": out}
    return _tree64(case, s)


def _tree64(case, s):
    new, kv = _lens(case)
    if work(case)["flops"] > 2e12:
        return None
    H, G, D, w = case["heads"], case["q_heads"] // case["heads"], case["dim"], case["window"]
    out = torch.zeros(sum(new), H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), H * G), -math.inf, dtype=torch.float64, device="cuda")
    kc, ks, vc, vs = s["parts"]
    row = 0
    for b, (n, L) in enumerate(zip(new, kv)):
        at = s["table"][b, :-(-L // case["page"])].long()
        hidden = torch.zeros(n, L, dtype=torch.bool)
        for i in range(n):      # up from node i: what is not on the way is hidden
            hidden[i, L - n:] = True
            depth, j = 0, i
            hidden[i, L - n + j] = False
            while j > 0:
                j, depth = (j - 1) // case["branch"], depth + 1
                hidden[i, L - n + j] = False
            if w:
                hidden[i, :max(0, min(L - n, L - n + depth - w + 1))] = True
        hidden = hidden.cuda()
        for h in range(H):
            k = _decode64(kc[at, h], ks[at, h], case["fmt"]).reshape(-1, D)[:L]
            v = _decode64(vc[at, h], vs[at, h], case["fmt"]).reshape(-1, D)[:L]
            kt = k.t().contiguous()
            q = s["q"][row:row + n, h * G:(h + 1) * G].double().transpose(0, 1)
            x = torch.stack([torch.mm(q[j], kt) for j in range(G)]) / math.sqrt(D)
            x.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            x = torch.exp(x - z[..., None])
            out[row:row + n, h * G:(h + 1) * G] = torch.stack([torch.mm(x[j], v) for j in range(G)], 1)
            lse[row:row + n, h * G:(h + 1) * G] = z.t()
        row += n
    return {"out": out, "lse": lse}
