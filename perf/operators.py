"""Workloads of the decode step's operators that shape or compress the masked LM head, and
their plain forms.

Four operators, as a serving process calls them between two forward passes of a diffusion LLM:

  counts  how often each token stands in each sequence's unmasked positions (what repetition,
          presence and frequency penalties need)
  quant   a matrix to microscaled 4-bit floating point (MXFP4: e2m1 codes, one power-of-two
          scale per 32 elements) and the values it then stands for
  rules   the mask-only LM head in bf16 with penalties, biases and grammar masks on the logits
  mx4     the same with W and the masked rows of H in MXFP4, with or without those rules

``own`` chooses between the plain forms (elementary torch operations) and the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _head(name, op, B, L, d, V, rows, rules, ext):
    """A masked LM-head case: `rows` masked positions at the end of each of the B sequences."""
    return dict(name=name, op=op, B=B, L=L, d=d, V=V, rows=rows, rules=rules, ext=ext)


def listed():
    return [
        # a short request: prompt and answer of a small-vocabulary model
        dict(name="counts_short", op="counts", B=1, L=256, V=4096),
        # eight requests of 8k positions, a large vocabulary (the block-decoding batch)
        dict(name="counts_batch", op="counts", B=8, L=8192, V=151936),
        # hidden rows of a ragged batch, quantised on their own
        dict(name="quant_rows", op="quant", R=1003, K=2048, dtype="bfloat16"),
        # the whole vocabulary projection, once per model load
        dict(name="quant_projection", op="quant", R=126464, K=4096, dtype="bfloat16"),
        # one token left to decode, every rule on: streaming W bounds it
        _head("rules_token", "rules", 1, 4096, 4096, 126464, 1, "all", False),
        # eight requests, each on its current 32-token block, every rule and every score
        _head("rules_block", "rules", 8, 8192, 2048, 151936, 32, "all", True),
        # one request with 1024 positions to fill, penalties and one shared bias
        _head("rules_answer", "rules", 1, 4096, 4096, 126464, 1024, "shared", False),
        # odd sizes: vocabulary tail, sequences that end inside a tile
        _head("rules_ragged", "rules", 3, 97, 192, 777, 41, "all", True),
        # the single-token and block steps with W in 4 bits
        _head("mx4_token", "mx4", 1, 4096, 4096, 126464, 1, "none", False),
        _head("mx4_block", "mx4", 8, 8192, 2048, 151936, 32, "all", True),
        # a long answer decoded from scratch: the tensor cores bound it
        _head("mx4_long", "mx4", 1, 8192, 4096, 126464, 7373, "none", True),
        _head("mx4_ragged", "mx4", 5, 131, 320, 5003, 77, "grammar", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["counts", "quant", "rules", "rules", "mx4", "mx4", "mx4"])
    if op == "counts":
        B = _log(rng, 1, 16)
        return dict(op=op, B=B, L=_log(rng, 1, 131072 // B), V=_log(rng, 500, 160000))
    if op == "quant":
        K = 32 * _log(rng, 2, 160)
        return dict(op=op, R=_log(rng, 1, min(126464, 400_000_000 // K)), K=K,
                    dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))
    B = _log(rng, 1, 12)
    d = 64 * _log(rng, 1, 64)
    V = _log(rng, 300, 160000)
    most = 1024 if op == "rules" else 4096
    rows = _log(rng, 1, max(1, most // B))
    L = rows + rng.randint(0, 2000)
    return dict(op=op, B=B, L=L, d=d, V=V, rows=rows,
                rules=rng.choice(["all", "shared", "grammar", "penalties"]
                                 + (["none"] if op == "mx4" else [])),
                ext=rng.random() < 0.5)


def _rule_parts(rules):
    """(per-sequence bias, shared bias, penalties, grammar) of a rule set."""
    return dict(none=(False, False, False, False), all=(True, False, True, True),
                shared=(False, True, True, False), grammar=(False, False, False, True),
                penalties=(False, False, True, False))[rules]


GRAMMAR_STATES = 12


def work(case):
    op = case["op"]
    if op == "counts":
        B, L, V = case["B"], case["L"], case["V"]
        return dict(bytes=5.0 * B * L + 4.0 * B * V + B * 4.0 * ((V + 31) // 32), flops=float(B * L))
    if op == "quant":
        n = case["R"] * case["K"]
        size = 4 if case["dtype"] == "float32" else 2
        # read once, the codes and scales written and read, the values written in bf16
        return dict(bytes=n * (size + 2 * (0.5 + 1 / 32) + 2.0), flops=3.0 * n)
    B, L, d, V, M = case["B"], case["L"], case["d"], case["V"], case["B"] * case["rows"]
    per_w = 0.5 + 1 / 32 if op == "mx4" else 2.0
    nbytes = V * d * per_w + M * d * 2.0 + B * L + M * (12 + (8 if case["ext"] else 0))
    seq_bias, shared_bias, pen, gram = _rule_parts(case["rules"])
    words = (V + 31) // 32
    nbytes += 4.0 * V * (B if seq_bias else 1 if shared_bias else 0)
    nbytes += B * 4.0 * (words + min(V, L - case["rows"])) if pen else 0   # counts of seen tokens
    nbytes += 4.0 * (words * GRAMMAR_STATES + M) if gram else 0
    return dict(bytes=nbytes, flops=2.0 * M * V * d)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _tokens(g, B, L, V):
    """Token ids with the skew of text: few ids very often, most never."""
    u = torch.rand(B, L, generator=g, device=DEV, dtype=torch.float64)
    return ((float(V) ** u) - 1).to(torch.int32).clamp_(0, V - 1)


def _make(case, seed):
    """The inputs alone, the same whichever side runs them."""
    g = _generator(seed)
    op = case["op"]
    if op == "counts":
        B, L, V = case["B"], case["L"], case["V"]
        return dict(tokens=_tokens(g, B, L, V),
                    M=(torch.rand(B, L, generator=g, device=DEV) < 0.3).to(torch.uint8))
    if op == "quant":
        R, K = case["R"], case["K"]
        x = torch.randn(R, K, generator=g, device=DEV, dtype=torch.bfloat16)
        # channels of very different size, as in hidden states and projections
        x *= torch.exp2(torch.randint(-6, 3, (1, K), generator=g, device=DEV).float()).to(x.dtype)
        x[torch.rand(R, generator=g, device=DEV) < 0.01] = 0         # padding rows
        return dict(X=x.to(getattr(torch, case["dtype"])))
    B, L, d, V, rows = case["B"], case["L"], case["d"], case["V"], case["rows"]
    W = torch.empty(V, d, device=DEV, dtype=torch.bfloat16)
    W.normal_(0.0, 0.02, generator=g)
    M = torch.zeros(B, L, dtype=torch.uint8, device=DEV)
    M[:, L - rows:] = 1
    H = torch.empty(B * L, d, device=DEV, dtype=torch.bfloat16)
    H.normal_(0.0, 1.0, generator=g)
    # a trained model's rows: each masked row leans towards one token, most of them clearly
    target = _tokens(g, B, rows, V).long()
    lean = torch.rand(B, rows, 1, generator=g, device=DEV) * 16 + 10
    unit = W[target].float()
    unit = unit / unit.norm(dim=-1, keepdim=True)
    H.view(B, L, d)[:, L - rows:] += (lean * unit).to(torch.bfloat16)
    s = dict(H=H, M=M, W=W, rows=rows)
    seq_bias, shared_bias, pen, gram = _rule_parts(case["rules"])
    if seq_bias or shared_bias:
        nb = B if seq_bias else 1
        Vp = (V + 3) // 4 * 4                       # rows start on 16 bytes
        bias = torch.randn(nb, Vp, generator=g, device=DEV) * 0.25
        u = torch.rand(nb, Vp, generator=g, device=DEV)
        bias = torch.where(u < 0.01, torch.full_like(bias, -math.inf), bias)       # banned tokens
        bias = torch.where(u > 0.995, torch.full_like(bias, torch.finfo(torch.float32).min), bias)
        s["bias"] = bias[:, :V] if seq_bias else bias[0, :V]
    if pen:
        tokens = _tokens(g, B, L, V)
        keep = (M == 0).to(torch.int32)
        counts = torch.zeros(B, V, dtype=torch.int32, device=DEV)
        counts.scatter_add_(1, tokens.long(), keep)
        s["counts"] = counts
        s["repetition"] = 1.0 + 0.5 * torch.rand(B, generator=g, device=DEV)
        s["presence"] = torch.rand(B, generator=g, device=DEV)
        s["frequency"] = 0.2 * torch.rand(B, generator=g, device=DEV)
    if gram:
        words = (V + 31) // 32
        # bitmaps of a grammar's states: nothing, everything, and sparse to dense sets
        share = torch.linspace(-4.0, 0.0, GRAMMAR_STATES - 2, device=DEV)[:, None]
        bits = torch.rand(GRAMMAR_STATES - 2, V, generator=g, device=DEV) < torch.exp(2.0 * share)
        # the state of a position; -1 = no restriction there, state 0 allows nothing
        state = torch.randint(1, GRAMMAR_STATES, (B, L), generator=g, device=DEV, dtype=torch.int32)
        u = torch.rand(B, L, generator=g, device=DEV)
        state = torch.where(u < 0.1, torch.full_like(state, -1), state)
        state = torch.where(u > 0.98, torch.zeros_like(state), state)
        bits = torch.cat([torch.zeros(1, V, dtype=torch.bool, device=DEV),
                          torch.ones(1, V, dtype=torch.bool, device=DEV), bits])
        # most positions' states allow what the model leans towards
        at = state[:, L - rows:].long()
        hit = (at > 1) & (torch.rand(B, rows, generator=g, device=DEV) < 0.9)
        bits[at[hit], target[hit]] = True
        pad = torch.zeros(GRAMMAR_STATES, words * 32 - V, dtype=torch.bool, device=DEV)
        shift = torch.arange(32, device=DEV)
        packed = (torch.cat([bits, pad], 1).view(GRAMMAR_STATES, words, 32).long() << shift).sum(-1)
        s["allow"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
        s["state"] = state
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = case
    op = case["op"]
    if not own:
        if op == "mx4":                             # the weights are quantised once
            s["Wq"] = _mx4_values(s.pop("W").float())
        return s
    import mask_only_logits_b200 as dl
    i32 = dict(dtype=torch.int32, device=DEV)
    if op == "counts":
        B, V = case["B"], case["V"]
        s["counts"], s["seen"] = torch.empty(B, V, **i32), torch.empty(B, (V + 31) // 32, **i32)
        return s
    if op == "quant":
        R, K = case["R"], case["K"]
        s["q"] = torch.empty(R, K // 2, dtype=torch.uint8, device=DEV)
        s["s"] = torch.empty(dl.mx4_scale_bytes(R, K), dtype=torch.uint8, device=DEV)
        s["Y"] = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
        return s
    B, L, d, V = case["B"], case["L"], case["d"], case["V"]
    n = B * L
    for name in ("conf", "lse", "entropy", "margin"):
        s[name] = torch.empty(n, dtype=torch.float32, device=DEV)
    s["tok"], s["row_idx"] = torch.empty(n, **i32), torch.empty(n, **i32)
    s["seq_off"], s["count"] = torch.empty(B + 1, **i32), torch.empty(4, **i32)
    if not case["ext"]:
        s["entropy"] = s["margin"] = None
    if "counts" in s:                               # the bitmap that goes with the counts
        s["seen"] = torch.empty(B, (V + 31) // 32, **i32)
        _pack_seen(s["counts"], s["seen"])
    s["handle"] = None
    if case["rules"] != "none":
        s["handle"] = dl.LogitRules(B, L, V, bias=s.get("bias"), counts=s.get("counts"),
                                    seen=s.get("seen"), repetition=s.get("repetition"),
                                    presence=s.get("presence"), frequency=s.get("frequency"),
                                    allow=s.get("allow"), allow_id=s.get("state"))
    if op == "mx4":
        s["W"] = dl.Mx4Matrix.quantize(s["W"])
        nbytes = dl.workspace_bytes_mx4(B, L, d, V, B * s["rows"])
    else:
        nbytes = dl.workspace_bytes_rows(B, L, d, V, B * s["rows"])
    s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return s


def _pack_seen(counts, seen):
    B, V = counts.shape
    words = seen.shape[1]
    bits = torch.zeros(B, words * 32, dtype=torch.int64, device=DEV)
    bits[:, :V] = (counts > 0).long()
    packed = (bits.view(B, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    seen.copy_(torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32))


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import mask_only_logits_b200 as dl
        if op == "counts":
            dl.token_counts(s["tokens"], s["counts"], s["seen"], M=s["M"])
            return dict(counts=s["counts"], seen=s["seen"])
        if op == "quant":
            dl.mx4_quantize(s["X"], s["q"], s["s"])
            dl.mx4_dequantize(s["q"], s["s"], s["Y"])
            return dict(values=s["Y"])
        call = dl.masked_logits_mx4 if op == "mx4" else dl.masked_logits_rules
        stats = dl.STAT_ENTROPY | dl.STAT_MARGIN if case["ext"] else 0
        call(s["H"], s["M"], s["W"], s["handle"], stats, s["tok"], s["conf"], s["lse"],
             s["entropy"], s["margin"], s["row_idx"], s["seq_off"], s["count"], s["ws"])
        m = case["B"] * s["rows"]                   # known to the loop that laid out the mask
        out = dict(tok=s["tok"][:m], conf=s["conf"][:m], lse=s["lse"][:m])
        if case["ext"]:
            out.update(entropy=s["entropy"][:m], margin=s["margin"][:m])
        return out
    if op == "counts":
        return _plain_counts(s)
    if op == "quant":
        return dict(values=_mx4_values(s["X"].float()).to(torch.bfloat16))
    return _plain_head(s)


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _plain_counts(s):
    V = s["case"]["V"]
    B = s["tokens"].shape[0]
    counts = torch.zeros(B, V, dtype=torch.int32, device=DEV)
    counts.scatter_add_(1, s["tokens"].long(), (s["M"] == 0).to(torch.int32))
    seen = torch.empty(B, (V + 31) // 32, dtype=torch.int32, device=DEV)
    _pack_seen(counts, seen)
    return dict(counts=counts, seen=seen)


def _mx4_values(x):
    """What x (fp32 [R, K]) stands for in MXFP4.  Blocks of 32: scale 2^(floor(log2 amax) - 2),
    elements to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), at most 6.
    Every step is exact in fp32: powers of two, and rounding to a multiple of the step."""
    R, K = x.shape
    xb = x.view(R, K // 32, 32)
    amax = xb.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)        # frexp: amax = f * 2^e', f in [.5, 1)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(xb, -e).clamp(-6.0, 6.0)
    a = y.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = torch.round(y / step) * step                             # ties to even: as the codes'
    return torch.ldexp(q, e).view(R, K)


def _plain_head(s):
    case = s["case"]
    B, L, V, rows = case["B"], case["L"], case["V"], case["rows"]
    pos = torch.nonzero_static(s["M"].view(-1), size=B * rows).view(-1)
    h = s["H"][pos].float()
    if case["op"] == "mx4":
        z = _mx4_values(h) @ s["Wq"].t()
    else:
        z = h @ s["W"].float().t()
    seq = pos // L
    if "counts" in s:
        c = s["counts"][seq]
        theta = s["repetition"][seq][:, None]
        cut = torch.where(z > 0, z / theta, z * theta)
        cut = cut - s["presence"][seq][:, None] - s["frequency"][seq][:, None] * c.float()
        z = torch.where(c > 0, cut, z)
    if "bias" in s:
        z = z + (s["bias"][seq] if s["bias"].dim() == 2 else s["bias"])
    if "allow" in s:
        v = torch.arange(V, device=DEV)
        table = ((s["allow"][:, v >> 5] >> (v & 31)) & 1).bool()
        state = s["state"].view(-1)[pos].long()
        free = state < 0
        ok = table[state.clamp(min=0)] | free[:, None]
        z = torch.where(ok, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    none = m == -math.inf
    ids = torch.arange(V, device=DEV, dtype=torch.int32)
    first = torch.where(z == m, ids, torch.full_like(ids, V)).amin(-1, keepdim=True)
    x = z - torch.where(none, torch.zeros_like(m), m)
    p = torch.exp(x)
    tot = p.sum(-1, keepdim=True)
    safe = torch.where(none, torch.ones_like(tot), tot)
    out = dict(tok=torch.where(none, torch.full_like(first, -1), first).view(-1),
               conf=torch.where(none, torch.zeros_like(m), 1 / safe).view(-1),
               lse=torch.where(none, m, m + torch.log(safe)).view(-1))
    if case["ext"]:
        t = torch.where(p > 0, p * x, torch.zeros_like(x)).sum(-1, keepdim=True)
        ent = torch.log(safe) - t / safe
        second = torch.where(ids == first, torch.full_like(z, -math.inf), z).amax(-1, keepdim=True)
        margin = (1 - torch.exp(second - torch.where(none, torch.zeros_like(m), m))) / safe
        out["entropy"] = torch.where(none, torch.full_like(ent, math.inf), ent).view(-1)
        out["margin"] = torch.where(none, torch.zeros_like(margin), margin).view(-1)
    return out


# ---------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------
def _mx4_exact(x):
    """MXFP4 of x by its table of values: the nearest one, of two as near the one with the
    even code."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV, dtype=torch.float64)
    edges = (table[1:] + table[:-1]) / 2
    R, K = x.shape
    out = torch.empty(R, K, dtype=torch.float64, device=DEV)
    for r0 in range(0, R, 8192):
        b = x[r0:r0 + 8192].double().reshape(-1, 32)
        top = b.abs().max(dim=1, keepdim=True).values
        # floor(log2 top) is the exponent field of the 64-bit number (0 and the tiniest: -1023)
        power = (top.view(torch.int64) >> 52) - 1023
        scale = torch.exp2((power - 2).clamp(-127, 127).double())
        a = b.abs() / scale
        low = torch.bucketize(a, edges)                   # number of edges below a
        high = torch.bucketize(a, edges, right=True)      # one more where a is an edge
        code = torch.where((low != high) & (low % 2 == 1), high, low)
        out[r0:r0 + 8192] = (torch.sign(b) * table[code] * scale).reshape(-1, K)
    return out


def exact(case, seed):
    s = _make(case, seed)
    op = case["op"]
    if op == "counts":
        return None
    if op == "quant":
        return dict(values=_mx4_exact(s["X"]))
    B, L, d, V, rows = case["B"], case["L"], case["d"], case["V"], case["rows"]
    W = _mx4_exact(s["W"]) if op == "mx4" else s["W"].double()
    H = s["H"].view(B, L, d)[:, L - rows:].reshape(B * rows, d)
    H = _mx4_exact(H) if op == "mx4" else H.double()
    allowed = None
    if "allow" in s:
        word = torch.arange(V, device=DEV) // 32
        bit = 2 ** (torch.arange(V, device=DEV) % 32)
        allowed = (s["allow"].long() % 2 ** 32)[:, word] // bit % 2 == 1
        state = s["state"][:, L - rows:].reshape(-1).long()
    parts = []
    for r0 in range(0, B * rows, 1024):
        r = torch.arange(r0, min(r0 + 1024, B * rows), device=DEV)
        b = r // rows
        z = torch.matmul(H[r], W.T)
        if "counts" in s:
            n = s["counts"][b].double()
            theta = s["repetition"][b].double().view(-1, 1)
            scaled = torch.minimum(z / theta, z * theta)  # theta >= 1: both signs move down
            scaled -= s["presence"][b].double().view(-1, 1) + s["frequency"][b].double().view(-1, 1) * n
            z = torch.where(n > 0, scaled, z)
        if "bias" in s:
            z = z + (s["bias"].double()[b] if s["bias"].dim() == 2 else s["bias"].double())
        if allowed is not None:
            z[~(allowed[state[r].clamp(min=0)] | (state[r] < 0).view(-1, 1))] = -math.inf
        lse = torch.logsumexp(z, dim=-1)
        p = torch.exp(z - lse.view(-1, 1))
        top = torch.topk(p, 2, dim=-1).values
        ent = -torch.xlogy(p, p).sum(-1)
        parts.append((lse, top, ent))
    lse, top, ent = (torch.cat(x) for x in zip(*parts))
    empty = torch.isneginf(lse)
    zero = torch.zeros_like(lse)
    out = dict(tok=None, conf=torch.where(empty, zero, top[:, 0]), lse=lse)
    if case["ext"]:
        out["entropy"] = torch.where(empty, zero + math.inf, ent)
        out["margin"] = torch.where(empty, zero, top[:, 0] - top[:, 1])
    return out
