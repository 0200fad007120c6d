"""Rules on logits and MXFP4 on the GPU against the fp64 reference: token counts, quantisation,
and the masked LM head with rules in bf16 and MXFP4 - small shapes where the kernels' edges lie
(odd vocabularies, one row, no row, rows with nothing allowed, strided tables).

Tolerances.  The tensor cores add d products per logit in fp32, each addition off by at most one
unit in the last place of the running sum (truncation), so |dz| <= d * 2^-23 * S with S the
largest sum_k |h_k w_k| of the row; MXFP4 products and their sums are exact here (a few bits
each).  The rules round at most six times: 6 * 2^-24 * (max|z| + what they add).  The sum of
exponentials adds V / 4 terms one after another at most (relative V / 4 * 2^-24), each with a
relative error below 2^-20 (2^x approximated to 2^-22, its argument rounded)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.shaped as S

pytestmark = pytest.mark.gpu
ALL = 3                                             # both extra scores


@pytest.fixture(scope="module")
def dl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mask_only_logits_b200 as dl
    return dl


def i32(*shape, fill=-7):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------
# token counts
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("B,n,V", [(1, 0, 5), (1, 1, 1), (2, 37, 31), (3, 1000, 33), (5, 513, 4096),
                                   (1, 20000, 160001), (150, 9, 70), (2, 4100, 70000)])
@pytest.mark.parametrize("masked", [False, True])
def test_token_counts(dl, B, n, V, masked):
    rng = np.random.default_rng(B * 1000 + n)
    tokens = rng.integers(-2, V + 2, (B, n)).astype(np.int32)
    M = (rng.random((B, n)) < 0.4).astype(np.uint8) * 3
    n_valid = rng.integers(-1, n + 2, B).astype(np.int32)
    counts, seen = i32(B, V), i32(B, (V + 31) // 32)
    t = torch.from_numpy(tokens).cuda()
    kw = dict(M=torch.from_numpy(M).cuda(), n_valid=torch.from_numpy(n_valid).cuda()) if masked else {}
    dl.token_counts(t, counts, seen, **kw)
    ref = np.zeros((B, V), dtype=np.int64)
    for b in range(B):
        for j in range(n):
            if 0 <= tokens[b, j] < V and not (masked and (M[b, j] or j >= n_valid[b])):
                ref[b, tokens[b, j]] += 1
    assert dl.get_status() == 0
    np.testing.assert_array_equal(counts.cpu().numpy(), ref)
    np.testing.assert_array_equal(seen.cpu().numpy(), S.pack_bits(ref > 0))
    # adding the same tokens again doubles the counts and leaves the bitmap
    dl.token_counts(t, counts, seen, accumulate=True, **kw)
    np.testing.assert_array_equal(counts.cpu().numpy(), 2 * ref)
    np.testing.assert_array_equal(seen.cpu().numpy(), S.pack_bits(ref > 0))


def test_token_counts_of_the_longest_sequence(dl):
    """n = 2^31 - 1: strides past the last token stay ahead of 31 bits."""
    n, V = 2**31 - 1, 70
    tokens = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    at = [0, 511, 2**31 - 37000, n - 300, n - 1]
    for v, j in enumerate(at):
        tokens[0, j] = v
    counts, seen = i32(1, V), i32(1, (V + 31) // 32)
    dl.token_counts(tokens, counts, seen)
    dl.token_counts(tokens, counts, seen, accumulate=True)
    ref = torch.zeros(1, V, dtype=torch.int32)
    ref[0, :len(at)] = 2
    assert dl.get_status() == 0
    assert torch.equal(counts.cpu(), ref)
    assert seen.cpu().tolist() == [[2**len(at) - 1, 0, 0]]


# ---------------------------------------------------------------------------------------
# MXFP4
# ---------------------------------------------------------------------------------------
def special_matrix(R, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-12, 12, (R, 1), generator=g).float())
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, -0.25, -2.5, -0.0, 0.0])
    x[0] = grid[torch.arange(K) % 14]               # ties, saturation, signed zeros
    if R > 2:
        x[1] = 0.0
        x[2, :32] = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -130   # subnormal
    if R > 4:
        x[3, 5] = float("nan")
        x[4, K - 1] = float("inf")
    x = x.to(dtype)
    return x


@pytest.mark.parametrize("R,K", [(1, 32), (1, 64), (5, 96), (127, 128), (129, 320), (300, 1056)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_mx4_quantize_and_back(dl, R, K, dtype):
    x = special_matrix(R, K, dtype, R + K)
    wide = torch.full((R, K + 8), 9.0, dtype=dtype, device="cuda")      # rows 8 elements further apart
    wide[:, :K] = x.cuda()
    codes, scales = S.mx4_codes(x.double().numpy())
    for X in (x.cuda(), wide[:, :K]):
        q = torch.full((R, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
        s = torch.full((dl.mx4_scale_bytes(R, K),), 0xEE, dtype=torch.uint8, device="cuda")
        dl.mx4_quantize(X, q, s)
        got = q.cpu().numpy()
        np.testing.assert_array_equal(dl.mx4_row_scales(s, R, K).cpu().numpy(), scales)
        np.testing.assert_array_equal(np.stack([got & 15, got >> 4], -1).reshape(R, K), codes)
        # the tiles hold nothing but those scales and zeros
        assert torch.equal(dl.mx4_tile_scales(torch.from_numpy(scales)), s.cpu())
    for out in (torch.bfloat16, torch.float32):
        y = dl.Mx4Matrix(q, s).dequantize(out)
        np.testing.assert_array_equal(y.double().cpu().numpy(), S.mx4_values(codes, scales))
    strided = torch.full((R, K + 8), 5.0, device="cuda")
    dl.mx4_dequantize(q, s, strided[:, :K])
    assert torch.equal(strided[:, K:], torch.full((R, 8), 5.0, device="cuda"))
    np.testing.assert_array_equal(strided[:, :K].double().cpu().numpy(), S.mx4_values(codes, scales))
    assert dl.get_status() == 0


# ---------------------------------------------------------------------------------------
# the masked LM head with rules
# ---------------------------------------------------------------------------------------
def make_rules(kinds, B, L, V, seed):
    """(NumPy rules for the reference, device tensors for LogitRules); tables are views of wider
    buffers, unused bits are set, and a NaN bias stands only where nothing is allowed."""
    rng = np.random.default_rng(seed)
    ref, dev = {}, {}
    words = (V + 31) // 32
    if "bias" in kinds or "shared" in kinds:
        nb = B if "bias" in kinds else 1
        bias = rng.normal(0, 1, (nb, V)).astype(np.float32)
        u = rng.random((nb, V))
        bias[u < 0.05] = -np.inf
        bias[u > 0.97] = np.finfo(np.float32).min
        wide = torch.full((nb, (V + 3) // 4 * 4 + 8), 1e30, device="cuda")
        wide[:, :V] = torch.from_numpy(bias).cuda()
        ref["bias"], dev["bias"] = (bias, wide[:, :V]) if "bias" in kinds else (bias[0], wide[0, :V])
    if "penalty" in kinds:
        counts = (rng.random((B, V)) < 0.3) * rng.integers(1, 9, (B, V))
        counts = counts.astype(np.int32)
        wide = i32(B, V + 3, fill=5)
        wide[:, :V] = torch.from_numpy(counts).cuda()
        bits = torch.full((B, words + 2), -1, dtype=torch.int32, device="cuda")
        sb = S.pack_bits(counts > 0)
        if V % 32:
            sb = sb | np.where(np.arange(words) == words - 1, -1 << (V % 32), 0).astype(np.int32)
        bits[:, :words] = torch.from_numpy(sb).cuda()
        ref["counts"], dev["counts"], dev["seen"] = counts, wide[:, :V], bits[:, :words]
        for name, lo, hi in (("repetition", 0.7, 2.0), ("presence", -0.5, 1.0), ("frequency", 0.0, 0.3)):
            if name in kinds or "only" not in kinds:
                ref[name] = rng.uniform(lo, hi, B).astype(np.float32)
                dev[name] = torch.from_numpy(ref[name]).cuda()
    if "grammar" in kinds or "allow_seq" in kinds:
        n = B if "allow_seq" in kinds else 6
        dens = np.array([0.0, 1.0, 0.5, 0.02, 0.9, 1.0 / V])[np.arange(n) % 6]
        bits = rng.random((n, V)) < dens[:, None]
        if n > 5:
            bits[5] = False
            bits[5, rng.integers(V)] = True          # one token only
        packed = S.pack_bits(bits)
        if V % 32:
            packed = packed | np.where(np.arange(words) == words - 1, -1 << (V % 32), 0).astype(np.int32)
        wide = torch.full((n, words + 1), -1, dtype=torch.int32, device="cuda")
        wide[:, :words] = torch.from_numpy(packed).cuda()
        ref["allow"], dev["allow"] = packed, wide[:, :words]
        if "grammar" in kinds:
            ids = rng.integers(-2, n, (B, L)).astype(np.int32)
            ref["allow_id"], dev["allow_id"] = ids, torch.from_numpy(ids).cuda()
        elif "bias" in kinds:                        # sequence 0 may take nothing: NaN is never seen
            dev["bias"][0, :].fill_(float("nan"))
            ref["bias"][0] = 0.0
    return ref, dev


def head_inputs(B, L, d, V, mask, seed):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, d, generator=g) * (1.5 / d ** 0.5)).to(torch.bfloat16)
    H = torch.randn(B * L, d, generator=g).to(torch.bfloat16)
    if mask == "none":
        M = torch.zeros(B, L, dtype=torch.uint8)
    elif mask == "one":
        M = torch.zeros(B, L, dtype=torch.uint8)
        M[B - 1, L // 2] = 7
    elif mask == "all":
        M = torch.ones(B, L, dtype=torch.uint8)
    else:
        M = (torch.rand(B, L, generator=g) < 0.5).to(torch.uint8)
    return H, M, W


def outputs(n, B, ext):
    f = lambda: torch.full((n,), -3.0, device="cuda")                  # noqa: E731
    return dict(tok=i32(n), conf=f(), lse=f(), entropy=f() if ext & 1 else None,
                margin=f() if ext & 2 else None, row_idx=i32(n), seq_off=i32(B + 1), count=i32(4))


def call(dl, mx4, H, M, W, rules, ext, o, ws, **kw):
    fn = dl.masked_logits_mx4 if mx4 else dl.masked_logits_rules
    fn(H, M, W, rules, ext, o["tok"], o["conf"], o["lse"], o["entropy"], o["margin"], o["row_idx"],
       o["seq_off"], o["count"], ws, **kw)


def dense(t, mx4):
    """What the products see of a bf16 matrix, in fp64."""
    return S.mx4_values(*S.mx4_codes(t.double().numpy())) if mx4 else t.double().numpy()


def reference(H, M, W, mx4, ref_rules, pos=None):
    B, L = M.shape
    V = W.shape[0]
    pos = np.flatnonzero(M.numpy().reshape(-1)) if pos is None else pos
    h, w = dense(H, mx4)[pos], dense(W, mx4)
    z0 = h @ w.T
    z = S.shape_logits(z0, pos // L, pos, V, **ref_rules)
    r = S.row_stats(z)
    mag = np.abs(h) @ np.abs(w).T
    dz = (0.0 if mx4 else h.shape[1] * 2.0 ** -23) * mag.max(-1, initial=0)
    added = 12.0                    # penalties and biases of make_rules but the lowest value
    r.update(pos=pos, z=z, dz=dz + 6 * 2.0 ** -24 * (2 * np.abs(z0).max(-1, initial=0) + added))
    return r


def check(o, r, V, ext, n_checked=None):
    c = len(r["pos"]) if n_checked is None else n_checked
    get = lambda k: o[k][:c].cpu().numpy()                             # noqa: E731
    rel = 2 * r["dz"] + V / 4 * 2.0 ** -24 + 2.0 ** -19
    tok, lse, conf = get("tok"), get("lse").astype(np.float64), get("conf").astype(np.float64)
    empty = r["tok"] < 0
    assert (tok[empty] == -1).all() and (conf[empty] == 0).all() and np.isneginf(lse[empty]).all()
    ok = ~empty
    assert (tok[ok] >= 0).all()
    best = r["z"].max(-1, initial=-np.inf)
    picked = r["z"][np.arange(c), np.maximum(tok, 0)]
    assert (picked[ok] >= best[ok] - 2 * r["dz"][ok] - 2.0 ** -24 * np.abs(best[ok])).all()
    # a logit at the lowest value swallows its own statistics' small terms: relative there
    scale = np.maximum(1.0, np.abs(r["lse"][ok]))
    assert (np.abs(lse[ok] - r["lse"][ok]) <= rel[ok] + 2.0 ** -23 * scale).all()
    assert (np.abs(conf[ok] - r["conf"][ok]) <= rel[ok] * r["conf"][ok]).all()
    if ext & 1:
        e = get("entropy").astype(np.float64)
        assert np.isposinf(e[empty]).all()
        tol = rel[ok] * (2 + r["entropy"][ok] + np.log(V))
        assert (np.abs(e[ok] - r["entropy"][ok]) <= tol).all()
    if ext & 2:
        m = get("margin").astype(np.float64)
        assert (m[empty] == 0).all()
        assert (np.abs(m[ok] - r["margin"][ok]) <= 3 * rel[ok]).all()


CASES = [
    # B, L, d, V, mask, rules, scores
    (1, 9, 64, 1, "all", "bias", ALL),
    (1, 9, 64, 1, "all", "grammar", 1),
    (2, 5, 64, 31, "half", "shared penalty", 0),
    (3, 40, 128, 33, "half", "penalty grammar bias", ALL),
    (3, 97, 192, 777, "half", "penalty grammar bias", 0),
    (3, 97, 192, 777, "all", "penalty grammar shared", ALL),
    (4, 11, 320, 1000, "half", "allow_seq bias", ALL),
    (1, 64, 256, 5003, "one", "penalty bias", 2),
    (1, 64, 256, 5003, "none", "penalty bias", ALL),
    (2, 200, 64, 5003, "all", "penalty only presence", 1),
    (1, 300, 1024, 2051, "half", "grammar", ALL),
    (1, 700, 64, 20011, "all", "shared grammar penalty", ALL),
    (5, 131, 448, 3000, "half", "penalty", 0),
]


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("variant", [0, 1, 2], ids=["auto", "single", "pair"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "+") for x in c))
def test_rows(dl, case, mx4, variant):
    B, L, d, V, mask, kinds, ext = case
    H, M, W = head_inputs(B, L, d, V, mask, seed=V + d)
    ref_rules, dev = make_rules(kinds.split(), B, L, V, seed=V)
    r = reference(H, M, W, mx4, ref_rules)
    n, c = B * L, len(r["pos"])
    o = outputs(n, B, ext)
    Wd = dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda()
    nbytes = dl.workspace_bytes_mx4(B, L, d, V) if mx4 else dl.workspace_bytes(B, L, d, V)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN wherever it is read unset
    rules = dl.LogitRules(B, L, V, **dev)
    dl.debug_set_gemm_variant(variant)
    try:
        call(dl, mx4, H.cuda(), M.cuda(), Wd, rules, ext, o, ws)
        assert dl.get_status() == 0
    finally:
        dl.debug_set_gemm_variant(0)
    assert int(o["count"][0]) == c
    np.testing.assert_array_equal(o["row_idx"][:c].cpu().numpy(), r["pos"])
    np.testing.assert_array_equal(o["seq_off"].cpu().numpy(), np.searchsorted(r["pos"], np.arange(B + 1) * L))
    check(o, r, V, ext)
    for k in ("tok", "conf", "lse", "entropy", "margin", "row_idx"):       # rows behind the last
        if o[k] is not None:
            assert (o[k][c:] == (-7 if o[k].dtype == torch.int32 else -3)).all(), k


@pytest.mark.parametrize("ext", [0, ALL])
@pytest.mark.parametrize("shape", [(1, 1, 64, 1), (2, 77, 192, 700), (1, 400, 512, 9000)])
def test_mx4_without_rules(dl, shape, ext):
    B, L, d, V = shape
    H, M, W = head_inputs(B, L, d, V, "all", seed=V)
    r = reference(H, M, W, True, {})
    o = outputs(B * L, B, ext)
    ws = torch.full((dl.workspace_bytes_mx4(B, L, d, V),), 0xFF, dtype=torch.uint8, device="cuda")
    call(dl, True, H.cuda(), M.cuda(), dl.Mx4Matrix.quantize(W.cuda()), None, ext, o, ws)
    assert dl.get_status() == 0
    check(o, r, V, ext)
    # sums of a few bits each: the first of equal maxima, exactly
    np.testing.assert_array_equal(o["tok"].cpu().numpy(), r["tok"])


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_mask_of_many_positions(dl, mx4):
    """As many positions as one launch stages (2048), one more, and several tiles of the mask; every
    position of the smallest masked, and a sequence of one position each."""
    d, V = 64, 300
    for B, L, k in ((2, 1024, 2048), (2048, 1, 700), (1, 2049, 2049), (3, 683, 1500), (2, 32768, 200)):
        H, M, W = head_inputs(B, L, d, V, "none", seed=9)
        pos = np.sort(np.random.default_rng(1).choice(B * L, k, replace=False))
        M.view(-1)[pos] = 1
        M[B - 1, L - 1] = 1
        pos = np.flatnonzero(M.numpy().reshape(-1))
        ref_rules, dev = make_rules(["penalty", "grammar"], B, L, V, seed=1)
        r = reference(H, M, W, mx4, ref_rules, pos)
        o = outputs(B * L, B, ALL)
        ws = torch.empty((dl.workspace_bytes_mx4 if mx4 else dl.workspace_bytes_rows)(B, L, d, V, k + 1),
                         dtype=torch.uint8, device="cuda")
        call(dl, mx4, H.cuda(), M.cuda(), dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda(),
             dl.LogitRules(B, L, V, **dev), ALL, o, ws)
        assert dl.get_status() == 0 and int(o["count"][0]) == len(pos)
        check(o, r, V, ALL)
        np.testing.assert_array_equal(o["row_idx"][:len(pos)].cpu().numpy(), pos)
        np.testing.assert_array_equal(o["seq_off"].cpu().numpy(), np.searchsorted(pos, np.arange(B + 1) * L))


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_windows_and_capacity(dl, mx4):
    """Rows of the windows only; a workspace for fewer rows computes those that fit, records the
    rest and touches nothing else."""
    B, L, d, V = 3, 50, 128, 600
    H, M, W = head_inputs(B, L, d, V, "half", seed=5)
    ref_rules, dev = make_rules(["penalty", "grammar"], B, L, V, seed=1)
    lo, hi = np.array([10, 60, 5], dtype=np.int32), np.array([40, 70, 5], dtype=np.int32)
    lo[2], hi[2] = 20, 50
    flat = np.flatnonzero(M.numpy().reshape(-1))
    pos = np.array([p for p in flat if lo[p // L] <= p % L < hi[p // L]])
    r = reference(H, M, W, mx4, ref_rules, pos)
    rules = dl.LogitRules(B, L, V, **dev)
    Wd = dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda()
    size = dl.workspace_bytes_mx4 if mx4 else dl.workspace_bytes_rows
    win = dict(win_lo=torch.from_numpy(lo).cuda(), win_hi=torch.from_numpy(hi).cuda())
    nbytes = size(B, L, d, V, len(pos))
    room = torch.full((nbytes + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o = outputs(B * L, B, ALL)
    call(dl, mx4, H.cuda(), M.cuda(), Wd, rules, ALL, o, room[:nbytes], **win)
    assert dl.get_status() == 0 and int(o["count"][0]) == len(pos)
    check(o, r, V, ALL)
    assert (room[nbytes:] == 0xA5).all()
    few = 5
    nbytes = size(B, L, d, V, few)
    cap = (dl.workspace_rows_mx4 if mx4 else dl.workspace_rows)(B, L, d, V, nbytes)
    room.fill_(0xA5)
    o = outputs(B * L, B, ALL)
    call(dl, mx4, H.cuda(), M.cuda(), Wd, rules, ALL, o, room[:nbytes], **win)
    if cap < len(pos):
        assert dl.get_status() == -11
        assert (o["tok"][cap:] == -7).all() and (room[nbytes:] == 0xA5).all()
        part = {k: v[:cap] for k, v in r.items()}
        check(o, part, V, ALL, n_checked=cap)


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_lowest_value_everywhere(dl, mx4):
    """A bias of the lowest finite value on every token is a number, not a ban: the row's
    softmax is uniform over its tokens and the first of them wins."""
    B, L, d, V = 1, 3, 64, 1000
    H, M, W = head_inputs(B, L, d, V, "all", seed=2)
    bias = torch.full((V,), torch.finfo(torch.float32).min, device="cuda")
    o = outputs(L, B, ALL)
    ws = torch.empty(max(dl.workspace_bytes(B, L, d, V), dl.workspace_bytes_mx4(B, L, d, V)),
                     dtype=torch.uint8, device="cuda")
    call(dl, mx4, H.cuda(), M.cuda(), dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda(),
         dl.LogitRules(B, L, V, bias=bias), ALL, o, ws)
    assert dl.get_status() == 0
    assert (o["tok"] == 0).all()
    # 1000 equal terms: exact sums, a reciprocal and a logarithm
    np.testing.assert_allclose(o["conf"].cpu().numpy(), 1 / V, rtol=2.0 ** -22)
    np.testing.assert_allclose(o["entropy"].cpu().numpy(), np.log(V), rtol=2.0 ** -21)
    assert (o["margin"] == 0).all() and (o["lse"] == torch.finfo(torch.float32).min).all()


@pytest.mark.parametrize("variant", [0, 1, 2], ids=["auto", "single", "pair"])
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_first_of_equal_maxima(dl, mx4, variant):
    """Equal logits in tiles that different CTAs, and one CTA in any order, walk over: the lowest
    allowed token wins.  Row l's largest logit stands at five tokens; where all are equal the
    first token does."""
    B, L, d, V = 1, 130, 64, 90001
    rng = np.random.default_rng(0)
    W = torch.zeros(V, d, dtype=torch.bfloat16)
    H = torch.zeros(L, d, dtype=torch.bfloat16)
    want = np.zeros(L, dtype=np.int64)
    allow = np.ones((L, V), dtype=bool)
    for l in range(L - 2):                           # the last two rows are zero: all logits equal
        H[l, l % d] = 2.0 if l < d else -2.0
        if l < d:
            at = np.sort(rng.choice(V, 10, replace=False))
            W[at[:5], l], W[at[5:], l] = 4.0, -4.0   # rows l and l + d: the same column, two signs
        at = np.flatnonzero(W[:, l % d].float().numpy() == (4.0 if l < d else -4.0))
        allow[l, at[0]] = l % 3 != 0                 # some rows may not take the first of them
        want[l] = at[0] if allow[l, at[0]] else at[1]
    rules = dl.LogitRules(B, L, V, allow=torch.from_numpy(S.pack_bits(allow)).cuda(),
                          allow_id=torch.arange(L, dtype=torch.int32, device="cuda")[None])
    M = torch.ones(B, L, dtype=torch.uint8, device="cuda")
    ws = torch.empty(max(dl.workspace_bytes(B, L, d, V), dl.workspace_bytes_mx4(B, L, d, V)),
                     dtype=torch.uint8, device="cuda")
    Wd = dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda()
    o = outputs(L, B, ALL)
    dl.debug_set_gemm_variant(variant)
    try:
        call(dl, mx4, H.cuda(), M, Wd, rules, ALL, o, ws)
        assert dl.get_status() == 0
    finally:
        dl.debug_set_gemm_variant(0)
    np.testing.assert_array_equal(o["tok"].cpu().numpy(), want)
    assert (o["margin"] == 0).all()


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_nan_and_infinity_stay_where_they_are(dl, mx4):
    """A hidden row with a NaN has NaN statistics (not those of a row that may take nothing), the
    rows beside it theirs; a NaN bias on a banned token is never seen; unmasked rows are not read."""
    B, L, d, V = 1, 40, 128, 700
    H, M, W = head_inputs(B, L, d, V, "half", seed=6)
    pos = np.flatnonzero(M.numpy().reshape(-1))
    clean = H.clone()
    H[np.setdiff1d(np.arange(L), pos)] = float("nan")
    H[pos[3], 5] = float("nan")
    H[pos[4], 7] = float("inf")
    bits = np.ones((1, V), dtype=bool)
    bits[0, ::7] = False
    bias = np.zeros(V, dtype=np.float32)
    bias[::7] = np.nan
    r = reference(clean, M, W, mx4, dict(allow=S.pack_bits(bits)))
    rules = dl.LogitRules(B, L, V, bias=torch.from_numpy(bias).cuda(),
                          allow=torch.from_numpy(S.pack_bits(bits)).cuda())
    o = outputs(L, B, ALL)
    ws = torch.full((max(dl.workspace_bytes(B, L, d, V), dl.workspace_bytes_mx4(B, L, d, V)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    call(dl, mx4, H.cuda(), M.cuda(), dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda(), rules, ALL, o, ws)
    assert dl.get_status() == 0
    for k in ("conf", "lse", "entropy"):
        assert torch.isnan(o[k][3:5]).all(), k
    keep = np.delete(np.arange(len(pos)), [3, 4])
    check({k: (v if v is None else v[:len(pos)][torch.from_numpy(keep).cuda()]) for k, v in o.items()
           if k in ("tok", "conf", "lse", "entropy", "margin")}, {k: v[keep] for k, v in r.items()}, V, ALL)


def test_bitmap_number_out_of_range_is_recorded(dl):
    """A bitmap number past the table is reported and its row left unrestricted; the others keep
    their bitmaps."""
    B, L, d, V = 1, 4, 64, 100
    H, M, W = head_inputs(B, L, d, V, "all", seed=3)
    allow = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    ids = torch.tensor([[0, 5, -1, 1]], dtype=torch.int32, device="cuda")
    o = outputs(L, B, 0)
    ws = torch.empty(dl.workspace_bytes(B, L, d, V), dtype=torch.uint8, device="cuda")
    call(dl, False, H.cuda(), M.cuda(), W.cuda(), dl.LogitRules(B, L, V, allow=allow, allow_id=ids), 0, o, ws)
    assert dl.get_status() == -8 and dl.get_status() == 0
    tok = o["tok"].cpu().numpy()
    assert (tok >= 0).tolist() == [False, True, True, False]


# ---------------------------------------------------------------------------------------
# as they are used together
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("weights", ["bf16", "mx4"])
@pytest.mark.parametrize("policy", ["confidence", "entropy", "margin"])
def test_decode_loop(dl, weights, policy):
    """A whole decode with penalties and a grammar: counts, steps that unmask k positions, the
    counts brought up to date from each selection.  Every step's rows match the reference on the
    state at that step, no banned token is ever taken, and the running counts equal a count from
    scratch."""
    B, L, d, V, k = 2, 24, 128, 500, 5
    mx4 = weights == "mx4"
    H, _, W = head_inputs(B, L, d, V, "all", seed=11)
    rng = np.random.default_rng(4)
    tokens = rng.integers(0, V, (B, L)).astype(np.int32)
    M = np.zeros((B, L), dtype=np.uint8)
    M[:, 8:] = 1
    allow = rng.random((3, V)) < 0.3
    ids = rng.integers(-1, 3, (B, L)).astype(np.int32)
    pen = dict(repetition=np.float32([1.3, 0.9]), presence=np.float32([0.2, 0.0]),
               frequency=np.float32([0.1, 0.5]))
    Hd, Wd = H.cuda(), dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda()
    counts, seen = i32(B, V), i32(B, (V + 31) // 32)
    td, Md = torch.from_numpy(tokens).cuda(), torch.from_numpy(M).cuda()
    dl.token_counts(td, counts, seen, M=Md)
    rules = dl.LogitRules(B, L, V, counts=counts, seen=seen, allow=torch.from_numpy(S.pack_bits(allow)).cuda(),
                          allow_id=torch.from_numpy(ids).cuda(),
                          **{n: torch.from_numpy(v).cuda() for n, v in pen.items()})
    step = dl.DecodeStep(B, L, d, V, k, policy=policy, weights=weights)
    steps = 0
    while M.any():
        ref_counts = np.stack([np.bincount(tokens[b][M[b] == 0], minlength=V) for b in range(B)])
        r = reference(H, torch.from_numpy(M), W, mx4,
                      dict(counts=ref_counts, allow=S.pack_bits(allow), allow_id=ids, **pen))
        out = step.run(Hd, Md, Wd, rules=rules)
        assert dl.get_status() == 0
        ext = {"confidence": 0, "entropy": 1, "margin": 2}[policy]
        check(out if ext else dict(out, entropy=None, margin=None), r, V, ext)
        n_sel, idx, tok_sel = out["n_sel"].cpu(), out["idx"].cpu(), out["tok_sel"].cpu()
        for b in range(B):
            assert int(n_sel[b]) == min(k, int(M[b].sum()))
            for j in range(int(n_sel[b])):
                l, t = int(idx[b, j]), int(tok_sel[b, j])
                assert M[b, l] and (ids[b, l] < 0 or allow[ids[b, l], t])
                tokens[b, l], M[b, l] = t, 0
        dl.token_counts(out["tok_sel"], counts, seen, n_valid=out["n_sel"], accumulate=True)
        td.copy_(torch.from_numpy(tokens))
        Md.copy_(torch.from_numpy(M))
        fresh, fseen = i32(B, V), i32(B, (V + 31) // 32)
        dl.token_counts(td, fresh, fseen, M=Md)
        assert torch.equal(fresh, counts) and torch.equal(fseen, seen)
        steps += 1
    assert steps == 4


@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_capture_other_stream_and_host_inputs(dl, weights):
    """The same step eagerly, replayed from a graph after every input and rule has changed in
    place, on another stream, and from page-locked host memory: equal outputs."""
    B, L, d, V, k = 2, 60, 192, 901, 6
    mx4 = weights == "mx4"
    H, M, W = head_inputs(B, L, d, V, "half", seed=21)
    H2, M2, _ = head_inputs(B, L, d, V, "half", seed=22)
    _, dev = make_rules(["bias", "penalty", "grammar"], B, L, V, seed=3)
    _, dev2 = make_rules(["bias", "penalty", "grammar"], B, L, V, seed=4)
    Wd = dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda()
    step = dl.DecodeStep(B, L, d, V, k, weights=weights)

    def snap(out):
        c = int(out["count"][0])
        return [out[n].clone() for n in ("idx", "n_sel", "tok_sel", "conf_sel")] + \
            [out[n][:c].clone() for n in ("tok", "conf", "lse", "row_idx")]

    want = snap(step.run(H2.cuda(), M2.cuda(), Wd, rules=dl.LogitRules(B, L, V, **dev2)))
    Hd, Md = H.cuda(), M.cuda()
    rules = dl.LogitRules(B, L, V, **dev)
    step.capture(Hd, Md, Wd, rules=rules)
    Hd.copy_(H2)
    Md.copy_(M2)
    for name, t in dev.items():
        t.copy_(dev2[name])
    assert all(torch.equal(a, b) for a, b in zip(snap(step.replay()), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = step.run(Hd, Md, Wd, stream=side, rules=rules)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(snap(out), want))
    out = step.run(H2.pin_memory(), M2.pin_memory(), Wd, rules=rules)
    assert all(torch.equal(a, b) for a, b in zip(snap(out), want))
    host = step.run_host(H2, M2, Wd, rules=rules)
    assert all(torch.equal(host[n], w.cpu()) for n, w in zip(("idx", "n_sel", "tok_sel", "conf_sel"), want))
    arena = dl.DecodeStep(B, L, d, V, k, weights=weights, arena=True)
    assert all(torch.equal(a, b) for a, b in zip(snap(arena.run(Hd, Md, Wd, rules=rules)), want))
    assert dl.get_status() == 0


def test_captured_step_keeps_its_rules(dl):
    """Rules that nothing but the graph refers to: their tensors are not given to others."""
    B, L, d, V, k = 1, 40, 64, 500, 4
    H, M, W = (t.cuda() for t in head_inputs(B, L, d, V, "half", seed=9))

    def rules():
        bias = torch.zeros(V, device="cuda")
        bias[123] = 1000.0
        return dl.LogitRules(B, L, V, bias=bias)

    step = dl.DecodeStep(B, L, d, V, k)
    step.capture(H, M, W, rules=rules())
    junk = [torch.full((V,), float(i), device="cuda") for i in range(64)]
    c = int(step.replay()["count"][0])
    assert c > 0 and step.tok[:c].tolist() == [123] * c
    assert len(junk) == 64 and dl.get_status() == 0


def test_two_steps_on_two_streams(dl):
    """Two steps at once, each with its own buffers and rules, on two streams."""
    B, L, d, V = 1, 200, 256, 3000
    res = []
    for seed in (1, 2):
        H, M, W = head_inputs(B, L, d, V, "half", seed=seed)
        _, dev = make_rules(["penalty", "grammar"], B, L, V, seed=seed)
        res.append((H.cuda(), M.cuda(), dl.Mx4Matrix.quantize(W.cuda()), dl.LogitRules(B, L, V, **dev),
                    dl.DecodeStep(B, L, d, V, 4, weights="mx4"), torch.cuda.Stream()))
    want = [r[4].run(r[0], r[1], r[2], rules=r[3])["conf_sel"].clone() for r in res]
    torch.cuda.synchronize()
    for _ in range(5):
        for H, M, W, rules, step, stream in res:
            step.run(H, M, W, stream=stream, rules=rules)
    torch.cuda.synchronize()
    assert all(torch.equal(r[4].conf_sel, w) for r, w in zip(res, want))
    assert dl.get_status() == 0


def test_c_struct_layout(dl):
    """The binding's struct is the header's: eight pointers, four 64-bit strides, one int."""
    from mask_only_logits_b200 import _abi
    assert ctypes.sizeof(_abi.LogitRulesStruct) == 13 * 8


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("variant", [1, 2], ids=["single", "pair"])
def test_unarmed_stage_times_out(dl, mx4, variant):
    """A copy of the library that leaves one stage of the ring unarmed: the waits give up after a
    second, every role unwinds, the host reads DLLM_ERR_TIMEOUT, and the regular library computes
    right afterwards.  Nothing faults or hangs."""
    import os

    from mask_only_logits_b200 import _abi, build
    out = os.path.join(build.PKG_DIR, "libdllm_fault_skip_stage.so")
    if not os.path.exists(out) or os.path.getmtime(out) < os.path.getmtime(build.LIB_PATH):
        build.build(extra_flags=["-DDLLM_FAULT_SKIP_STAGE=1"], out=out)
    lib = _abi.load_from(out)
    B, L, d, V = 1, 300, 512, 2000
    H, M, W = head_inputs(B, L, d, V, "all", seed=1)
    ref_rules, dev = make_rules(["penalty"], B, L, V, seed=1)
    rules = dl.LogitRules(B, L, V, **dev)
    Wd = dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda()
    Hd, Md, o = H.cuda(), M.cuda(), outputs(L, B, 0)
    ws = torch.empty(max(dl.workspace_bytes(B, L, d, V), dl.workspace_bytes_mx4(B, L, d, V)),
                     dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())                        # noqa: E731
    nul, stream = ctypes.c_void_p(None), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    head = [p(Hd), p(Md)] + ([p(Wd.q), p(Wd.s)] if mx4 else [p(Wd)]) + [B, L, d, V, nul, nul]
    tail = [0, p(o["tok"]), p(o["conf"]), p(o["lse"]), nul, nul, p(o["row_idx"]), p(o["seq_off"]),
            p(o["count"]), p(ws), ws.numel(), stream]
    fn = lib.dllm_masked_logits_mx4 if mx4 else lib.dllm_masked_logits_rules
    assert lib.dllm_debug_set_gemm_variant(variant) == 0
    assert fn(*head, ctypes.byref(rules._struct), *tail) == 0
    assert lib.dllm_get_status(stream) == -6 and lib.dllm_get_status(stream) == 0
    call(dl, mx4, Hd, Md, Wd, rules, 0, o, ws)
    assert dl.get_status() == 0
    check(o, reference(H, M, W, mx4, ref_rules), V, 0)


# ---------------------------------------------------------------------------------------
# buffers that the package makes itself
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_mx4_matrix_on_another_stream(dl, handle):
    """Quantising and dequantising on a side stream leave alone what the current stream still reads
    of memory given back to the allocator, and what it gets of theirs when they are dropped."""
    R, K = 8192, 4096
    side = torch.cuda.Stream()
    on = side.cuda_stream if handle else side
    X = torch.randn(R, K, device="cuda", dtype=torch.bfloat16)
    want = dl.Mx4Matrix.quantize(X)
    back = want.dequantize()
    kept = [torch.empty(R, K // 2, dtype=torch.uint8, device="cuda"), torch.empty_like(X)]
    torch.cuda.synchronize()
    # memory of the results' sizes, given back while the current stream has yet to read it
    old = [torch.full_like(kept[0], 7), torch.full_like(kept[1], 7)]
    torch.cuda._sleep(100_000_000)
    for k, o in zip(kept, old):
        k.copy_(o)
    del old, o
    got = dl.Mx4Matrix.quantize(X, stream=on)
    again = got.dequantize(stream=on)
    torch.cuda.synchronize()
    assert (kept[0] == 7).all() and (kept[1] == 7).all()
    assert torch.equal(got.q, want.q) and torch.equal(got.s, want.s) and torch.equal(again, back)
    # results dropped before the side stream has written them
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    dl.Mx4Matrix.quantize(X, stream=on).dequantize(stream=on)
    new = [torch.full_like(kept[0], 9), torch.full_like(kept[1], 9)]
    torch.cuda.synchronize()
    assert (new[0] == 9).all() and (new[1] == 9).all()
    assert dl.get_status() == 0


@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_an_earlier_graph_stays_valid(dl, weights):
    """Two captures of one step with rules and weights that only the graphs refer to: each graph
    replays its own."""
    B, L, d, V, k = 1, 40, 64, 500, 4
    H, M, W = (t.cuda() for t in head_inputs(B, L, d, V, "half", seed=9))
    step = dl.DecodeStep(B, L, d, V, k, weights=weights)
    graphs = []
    for best in (123, 321):
        bias = torch.zeros(V, device="cuda")
        bias[best] = 1000.0
        Wd = dl.Mx4Matrix.quantize(W) if weights == "mx4" else W.clone()
        graphs.append(step.capture(H, M, Wd, rules=dl.LogitRules(B, L, V, bias=bias)))
        del Wd, bias
    junk = [torch.full((n,), float(i), device="cuda") for i in range(64) for n in (V, V * d // 4)]
    for g, best in zip(graphs + graphs[:1], (123, 321, 123)):
        g.replay()
        c = int(step.count[0])
        assert c > 0 and step.tok[:c].tolist() == [best] * c
    assert len(junk) == 128 and dl.get_status() == 0


# ---------------------------------------------------------------------------------------
# rows that no token is left for, in a selection
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [40, 300, 5000], ids=["ranked", "staged", "long"])
@pytest.mark.parametrize("policy", ["confidence", "entropy", "margin"])
@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_rows_without_a_token_come_last(dl, weights, policy, n):
    """Every second position may take nothing, and all logits of the others are equal (margin 0,
    the least confidence): a selection of as many as can be filled takes those, in order, and a
    selection of more the others after them.  n: each of the selection's ways."""
    L, d, V = n, 64, 40
    H = torch.zeros(L, d, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    M = torch.ones(1, L, dtype=torch.uint8, device="cuda")
    allow = torch.from_numpy(S.pack_bits(np.stack([np.zeros(V, bool), np.ones(V, bool)]))).cuda()
    ids = (torch.arange(L, dtype=torch.int32, device="cuda") % 2)[None].contiguous()
    rules = dl.LogitRules(1, L, V, allow=allow, allow_id=ids)
    Wd = dl.Mx4Matrix.quantize(W) if weights == "mx4" else W
    full = list(range(1, L, 2))
    for k, threshold in ((L // 2, None), (L // 2 + 7, None),
                         (L // 2 + 7, dict(confidence=0.0, entropy=np.inf, margin=0.0)[policy])):
        k = min(k, dl.MAX_K)
        step = dl.DecodeStep(1, L, d, V, k, policy=policy, threshold=threshold, weights=weights)
        out = step.run(H, M, Wd, rules=rules)
        assert dl.get_status() == 0 and int(out["n_sel"][0]) == k
        want = (full + [0, 2, 4, 6, 8, 10, 12])[:k]
        assert out["idx"][0].tolist() == want
        assert out["tok_sel"][0].tolist() == [0 if l % 2 else -1 for l in want]


@pytest.mark.parametrize("n", [5, 300, 5000])
@pytest.mark.parametrize("ascending", [False, True])
def test_a_threshold_of_zero_takes_zeros_of_either_sign(dl, ascending, n):
    """Scores at least as good as the threshold in the numbers' order, where zeros are equal."""
    rng = np.random.default_rng(n)
    score = rng.choice(np.float32([-1.0, -0.0, 0.0, 1.0]), n)
    passing = int((score <= 0).sum() if ascending else (score >= 0).sum())
    for tau in (0.0, -0.0):
        idx, n_sel = i32(1, 1024), i32(1)
        dl.select_unmask_ex(torch.from_numpy(score).cuda(), torch.arange(n, dtype=torch.int32, device="cuda"),
                            torch.tensor([0, n], dtype=torch.int32, device="cuda"), 1, n, 1024, tau, 0, idx,
                            n_sel, ascending)
        assert int(n_sel[0]) == min(passing, 1024), tau
        taken = idx[0, :int(n_sel[0])].cpu().numpy()
        assert (score[taken] <= 0).all() if ascending else (score[taken] >= 0).all()
    assert dl.get_status() == 0


# ---------------------------------------------------------------------------------------
# a build whose registers do not fit
# ---------------------------------------------------------------------------------------
def test_a_build_with_other_registers_refuses_one_kernel_only(dl):
    """A copy of the library that expects another register count of the bf16 kernel with rules: that
    call is refused before anything is launched, and every other one runs."""
    import os

    from mask_only_logits_b200 import _abi, build
    out = os.path.join(build.PKG_DIR, "libdllm_other_registers.so")
    if not os.path.exists(out) or os.path.getmtime(out) < os.path.getmtime(build.LIB_PATH):
        build.build(extra_flags=["-DDLLM_SHAPED_LAUNCH_REGS=176"], out=out)
    lib = _abi.load_from(out)
    B, L, d, V, k = 1, 60, 128, 700, 4
    H, M, W = head_inputs(B, L, d, V, "half", seed=1)
    Hd, Md, Wd, Q = H.cuda(), M.cuda(), W.cuda(), dl.Mx4Matrix.quantize(W.cuda())
    o = outputs(L, B, 0)
    ws = torch.empty(max(dl.workspace_bytes(B, L, d, V), dl.workspace_bytes_mx4(B, L, d, V)),
                     dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())                        # noqa: E731
    nul, stream = ctypes.c_void_p(None), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rules = dl.LogitRules(B, L, V, bias=torch.zeros(V, device="cuda"))._struct
    tail = [0, p(o["tok"]), p(o["conf"]), p(o["lse"]), nul, nul, p(o["row_idx"]), p(o["seq_off"]),
            p(o["count"]), p(ws), ws.numel(), stream]
    dims = [B, L, d, V, nul, nul, ctypes.byref(rules)]
    assert lib.dllm_masked_logits_rules(p(Hd), p(Md), p(Wd), *dims, *tail) == -7       # DLLM_ERR_DEVICE
    assert lib.dllm_get_status(stream) == 0 and (o["count"] == -7).all() and (o["tok"] == -7).all()
    assert lib.dllm_masked_logits_mx4(p(Hd), p(Md), p(Q.q), p(Q.s), *dims, *tail) == 0
    assert lib.dllm_get_status(stream) == 0
    check(o, reference(H, M, W, True, {}), V, 0)
    want = dl.DecodeStep(B, L, d, V, k).run(Hd, Md, Wd)["idx"]
    idx, n_sel = i32(B, k), i32(4)
    assert lib.dllm_decode_step(p(Hd), p(Md), p(Wd), B, L, d, V, k, nul, nul, *tail[1:4], *tail[6:9], p(idx),
                                p(n_sel), nul, nul, p(ws), ws.numel(), stream) == 0
    assert lib.dllm_get_status(stream) == 0 and torch.equal(idx, want)


# ---------------------------------------------------------------------------------------
# accuracy
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("variant,first", [(1, 128), (2, 1024)], ids=["single", "pair"])
def test_bf16_sums_are_taken_in_pieces(dl, variant, first):
    """A product of 16 (or 8), then, from k = first on, products of 2^-24 (2^-25): beside the large
    one each of them is below fp32's last place and lost, in pieces of their own they add up to
    multiples of 2^-17 (2^-18), which the large one takes exactly.  So the logit is exact, and the
    log-sum-exp off by its own rounding, half of 2^-19, and less than 2^-21 for the logarithm;
    summed in one go it would be 1.8e-4 lower."""
    d, V, n = 4096, 600, 3 if variant == 1 else 300
    H, W = torch.zeros(n, d), torch.zeros(V, d)
    H[:, 0] = W[5, 0] = 4.0
    H[:, first:] = W[5, first:] = 2.0 ** -12
    H[1::2] *= 0.5
    z = 16.0 + (d - first) * 2.0 ** -24
    z = np.where(np.arange(n) % 2, z / 2, z)
    o = outputs(n, 1, ALL)
    ws = torch.empty(dl.workspace_bytes(1, n, d, V), dtype=torch.uint8, device="cuda")
    rules = dl.LogitRules(1, n, V, bias=torch.zeros(V, device="cuda"))
    dl.debug_set_gemm_variant(variant)
    try:
        call(dl, False, H.bfloat16().cuda(), torch.ones(1, n, dtype=torch.uint8, device="cuda"),
             W.bfloat16().cuda(), rules, ALL, o, ws)
        assert dl.get_status() == 0
    finally:
        dl.debug_set_gemm_variant(0)
    lse = z + np.log1p((V - 1) * np.exp(-z))
    assert (o["tok"] == 5).all()
    assert np.abs(o["lse"].double().cpu().numpy() - lse).max() <= 2.0 ** -20 + 2.0 ** -21


@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("variant,n", [(1, 3), (2, 300)], ids=["single", "pair"])
def test_every_column_counts_once(dl, mx4, variant, n):
    """V equal logits: the sum of their exponentials is the number V, exactly, so conf is 1 / V to a
    rounding (a column lost or counted twice is a hundred of them) and the entropy ln V."""
    d, V = 64, 151937
    H, _, _ = head_inputs(1, n, d, 8, "all", seed=3)
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    o = outputs(n, 1, ALL)
    ws = torch.empty(max(dl.workspace_bytes(1, n, d, V), dl.workspace_bytes_mx4(1, n, d, V)),
                     dtype=torch.uint8, device="cuda")
    M = torch.ones(1, n, dtype=torch.uint8, device="cuda")
    for rules in ([None] if mx4 else []) + [dl.LogitRules(1, n, V, bias=torch.full((V,), 2.0, device="cuda"))]:
        dl.debug_set_gemm_variant(variant)
        try:
            call(dl, mx4, H.cuda(), M, dl.Mx4Matrix.quantize(W) if mx4 else W, rules, ALL, o, ws)
            assert dl.get_status() == 0
        finally:
            dl.debug_set_gemm_variant(0)
        assert (o["tok"] == 0).all() and (o["margin"] == 0).all()
        np.testing.assert_allclose(o["conf"].double().cpu().numpy(), 1 / V, rtol=2.0 ** -23)
        # ln V = 11.9: the logarithm's rounding (2^-22 of it at most) and one of the sum with 2
        np.testing.assert_allclose(o["entropy"].double().cpu().numpy(), np.log(V), rtol=2.0 ** -22)
        np.testing.assert_allclose(o["lse"].double().cpu().numpy(), np.log(V) + (2.0 if rules else 0.0),
                                   rtol=2.0 ** -22 + 2.0 ** -24)


@pytest.mark.parametrize("variant,n", [(1, 40), (2, 200)], ids=["single", "pair"])
@pytest.mark.parametrize("span", [(12, 0), (6, 6), (12, 12)], ids=["rows", "both", "wide"])
def test_mx4_sums_of_blocks_of_very_different_size(dl, span, variant, n):
    """Blocks of 32 channels whose scales lie up to 2^24 apart, in the rows, in W or in both (outlier
    channels): such sums do not fit fp32.  Each of the d / 64 tensor-core steps may then cut off the
    running sum's last place: dz <= d / 64 * 2^-23 * the largest running sum, and the statistics
    add what check counts."""
    d, V = 4096, 1030
    g = torch.Generator().manual_seed(n + span[1])
    H, W = torch.randn(n, d, generator=g), torch.randn(V, d, generator=g)
    for t, e in ((H, span[0]), (W, span[1])):
        t *= torch.exp2(torch.randint(-e, e + 1, (d // 32,), generator=g).float()).repeat_interleave(32)
    W = (W.double() * (20 / (H.double() @ W.double().T).abs().max())).bfloat16()
    H = H.bfloat16()
    h, w = dense(H, True), dense(W, True)
    z, largest = np.zeros((n, V)), np.zeros(n)
    for k in range(0, d, 64):
        z += h[:, k:k + 64] @ w[:, k:k + 64].T
        largest = np.maximum(largest, np.abs(z).max(-1))
    r = S.row_stats(z)
    dz = d // 64 * 2.0 ** -23 * largest
    r.update(pos=np.arange(n), z=z, dz=dz)
    o = outputs(n, 1, ALL)
    ws = torch.empty(dl.workspace_bytes_mx4(1, n, d, V), dtype=torch.uint8, device="cuda")
    dl.debug_set_gemm_variant(variant)
    try:
        call(dl, True, H.cuda(), torch.ones(1, n, dtype=torch.uint8, device="cuda"),
             dl.Mx4Matrix.quantize(W.cuda()), None, ALL, o, ws)
        assert dl.get_status() == 0
    finally:
        dl.debug_set_gemm_variant(0)
    check(o, r, 1, ALL)                              # V = 1: no allowance for a plain sum's roundings


# ---------------------------------------------------------------------------------------
# larger problems
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("B,L,d,V", [(2, 2600, 64, 6007),       # two groups of m-tiles, paced
                                     (1, 300, 2624, 700),       # K in four pieces of 11 stages
                                     (1, 20, 4160, 520)], ids=["rows", "d2624", "d4160"])
def test_larger_problems(dl, B, L, d, V, mx4):
    H, M, W = head_inputs(B, L, d, V, "all", seed=V)
    ref_rules, dev = make_rules(["penalty", "grammar", "bias"], B, L, V, seed=V)
    r = reference(H, M, W, mx4, ref_rules)
    o = outputs(B * L, B, ALL)
    nbytes = dl.workspace_bytes_mx4(B, L, d, V) if mx4 else dl.workspace_bytes(B, L, d, V)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    call(dl, mx4, H.cuda(), M.cuda(), dl.Mx4Matrix.quantize(W.cuda()) if mx4 else W.cuda(),
         dl.LogitRules(B, L, V, **dev), ALL, o, ws)
    assert dl.get_status() == 0 and int(o["count"][0]) == B * L
    check(o, r, V, ALL)


@pytest.mark.parametrize("weights", ["bf16", "mx4"])
@pytest.mark.parametrize("B,L", [(2, 40), (3, 3000)], ids=["staged", "compacted"])
def test_steps_that_follow_each_other_at_once(dl, weights, B, L):
    """Steps whose penalties read what the step before has just counted, queued without a pause and
    replayed from one graph: the selections of the same steps taken one at a time."""
    d, V, k, steps = 128, 5003, 8, 24
    H, M, W = head_inputs(B, L, d, V, "none", seed=4)
    M[:, 5:L:L // 30] = 1
    Hd, Md = H.cuda(), M.cuda()
    Wd = dl.Mx4Matrix.quantize(W.cuda()) if weights == "mx4" else W.cuda()
    counts, seen = i32(B, V), i32(B, (V + 31) // 32)
    pen = {n: torch.full((B,), v, device="cuda") for n, v in
           (("repetition", 1.2), ("presence", 0.3), ("frequency", 0.5))}
    rules = dl.LogitRules(B, L, V, counts=counts, seen=seen, **pen)
    step = dl.DecodeStep(B, L, d, V, k, weights=weights)

    def start():
        dl.token_counts(torch.empty(B, 0, dtype=torch.int32, device="cuda"), counts, seen)

    def once():
        step.run(Hd, Md, Wd, rules=rules)
        dl.token_counts(step.tok_sel, counts, seen, n_valid=step.n_sel, accumulate=True)

    start()
    want = []
    for _ in range(steps):
        step.run(Hd, Md, Wd, rules=rules)
        torch.cuda.synchronize()
        dl.token_counts(step.tok_sel, counts, seen, n_valid=step.n_sel, accumulate=True)
        torch.cuda.synchronize()
        want.append(step.sel_buf.clone())
    last = counts.clone()
    assert len({tuple(w.tolist()) for w in want}) > steps // 2     # the penalties do change them
    for _ in range(3):
        start()
        got = []
        for _ in range(steps):
            once()
            got.append(step.sel_buf.clone())
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(counts, last)
        start()
        for _ in range(steps):                       # nothing of another library between the kernels
            once()
        assert torch.equal(step.sel_buf, want[-1]) and torch.equal(counts, last)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            once()
    start()
    for _ in range(steps // 4):
        graph.replay()
    assert torch.equal(step.sel_buf, want[-1]) and torch.equal(counts, last)
    assert dl.get_status() == 0
