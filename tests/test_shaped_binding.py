"""Rules on logits and MXFP4 without a GPU: what the binding refuses before it calls the library,
the arity of each wrapper, and the library's own host-side validation."""
import ctypes

import numpy as np
import pytest
import torch

import mask_only_logits_b200 as dl
from mask_only_logits_b200 import _abi, build
from test_binding import FakeLib, S, f32, fake, i32  # noqa: F401  (fake: the fixture)

B, L, d, V = 2, 40, 64, 100
N, WORDS = B * L, 4


def tables():
    return dict(bias=torch.zeros(B, V), counts=torch.zeros(B, V, dtype=torch.int32),
                seen=torch.zeros(B, WORDS, dtype=torch.int32), repetition=f32(B), presence=f32(B),
                frequency=f32(B), allow=torch.zeros(3, WORDS, dtype=torch.int32),
                allow_id=torch.zeros(B, L, dtype=torch.int32))


def bufs():
    return dict(H=torch.zeros(N, d, dtype=torch.bfloat16), M=torch.zeros(B, L, dtype=torch.uint8),
                W=torch.zeros(V, d, dtype=torch.bfloat16), tok=i32(N), conf=f32(N), lse=f32(N),
                ent=f32(N), mar=f32(N), row_idx=i32(N), seq_off=i32(B + 1), count=i32(4), lo=i32(B),
                hi=i32(B), ws=torch.zeros(64, dtype=torch.uint8),
                q=torch.zeros(V, d // 2, dtype=torch.uint8), s=torch.zeros(512, dtype=torch.uint8))


def logits(b, mx4, rules):
    out = (3, b["tok"], b["conf"], b["lse"], b["ent"], b["mar"], b["row_idx"], b["seq_off"], b["count"],
           b["ws"], S, b["lo"], b["hi"])
    if mx4:
        dl.masked_logits_mx4(b["H"], b["M"], dl.Mx4Matrix(b["q"], b["s"]), rules, *out)
    else:
        dl.masked_logits_rules(b["H"], b["M"], b["W"], rules, *out)


@pytest.mark.parametrize("mx4", [False, True])
def test_logits_arity_and_sizes(fake, mx4):                              # noqa: F811
    rules = dl.LogitRules(B, L, V, **tables())
    logits(bufs(), mx4, rules)
    assert fake.calls == ["dllm_masked_logits_mx4" if mx4 else "dllm_masked_logits_rules"]
    if mx4:
        logits(bufs(), mx4, None)
        fake.calls.pop()
    for key in ("H", "tok", "conf", "lse", "ent", "mar", "row_idx", "seq_off", "lo", "hi"):
        b = bufs()
        b[key] = b[key].reshape(-1)[:-1]
        with pytest.raises(ValueError, match="needs at least"):
            logits(b, mx4, rules)
    with pytest.raises(ValueError, match="rules: made for"):
        logits(bufs(), mx4, dl.LogitRules(B, L, V + 1, bias=torch.zeros(V + 1)))
    assert len(fake.calls) == 1


def test_rules_describe_their_tensors(fake):                             # noqa: F811
    t = tables()
    t["bias"] = torch.zeros(B, 112)[:, :V]
    t["counts"] = torch.zeros(B, V + 5, dtype=torch.int32)[:, :V]
    r = dl.LogitRules(B, L, V, **t)._struct
    assert (r.bias, r.bias_stride, r.counts_stride, r.seen_stride) == (t["bias"].data_ptr(), 112, V + 5, WORDS)
    assert (r.allow_stride, r.allow_rows, r.allow_id) == (WORDS, 3, t["allow_id"].data_ptr())
    assert r.repetition == t["repetition"].data_ptr()
    shared = dl.LogitRules(B, L, V, bias=torch.zeros(V))._struct
    assert shared.bias_stride == 0 and shared.counts is None and shared.allow is None


@pytest.mark.parametrize("change,text", [
    (dict(seen=None), "go together"),
    (dict(counts=None), "go together"),
    (dict(counts=None, seen=None), "penalties need counts"),
    (dict(allow=None), "allow_id needs allow"),
    (dict(allow_id=None), "need allow_id"),
    (dict(allow_id=torch.zeros(B, L - 1, dtype=torch.int32)), "needs at least"),
    (dict(allow=torch.zeros(3, WORDS - 1, dtype=torch.int32)), "expected at least"),
    (dict(allow=torch.zeros(3, WORDS, dtype=torch.int64)), "expected torch.int32"),
    (dict(bias=torch.zeros(B, V - 1)), "expected at least"),
    (dict(bias=torch.zeros(B, V, dtype=torch.bfloat16)), "expected torch.float32"),
    (dict(bias=torch.zeros(B, V + 2)[:, :V]), "multiple of 4"),
    (dict(bias=torch.zeros(V, B).t()), "contiguous rows"),
    (dict(bias=torch.zeros(1, V).expand(B, V)), "overlap"),
    (dict(counts=torch.zeros(B - 1, V, dtype=torch.int32)), "expected at least"),
    (dict(repetition=f32(B - 1)), "needs at least"),
    (dict(presence=f32(B).double()), "expected torch.float32"),
])
def test_rules_refuse(fake, change, text):                               # noqa: F811
    with pytest.raises(ValueError, match=text):
        dl.LogitRules(B, L, V, **dict(tables(), **change))


def test_counts_and_mx4_arity_and_refusals(fake):                        # noqa: F811
    tokens, counts, seen = (torch.zeros(B, 7, dtype=torch.int32), torch.zeros(B, V, dtype=torch.int32),
                            torch.zeros(B, WORDS, dtype=torch.int32))
    dl.token_counts(tokens, counts, seen, M=torch.zeros(B, 7, dtype=torch.uint8), n_valid=i32(B),
                    accumulate=True, stream=S)
    for bad in (dict(counts=counts[:1]), dict(seen=seen[:, :-1]), dict(seen=seen.long()),
                dict(M=torch.zeros(B, 6, dtype=torch.uint8)), dict(n_valid=i32(1)),
                dict(tokens=tokens.long())):
        a = dict(dict(tokens=tokens, counts=counts, seen=seen), **bad)
        with pytest.raises(ValueError):
            dl.token_counts(stream=S, **a)
    X = torch.zeros(130, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(130, 32, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8)
    dl.mx4_quantize(X, q, s, S)
    dl.mx4_dequantize(q, s, X, S)
    with pytest.raises(ValueError, match="multiple of 32"):
        dl.mx4_quantize(X[:, :40], q, s, S)
    with pytest.raises(ValueError, match="s: needs at least"):
        dl.mx4_quantize(X, q, s[:-1], S)
    with pytest.raises(ValueError, match="q: needs at least"):
        dl.mx4_dequantize(q[:-1], s, X, S)
    with pytest.raises(ValueError, match="expected"):
        dl.mx4_dequantize(q, s, X.half(), S)
    with pytest.raises(ValueError, match="q: expected uint8"):
        dl.Mx4Matrix(q.int(), s)
    with pytest.raises(ValueError, match="s: expected uint8"):
        dl.Mx4Matrix(q, s[:-1])
    assert fake.calls == ["dllm_token_counts", "dllm_mx4_quantize", "dllm_mx4_dequantize"]


def test_scale_tiles_round_trip():
    """The tile order written out: byte of (row, block) as the header gives it."""
    R, K = 131, 160
    g = np.random.default_rng(0).integers(0, 256, (R, K // 32)).astype(np.uint8)
    s = dl.mx4_tile_scales(torch.from_numpy(g))
    assert s.numel() == 2 * 2 * 512
    for r, j in [(0, 0), (31, 1), (32, 2), (127, 3), (128, 4), (130, 0), (77, 4)]:
        at = ((r // 128) * 2 + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4
        assert int(s[at]) == g[r, j]
    assert torch.equal(dl.mx4_row_scales(s, R, K), torch.from_numpy(g))


def test_decode_step_takes_the_weights_it_was_made_for(fake):            # noqa: F811
    fake.dllm_workspace_bytes_mx4 = lambda *a: 4096
    W, Q = torch.zeros(V, d, dtype=torch.bfloat16), dl.Mx4Matrix(bufs()["q"], bufs()["s"])
    H, M = bufs()["H"], bufs()["M"]
    step = dl.DecodeStep(B, L, d, V, 4, device="cpu", weights="mx4")
    step.run(H, M, Q, stream=S)
    assert fake.calls == ["dllm_masked_logits_mx4", "dllm_select_unmask"]
    with pytest.raises(ValueError, match="Mx4Matrix"):
        step.run(H, M, W, stream=S)
    with pytest.raises(ValueError, match="Mx4Matrix"):
        dl.DecodeStep(B, L, d, V, 4, device="cpu").run(H, M, Q, stream=S)
    with pytest.raises(ValueError, match="weights must be"):
        dl.DecodeStep(B, L, d, V, 4, device="cpu", weights="fp8")
    with pytest.raises(RuntimeError, match="overlapped"):
        step._double()
    with pytest.raises(ValueError, match="expected shape"):
        step.run(H, M[:, :-1], Q, stream=S)


# ---------------------------------------------------------------------------------------
# the library's own validation (no CUDA call is reached)
# ---------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def _p(x):
    return ctypes.c_void_p(x)


A = 1 << 20
NUL = _p(None)


def c_rules(**kw):
    r = _abi.LogitRulesStruct()
    for k, v in kw.items():
        setattr(r, k, v)
    return ctypes.byref(r)


@pytest.mark.parametrize("kw,status", [
    (dict(counts=A, counts_stride=4096), -1),
    (dict(seen=A, seen_stride=128), -1),
    (dict(repetition=A), -1),
    (dict(allow_id=A), -1),
    (dict(bias=A + 4), -2),
    (dict(allow=A + 8, allow_rows=1, allow_stride=128), -2),
    (dict(bias=A, bias_stride=4000), -3),
    (dict(bias=A, bias_stride=4098), -3),
    (dict(counts=A, seen=A, counts_stride=4095, seen_stride=128), -3),
    (dict(counts=A, seen=A, counts_stride=4096, seen_stride=127), -3),
    (dict(allow=A, allow_rows=0, allow_stride=128), -3),
    (dict(allow=A, allow_rows=3, allow_stride=128), -3),
    (dict(allow=A, allow_rows=2, allow_stride=127), -3),
    (dict(allow=A, allow_rows=2, allow_stride=128), -4),      # fits: the workspace is looked at next
    (dict(bias=A), -4),
])
def test_rules_validate_on_host(lib, kw, status):
    ins = [_p(A), _p(A), _p(A), 2, 256, 256, 4096, NUL, NUL]
    outs = [_p(A), _p(A), _p(A), NUL, NUL, _p(A), _p(A), _p(A), _p(A), 10, NUL]
    assert lib.dllm_masked_logits_rules(*ins, c_rules(**kw), 0, *outs) == status
    mx = [_p(A), _p(A), _p(A), _p(A), 2, 256, 256, 4096, NUL, NUL]
    assert lib.dllm_masked_logits_mx4(*mx, c_rules(**kw), 0, *outs) == status


def test_other_entry_points_validate_on_host(lib):
    ins = [_p(A), _p(A), _p(A), 1, 256, 256, 4096]
    outs = [_p(A), _p(A), _p(A), NUL, NUL, _p(A), _p(A), _p(A), _p(A), 1 << 30, NUL]
    call = lib.dllm_masked_logits_rules
    assert call(*ins, NUL, NUL, None, 0, *outs) == -1                     # rules are required here
    assert call(*ins, _p(A), NUL, c_rules(), 0, *outs) == -1
    assert call(*ins, NUL, NUL, c_rules(), 1, *outs) == -1                # entropy asked for, not given
    assert call(*ins, NUL, NUL, c_rules(), 8, *outs) == -3
    bad = list(ins)
    bad[5] = 100
    assert call(*bad, NUL, NUL, c_rules(), 0, *outs) == -3
    mx = lib.dllm_masked_logits_mx4
    assert mx(_p(A), _p(A), NUL, _p(A), *ins[3:], NUL, NUL, None, 0, *outs) == -1
    assert mx(_p(A), _p(A), _p(A), _p(A + 4), *ins[3:], NUL, NUL, None, 0, *outs) == -2
    tc = lib.dllm_token_counts
    assert tc(NUL, NUL, NUL, 1, 5, 10, 0, _p(A), _p(A), NUL) == -1
    assert tc(_p(A), NUL, NUL, 0, 5, 10, 0, _p(A), _p(A), NUL) == -3
    assert tc(_p(A), NUL, NUL, 65536, 5, 10, 0, _p(A), _p(A), NUL) == -3
    assert tc(_p(A), NUL, NUL, 1, -1, 10, 0, _p(A), _p(A), NUL) == -3
    assert tc(_p(A), NUL, NUL, 1, 5, 10, 2, _p(A), _p(A), NUL) == -3
    assert tc(_p(A + 4), NUL, NUL, 1, 5, 10, 0, _p(A), _p(A), NUL) == -2
    q, dq = lib.dllm_mx4_quantize, lib.dllm_mx4_dequantize
    assert q(NUL, 0, 4, 64, 64, _p(A), _p(A), NUL) == -1
    assert q(_p(A), 3, 4, 64, 64, _p(A), _p(A), NUL) == -3
    assert q(_p(A), 0, 4, 48, 64, _p(A), _p(A), NUL) == -3
    assert q(_p(A), 0, 0, 64, 64, _p(A), _p(A), NUL) == -3
    assert q(_p(A), 0, 4, 64, 32, _p(A), _p(A), NUL) == -3
    assert q(_p(A), 0, 4, 64, 68, _p(A), _p(A), NUL) == -2
    assert q(_p(A + 8), 2, 4, 64, 68, _p(A), _p(A), NUL) == -2
    assert dq(_p(A), _p(A), 4, 64, 1, _p(A), 64, NUL) == -3
    assert lib.dllm_mx4_scale_bytes(1, 32) == 512 and lib.dllm_mx4_scale_bytes(129, 160) == 2048
    assert lib.dllm_mx4_scale_bytes(0, 32) == 0 and lib.dllm_mx4_scale_bytes(5, 33) == 0


def test_mx4_workspace_arithmetic(lib):
    size, cap = lib.dllm_workspace_bytes_mx4, lib.dllm_workspace_rows_mx4
    for b, l, dd, v in [(1, 4096, 4096, 126464), (3, 97, 192, 777)]:
        prev = 0
        for r in (1, 2, 127, 128, 129, b * l - 1, b * l, 10 * b * l):
            n = size(b, l, dd, v, r)
            assert n >= prev and n >= min(r, b * l) * dd // 2
            prev = n
            assert cap(b, l, dd, v, n) >= min(r, b * l)
        assert cap(b, l, dd, v, size(b, l, dd, v, 1) - 1) == 0
        assert cap(b, l, dd, v, 1 << 60) == b * l
    assert size(1, 8, 100, 10, 1) == 0 and size(1, 8, 64, 10, 0) == 0 and cap(1, 8, 100, 10, 1 << 20) == 0


def test_mx4_matrix_on_another_stream_owns_its_buffers(fake, monkeypatch):   # noqa: F811
    """Buffers that a call on `stream` makes come from that stream's memory and stay allocated for
    the current stream too; what it reads stays allocated until `stream` is done."""
    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

        def __enter__(self):
            active.append(self)

        def __exit__(self, *_):
            active.pop()

    here, side = Stream(1), Stream(2)
    active, made, kept = [here], [], []
    empty = torch.empty

    def logged_empty(*a, **kw):
        t = empty(*a, **kw)
        made.append((t.data_ptr(), active[-1]))
        return t

    monkeypatch.setattr(torch, "empty", logged_empty)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.data_ptr(), s)))
    X = torch.zeros(130, 64, dtype=torch.bfloat16)
    W = dl.Mx4Matrix.quantize(X, stream=side)
    q, s = W.q.data_ptr(), W.s.data_ptr()
    assert made == [(q, side), (s, side)]
    assert set(kept) == {(X.data_ptr(), side), (q, here), (s, here)}
    made.clear()
    kept.clear()
    Y = W.dequantize(stream=side)
    assert made == [(Y.data_ptr(), side)]
    assert set(kept) == {(q, side), (s, side), (Y.data_ptr(), here)}
    assert fake.calls == ["dllm_mx4_quantize", "dllm_mx4_dequantize"] and active == [here]


def test_each_captured_graph_keeps_what_it_reads(fake, monkeypatch):      # noqa: F811
    """Two captures of one step: the first graph still holds its own rules and tensors."""
    import contextlib
    import gc
    import weakref

    class Stream:
        cuda_stream = 1

        def wait_stream(self, other):
            pass

    class Graph:
        pass

    monkeypatch.setattr(torch.cuda, "Stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "graph", lambda g, **kw: contextlib.nullcontext())
    b = bufs()
    step = dl.DecodeStep(B, L, d, V, 4, device="cpu")
    bias = [torch.zeros(V), torch.zeros(V)]
    refs = [weakref.ref(t) for t in bias]
    graphs = [step.capture(b["H"], b["M"], b["W"], rules=dl.LogitRules(B, L, V, bias=t)) for t in bias]
    del bias
    gc.collect()
    assert all(r() is not None for r in refs)
    del graphs[0]
    gc.collect()
    assert refs[0]() is None and refs[1]() is not None    # and no longer than that


def test_rows_of_another_length_are_refused(fake):                       # noqa: F811
    """A mask or a table of positions with longer rows holds enough elements, but not in the rows
    that the kernels read; flat ones are taken as they are."""
    tokens, counts, seen = (torch.zeros(B, 7, dtype=torch.int32), torch.zeros(B, V, dtype=torch.int32),
                            torch.zeros(B, WORDS, dtype=torch.int32))
    with pytest.raises(ValueError, match="M: expected rows of 7"):
        dl.token_counts(tokens, counts, seen, M=torch.zeros(B, 8, dtype=torch.uint8), stream=S)
    with pytest.raises(ValueError, match="allow_id: expected rows of 40"):
        dl.LogitRules(B, L, V, **dict(tables(), allow_id=torch.zeros(B, L + 1, dtype=torch.int32)))
    assert fake.calls == []
    dl.token_counts(tokens, counts, seen, M=torch.zeros(B * 7, dtype=torch.uint8), stream=S)
    dl.LogitRules(B, L, V, **dict(tables(), allow_id=torch.zeros(N, dtype=torch.int32)))


def test_block_only_needs_its_windows(fake):                             # noqa: F811
    """Without them the step would compute every masked row."""
    fake.dllm_workspace_bytes_mx4 = lambda *a: 4096
    b = bufs()
    rules = dl.LogitRules(B, L, V, bias=torch.zeros(V))
    for step, W, kw in ((dl.DecodeStep(B, L, d, V, 4, device="cpu"), b["W"], dict(rules=rules)),
                        (dl.DecodeStep(B, L, d, V, 4, device="cpu", weights="mx4"), dl.Mx4Matrix(b["q"], b["s"]), {})):
        for win in ((None, None), (b["lo"], None), (None, b["hi"])):
            with pytest.raises(ValueError, match="block_only=True needs"):
                step.run(b["H"], b["M"], W, *win, stream=S, block_only=True, **kw)
        assert fake.calls == []
        step.run(b["H"], b["M"], W, b["lo"], b["hi"], stream=S, block_only=True, **kw)
        fake.calls.clear()


def test_scale_tiles_take_bytes_or_e8m0():
    """A checkpoint's scales as torch's E8M0 numbers are the same bytes, not their values rounded to
    integers; other types are refused."""
    g = torch.arange(3 * 5, dtype=torch.uint8).view(3, 5) * 17
    want = dl.mx4_tile_scales(g)
    assert torch.equal(dl.mx4_tile_scales(g.view(torch.float8_e8m0fnu)), want)
    assert torch.equal(dl.mx4_row_scales(want, 3, 160), g)
    for t in (torch.int8, torch.int32, torch.float32):
        with pytest.raises(ValueError, match="scales: expected"):
            dl.mx4_tile_scales(g.to(t))
