"""GPU checks of ls_process_logits against its definition in 64 bits: both
types, vocabularies from one entry up, rows at every alignment, histories of
every length, masks, biases, gathered rows, in-place calls, special values and
bad rows."""
import numpy as np
import pytest

import row_ops_ref as R

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


@pytest.fixture(autouse=True, params=[1, 2], ids=["one-kernel", "pair"])
def policy(request):
    """Every test runs with either choice of kernels forced."""
    import logits_sampling_gb300 as ls
    ls.set_process_policy(request.param)
    yield
    ls.set_process_policy(0)


def _i32(v):
    import torch
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def _f32(v):
    import torch
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda()


def _compare(got, x_rows, refs, dtype, where=""):
    """got: the call's rows; x_rows: the logits that each row read; refs: process_row's answers."""
    for i, (y, touched, tol) in enumerate(refs):
        g = got[i]
        same = ~touched
        assert np.array_equal(g[same].view(np.int32), x_rows[i][same].view(np.int32)), (where, i, "untouched entries")
        yt, gt, tt = y[touched], g[touched].astype(np.float64), tol[touched]
        fin = np.isfinite(yt)
        assert np.array_equal(gt[~fin], yt[~fin]), (where, i, "infinities")
        ok = R.within(gt[fin], yt[fin], tt[fin], dtype)
        assert ok.all(), (where, i, gt[fin][~ok][:4], yt[fin][~ok][:4])


def _case(rng, n, V, cap, dtype, bias=0, requests=None):
    requests = requests or n
    x = R.to_dtype(rng.standard_normal((n, V)) * 3, dtype)
    tokens = rng.integers(0, V, (requests, cap)).astype(np.int32)
    if cap:
        tokens[:, ::3] = tokens[:, :1]  # one id many times over
        tokens[rng.random((requests, cap)) < 0.05] = -1
        tokens[rng.random((requests, cap)) < 0.02] = V
    seq = rng.integers(0, cap + 1, requests).astype(np.int32)
    prompt = (seq * rng.random(requests)).astype(np.int32)
    c = {"x": x, "tokens": tokens, "seq": seq, "prompt": prompt,
         "rho": R.to_dtype(1 + rng.random(requests), "f32"), "pres": R.to_dtype(rng.random(requests), "f32"),
         "freq": R.to_dtype(rng.random(requests) * 0.5, "f32"), "biases": None}
    if bias:
        c["biases"] = [dict(zip(rng.permutation(V)[:min(bias, V)].tolist(),
                                R.to_dtype(rng.standard_normal(min(bias, V)) * 4, "f32").tolist()))
                       if r % 3 != 1 else {} for r in range(requests)]
    return c


def _params(c):
    import logits_sampling_gb300 as ls
    b = c["biases"]
    off = ids = val = None
    if b is not None:
        off = _i32(np.cumsum([0] + [len(d) for d in b]))
        ids = _i32([j for d in b for j in d])
        val = _f32([v for d in b for v in d.values()])
    return ls.LogitsParams(tokens=_i32(c["tokens"]), prompt_lens=_i32(c["prompt"]), seq_lens=_i32(c["seq"]),
                           repetition_penalty=_f32(c["rho"]), presence_penalty=_f32(c["pres"]),
                           frequency_penalty=_f32(c["freq"]), bias_offsets=off, bias_ids=ids, bias_values=val)


def _ref(c, row, request, length, allowed=None):
    return R.process_row(c["x"][row], c["tokens"][request][:length], c["prompt"][request], float(c["rho"][request]),
                         float(c["pres"][request]), float(c["freq"][request]),
                         c["biases"][request] if c["biases"] is not None else None, allowed)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,cap,bias,mask", [(1, 5, 1, True), (2, 0, 0, True), (31, 40, 3, True), (33, 200, 0, False),
                                             (1000, 300, 20, True), (4097, 3000, 300, False), (8191, 64, 5, True),
                                             (32003, 2000, 33, True), (128256, 5000, 16, True),
                                             (262144, 40000, 9, True)])
def test_against_the_definition(dtype, V, cap, bias, mask):
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(V + cap)
    n = 5 if V < 100000 else 3
    c = _case(rng, n, V, cap, dtype, bias)
    c["seq"][0] = cap  # a full history, and
    c["seq"][1] = 0    # none
    allowed = rng.random((n, V)) < rng.choice([0.01, 0.5, 0.99], (n, 1))
    index = np.arange(n, dtype=np.int32)
    index[-1] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ls.process_logits(R.device_matrix(c["x"], dtype), n, _params(c),
                            allowed_mask=_i32(R.pack_mask(allowed)) if mask else None,
                            mask_index=_i32(index) if mask else None, error_word=err)
    refs = [_ref(c, i, i, c["seq"][i], allowed[i] if mask and index[i] >= 0 else None) for i in range(n)]
    _compare(out.float().cpu().numpy(), c["x"], refs, dtype)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("in_off,in_pad,out_off,out_pad", [(0, 0, 0, 0), (1, 0, 0, 0), (3, 5, 3, 5), (7, 1, 2, 0),
                                                           (0, 3, 5, 7), (4, 4, 4, 4), (8, 8, 0, 8)])
def test_strides_and_alignments(dtype, in_off, in_pad, out_off, out_pad):
    """Rows of the input and of the output start at their own alignments; what
    lies between the output's rows keeps its values."""
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(in_off + 10 * out_off)
    n, V = 4, 9001
    c = _case(rng, n, V, 500, dtype, 20)
    allowed = rng.random((n, V)) < 0.5
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    whole = torch.full((n, out_off + V + out_pad), 7.0, dtype=t, device="cuda")
    out = whole[:, out_off:out_off + V]
    got = ls.process_logits(R.device_matrix(c["x"], dtype, in_off, in_pad), n, _params(c),
                            allowed_mask=_i32(R.pack_mask(allowed, 300)), out=out)
    assert got is out
    refs = [_ref(c, i, i, c["seq"][i], allowed[i]) for i in range(n)]
    _compare(out.float().cpu().numpy(), c["x"], refs, dtype)
    side = torch.cat([whole[:, :out_off], whole[:, out_off + V:]], 1)
    assert bool((side == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mask", [False, True])
def test_in_place(dtype, mask):
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(4)
    n, V = 6, 20011
    c = _case(rng, n, V, 700, dtype, 40)
    allowed = rng.random((n, V)) < 0.7
    words = _i32(R.pack_mask(allowed)) if mask else None
    x = R.device_matrix(c["x"], dtype, 3, 2)
    away = ls.process_logits(x, n, _params(c), allowed_mask=words)
    got = ls.process_logits(x, n, _params(c), allowed_mask=words, out=x)
    assert got is x
    assert np.array_equal(got.float().cpu().numpy(), away.float().cpu().numpy())
    refs = [_ref(c, i, i, c["seq"][i], allowed[i] if mask else None) for i in range(n)]
    _compare(got.float().cpu().numpy(), c["x"], refs, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_speculative_rows_gathered(dtype):
    """Rows of a request see one draft more each; rows come gathered out of a larger buffer."""
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(12)
    requests, per, V, cap = 7, 4, 5003, 90
    n = requests * per
    c = _case(rng, n + 9, V, cap, dtype, 6, requests)
    gather = rng.permutation(n + 9)[:n].astype(np.int32)
    t2r = np.repeat(np.arange(requests), per).astype(np.int32)
    lens = (rng.integers(0, cap - per, requests).repeat(per) + np.tile(np.arange(per), requests)).astype(np.int32)
    out = ls.process_logits(R.device_matrix(c["x"], dtype), n, _params(c), gather_indices=_i32(gather),
                            token_to_request_index=_i32(t2r), row_lens=_i32(lens))
    refs = [_ref(c, gather[i], t2r[i], lens[i]) for i in range(n)]
    _compare(out.float().cpu().numpy(), c["x"][gather], refs, dtype)


def test_parts_alone():
    """Each part of the parameters may be absent; a mask needs no parameters."""
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(1)
    n, V = 3, 3001
    c = _case(rng, n, V, 100, "f32", 10)
    x = R.device_matrix(c["x"], "f32")
    tok = {"tokens": _i32(c["tokens"]), "seq_lens": _i32(c["seq"])}
    for kw, ref in [
            ({"frequency_penalty": _f32(c["freq"])}, lambda i: dict(frequency=float(c["freq"][i]))),
            ({"presence_penalty": _f32(c["pres"])}, lambda i: dict(presence=float(c["pres"][i]))),
            ({"repetition_penalty": _f32(c["rho"])}, lambda i: dict(rho=float(c["rho"][i])))]:
        out = ls.process_logits(x, n, ls.LogitsParams(**tok, **kw))
        refs = [R.process_row(c["x"][i], c["tokens"][i][:c["seq"][i]], 0, **ref(i)) for i in range(n)]
        _compare(out.cpu().numpy(), c["x"], refs, "f32", str(list(kw)))
    only_bias = ls.LogitsParams.from_host(biases=c["biases"])
    refs = [R.process_row(c["x"][i], bias=c["biases"][i]) for i in range(n)]
    _compare(ls.process_logits(x, n, only_bias).cpu().numpy(), c["x"], refs, "f32", "bias")
    allowed = rng.random((2, V)) < 0.5
    out = ls.process_logits(x, n, allowed_mask=_i32(R.pack_mask(allowed)), mask_index=_i32([1, -1, 1]))
    refs = [R.process_row(c["x"][i], allowed=allowed[1] if i != 1 else None) for i in range(n)]
    _compare(out.cpu().numpy(), c["x"], refs, "f32", "mask")
    assert np.array_equal(ls.process_logits(x, n).cpu().numpy(), c["x"])
    assert ls.process_logits(x, 0).shape == (0, V)


def test_from_host_defaults_to_prompts():
    import logits_sampling_gb300 as ls
    p = ls.LogitsParams.from_host(histories=[[1, 2], [], [5]], capacity=9, frequency_penalty=[1, 1, 1])
    assert p.tokens.shape == (3, 9) and p.seq_lens.tolist() == [2, 0, 1] and p.prompt_lens.tolist() == [2, 0, 1]


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_values(dtype):
    """Infinities and NaN in touched, untouched and masked places, and the type's
    lowest value."""
    import torch
    import logits_sampling_gb300 as ls
    V = 300
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    vals = [np.inf, -np.inf, np.nan, low, 0.0, -0.0, 1e-40, 2.0]
    x = np.zeros((1, V), np.float32)
    x[0, :8] = vals          # in the history
    x[0, 100:108] = vals     # untouched
    x[0, 200:208] = vals     # masked
    x[0, 220:228] = vals     # bias +inf
    x[0, 240:248] = vals     # bias -inf
    x[0, 260:268] = vals     # bias NaN
    x = R.to_dtype(x, dtype)
    hist = list(range(8)) + list(range(200, 208))
    bias = {**{j: np.inf for j in range(220, 228)}, **{j: -np.inf for j in range(240, 248)},
            **{j: np.nan for j in range(260, 268)}}
    allowed = np.ones((1, V), bool)
    allowed[0, 200:208] = False
    p = ls.LogitsParams.from_host(histories=[hist], prompt_lens=[4], repetition_penalty=[2.0],
                                  presence_penalty=[0.5], frequency_penalty=[0.25], biases=[bias])
    out = ls.process_logits(R.device_matrix(x, dtype), 1, p, allowed_mask=_i32(R.pack_mask(allowed)))
    ref = R.process_row(x[0], hist, 4, 2.0, 0.5, 0.25, bias, allowed[0])
    got = out.float().cpu().numpy()
    _compare(got, x, [ref], dtype)
    assert np.isneginf(got[0, 260:268]).all() and np.isneginf(got[0, 2])


def test_mask_that_allows_nothing_leaves_no_token():
    import torch
    import logits_sampling_gb300 as ls
    x = torch.randn(3, 1000, device="cuda")
    out = ls.process_logits(x, allowed_mask=torch.zeros((3, 32), dtype=torch.int32, device="cuda"))
    assert bool(torch.isneginf(out).all())
    prm = ls.SamplingParams.from_host([1.0] * 3, [0] * 3, [1.0] * 3, [0] * 3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert ls.sample(out, 3, prm, 0, True, True, error_word=err).tolist() == [-1] * 3
    assert int(err.item()) == ls.LS_ROW_ERR_NO_FINITE


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_rows(dtype):
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(3)
    n, V = 6, 9000
    c = _case(rng, n, V, 50, dtype, 0)
    x = R.device_matrix(c["x"], dtype)
    allowed = np.ones((n, V), bool)
    for kw, bit in [({"gather_indices": _i32([0, 1, 6, -1, 4, 5])}, ls.LS_ROW_ERR_BAD_GATHER),
                    ({"token_to_request_index": _i32([0, 1, 6, -1, 4, 5])}, ls.LS_ROW_ERR_BAD_REQUEST),
                    ({"allowed_mask": _i32(R.pack_mask(allowed)), "mask_index": _i32([0, 1, 6, -2, 4, 5])},
                     ls.LS_ROW_ERR_BAD_MASK)]:
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = ls.process_logits(x, n, _params(c), error_word=err, **kw).float().cpu().numpy()
        assert int(err.item()) == bit
        assert np.isnan(out[2:4]).all()
        refs = [_ref(c, i, i, c["seq"][i]) for i in (0, 1, 4, 5)]
        _compare(out[[0, 1, 4, 5]], c["x"][[0, 1, 4, 5]], refs, dtype)


def test_lengths_beyond_the_buffer_are_clamped():
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(8)
    c = _case(rng, 3, 500, 20, "f32")
    c["seq"][:] = [1000, -5, 20]
    out = ls.process_logits(R.device_matrix(c["x"], "f32"), 3, _params(c))
    refs = [_ref(c, i, i, (20, 0, 20)[i]) for i in range(3)]
    _compare(out.cpu().numpy(), c["x"], refs, "f32")


def test_bias_offsets_outside_the_list_are_clamped():
    import logits_sampling_gb300 as ls
    V = 500
    x = R.to_dtype(np.random.default_rng(3).standard_normal((5, V)), "f32")
    # row 0 begins past the list, 1 is empty, 2 ends before it begins, 3 is the whole list, 4 is empty
    off = _i32([0x7FFFFFF0, 3, 3, -5, 1000, 3])
    ids, val = [7, 499, 250], [1.0, -2.0, 0.5]
    got = ls.process_logits(R.device_matrix(x, "f32"), 5,
                            ls.LogitsParams(bias_offsets=off, bias_ids=_i32(ids), bias_values=_f32(val))).cpu().numpy()
    want = x.copy()
    want[3, ids] += np.array(val, np.float32)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("cap", [32000, 70000])
def test_one_id_repeated_through_a_long_history(cap):
    """Counts past 16 bits."""
    import logits_sampling_gb300 as ls
    V = 2000
    x = R.to_dtype(np.random.default_rng(0).standard_normal((1, V)), "f32")
    c = {"x": x, "tokens": np.full((1, cap), 77, np.int32), "seq": [cap], "prompt": [1], "rho": [1.5], "pres": [0.1],
         "freq": [0.01], "biases": None}
    out = ls.process_logits(R.device_matrix(x, "f32"), 1, _params(c))
    _compare(out.cpu().numpy(), x, [_ref(c, 0, 0, cap)], "f32")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cap", [3000, 9000, 30000, 33000])
def test_many_distinct_ids(dtype, cap):
    """Histories of mostly distinct ids in a batch large enough that a CTA takes a long run of the row."""
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(cap)
    n, V = 640, 33000
    x = R.to_dtype(rng.standard_normal((1, V)), dtype)
    tokens = np.stack([rng.permutation(V)[:cap] for _ in range(2)]).astype(np.int32)
    bias = {int(j): float(np.float32(v)) for j, v in zip(rng.permutation(V)[:300], rng.standard_normal(300))}
    c = {"x": x, "tokens": tokens, "seq": np.array([cap, cap // 2]), "prompt": np.array([100, cap]), "rho": [1.5, 1.25],
         "pres": [0.1, 0.2], "freq": [0.01, 0.3], "biases": [bias, {}]}
    t2r = np.arange(n) % 2
    allowed = rng.random((1, V)) < 0.8
    out = ls.process_logits(R.device_matrix(x, dtype), n, _params(c), gather_indices=_i32(np.zeros(n)),
                            token_to_request_index=_i32(t2r), allowed_mask=_i32(R.pack_mask(allowed)),
                            mask_index=_i32(np.where(np.arange(n) < 4, 0, -1)))
    got = out[[0, 1, n - 2, n - 1]].float().cpu().numpy()
    refs = [_ref(c, 0, r, c["seq"][r], m) for m in (allowed[0], None) for r in (0, 1)]
    _compare(got, np.repeat(x, 4, 0), refs, dtype)
    assert bool((out[4:] == out[4:6].repeat(n // 2 - 2, 1)).all())


def test_offsets_past_32_bits():
    """A logits matrix of more than 2^32 entries: its last rows, gathered."""
    import torch
    import logits_sampling_gb300 as ls
    V, rows = 262144, 16640
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, V, device="cuda").to(torch.bfloat16)
    host = x[-3:].float().cpu().numpy()
    rng = np.random.default_rng(2)
    c = _case(rng, 3, V, 100, "bf16")
    c["x"] = host
    out = ls.process_logits(x, 3, _params(c), gather_indices=_i32([rows - 3, rows - 2, rows - 1]))
    _compare(out.float().cpu().numpy(), host, [_ref(c, i, i, c["seq"][i]) for i in range(3)], "bf16")
    del out
    p = ls.LogitsParams.from_host(biases=[{V - 1: 1.5}])
    t2r = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ls.process_logits(x, rows, p, token_to_request_index=t2r, out=x)
    got = x[-3:].float().cpu().numpy()
    _compare(got, host, [R.process_row(h, bias={V - 1: 1.5}) for h in host], "bf16")


def test_the_choice_by_batch_size_changes_nothing():
    import torch
    import logits_sampling_gb300 as ls
    x = (torch.randn(400, 128256, device="cuda") * 3).to(torch.bfloat16)
    hist = torch.randint(0, 128256, (400, 50), dtype=torch.int32, device="cuda")
    ones = torch.ones(400, device="cuda")
    p = ls.LogitsParams(tokens=hist, seq_lens=(ones * 50).int(), repetition_penalty=ones * 1.25, frequency_penalty=ones)
    forced = ls.process_logits(x, 400, p)
    ls.set_process_policy(0)
    assert torch.equal(ls.process_logits(x, 400, p), forced)
    assert torch.equal(ls.process_logits(x[:3], 3, ls.LogitsParams(
        tokens=hist[:3], seq_lens=(ones[:3] * 50).int(), repetition_penalty=ones[:3] * 1.25,
        frequency_penalty=ones[:3])), forced[:3])


def test_on_another_stream_and_in_a_graph():
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(5)
    c = _case(rng, 4, 8000, 100, "bf16", 8)
    x, p = R.device_matrix(c["x"], "bf16"), _params(c)
    ref = ls.process_logits(x, 4, p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = ls.process_logits(x, 4, p, stream=s)
    s.synchronize()
    assert torch.equal(a, ref)
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ls.process_logits(x, 4, p, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
