"""arcs_adjust_logits against the definition.

The penalties and the biases are sequences of binary32 operations, the same as numpy's
float32 ones in the same order, so results are compared bit for bit (-0 and +0 as they come).
"""

import numpy as np
import pytest

from _util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, V, dtype, seed, hist=0, bias=0, masks=None, odd_ids=True):
    """Host lists and the device tensors of a call.  Rows have lists of different lengths, some
    empty, with ids outside the vocabulary and ids that come several times."""
    import torch
    from workloads import make_params
    rng = np.random.default_rng(seed)
    c = dict(B=B, V=V)
    logits = torch.from_numpy((3 * rng.standard_normal((B, V))).astype(np.float32)).to(types()[dtype])
    c["z"] = logits.float().numpy()
    c["logits"] = logits.cuda()
    off = rng.random(B) < 0.2
    params = make_params(B, temperature=0.7, presence=np.where(off, 0, 0.5).astype(np.float32),
                         frequency=np.where(off, 0, rng.uniform(-0.2, 0.6, B)).astype(np.float32),
                         repetition=np.where(off, rng.choice([0.0, 1.0], B), rng.uniform(0.8, 1.5, B)).astype(np.float32))
    c["p"] = params
    import decode_step_token_row_amd as arcs
    c["params"] = arcs.params_to_device(params)

    def lists(most):
        lengths = rng.integers(0, most + 1, B)
        lengths[rng.random(B) < 0.2] = 0
        lengths[rng.integers(0, B)] = most
        ids = [(rng.random(n) ** 3 * (V + (4 if odd_ids else 0))).astype(np.int32) - (2 if odd_ids else 0) for n in lengths]
        if odd_ids and most > 2:
            ids[int(np.argmax(lengths))][:2] = (-2**31, 2**31 - 1)
        return ids

    c["hist"] = lists(hist) if hist else None
    c["bias"] = lists(bias) if bias else None
    c["values"] = [rng.standard_normal(len(x)).astype(np.float32) for x in c["bias"]] if bias else None

    def csr(x):
        return torch.from_numpy(np.concatenate([[0], np.cumsum([len(i) for i in x])]).astype(np.int64)).cuda()

    c["args"] = dict(params=c["params"])
    if hist:
        c["args"].update(hist_ids=torch.from_numpy(np.concatenate(c["hist"])).cuda(), hist_offsets=csr(c["hist"]))
    if bias:
        c["args"].update(bias_ids=torch.from_numpy(np.concatenate(c["bias"])).cuda(), bias_offsets=csr(c["bias"]),
                         bias_values=torch.from_numpy(np.concatenate(c["values"])).cuda())
    c["rows"] = np.full(B, -1)
    if masks is not None:
        words = (V + 31) // 32
        density = rng.choice([0.0, 0.001, 0.5, 0.99, 1.0], masks)
        bits = rng.random((masks, words * 32)) < density[:, None]
        c["bits"] = bits[:, :V]
        packed = np.packbits(bits.reshape(masks, words, 32), axis=2, bitorder="little").reshape(masks, words * 4).view(np.int32)
        c["args"]["mask"] = torch.from_numpy(np.ascontiguousarray(packed)).cuda()
        c["rows"] = rng.integers(-1, masks, B)
        c["args"]["mask_rows"] = torch.from_numpy(c["rows"].astype(np.int32)).cuda()
    return c


def reference(c):
    f = np.float32
    y = c["z"].copy()
    status = np.zeros(c["B"], np.int32)
    with np.errstate(all="ignore"):
        for b in range(c["B"]):
            p = c["p"][b]
            rep = f(1) if p["repetition"] in (0, 1) else p["repetition"]
            if c["hist"] is not None and (rep != 1 or p["frequency"] != 0 or p["presence"] != 0):
                ids, n = np.unique(c["hist"][b], return_counts=True)
                ok = (ids >= 0) & (ids < c["V"])
                ids, n = ids[ok], n[ok]
                z = y[b, ids]
                z = np.where(z > 0, z / rep, z * rep).astype(f)
                z = (z - (p["frequency"] * n.astype(f)).astype(f)).astype(f)
                y[b, ids] = (z - p["presence"]).astype(f)
            if c["bias"] is not None:
                total = {}
                for i, v in zip(c["bias"][b].tolist(), c["values"][b]):
                    if 0 <= i < c["V"]:
                        total[i] = f(total[i] + v) if i in total else v
                for i, v in total.items():
                    y[b, i] = f(y[b, i] + v)
            if c["rows"][b] >= 0:
                allowed = c["bits"][c["rows"][b]]
                y[b, ~allowed] = -np.inf
                if not allowed.any():
                    status[b] = 10
    return y, status


def same(got, want):
    """Bit for bit, -0 and +0 apart from each other, NaN equal to NaN."""
    import torch
    want = torch.from_numpy(want).to(got.dtype)
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    bits = torch.int16 if got.element_size() == 2 else torch.int32
    ok = ~want.isnan()
    assert torch.equal(got[ok].view(bits), want[ok].view(bits))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,V,hist,bias,masks", [
    (1, 1, 3, 2, 1), (1, 31, 0, 0, 2), (3, 32, 40, 0, None), (2, 33, 0, 9, 3), (5, 1000, 300, 60, 4), (7, 4095, 50, 0, 2),
    (4, 4096, 0, 600, None), (3, 4097, 5000, 300, 3), (6, 20003, 1024, 100, 5), (2, 129280, 2000, 300, 2), (40, 777, 20, 5, 9),
    (3, 8192, 0, 0, None),
])
def test_against_the_definition(arcs, B, V, hist, bias, masks, dtype, out):
    import torch
    c = make(B, V, dtype, B * 1000 + V, hist, bias, masks)
    want, status = reference(c)
    st = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    got = arcs.adjust_logits(c["logits"], out_dtype=types()[out], out_status=st, **c["args"])
    same(got, want)
    assert (st.cpu().numpy() == status).all()
    assert torch.equal(c["logits"].float().cpu(), torch.from_numpy(c["z"]))
    if dtype == out:
        x = c["logits"].clone()
        assert arcs.adjust_logits(x, out=x, **c["args"]) is x
        same(x, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 5, 8])
def test_strided_rows(arcs, dtype, pad):
    """Rows off the 16-byte grid; what lies between them stays, in place too."""
    import torch
    c = make(5, 4999, dtype, 3, 200, 40, 3)
    want, _ = reference(c)
    wide = torch.full((5, 4999 + pad), 77.0, dtype=c["logits"].dtype, device="cuda")
    wide[:, :4999] = c["logits"]
    words = torch.full((3, (4999 + 31) // 32 + 3), -1, dtype=torch.int32, device="cuda")
    words[:, :-3] = c["args"]["mask"]
    c["args"]["mask"] = words[:, :-3]
    for o in types().values():
        to = torch.full((5, 4999 + 2 * pad), 55.0, dtype=o, device="cuda")
        same(arcs.adjust_logits(wide[:, :4999], out=to[:, :4999], **c["args"]), want)
        assert (to[:, 4999:] == 55.0).all() and (wide[:, 4999:] == 77.0).all()
    same(arcs.adjust_logits(wide[:, :4999], out=wide[:, :4999], **c["args"]), want)
    assert (wide[:, 4999:] == 77.0).all()


def test_rows_between_each_others(arcs):
    """Two halves of one buffer's rows do not overlap."""
    import torch
    c = make(4, 512, "f32", 3, 20, 10, 2)
    buf = torch.cat([c["logits"], torch.zeros_like(c["logits"])], dim=1)
    same(arcs.adjust_logits(buf[:, :512], out=buf[:, 512:], **c["args"]), reference(c)[0])
    assert torch.equal(buf[:, :512], c["logits"])


@pytest.mark.parametrize("n,V", [(257, 10), (1500, 3), (700, 5000)])
def test_biases_of_the_same_token_add_up_in_order(arcs, n, V):
    """Values whose sum depends on the order, one token listed hundreds of times."""
    import torch
    c = make(2, V, "f32", 1, 0, n, None, odd_ids=False)
    rng = np.random.default_rng(n)
    for b in range(2):
        c["bias"][b] = rng.integers(0, min(V, 4), n).astype(np.int32)
        c["values"][b] = (rng.standard_normal(n) * 10.0 ** rng.integers(-4, 5, n)).astype(np.float32)
    c["args"].update(bias_ids=torch.from_numpy(np.concatenate(c["bias"])).cuda(),
                     bias_values=torch.from_numpy(np.concatenate(c["values"])).cuda(),
                     bias_offsets=torch.tensor([0, n, 2 * n], device="cuda"))
    same(arcs.adjust_logits(c["logits"], **c["args"]), reference(c)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_special_values(arcs, dtype, in_place):
    """NaN, infinities, -0 and the type's lowest value: kept where nothing applies, -inf where the
    mask takes the token, IEEE results where penalties and biases meet them."""
    import torch
    c = make(3, 300, dtype, 2, 30, 30, 2)
    special = [np.nan, np.inf, -np.inf, -0.0, torch.finfo(types()[dtype]).min, torch.finfo(types()[dtype]).max]
    for b in range(3):
        c["z"][b, : 300 // 6 * 6] = np.tile(np.float32(special), 300 // 6)
    c["logits"] = torch.from_numpy(c["z"]).to(types()[dtype]).cuda()
    c["values"][0][:] = np.resize(np.float32([np.inf, -np.inf, np.nan, 0.0, -0.0]), len(c["values"][0]))
    c["args"]["bias_values"] = torch.from_numpy(np.concatenate(c["values"])).cuda()
    want, _ = reference(c)
    same(arcs.adjust_logits(c["logits"], out=c["logits"] if in_place else None, **c["args"]), want)


@pytest.mark.parametrize("in_place", [False, True])
def test_refused_rows(arcs, in_place):
    import torch
    c = make(6, 5000, "bf16", 4, 100, 20, 3)
    c["rows"][:] = (0, 3, -2, -1, 2**31 - 1, 1)
    c["args"]["mask_rows"] = torch.from_numpy(c["rows"].astype(np.int32)).cuda()
    c["p"]["frequency"][5], c["p"]["repetition"][3] = np.nan, -1.0
    c["args"]["params"] = arcs.params_to_device(c["p"])
    st = torch.full((6,), 99, dtype=torch.int32, device="cuda")
    got = arcs.adjust_logits(c["logits"], out=c["logits"] if in_place else None, out_status=st, **c["args"])
    c["rows"][[1, 2, 4]] = -1
    want, status = reference(c)
    want[1:] = np.nan
    status[1:] = (9, 9, 4, 9, 4)
    same(got, want)
    assert (st.cpu().numpy() == status).all()


def test_lists_without_elements_and_no_mask_rows(arcs):
    import torch
    c = make(4, 1000, "f32", 4, 0, 0, 4)
    none, zero = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda")
    c["rows"] = np.arange(4)
    args = dict(c["args"], mask_rows=None, hist_ids=none, hist_offsets=zero, bias_ids=none, bias_offsets=zero,
                bias_values=torch.empty(0, device="cuda"))
    same(arcs.adjust_logits(c["logits"], **args), reference(c)[0])
    same(arcs.adjust_logits(c["logits"]), c["z"])
    # offsets that run backwards are empty lists
    back = torch.tensor([5, 4, 3, 2, 1], device="cuda")
    ids = torch.zeros(8, dtype=torch.int32, device="cuda")
    same(arcs.adjust_logits(c["logits"], params=c["params"], hist_ids=ids, hist_offsets=back), c["z"])


@pytest.mark.parametrize("V", [5000, 129280])
def test_sampling_adjusted_rows_is_sampling_with_a_history(arcs, V):
    """float32 rows adjusted first draw the tokens that arcs_sample draws with the history."""
    import torch
    from workloads import make_params
    c = make(8, V, "f32", 21, 700, 0, None)
    p = c["p"]
    p["top_k"], p["top_p"] = 40, 0.9
    params = arcs.params_to_device(p)
    a = {k: c["args"][k] for k in ("hist_ids", "hist_offsets")}
    z = arcs.adjust_logits(c["logits"], params, **a)
    for step in range(3):
        want = arcs.sample(c["logits"], params, seed=5, step=step, **a)
        assert torch.equal(arcs.sample(z, params, seed=5, step=step), want)


def test_masked_rows_sample_allowed_tokens_only(arcs):
    import torch
    c = make(16, 20000, "bf16", 8, 100, 30, 16)
    c["rows"] = np.arange(16)
    args = dict(c["args"], mask_rows=None)
    st = torch.empty(16, dtype=torch.int32, device="cuda")
    z = arcs.adjust_logits(c["logits"], out_status=st, **args)
    ids = arcs.sample(z, c["params"], seed=1, step=2).cpu().numpy()
    for b in range(16):
        if int(st[b]) == arcs.ROW_OK:
            assert c["bits"][b, ids[b]]
        else:
            assert int(st[b]) == arcs.ROW_NOTHING_ALLOWED and not c["bits"][b].any()


def test_a_mask_without_rows_is_refused(arcs):
    """torch has no address for it, and it is not the same as no mask."""
    import torch
    x = torch.zeros(2, 64, device="cuda")
    for rows in (None, torch.full((2,), -1, dtype=torch.int32, device="cuda")):
        with pytest.raises(arcs.ArcsError):
            arcs.adjust_logits(x, mask=torch.empty(0, 2, dtype=torch.int32, device="cuda"), mask_rows=rows)


def test_side_stream_and_replays(arcs):
    import torch
    c = make(9, 7000, "bf16", 9, 200, 50, 4)
    want, _ = reference(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = arcs.adjust_logits(c["logits"], stream=side, **c["args"])
    side.synchronize()
    same(got, want)
    out = torch.empty_like(c["logits"])
    st = torch.empty(9, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        arcs.adjust_logits(c["logits"], out=out, out_status=st, **c["args"])
    for i in range(4):
        c["logits"].copy_(torch.randn(9, 7000, device="cuda", generator=torch.Generator("cuda").manual_seed(i)))
        eager = arcs.adjust_logits(c["logits"], **c["args"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_rows_past_32_bits(arcs):
    """Logits whose last rows begin past 2^32 bytes."""
    import torch
    V, B = 131072 * 8, 2100
    x = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    n[-1] = 2
    ids = torch.tensor([V - 1, 3], dtype=torch.int32, device="cuda")
    arcs.adjust_logits(x, bias_ids=ids, bias_values=torch.tensor([2.0, 1.0], device="cuda"), bias_offsets=n, out=x)
    assert float(x[-1, -1]) == 2.0 and float(x[-1, 3]) == 1.0 and float(x[-1].sum()) == 3.0 and not x[:-1].any()


@pytest.mark.parametrize("own_masks", [False, True])
def test_more_rows_than_one_launch_takes(arcs, own_masks):
    """2^24 rows of 20 tokens, in place and with another type: each has a bias for one token, and a mask (two by
    number, or its own) that takes another."""
    import torch
    B, V = 2 ** 24 + 3, 20
    row = torch.arange(B, device="cuda")
    x = (row % 128)[:, None].to(torch.bfloat16).expand(B, V).contiguous()
    masks = torch.tensor([~1, ~2], dtype=torch.int32, device="cuda")[:, None]  # without token 0, without token 1
    c = dict(bias_ids=(row % V).to(torch.int32), bias_values=(row % 64).float(), bias_offsets=torch.arange(B + 1, device="cuda"))
    c.update(dict(mask=masks[row % 2].contiguous()) if own_masks else dict(mask=masks.contiguous(), mask_rows=(row % 2).to(torch.int32)))
    want = x.clone()
    want[row, row % V] += (row % 64).to(torch.bfloat16)
    want[row, row % 2] = float("-inf")
    st = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    assert torch.equal(arcs.adjust_logits(x, out_dtype=torch.float32, out_status=st, **c), want.float()) and not st.any()
    arcs.adjust_logits(x, out=x, **c)
    assert torch.equal(x, want)
