"""The training-step operators on the GPU against their FP64 statements (oracle/train_ops.py).

Bounds, derived before the first run (u = eps / 2 of a type, the largest relative error of
one rounding: bf16 2^-8, fp32 2^-24):

logits   The tensor cores add sixteen products at a time to an FP32 accumulator, rounding
         towards zero: at most 2^-23 of the magnitudes added per step, 32 steps a segment of
         512, and the segments added to nearest.  |error of z| <= E = (32 + H / 512 + 2)
         2^-23 reach, reach = the largest sum_k |h_k w_k|.
lse      within E, the 2^-21 of the exponentials, their sum and the logarithm, and the
         rounding of the value itself: E + 2^-20 + 2^-22 |lse|.  CE: E more.
dz       p (relative) within P = 2 (E' + E) + 2^-20 (E' = the unsegmented product's error,
         (H / 16 + 2) 2^-23 reach, against lse's E); dz = p - onehot is then off by P p, which
         at the label of a nearly right row is more than P |dz|: p - 1 cancels what p's error
         does not.  Rounding adds u(bf16) |dz|.
dhidden  P sum |p w| + u(bf16) sum |dz w|, the accumulation ((n / 16 + 2) 2^-23 sum |dz w|, n
dweight  the contracted length), and u of the result's own rounding.
"""

import pytest
import torch

from oracle import train_ops as O

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def T():
    from speculative_decoding_draft_vocab_b200 import build as _build
    _build.build()
    from speculative_decoding_draft_vocab_b200 import torch_api
    return torch_api


def _u(dtype):
    return U16 if dtype == torch.bfloat16 else U32


# ------------------------------------------------------------- linear cross entropy
def lce_inputs(R, V, H, ignored=0, seed=0, std=3.0, hidden_pad=0, weight_pad=0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    hidden = torch.randn(R, H + hidden_pad, generator=g, device="cuda").to(torch.bfloat16)[:, :H]
    weight = (torch.randn(V, H + weight_pad, generator=g, device="cuda") * (std / H ** 0.5)).to(torch.bfloat16)[:, :H]
    targets = torch.randint(0, V, (R,), generator=g, device="cuda")
    targets[torch.randperm(R, generator=g, device="cuda")[:ignored]] = -100
    row_weight = torch.rand(R, generator=g, device="cuda") + 0.1
    return hidden, weight, targets, row_weight


def lce_compare(call, ref, H, V, g=1.0, base=None):
    R = call.ce_rows.numel()
    E = (32 + H / 512 + 2) * 2.0 ** -23 * ref["reach"]
    assert int(call.num_tokens) == ref["num_tokens"]
    lse, ce = call.lse_rows.double(), call.ce_rows.double()
    tol = E + 2.0 ** -20 + 2.0 ** -22 * ref["lse_rows"].abs()
    assert bool(((lse - ref["lse_rows"]).abs() <= tol).all())
    assert bool(((ce - ref["ce_rows"]).abs() <= tol + E).all())
    dead = ref["lse_rows"] == 0
    assert bool((lse[dead] == 0).all()) and bool((ce[dead] == 0).all())
    if call.grads is None:
        return
    P = 2 * ((H / 16 + 2) * 2.0 ** -23 * ref["reach"] + E) + 2.0 ** -20
    if call.dhidden is not None:
        want, mag = ref["dhidden"], ref["dh_mag"]
        tol = P * ref["dh_pmag"] + (U16 + (V / 16 + 2) * 2.0 ** -23) * mag + U16 * want.abs()
        assert bool(((call.dhidden.double() - want).abs() <= tol * 1.01).all())
        none = call.dhidden[mag.sum(1) == 0]
        assert bool((none == 0).all())
    if call.dweight is not None:
        want, mag = ref["dweight"], ref["dw_mag"]
        got = call.dweight.double() - (0 if base is None else base.double())
        tol = P * ref["dw_pmag"] + (U16 + (R / 16 + 2) * 2.0 ** -23) * mag + _u(call.dweight.dtype) * want.abs()
        if base is not None:
            tol = tol + U32 * (base.double().abs() + want.abs())
        assert bool(((got - want).abs() <= tol * 1.01).all())


@pytest.mark.parametrize("R,V,H,ignored", [
    (1, 1, 8, 0), (1, 500, 64, 0), (1, 7, 8, 1), (3, 33, 16, 1),
    (7, 8192, 512, 0), (56, 8192, 512, 9), (64, 257, 72, 0), (65, 255, 136, 1),
    (127, 1000, 200, 3), (128, 1024, 128, 0), (129, 1025, 520, 2), (130, 700, 72, 130),
    (255, 3001, 264, 100), (256, 2048, 256, 0), (257, 777, 1032, 5), (448, 5000, 1024, 205),
    (1021, 4003, 1000, 100), (2049, 769, 328, 1000), (8300, 1500, 64, 5000),
])
@pytest.mark.parametrize("z_alpha", [0.0, 1e-3])
def test_linear_ce_matches_the_statement(T, R, V, H, ignored, z_alpha):
    h, w, t, a = lce_inputs(R, V, H, ignored, seed=R + V)
    call = T.LinearCE(h, w, t, row_weight=a, z_alpha=z_alpha)
    call.grad_scale.fill_(0.75)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    ref = O.linear_ce(h, w, t, a, z_alpha=z_alpha, grad_scale=0.75)
    lce_compare(call, ref, H, V)
    n = max(ref["num_tokens"], 1)
    E = (32 + H / 512 + 2) * 2.0 ** -23 * ref["reach"]
    lse = float(ref["lse_rows"].abs().max())
    tol = n * 1.1 * (2 * E + 2.0 ** -19 + z_alpha * 2 * lse * (E + 2.0 ** -20)) + 2.0 ** -21 * float(
        (a * ref["ce_rows"].abs()).sum() + z_alpha * (a * ref["lse_rows"] ** 2).sum())
    assert abs(float(call.loss_num) - float(ref["loss_num"])) <= tol


def test_linear_ce_over_several_pieces(T):
    """More rows and columns than one piece of dz holds (256 MiB): the hidden gradient is
    added up over the pieces, and the last piece is short."""
    R, V, H = 8192, 20011, 64
    h, w, t, a = lce_inputs(R, V, H, 500, seed=1)
    call = T.LinearCE(h, w, t, row_weight=a, dweight_dtype=torch.float32)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    lce_compare(call, O.linear_ce(h, w, t, a), H, V)


def test_linear_ce_split_and_in_pieces(T):
    """Few row tiles, so the hidden gradient's K range is split, and two pieces, the second
    shorter: every split's plane is added to."""
    R, V, H = 1024, 140003, 64
    h, w, t, a = lce_inputs(R, V, H, 300, seed=11)
    call = T.LinearCE(h, w, t, row_weight=a)
    call.forward()
    call.backward()
    ref = O.linear_ce(h, w, t, a)
    lce_compare(call, ref, H, V)
    gathered = T.LinearCE(h, w, t, row_weight=a, dweight=False)
    gathered.forward()
    gathered.backward()
    lce_compare(gathered, ref, H, V)


@pytest.mark.parametrize("R,V,kept", [(448, 151936, True), (600, 151936, False)])
def test_linear_ce_kept_logits_or_not(T, R, V, kept):
    """On both sides of the bound up to which the logits stay in the workspace; the same rows'
    gradients agree to the bounds of either."""
    H = 64
    h, w, t, a = lce_inputs(R, V, H, 100, seed=12)
    call = T.LinearCE(h, w, t, row_weight=a, z_alpha=1e-3)
    assert (call.ws.numel() > 4 * R * V) == kept
    call.forward()
    call.backward()
    assert call.check_status() == 0
    lce_compare(call, O.linear_ce(h, w, t, a, z_alpha=1e-3), H, V)


@pytest.mark.parametrize("R", [40, 300])
def test_linear_ce_strides_scores_and_partial_gradients(T, R):
    V, H = 1003, 144
    h, w, t, a = lce_inputs(R, V, H, 7, seed=2, hidden_pad=24, weight_pad=8)
    ref = O.linear_ce(h, w, t)
    dh = torch.full((R, H + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((V + 1, H + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    both = T.LinearCE(h, w, t, dhidden=dh[:, :H], dweight=dw[:V, :H])
    both.forward()
    both.backward()
    lce_compare(both, ref, H, V)
    assert bool((dh[:, H:] == 7).all()) and bool((dw[:, H:] == 7).all()) and bool((dw[V] == 7).all())
    only_h = T.LinearCE(h, w, t, dweight=False)
    only_h.forward()
    only_h.backward()
    assert torch.equal(only_h.dhidden, dh[:, :H])
    only_w = T.LinearCE(h, w, t, dhidden=False)
    only_w.forward()
    only_w.backward()
    assert torch.equal(only_w.dweight, dw[:V, :H])
    score = T.LinearCE(h, w, t, dhidden=False, dweight=False)
    score.forward()
    assert torch.equal(score.ce_rows, both.ce_rows) and torch.equal(score.loss_num, both.loss_num)
    with pytest.raises(ValueError, match="without gradients"):
        score.backward()
    with pytest.raises(ValueError, match="follows a forward"):
        T.LinearCE(h, w, t).backward()


@pytest.mark.parametrize("R", [50, 200])
def test_linear_ce_accumulates_fp32(T, R):
    V, H = 901, 136
    h, w, t, a = lce_inputs(R, V, H, 3, seed=3)
    base = torch.randn(V, H, device="cuda")
    dw = base.clone()
    call = T.LinearCE(h, w, t, row_weight=a, dhidden=False, dweight=dw, accumulate=True)
    call.forward()
    call.backward()
    lce_compare(call, O.linear_ce(h, w, t, a), H, V, base=base)
    # no labelled row: nothing is added
    none = T.LinearCE(h, w, torch.full_like(t, -100), dhidden=False, dweight=dw, accumulate=True)
    before = dw.clone()
    none.forward()
    none.backward()
    assert torch.equal(dw, before) and float(none.loss_num) == 0.0


def test_linear_ce_rows_without_a_label_are_not_read(T):
    """NaN and infinities in ignored rows, an id out of range, an ignore_index inside the
    vocabulary; everything else as without them."""
    R, V, H = 200, 600, 64
    h, w, t, a = lce_inputs(R, V, H, 20, seed=4)
    clean = T.LinearCE(h, w, t)
    clean.forward()
    clean.backward()
    assert clean.check_status() == 0
    dirty = h.clone()
    dirty[t == -100] = float("nan")
    dirty[(t == -100).nonzero()[0]] = float("inf")
    aw = torch.ones(R, device="cuda")
    aw[t == -100] = float("nan")
    call = T.LinearCE(dirty, w, t, row_weight=aw)
    call.forward()
    call.backward()
    for k in ("loss_num", "num_tokens", "ce_rows", "lse_rows", "dhidden", "dweight"):
        assert torch.equal(getattr(call, k), getattr(clean, k)), k
    bad = t.clone()
    bad[t == -100] = V  # out of range: flagged, and no label
    call = T.LinearCE(dirty, w, bad)
    call.forward()
    call.backward()
    assert call.check_status() == 3  # DSPARK_ERR_ID_OUT_OF_RANGE
    assert torch.equal(call.dweight, clean.dweight) and torch.equal(call.loss_num, clean.loss_num)
    inside = torch.where(t == -100, torch.full_like(t, 5), torch.where(t == 5, torch.full_like(t, 6), t))
    call = T.LinearCE(dirty, w, inside, ignore_index=5)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    lce_compare(call, O.linear_ce(dirty, w, inside, ignore_index=5), H, V)


def test_linear_ce_extreme_logits(T):
    """Logits of +-1000, where every exponential under- or overflows without the row's own
    maximum; and a labelled row of NaN, which spoils its own outputs and the sums only."""
    R, V, H = 140, 515, 8
    h = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = 1.0
    h[1::2, 0] = -1.0
    w[:, 0] = 1000.0
    w[7, 0] = 1008.0
    t = torch.arange(R, device="cuda") % V
    call = T.LinearCE(h, w, t)
    call.forward()
    call.backward()
    lce_compare(call, O.linear_ce(h, w, t), H, V)
    h[3, 1] = float("nan")
    call.forward()
    call.backward()
    bad = torch.isnan(call.ce_rows)
    assert bool(bad[3]) and int(bad.sum()) == 1 and bool(torch.isnan(call.loss_num))
    assert not bool(torch.isnan(call.dhidden[torch.arange(R, device="cuda") != 3]).any())


@pytest.mark.parametrize("R,V", [(100, 4000), (600, 9000)])
def test_linear_ce_repeats_replays_and_keeps_to_its_stream(T, R, V):
    H = 256
    h, w, t, a = lce_inputs(R, V, H, 11, seed=5)
    call = T.LinearCE(h, w, t, row_weight=a)
    keys = ("loss_num", "num_tokens", "ce_rows", "lse_rows", "dhidden", "dweight")

    def snap():
        return [getattr(call, k).clone() for k in keys]
    call.forward()
    call.backward()
    call.backward()  # again after one forward
    first = snap()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call.forward()
        call.backward()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, snap()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.forward()
        call.backward()
    h2, _, t2, _ = lce_inputs(R, V, H, 60, seed=6)
    h.copy_(h2)
    t.copy_(t2)  # the same buffers, other rows without a label
    g.replay()
    replayed = snap()
    call.forward()
    call.backward()
    assert all(torch.equal(x, y) for x, y in zip(replayed, snap()))
    lce_compare(call, O.linear_ce(h, w, t, a), H, V)


def test_linear_ce_two_calls_at_once(T):
    """Two calls with workspaces of their own, on two streams at the same time."""
    made = []
    for seed, (R, V, H) in enumerate([(300, 9000, 256), (90, 12000, 512)]):
        h, w, t, a = lce_inputs(R, V, H, 9, seed=20 + seed)
        alone = T.LinearCE(h, w, t, row_weight=a)
        alone.forward()
        alone.backward()
        made.append((T.LinearCE(h, w, t, row_weight=a), alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for call, _, s in made:
            with torch.cuda.stream(s):
                call.forward()
                call.backward()
    torch.cuda.synchronize()
    for call, alone, _ in made:
        assert call.check_status() == 0
        for k in ("loss_num", "ce_rows", "dhidden", "dweight"):
            assert torch.equal(getattr(call, k), getattr(alone, k)), k


def test_linear_ce_gradient_against_differences(T):
    """The kernels' own loss, moved along a direction, against their gradient: hidden rows
    are perturbed in exact bf16 steps."""
    R, V, H = 96, 400, 64
    h, w, t, a = lce_inputs(R, V, H, 5, seed=7)
    call = T.LinearCE(h, w, t, row_weight=a, z_alpha=1e-3)
    call.forward()
    call.backward()
    ref = O.linear_ce(h, w, t, a, z_alpha=1e-3)
    d = torch.zeros(R, H, device="cuda", dtype=torch.float64)
    d[:, :] = ref["dhidden"].sign()
    step = 2.0 ** -6
    losses = []
    for s in (+1, -1):
        hs = (h.double() + s * step * d).to(torch.bfloat16)
        c = T.LinearCE(hs, w, t, row_weight=a, z_alpha=1e-3, dhidden=False, dweight=False)
        c.forward()
        losses.append((float(c.loss_num), hs))
    moved = losses[0][1].double() - losses[1][1].double()  # what the rounding left of the step
    want = float((call.dhidden.double() * moved).sum())
    # second-order terms cancel between the two sides but for the rounding of h; third order
    # and that: a hundredth of the change at this step
    assert abs((losses[0][0] - losses[1][0]) - want) <= 0.02 * abs(want)


# ----------------------------------------------------------------------- embedding
def _ids(R, Vt, hot, g):
    ids = torch.randint(0, Vt, (R,), generator=g, device="cuda")
    if hot:
        ids[torch.rand(R, generator=g, device="cuda") < hot] = Vt // 2
    return ids


EMB = [(1, 1, 8), (1, 100, 64), (5, 3, 8), (33, 50, 24), (448, 5000, 264), (1000, 7, 512), (4096, 4097, 128),
       (4097, 100000, 32), (9001, 600, 1032)]


@pytest.mark.parametrize("R,Vt,D", EMB + [(8193, 50, 8), (20003, 300, 248), (9001, 100, 264), (70001, 1000, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_embedding_matches_the_statement(T, R, Vt, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(R + D)
    table = torch.randn(Vt, D + 8, generator=g, device="cuda").to(dtype)[:, :D]
    ids = _ids(R, Vt, 0.3, g)
    valid = (torch.rand(R, generator=g, device="cuda") < 0.8).to(torch.uint8)
    ids[valid == 0] = -7  # not looked at
    out = torch.full((R, D + 16), 3.0, dtype=dtype, device="cuda")
    call = T.Embedding(ids, table, scale=D ** 0.5, valid=valid, out=out[:, :D])
    call.launch()
    assert call.check_status() == 0
    ref = O.embed(ids, table, float(torch.tensor(D ** 0.5, dtype=torch.float32)), valid)
    # the product in FP32, then the type's rounding
    assert bool(((out[:, :D].double() - ref).abs() <= (U32 + _u(dtype)) * 1.01 * ref.abs()).all())
    assert bool((out[:, D:] == 3.0).all())
    last = R - 1
    ids[last] = Vt
    valid[last] = 1
    call.launch()
    assert call.check_status() == 3 and bool((out[last, :D] == 0).all())
    valid[last] = 0  # the status is the last call's
    call.launch()
    assert call.check_status() == 0


@pytest.mark.parametrize("R,Vt,D", EMB + [(40000, 11, 64), (70001, 151936, 16), (50, 300001, 8), (5000, 300001, 8),
                                          (140001, 300001, 8), (140001, 97, 40)])
@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                        (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("hot", [0.0, 0.4])
def test_embedding_gradient_matches_the_statement(T, R, Vt, D, dtype, grad, hot):
    g = torch.Generator(device="cuda").manual_seed(R + D + 1)
    dout = torch.randn(R, D + 8, generator=g, device="cuda").to(dtype)[:, :D]
    ids = _ids(R, Vt, hot, g)
    valid = (torch.rand(R, generator=g, device="cuda") < 0.8).to(torch.uint8)
    ids[valid == 0] = 1 << 40
    dout[valid == 0] = float("nan")  # not read
    buf = torch.full((Vt, D + 8), 5.0, dtype=grad, device="cuda")
    call = T.EmbeddingGrad(ids, dout, Vt, scale=1.5, valid=valid, out=buf[:, :D])
    call.launch()
    assert call.check_status() == 0
    ref, mag, n = O.embed_grad(ids, dout, Vt, 1.5, valid)
    # n additions in FP32 and the scale's rounding, then the type's
    tol = (n[:, None] + 2) * U32 * mag + _u(grad) * ref.abs()
    assert bool(((buf[:, :D].double() - ref).abs() <= tol * 1.01).all())
    assert bool((buf[:, :D][n == 0] == 0).all()) and bool((buf[:, D:] == 5.0).all())
    first = buf.clone()
    call.launch()
    assert torch.equal(buf, first)


@pytest.mark.parametrize("R,Vt,D", [(1, 9, 8), (500, 40, 136), (9001, 600, 64)])
def test_embedding_gradient_accumulates(T, R, Vt, D):
    g = torch.Generator(device="cuda").manual_seed(R)
    dout = torch.randn(R, D, generator=g, device="cuda").to(torch.bfloat16)
    ids = _ids(R, Vt, 0.2, g)
    ids[ids == 3] = 4  # a row that nothing is added to
    base = torch.randn(Vt, D, generator=g, device="cuda")
    base[3] = float("nan")
    table = base.clone()
    call = T.EmbeddingGrad(ids, dout, Vt, out=table, accumulate=True)
    call.launch()
    ref, mag, n = O.embed_grad(ids, dout, Vt)
    on = torch.arange(Vt, device="cuda") != 3
    tol = (n[:, None] + 2) * U32 * mag + U32 * (base.double().abs() + mag)
    assert bool(((table.double() - base.double() - ref).abs() <= tol * 1.01)[on].all())
    assert bool(torch.isnan(table[3]).all())  # left as it was
    with pytest.raises(Exception, match="not supported"):
        T.EmbeddingGrad(ids, dout, Vt, dtype=torch.bfloat16, accumulate=True).launch()


def test_embedding_gradient_edges(T):
    """Nothing valid; every row the same id; an id out of range; a replayed capture."""
    R, Vt, D = 5000, 64, 40
    dout = torch.randn(R, D, device="cuda")
    ids = torch.full((R,), 63, device="cuda")
    call = T.EmbeddingGrad(ids, dout, Vt, valid=torch.zeros(R, dtype=torch.uint8, device="cuda"))
    call.launch()
    assert call.check_status() == 0 and not bool(call.out.any())
    call = T.EmbeddingGrad(ids, dout, Vt)
    call.launch()
    ref, mag, n = O.embed_grad(ids, dout, Vt)
    assert bool(((call.out.double() - ref).abs() <= 1.01 * (n[:, None] + 2) * U32 * mag).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.launch()
    ids.copy_(torch.randint(0, Vt, (R,), device="cuda"))
    ids[17] = -1
    graph.replay()
    assert call.check_status() == 3
    ref, mag, n = O.embed_grad(ids, dout, Vt)
    assert bool(((call.out.double() - ref).abs() <= 1.01 * (n[:, None] + 2) * U32 * mag).all())


# ------------------------------------------------------------------------ clipping
def _flat(sizes, dtype, off, scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = (torch.randn(sum(sizes) + off + 8, generator=g, device="cuda") * scale).to(dtype)
    out, at = [], off
    for n in sizes:
        out.append(buf[at:at + n])
        at += n
    return buf, out


SIZES = [[1], [0, 5, 0], [8191, 8192, 8193], [1, 2, 3, 5, 7, 100001, 13], [17] * 700, [3000001],
         [3, 0, 9001] * 700]  # (the last: more tensors than one launch describes)


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("factor", [0.3, 4.0])
def test_clip_matches_the_statement(T, sizes, dtype, off, factor):
    buf, grads = _flat(sizes, dtype, off, seed=len(sizes))
    max_norm = factor * float(torch.cat([g.double() for g in grads]).norm())
    norm, coef, want = O.clip(grads, max_norm)
    dst, outs = _flat(sizes, dtype, off + 1 if factor < 1 else off, seed=9)
    for into in (outs, None):  # to buffers that meet 16 bytes elsewhere, then in place
        call = T.GradClip(grads, max_norm, outs=into)
        edges = [buf[:off].clone(), buf[off + sum(sizes):].clone()]
        call.launch()
        assert call.check_status() == 0
        # FP64 sums of squares each right to 2^-22, one square root and three FP32 roundings
        assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
        assert abs(float(call.coef) - coef) <= 2.0 ** -20 * coef
        for g, w in zip(call.outs, want):
            assert bool(((g.double() - w).abs() <= (2.0 ** -20 + 1.01 * _u(dtype)) * w.abs() + 1e-45).all())
        assert torch.equal(buf[:off], edges[0]) and torch.equal(buf[off + sum(sizes):], edges[1])


def test_clip_values_out_of_the_ordinary(T):
    big = torch.full((1000,), 1e25, device="cuda")      # squares overflow FP32
    small = torch.full((1000,), 1e-25, device="cuda")   # and underflow
    zero = torch.zeros(5000, device="cuda")
    for g in (big, small, zero):
        norm, coef, want = O.clip([g], 1.0)
        call = T.GradClip([g.clone()], 1.0)
        call.launch()
        assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
        assert bool(((call.outs[0].double() - want[0]).abs() <= 2.0 ** -19 * want[0].abs()).all())
    for bad in (float("inf"), float("nan")):
        g = torch.randn(3001, device="cuda")
        g[1234] = bad
        before = g.clone()
        out = torch.empty_like(g)
        call = T.GradClip([g], 0.5, outs=[out])
        call.launch()
        assert not bool(torch.isfinite(call.norm)) and float(call.coef) == 1.0
        assert torch.equal(torch.nan_to_num(out, 9.0, 8.0), torch.nan_to_num(before, 9.0, 8.0))


def test_clip_repeats_and_replays(T):
    _, grads = _flat([100003, 77, 4096 * 5], torch.float32, 1, seed=3)
    _, more = _flat([60001, 12], torch.bfloat16, 1, seed=4)
    grads = grads + more
    outs = [torch.empty_like(g) for g in grads]
    call = T.GradClip(grads, 3.0, outs=outs)
    call.launch()
    first = [o.clone() for o in outs] + [call.norm.clone()]
    call.launch()
    assert all(torch.equal(x, y) for x, y in zip(first, outs + [call.norm]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.launch()
    for g in grads:
        g.mul_(-2.0)
    graph.replay()
    norm, coef, want = O.clip(grads, 3.0)
    assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
    for g, w in zip(outs, want):
        assert bool(((g.double() - w).abs() <= (2.0 ** -20 + 1.01 * _u(g.dtype)) * w.abs()).all())
    with pytest.raises(ValueError, match="twice"):
        T.GradClip([grads[0], grads[0]], 1.0)


def test_clip_of_nothing(T):
    empty = torch.empty(0, device="cuda")
    call = T.GradClip([empty, empty], 1.0)
    call.launch()
    assert float(call.norm) == 0.0 and float(call.coef) == 1.0 and call.check_status() == 0


def test_clip_over_a_group(T, monkeypatch):
    """With a process group the FP64 sum goes through one all-reduce before the scaling (here
    a stand-in that adds another rank's sum)."""
    import torch.distributed as dist
    seen = []

    def all_reduce(x, op=None, group=None):
        seen.append((x.dtype, x.numel(), group))
        x += 3.0
    monkeypatch.setattr(dist, "all_reduce", all_reduce)
    g = torch.full((100,), 0.1, device="cuda")
    call = T.GradClip([g], 1.0, outs=[torch.empty_like(g)], group="ranks")
    call.launch()
    assert seen == [(torch.float64, 1, "ranks")]
    norm = (float(g.double().pow(2).sum()) + 3.0) ** 0.5
    assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
    want = g.double() / (norm + 1e-6)
    assert bool(((call.outs[0].double() - want).abs() <= 2.0 ** -20 * want).all())
    with pytest.raises(ValueError, match="current stream"):
        call.launch(stream=0)


def test_clip_in_two_steps(T):
    """dspark_grad_sumsq and dspark_grad_scale, as ranks use them around an all-reduce: two
    halves of a gradient clipped by the norm of the whole equal the whole clipped at once."""
    import ctypes
    from speculative_decoding_draft_vocab_b200 import abi
    g = torch.randn(50000, device="cuda")
    whole = T.GradClip([g], 2.0, outs=[torch.empty_like(g)])
    whole.launch()
    halves = [T.GradClip([h], 2.0, outs=[torch.empty_like(h)]) for h in (g[:30000], g[30000:])]
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for h in halves:
        abi.check(abi.dspark_grad_sumsq(h.tensors, 1, h.sumsq.data_ptr(), h.ws_ptr, h.ws_len, s), "sumsq")
    total = halves[0].sumsq + halves[1].sumsq
    for h in halves:
        abi.check(abi.dspark_grad_scale(h.tensors, 1, total.data_ptr(), 2.0, h.norm.data_ptr(), h.coef.data_ptr(),
                                        h.ws_ptr, h.ws_len, s), "scale")
        assert h.check_status() == 0
        assert abs(float(h.norm) - float(whole.norm)) <= 2.0 ** -22 * float(whole.norm)
    both = torch.cat([h.outs[0] for h in halves])
    assert bool(((both - whole.outs[0]).abs() <= 2.0 ** -21 * whole.outs[0].abs()).all())


# ------------------------------------------------------------------ used together
def test_a_training_step_of_all_of_them(T):
    """Tokens -> scaled embedding -> linear cross entropy with a tied head -> both gradients
    of the table in one FP32 buffer -> clipping; against the same chain in FP64 from the
    kernels' own bf16 activations.  Then the heads' gradients of the fused loss, clipped."""
    from speculative_decoding_draft_vocab_b200.synthetic import make_inputs
    R, V, H, scale = 300, 2003, 128, 2.0
    g = torch.Generator(device="cuda").manual_seed(8)
    table = (torch.randn(V, H, generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    ids = _ids(R, V, 0.2, g)
    targets = torch.roll(ids, -1)
    targets[-1] = -100
    emb = T.Embedding(ids, table, scale=scale)
    emb.launch()
    dtable = torch.empty(V, H, device="cuda")
    ce = T.LinearCE(emb.out, table, targets, dweight=dtable, accumulate=False)
    ce.forward()
    ce.backward()
    back = T.EmbeddingGrad(ids, ce.dhidden, V, scale=scale, out=dtable, accumulate=True)
    back.launch()
    clip = T.GradClip([dtable], 0.5)
    head = dtable.clone()
    clip.launch()
    torch.cuda.synchronize()
    assert emb.check_status() == ce.check_status() == back.check_status() == clip.check_status() == 0
    ref = O.linear_ce(emb.out, table, targets)
    lce_compare(T_no_weight(ce), ref, H, V)
    want, mag, n = O.embed_grad(ids, ce.dhidden, V, scale)
    want = want + ref["dweight"]
    P = 2 * ((H / 16 + 2) + (32 + H / 512 + 2)) * 2.0 ** -23 * ref["reach"] + 2.0 ** -20
    tol = P * ref["dw_pmag"] + (U16 + (R / 16 + 2) * 2.0 ** -23) * ref["dw_mag"] + (n[:, None] + 4) * U32 * (mag + ref["dw_mag"])
    assert bool(((head.double() - want).abs() <= 1.01 * tol).all())
    norm, coef, clipped = O.clip([head], 0.5)
    assert abs(float(clip.norm) - norm) <= 2.0 ** -21 * norm and coef < 1.0
    assert bool(((dtable.double() - clipped[0]).abs() <= 2.0 ** -19 * clipped[0].abs()).all())

    inp = make_inputs("recipe_heads", device="cuda", B=1, N=3, K=7, V=2048, hidden=256, rank=64, seed=3)
    out = T.dspark_loss(inp)
    grads = out.head_grads()
    assert len(grads) == 4
    norm, coef, clipped = O.clip(grads, 0.1)
    call = T.GradClip(grads, 0.1)
    call.launch()
    assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
    for got, w in zip(grads, clipped):
        assert bool(((got.double() - w).abs() <= 2.0 ** -19 * w.abs()).all())


def T_no_weight(call):
    """`call` with its weight gradient set aside (another kernel added to that buffer)."""
    import copy
    c = copy.copy(call)
    c.dweight = None
    return c


# ------------------------------------------- hidden gradient gathered by the forward
@pytest.mark.parametrize("R,V,H,ignored", [(1, 16384, 64, 0), (5, 16400, 72, 5), (100, 20011, 136, 7),
                                           (128, 16385, 520, 0), (300, 17000, 256, 40), (700, 16640, 1032, 3),
                                           (8192, 20011, 64, 500)])
@pytest.mark.parametrize("z_alpha", [0.0, 1e-3])
def test_linear_ce_gathered_matches_the_statement(T, R, V, H, ignored, z_alpha):
    """Without a head gradient, from 16384 columns on, the forward gathers the hidden one.
    The bounds are those of the other way: exponentials are rounded to bf16 instead of dz
    (relative error 2^-8 of each term; the label's own term is not rounded)."""
    h, w, t, a = lce_inputs(R, V, H, ignored, seed=R + V + 1)
    call = T.LinearCE(h, w, t, row_weight=a, z_alpha=z_alpha, dweight=False)
    assert call.prob.hidden_grad_only == 1
    call.forward()
    call.grad_scale.fill_(-0.75)  # known only after the forward
    call.backward()
    assert call.check_status() == 0
    ref = O.linear_ce(h, w, t, a, z_alpha=z_alpha, grad_scale=-0.75)
    lce_compare(call, ref, H, V)
    both = T.LinearCE(h, w, t, row_weight=a, z_alpha=z_alpha)
    both.forward()
    assert int(both.num_tokens) == int(call.num_tokens)
    assert abs(float(both.loss_num) - float(call.loss_num)) <= 2.0 ** -18 * abs(float(both.loss_num)) + 1e-30
    first = [x.clone() for x in (call.loss_num, call.ce_rows, call.lse_rows, call.dhidden)]
    call.forward()
    call.backward()
    assert all(torch.equal(x, y) for x, y in zip(first, (call.loss_num, call.ce_rows, call.lse_rows, call.dhidden)))


@pytest.mark.parametrize("R", [60, 200])
def test_linear_ce_gathered_out_of_the_reference_range(T, R):
    """A logit past the sampled columns far above every sampled one (by 200 to 1000): the
    exponentials relative to the sample would overflow, and the call has to go the other way,
    rows that did not ask for it included.  Then the same buffers with ordinary logits."""
    V, H = 16500, 16
    h = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    w = (torch.randn(V, H, device="cuda") * 0.5).to(torch.bfloat16)
    w[:, 0] = 0.0
    w[V - 3, 0] = 200.0
    w[9000, 0] = 190.0
    h[:, 1:] = torch.randn(R, H - 1, device="cuda").to(torch.bfloat16)
    h[::3, 0] = 1.0   # a third of the rows leave the range
    h[1::3, 0] = 5.0  # a third by far more
    t = torch.arange(R, device="cuda") * 7 % V
    t[3] = V - 3
    call = T.LinearCE(h, w, t, dweight=False)
    call.grad_scale.fill_(0.5)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    lce_compare(call, O.linear_ce(h, w, t, grad_scale=0.5), H, V)
    h[:, 0] = 0.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.forward()
        call.backward()
    graph.replay()
    lce_compare(call, O.linear_ce(h, w, t, grad_scale=0.5), H, V)
    h[::2, 0] = 2.0
    graph.replay()
    lce_compare(call, O.linear_ce(h, w, t, grad_scale=0.5), H, V)
    h[4, 2] = float("nan")
    call.forward()
    call.backward()
    bad = torch.isnan(call.lse_rows)
    assert bool(bad[4]) and int(bad.sum()) == 1
    assert not bool(torch.isnan(call.dhidden[torch.arange(R, device="cuda") != 4]).any())


# --------------------------------------- a backward that forms the logits again
def forward_alone(call):
    """The forward with the workspace size that it needs by itself: it keeps no logits."""
    import ctypes
    from speculative_decoding_draft_vocab_b200 import abi
    n = abi.dspark_lce_workspace_size(ctypes.byref(call.prob), None)
    assert n < call.ws_len
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    abi.check(abi.dspark_lce_fwd(ctypes.byref(call.prob), ctypes.byref(call.out), call.ws_ptr, n, s), "dspark_lce_fwd")
    call._ran = True


@pytest.mark.parametrize("R,V,H", [(100, 1003, 72), (300, 5000, 136)])
def test_linear_ce_backward_goes_by_what_its_forward_kept(T, R, V, H):
    """A forward that was given no room for the logits, on a workspace that holds those of an
    earlier forward: the backward must not take these for its own."""
    h, w, t, a = lce_inputs(R, V, H, 9, seed=30)
    call = T.LinearCE(h, w, t, row_weight=a)
    call.forward()
    call.backward()
    lce_compare(call, O.linear_ce(h, w, t, a), H, V)
    h2, _, t2, _ = lce_inputs(R, V, H, 5, seed=31)
    h.copy_(h2)
    t.copy_(t2)
    ref = O.linear_ce(h, w, t, a)
    forward_alone(call)
    call.backward()
    assert call.check_status() == 0
    lce_compare(call, ref, H, V)
    call.forward()  # and kept again
    call.backward()
    lce_compare(call, ref, H, V)


@pytest.mark.parametrize("R,V,H,ignored", [(64, 1500, 4096, 3), (100, 3001, 328, 9), (129, 2000, 1000, 0),
                                           (300, 5003, 1000, 120), (700, 4100, 4096, 50)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_ce_forms_its_logits_again(T, R, V, H, ignored, dtype):
    """What larger batches do, at small ones: dz from the product again, over hidden sizes of
    several K chunks and segments, with a z-loss, strides and a scale."""
    h, w, t, a = lce_inputs(R, V, H, ignored, seed=R + H, hidden_pad=8, weight_pad=16)
    call = T.LinearCE(h, w, t, row_weight=a, z_alpha=1e-3, dweight_dtype=dtype)
    call.grad_scale.fill_(-1.25)
    forward_alone(call)
    call.backward()
    assert call.check_status() == 0
    ref = O.linear_ce(h, w, t, a, z_alpha=1e-3, grad_scale=-1.25)
    lce_compare(call, ref, H, V)
    first = [call.dhidden.clone(), call.dweight.clone()]
    call.backward()
    assert torch.equal(first[0], call.dhidden) and torch.equal(first[1], call.dweight)
    if dtype == torch.float32:  # added to what is there
        base = torch.randn(V, H, device="cuda")
        more = T.LinearCE(h, w, t, row_weight=a, z_alpha=1e-3, dhidden=False, dweight=base.clone(), accumulate=True)
        more.grad_scale.fill_(-1.25)
        forward_alone(more)
        more.backward()
        lce_compare(more, ref, H, V, base=base)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_ce_head_gradient_alone_in_pieces(T, dtype):
    R, V, H = 8192, 20011, 72
    h, w, t, a = lce_inputs(R, V, H, 700, seed=32)
    call = T.LinearCE(h, w, t, row_weight=a, dhidden=False, dweight_dtype=dtype)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    lce_compare(call, O.linear_ce(h, w, t, a), H, V)


def test_linear_ce_sums_over_many_rows_do_not_fall_short(T):
    """An FP32 head gradient over 100003 rows.  Logits of zero over four columns: dz is 1/4
    exactly where there is no label, so dz's rounding takes no part and the sums of positive
    terms stand alone.  Accumulators round towards zero within segments of 4096 rows (at most
    2^-23 of the sum at each of 4096 / 16 steps, and 2 more for the product), the segments are
    added to nearest."""
    R, V, H = 100003, 4, 64
    g = torch.Generator(device="cuda").manual_seed(33)
    h = (torch.rand(R, H, generator=g, device="cuda") + 1.0).to(torch.bfloat16)
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(R, dtype=torch.int64, device="cuda")
    call = T.LinearCE(h, w, t, dhidden=False, dweight_dtype=torch.float32)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    total = h.double().sum(0)
    want = torch.stack([-0.75 * total] + 3 * [0.25 * total])
    bound = (4096 / 16 + 2) * 2.0 ** -23 + (R / 4096 + 2) * 2.0 ** -24
    assert bool(((call.dweight.double() - want).abs() <= bound * want.abs()).all())


def test_linear_ce_long_hidden_rows(T):
    """dz from the product again over a hidden size of 2^18, all terms positive: its logits may
    be short by the rounding of a segment of 4096 and of the segments' sum, not by that of the
    whole length (bounds of the head of this file, with the segments' E')."""
    R, V, H = 20, 40, 1 << 18
    g = torch.Generator(device="cuda").manual_seed(34)
    h = ((torch.rand(R, H, generator=g, device="cuda") + 0.5) * 0.0276).to(torch.bfloat16)
    w = ((torch.rand(V, H, generator=g, device="cuda") + 0.5) * 0.0276).to(torch.bfloat16)
    t = torch.arange(R, device="cuda")
    call = T.LinearCE(h, w, t)
    forward_alone(call)
    call.backward()
    assert call.check_status() == 0
    ref = O.linear_ce(h, w, t)
    E = (32 + H / 512 + 2) * 2.0 ** -23 * ref["reach"]
    P = 2 * ((4096 / 16 + H / 4096 + 2) * 2.0 ** -23 * ref["reach"] + E) + 2.0 ** -20
    assert bool(((call.lse_rows.double() - ref["lse_rows"]).abs() <= E + 2.0 ** -20 + 2.0 ** -22 * ref["lse_rows"]).all())
    tol = P * ref["dw_pmag"] + (U16 + 4 * 2.0 ** -23) * ref["dw_mag"] + U16 * ref["dweight"].abs()
    assert bool(((call.dweight.double() - ref["dweight"]).abs() <= tol).all())


@pytest.mark.parametrize("R", [60, 200])
@pytest.mark.parametrize("big", [10, 50])
def test_linear_ce_gathered_with_a_large_head_column(T, R, big):
    """A head column of 2^56 against hidden values of 2^-50, and a logit past the sampled
    columns 80 octaves above them: 2^80 times 2^56 is beyond FP32, the gradient itself is not.
    (With 2^16 it stays in range.)"""
    V, H = 16500, 16
    g = torch.Generator(device="cuda").manual_seed(35)
    h = torch.randn(R, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, H, generator=g, device="cuda") * 0.5).to(torch.bfloat16)
    h[:, 0] = 2.0 ** -big
    w[:, 0] = 0.0
    w[V - 3, 0] = 62.0 * 2.0 ** big
    t = torch.arange(R, device="cuda") * 7 % V
    t[3] = V - 3
    call = T.LinearCE(h, w, t, dweight=False)
    assert call.prob.hidden_grad_only == 1
    for _ in range(2):  # the second forward begins anew
        call.forward()
        call.backward()
        assert call.check_status() == 0
        assert bool(torch.isfinite(call.dhidden).all())
        lce_compare(call, O.linear_ce(h, w, t), H, V)


# ----------------------------------------------------- norms past FP32's range
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,max_norm", [(2, 1.0), (50001, 1.0), (50001, 1e-30)])
def test_clip_by_a_norm_past_fp32(T, dtype, n, max_norm):
    """Finite values whose norm FP32 does not hold are clipped all the same; the coefficient
    may be far below FP32's range when the clipped values are not."""
    g = torch.full((n,), 3e38, device="cuda").to(dtype)
    g[::2] *= -1
    norm, coef, want = O.clip([g], max_norm)
    assert norm > torch.finfo(torch.float32).max and coef < torch.finfo(torch.float32).tiny
    for out in (torch.zeros(n + 1, dtype=dtype, device="cuda")[1:], None):  # other alignment, in place
        call = T.GradClip([g], max_norm, outs=None if out is None else [out])
        call.launch()
        assert call.check_status() == 0 and float(call.norm) == float("inf")
        assert abs(float(call.coef) - coef) <= 2.0 ** -150 + 2.0 ** -20 * coef
        # the sum of squares in FP64 and the product's and the type's roundings
        assert bool(((call.outs[0].double() - want[0]).abs() <= (2.0 ** -20 + 1.01 * _u(dtype)) * want[0].abs()).all())


def test_clip_of_many_launches_in_one_call_and_in_two_steps(T):
    """3000 tensors, more than one launch describes: one call adds the launches' partial sums up
    once, in the order the two steps do, and gives the same bits; replayed too."""
    import ctypes
    from speculative_decoding_draft_vocab_b200 import abi
    _, grads = _flat([9001, 0, 17] * 1000, torch.bfloat16, 1, seed=40)
    outs = [torch.empty_like(g) for g in grads]
    call = T.GradClip(grads, 2.0, outs=outs)
    call.launch()
    norm, coef, want = O.clip(grads, 2.0)
    assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm and call.check_status() == 0
    first = [call.norm.clone(), call.coef.clone(), torch.cat(outs)]
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    abi.check(abi.dspark_grad_sumsq(call.tensors, call.count, call.sumsq.data_ptr(), call.ws_ptr, call.ws_len, s), "sumsq")
    abi.check(abi.dspark_grad_scale(call.tensors, call.count, call.sumsq.data_ptr(), 2.0, call.norm.data_ptr(),
                                    call.coef.data_ptr(), call.ws_ptr, call.ws_len, s), "scale")
    assert all(torch.equal(x, y) for x, y in zip(first, (call.norm, call.coef, torch.cat(outs))))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.launch()
    for g in grads[:2000]:
        g.mul_(4.0)
    graph.replay()
    norm, coef, want = O.clip(grads, 2.0)
    assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
    got = torch.cat(outs).double()
    assert bool(((got - torch.cat(want)).abs() <= (2.0 ** -20 + 1.01 * U16) * torch.cat(want).abs()).all())


@pytest.mark.parametrize("shard", [True, False])
def test_clip_counts_replicated_gradients_once(T, monkeypatch, shard):
    """A vocabulary-parallel rank's gradients: its shard of dW2 beside its copies of dW1,
    dconf_w and dconf_b.  Both ranks of a group of two get the norm of the whole gradient, in
    which the copies count once (the collective is a stand-in that adds the other rank's sum)."""
    import torch.distributed as dist
    from speculative_decoding_draft_vocab_b200.synthetic import make_inputs
    inp = make_inputs("recipe_heads", device="cuda", B=1, N=3, K=7, V=2048, hidden=256, rank=64, seed=4)
    ranks = T.tp_group_emulated(inp, 2)
    torch.cuda.synchronize()
    sharded, copies = [], []
    for r in ranks:
        sharded.append([r.dW2[r.col0:r.col0 + r.width]] if shard else [])
        copies.append([r.dW1, r.dconf_w, r.dconf_b])
    sums = [sum(float(t.double().pow(2).sum()) for t in ts) for ts in (sharded[0] + copies[0], sharded[1])]
    norm, coef, _ = O.clip(sharded[0] + sharded[1] + copies[0], 0.05)
    assert norm > 0.05
    calls = []
    for k in range(2):
        monkeypatch.setattr(dist, "get_rank", lambda group=None, k=k: k)
        monkeypatch.setattr(dist, "all_reduce", lambda x, op=None, group=None, k=k: x.add_(sums[1 - k]))
        grads = copies[k][:1] + sharded[k] + copies[k][1:]
        call = T.GradClip(grads, 0.05, outs=[torch.empty_like(g) for g in grads], group="tp", replicated=copies[k])
        call.launch()
        assert call.check_status() == 0
        # FP64 sums of squares each right to 2^-22, one square root and three FP32 roundings
        assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm and abs(float(call.coef) - coef) <= 2.0 ** -20 * coef
        for g, o in zip(grads, call.outs):
            assert bool(((o.double() - g.double() * coef).abs() <= 2.0 ** -19 * (g.double() * coef).abs()).all())
        calls.append(call)
    with pytest.raises(ValueError, match="replicated"):
        T.GradClip([ranks[0].dW1], 1.0, group="tp", replicated=[ranks[0].dconf_b])


def test_clip_refuses_tensors_that_share_memory(T):
    """A part listed beside the whole, one output for two gradients, an output on another's
    gradient: each would be scaled twice or read half written."""
    buf, more = torch.randn(100, device="cuda"), torch.empty(100, device="cuda")
    a, b, c = buf[:40], buf[40:], buf[30:60]
    T.GradClip([a, b], 1.0).launch()
    T.GradClip([a, b], 1.0, outs=[a, more[:60]]).launch()
    T.GradClip([a, buf[40:40], b], 1.0, outs=[more[:40], more[10:10], more[40:]]).launch()
    for grads, outs in (([a, b, c], None), ([buf, a], None), ([a, buf[40:80]], [more[:40], more[:40]]),
                        ([a, buf[40:80]], [more[:40], more[39:79]]), ([a, buf[40:80]], [buf[40:80], a]),
                        ([a], [buf[8:48]])):
        with pytest.raises(ValueError, match="overlap|listed twice"):
            T.GradClip(grads, 1.0, outs=outs)


@pytest.mark.parametrize("R,V,H,kept", [(64, 151936, 64, True), (80, 151936, 64, False), (160, 151936, 448, False),
                                        (160, 151936, 512, True), (200, 151936, 640, False),
                                        (200, 151936, 704, True), (600, 151936, 704, False)])
def test_linear_ce_keeps_logits_where_that_is_faster(T, R, V, H, kept):
    """By the logits' size and the hidden size; the results hold either way."""
    h, w, t, a = lce_inputs(R, V, H, 7, seed=36)
    call = T.LinearCE(h, w, t, row_weight=a)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    head = call.ws[call.ws_ptr.value - call.ws.data_ptr():][:32].view(torch.int32).tolist()
    assert head[1] == R - 7 and head[4] == kept  # the workspace's header: labelled rows, logits kept
    lce_compare(call, O.linear_ce(h, w, t, a), H, V)


def test_empty_batches_are_refused(T):
    """No rows: refused by name before anything is launched; empty tensors among others to clip
    are not (also where they lie at another's first element)."""
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    table = torch.zeros(5, 8, device="cuda")
    with pytest.raises(ValueError, match="at least one"):
        T.Embedding(none, table)
    with pytest.raises(ValueError, match="at least one"):
        T.EmbeddingGrad(none, table[:0], 5)
    with pytest.raises(ValueError, match="at least one"):
        T.LinearCE(table[:0].to(torch.bfloat16), table.to(torch.bfloat16), none)
    buf = torch.ones(64, device="cuda")
    call = T.GradClip([buf[:0], buf, buf[64:]], 1.0)
    call.launch()
    assert abs(float(call.norm) - 8.0) <= 2.0 ** -20


@pytest.mark.parametrize("given", [False, True])
def test_what_a_dropped_call_allocated_waits_for_its_stream(T, given):
    """A call built on one stream, launched on another behind other work there and dropped:
    its memory goes to nobody before that launch is done."""
    h, w, t, a = lce_inputs(300, 5000, 256, 9, seed=37)
    ids = torch.randint(0, 700, (300,), device="cuda")
    g = torch.randn(100000, device="cuda")
    out = torch.empty_like(g)
    made = [lambda: T.LinearCE(h, w, t, row_weight=a, dhidden=False, dweight=False),
            lambda: T.EmbeddingGrad(ids, h, 700, dtype=torch.bfloat16), lambda: T.Embedding(ids, w),
            lambda: T.GradClip([g], 1.0, outs=[out])]
    side = torch.cuda.Stream()
    for make in made:  # once before, so that nothing below has to load code first
        call = make()
        (call.forward if isinstance(call, T.LinearCE) else call.launch)(stream=side.cuda_stream if given else None)
        torch.cuda.synchronize()
        del call
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)  # half a second of waiting
    for make in made:
        call = make()
        run = call.forward if isinstance(call, T.LinearCE) else call.launch
        if given:
            run(stream=side.cuda_stream)
        else:
            with torch.cuda.stream(side):
                run()
        held = {x.data_ptr(): x.numel() * x.element_size() for x in (call.ws, getattr(call, "out", None),
                                                                    getattr(call, "norm", None)) if isinstance(x, torch.Tensor)}
        assert not side.query()
        del call, run
        again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in held.values() for _ in range(3)]
        assert not side.query() and not held.keys() & {x.data_ptr() for x in again}
    torch.cuda.synchronize()


# ------------------------------------------------- offsets that 32 bits do not hold
def test_embedding_past_32_bits(T):
    """A table of 2.46e9 elements: rows at its end, looked up and given gradients."""
    Vt, D, R = 600001, 4096, 700
    g = torch.Generator(device="cuda").manual_seed(50)
    ids = torch.randint(0, Vt, (R,), generator=g, device="cuda")
    ids[:3] = torch.tensor([Vt - 1, Vt - 2, 524288], device="cuda")  # (524288 x 4096 = 2^31)
    table = torch.zeros(Vt, D, dtype=torch.bfloat16, device="cuda")
    table[ids] = torch.randn(R, D, generator=g, device="cuda").to(torch.bfloat16)
    look = T.Embedding(ids, table, scale=2.0)
    look.launch()
    assert look.check_status() == 0 and torch.equal(look.out, table[ids] * 2)
    grad = T.EmbeddingGrad(ids, look.out, Vt, out=table.fill_(7.0))
    grad.launch()
    assert grad.check_status() == 0
    touched, where = torch.unique(ids, return_inverse=True)
    want = torch.zeros(touched.numel(), D, dtype=torch.float64, device="cuda").index_add_(0, where, look.out.double())
    mag = torch.zeros_like(want).index_add_(0, where, look.out.double().abs())
    n = torch.bincount(where)[:, None]
    assert bool(((table[touched].double() - want).abs() <= 1.01 * ((n + 2) * U32 * mag + U16 * want.abs())).all())
    table[touched] = 0
    assert not bool(table.any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_clip_past_32_bits(T, dtype):
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=dtype, device="cuda")
    g[::4097] = -2.0
    more = n // 4097 + 1
    norm = (0.25 * (n - more) + 4.0 * more) ** 0.5
    call = T.GradClip([g, torch.zeros(3, device="cuda")], norm / 2)
    call.launch()
    assert call.check_status() == 0
    # FP64 sums of squares each right to 2^-22, one square root and three FP32 roundings
    assert abs(float(call.norm) - norm) <= 2.0 ** -21 * norm
    coef = norm / 2 / (norm + 1e-6)
    tol = (2.0 ** -20 + 1.01 * _u(dtype)) * coef
    assert float((g[::4097].double() + 2.0 * coef).abs().max()) <= 2.0 * tol
    g[::4097] = g[1]
    assert bool((g == g[1]).all()) and abs(float(g[1]) - 0.5 * coef) <= 0.5 * tol


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_ce_past_32_bits(T, dtype):
    """A head of 2.46e9 elements; its gradient compared in the rows of labels, around the
    places that 31 and 32 bits of elements and bytes end at, and at the end."""
    R, V, H = 70, 300001, 8192
    h, w, t, a = lce_inputs(R, V, H, 4, seed=51)
    t[:2] = torch.tensor([V - 1, 262144], device="cuda")
    call = T.LinearCE(h, w, t, row_weight=a, dweight_dtype=dtype)
    call.forward()
    call.backward()
    assert call.check_status() == 0
    live = t != -100
    hd, td = h[live].double(), t[live]
    z = torch.cat([hd @ p.double().T for p in w.split(20000)], dim=1)
    lse = torch.logsumexp(z, dim=1)
    reach = float(max((h[live].float().abs() @ p.float().abs().T).max() for p in w.split(20000)))
    E = (32 + H / 512 + 2) * 2.0 ** -23 * reach
    assert bool(((call.lse_rows[live].double() - lse).abs() <= E + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all())
    ad = a[live].double()[:, None]
    p = torch.exp(z - lse[:, None]) * ad
    dz = p.clone()
    dz[torch.arange(td.numel(), device="cuda"), td] -= ad[:, 0]
    P = 2 * ((H / 16 + 2) * 2.0 ** -23 * reach + E) + 2.0 ** -20
    rows = torch.cat([td, torch.arange(0, V, 9973, device="cuda"), torch.arange(131070, 131075, device="cuda"),
                      torch.arange(262142, 262147, device="cuda"), torch.arange(V - 300, V, device="cuda")])
    want, mag = dz[:, rows].T @ hd, dz[:, rows].abs().T @ hd.abs()
    tol = P * (p[:, rows].T @ hd.abs()) + (U16 + (R / 16 + 2) * 2.0 ** -23) * mag + _u(dtype) * want.abs()
    assert bool(((call.dweight[rows].double() - want).abs() <= tol * 1.01).all())
    dh = mag = pmag = 0
    for v0 in range(0, V, 20000):
        part = w[v0:v0 + 20000].double()
        dh = dh + dz[:, v0:v0 + 20000] @ part
        mag = mag + dz[:, v0:v0 + 20000].abs() @ part.abs()
        pmag = pmag + p[:, v0:v0 + 20000] @ part.abs()
    tol = P * pmag + (U16 + (V / 16 + 2) * 2.0 ** -23) * mag + U16 * dh.abs()
    assert bool(((call.dhidden[live].double() - dh).abs() <= tol * 1.01).all())
    assert not bool(call.dhidden[~live].any())
