"""The balance loss over sequences and its gradient on the GPU against the
formulas in 64 bits, against differences, and against the layer's own loss."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_53_b200 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

# A score is off by the special-function exponential (2^-22), the rounding of
# its argument (2^-24 |z - max| / ln 2, |z - max| below 25 where a score
# matters), the reciprocal and the sums over 256 experts by pairs (8 roundings):
# under 4e-6 of itself; the sums over a chunk of tokens add fewer than 128
# roundings of 2^-24.
REL = 1.2e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_layer_53_b200 import build
    build.build()
    M.library()
    assert torch.cuda.is_available()


def np64(t):
    return t.detach().double().cpu().numpy()


def scores_of(z, kind):
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if kind == "softmax":
            top = z.max(1, keepdims=True)
            p, m = np.exp(z - np.where(np.isfinite(top), top, 0)), np.ones_like(z)
        else:
            s = np.exp(-np.logaddexp(0, -z))
            p, m = s, np.exp(-np.logaddexp(0, z))
        t = p.sum(1, keepdims=True)
        return np.where(t > 0, p / np.where(t > 0, t, 1), 0), m


def reference(z, ids, cuts, mask, kind):
    """(loss, counts, weight, dz, how far dz may be off)."""
    N, E = z.shape
    S = len(cuts) - 1
    valid = np.ones(N, bool) if mask is None else mask
    z = np.where(valid[:, None], z, 0.0)
    p, m = scores_of(z, kind)
    counts, T, P = np.zeros((S, E), np.int64), np.zeros(S), np.zeros((S, E))
    for s in range(S):
        r = np.arange(cuts[s], cuts[s + 1])
        r = r[valid[r]]
        T[s] = len(r)
        got = ids[r].reshape(-1)
        counts[s] = np.bincount(got[(got >= 0) & (got < E)], minlength=E)
        P[s] = p[r].sum(0)
    full = (T > 0).sum()
    weight = np.where(T > 0, E / np.maximum(T, 1) ** 2 / max(full, 1), 0.0)
    loss = (weight * (counts * P).sum(1)).sum()
    dz, tol = np.zeros((N, E)), np.zeros((N, E))
    for s in range(S):
        r = np.arange(cuts[s], cuts[s + 1])
        r = r[valid[r]]
        c = weight[s] * counts[s]
        dot = (p[r] * c).sum(1, keepdims=True)
        dz[r] = p[r] * m[r] * (c - dot)
        tol[r] = REL * p[r] * m[r] * (c + dot)
    return loss, counts, weight, dz, tol


def inputs(N, E, k, S, dtype, seed, padded=False, ties=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = (2 * torch.randn((N, E), generator=g, device=DEV)).to(dtype)
    ids = torch.rand((N, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    cuts = np.sort(np.random.RandomState(seed).randint(0, N + 1, S - 1)) if S > 1 else np.zeros(0, int)
    cuts = np.concatenate([[0], cuts, [N]]).astype(np.int32)
    mask = torch.rand(N, generator=g, device=DEV) > 0.3 if padded else None
    return z, ids.contiguous(), cuts, mask


def run(z, ids, cuts, mask, kind, **kw):
    off = torch.from_numpy(cuts).to(DEV)
    fwd = M.moe_balance_loss(z, ids, seq_offsets=off, token_mask=mask, scores=kind)
    return fwd, M.moe_balance_loss_backward(z, fwd, seq_offsets=off, token_mask=mask, scores=kind, **kw)


def check(z, ids, cuts, mask, kind):
    fwd, dz = run(z, ids, cuts, mask, kind)
    loss, counts, weight, want, tol = reference(np64(z), ids.cpu().numpy(), cuts, None if mask is None else mask.cpu().numpy(), kind)
    assert np.array_equal(fwd["counts"].cpu().numpy(), counts)
    assert np.all(np.abs(np64(fwd["seq_weight"]) - weight) <= 2.0 ** -24 * weight)
    assert abs(float(fwd["loss"]) - loss) <= REL * abs(loss), (float(fwd["loss"]), loss)
    bad = ~(np.abs(np64(dz) - want) <= tol + 1e-37)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())
    assert int(fwd["status"]) == 0
    return fwd, dz


@pytest.mark.parametrize("E", [1, 3, 4, 6, 8, 16, 24, 33, 64, 100, 128, 200, 256])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_widths(E, kind, dtype):
    check(*inputs(301, E, min(E, 3), 5, dtype, E, padded=E % 2 == 0), kind)


@pytest.mark.parametrize("N,S", [(1, 1), (2, 7), (31, 1), (32, 2), (33, 33), (1000, 400), (5000, 3), (40000, 1), (70001, 9)])
@pytest.mark.parametrize("padded", [False, True])
def test_lengths(N, S, padded):
    check(*inputs(N, 60, 6, S, F32, N + S, padded), "softmax")
    check(*inputs(N, 8, 2, S, F32, N + S, padded), "sigmoid")


@pytest.mark.parametrize("E,k", [(100, 4), (33, 3), (200, 8), (7, 2)])
def test_millions_of_tokens_with_equal_scores(E, k):
    """Equal scores round the same way at every addition: runs of fp32 additions stay short however many tokens there are.
    Bound as for any length: REL, which has room for fewer than 128 roundings."""
    N = 8_000_000
    z = torch.zeros((N, E), device=DEV)
    ids = (torch.arange(N * k, device=DEV) % E).view(N, k).to(torch.int32)
    for kind in ("softmax", "sigmoid"):
        fwd = M.moe_balance_loss(z, ids, scores=kind)
        assert int(fwd["counts"].sum()) == N * k and int(fwd["status"]) == 0
        assert abs(float(fwd["loss"]) - k) <= REL * k, float(fwd["loss"])   # sum_e cnt_e / N * E / E = k


def test_no_tokens():
    for N, cuts, mask in ((0, [0, 0, 0], None), (9, [0, 0, 9], torch.zeros(9, dtype=torch.bool, device=DEV))):
        z, ids = torch.randn((N, 8), device=DEV), torch.zeros((N, 2), dtype=torch.int32, device=DEV)
        fwd, dz = run(z, ids, np.array(cuts, np.int32), mask, "softmax")
        assert float(fwd["loss"]) == 0 and not fwd["counts"].any() and not fwd["seq_weight"].any() and not dz.any()


def test_one_sequence_is_the_layers_loss():
    """Softmax scores of one unpadded sequence: moe_aux_loss of the same probabilities and ids; k at balance."""
    z, ids, cuts, _ = inputs(700, 64, 6, 1, F32, 5)
    fwd = M.moe_balance_loss(z, ids)
    cfg = M.make_config(700, 64, 64, 64, 6, dtype="f32")
    aux, counts, _ = M.moe_aux_loss(cfg, torch.softmax(z.double(), 1).float(), ids)
    assert abs(float(aux) - float(fwd["loss"])) <= REL * float(aux)
    assert torch.equal(counts, fwd["counts"][0])
    even = (torch.arange(64 * 6, device=DEV).view(64, 6) % 64).to(torch.int32)
    assert abs(float(M.moe_balance_loss(torch.zeros((64, 64), device=DEV), even)["loss"]) - 6) <= 6 * REL


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_masked_experts_and_rows_without_any(kind):
    z, ids, cuts, mask = inputs(200, 24, 4, 3, F32, 7)
    z[:, 5] = -float("inf")            # an expert that is switched off
    z[17] = -float("inf")              # a token with no expert left
    z[18, 1:] = -float("inf")          # a token with one
    z[19] = torch.finfo(F32).min       # the type's lowest value throughout: an even softmax
    if kind == "sigmoid":
        z[19] = -80.0                  # sigmoids far below 1, their ratios even
    fwd, dz = check(z, ids, cuts, mask, kind)
    assert not dz[torch.isinf(z)].any() and torch.isfinite(dz).all()


def test_very_negative_sigmoid_scores_keep_their_ratios():
    z, ids, cuts, _ = inputs(64, 16, 2, 1, F32, 8)
    check(z - 60.0, ids, cuts, None, "sigmoid")
    check(z - 120.0, ids, cuts, None, "sigmoid")   # beyond the exponent range of fp32


def test_what_padding_holds_does_not_matter():
    z, ids, cuts, mask = inputs(300, 33, 4, 4, F32, 9, padded=True)
    want, dz = check(z, ids, cuts, mask, "softmax")
    z2, ids2 = z.clone(), ids.clone()
    z2[~mask] = float("nan")
    ids2[~mask] = -1
    got, dz2 = run(z2, ids2, cuts, mask, "softmax")
    assert all(torch.equal(got[k], want[k]) for k in want) and torch.equal(dz, dz2)
    assert not dz2[~mask].any()


def test_tokens_of_no_sequence():
    z, ids, _, _ = inputs(100, 8, 2, 1, F32, 3)
    cuts = np.array([11, 40, 40, 77], np.int32)
    fwd, dz = check(z, ids, cuts, None, "softmax")
    assert not dz[:11].any() and not dz[77:].any()


def test_a_nan_logit_of_a_counted_token_shows():
    z, ids, cuts, _ = inputs(50, 8, 2, 2, F32, 4)
    z[3, 2] = float("nan")
    fwd, dz = run(z, ids, cuts, None, "softmax")
    assert torch.isnan(fwd["loss"]).all() and torch.isnan(dz[3]).all()


def test_bad_ids_and_repeated_ids():
    z, ids, cuts, _ = inputs(90, 8, 3, 2, F32, 6)
    ids[:, 1] = ids[:, 0]               # the same expert twice counts twice
    check(z, ids, cuts, None, "softmax")
    ids[5, 2], ids[60, 0] = 8, -1       # left out, and reported
    fwd, dz = run(z, ids, cuts, None, "softmax")
    loss, counts, _, want, tol = reference(np64(z), ids.cpu().numpy(), cuts, None, "softmax")
    assert np.array_equal(fwd["counts"].cpu().numpy(), counts) and int(fwd["status"]) == 6
    assert abs(float(fwd["loss"]) - loss) <= REL * loss and np.all(np.abs(np64(dz) - want) <= tol + 1e-37)


@pytest.mark.parametrize("cuts", [[0, 50, 20, 90], [0, 10, 20, 91], [-1, 10, 20, 90]])
def test_bad_offsets_are_reported(cuts):
    z, ids, _, _ = inputs(90, 8, 3, 1, F32, 6)
    fwd, dz = run(z, ids, np.array(cuts, np.int32), None, "softmax")
    assert int(fwd["status"]) == 1


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_against_differences(kind):
    """Central differences of the 64-bit loss: step 1e-4, error of the quotient h^2 |L'''| / 6 (below 1e-8 here)."""
    z, ids, cuts, mask = inputs(24, 6, 2, 3, F32, 12, padded=True)
    _, dz = run(z, ids, cuts, mask, kind)
    z64, i, m = np64(z), ids.cpu().numpy(), mask.cpu().numpy()
    h = 1e-4
    for n in range(24):
        for e in range(6):
            up, dn = z64.copy(), z64.copy()
            up[n, e] += h
            dn[n, e] -= h
            diff = (reference(up, i, cuts, m, kind)[0] - reference(dn, i, cuts, m, kind)[0]) / (2 * h)
            assert abs(diff - float(dz[n, e])) <= 1e-6


def test_coefficients():
    z, ids, cuts, _ = inputs(120, 16, 2, 2, F32, 2)
    _, dz = run(z, ids, cuts, None, "softmax")
    up = torch.tensor([4.0], device=DEV)
    assert torch.equal(run(z, ids, cuts, None, "softmax", coef=0.5)[1], dz * 0.5)   # powers of two: exact
    assert torch.equal(run(z, ids, cuts, None, "softmax", coef=0.5, dloss=up)[1], dz * 2.0)
    assert not run(z, ids, cuts, None, "softmax", coef=0.0)[1].any()


def test_equal_inputs_give_equal_bits():
    z, ids, cuts, mask = inputs(30011, 128, 8, 17, F32, 1, padded=True)
    first = run(z, ids, cuts, mask, "sigmoid")
    for _ in range(3):
        again = run(z, ids, cuts, mask, "sigmoid")
        assert all(torch.equal(first[0][k], again[0][k]) for k in first[0]) and torch.equal(first[1], again[1])


def test_captured_step_replayed_on_new_inputs():
    a, b = inputs(500, 24, 3, 4, F32, 1, padded=True), inputs(500, 24, 3, 4, F32, 2, padded=True)
    off = torch.from_numpy(a[2]).to(DEV)
    z, ids, mask = a[0].clone(), a[1].clone(), a[3].clone()
    step = lambda: (lambda f: (f, M.moe_balance_loss_backward(z, f, seq_offsets=off, token_mask=mask)))(  # noqa: E731
        M.moe_balance_loss(z, ids, seq_offsets=off, token_mask=mask))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd, dz = step()
    for x in (a, b, a):
        z.copy_(x[0])
        ids.copy_(x[1])
        mask.copy_(x[3])
        want, wdz = run(x[0], x[1], a[2], x[3], "softmax")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(fwd[k], want[k]) for k in want) and torch.equal(dz, wdz)


@pytest.mark.parametrize("E,dtype", [(6, F32), (6, BF), (4, BF), (8, F32), (33, BF)])
def test_a_part_of_the_tokens(E, dtype):
    """Logits that start inside a larger tensor, on whatever boundary its rows leave."""
    z, ids, cuts, mask = inputs(200, E, 2, 1, dtype, E)
    check(z[37:], ids[37:], np.array([0, 50, 163], np.int32), None, "softmax")


def test_on_a_side_stream_with_a_workspace():
    z, ids, cuts, mask = inputs(5000, 64, 6, 5, F32, 1, padded=True)
    want, wdz = run(z, ids, cuts, mask, "sigmoid")
    off, side = torch.from_numpy(cuts).to(DEV), torch.cuda.Stream()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    got = M.moe_balance_loss(z, ids, seq_offsets=off, token_mask=mask.to(torch.uint8), scores="sigmoid", ws=ws, stream=side)
    dz = M.moe_balance_loss_backward(z, got, seq_offsets=off, token_mask=mask, scores="sigmoid", stream=side)
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want) and torch.equal(dz, wdz)
    with pytest.raises(M.MoeError, match="WORKSPACE"):
        M.moe_balance_loss(z, ids, seq_offsets=off, ws=ws[:1024])


def test_the_layers_probabilities_as_logits():
    """log of moe_route's probabilities are logits of the same softmax scores."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x, Wg = torch.randn((300, 64), generator=g, device=DEV), torch.randn((16, 64), generator=g, device=DEV) * 0.2
    cfg = M.make_config(300, 64, 64, 16, 4, dtype="f32")
    ids, _, probs = M.moe_route(cfg, x, Wg, want_probs=True)
    aux, counts, _ = M.moe_aux_loss(cfg, probs, ids)
    fwd = M.moe_balance_loss(probs.log(), ids)
    assert abs(float(fwd["loss"]) - float(aux)) <= REL * float(aux) and torch.equal(fwd["counts"][0], counts)


def test_router_gradient_of_a_training_step():
    """The loss from the layer's own routing, its gradient carried to W_g and x by torch: differences in 64 bits."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    N, d, E, k = 40, 64, 8, 2
    x, Wg = torch.randn((N, d), generator=g, device=DEV), torch.randn((E, d), generator=g, device=DEV) * 0.1
    cfg = M.make_config(N, d, 64, E, k, dtype="f32")
    ids, _, _ = M.moe_route(cfg, x, Wg)
    off = torch.tensor([0, 25, 40], dtype=torch.int32, device=DEV)
    z = (x.double() @ Wg.double().t()).float()
    dz = M.moe_balance_loss_backward(z, M.moe_balance_loss(z, ids, seq_offsets=off), seq_offsets=off)
    dWg = dz.double().t() @ x.double()
    z64, dirn = np64(x) @ np64(Wg).T, np64(torch.randn((E, d), generator=g, device=DEV))
    L = lambda t: reference(z64 + t * (np64(x) @ dirn.T), ids.cpu().numpy(), off.cpu().numpy(), None, "softmax")[0]  # noqa: E731
    diff = (L(1e-5) - L(-1e-5)) / 2e-5
    got = float((dWg.cpu().numpy() * dirn).sum())
    assert abs(got - diff) <= 1e-5 * np.abs(np64(dz) * (np64(x) @ dirn.T)).sum() + 1e-7


def test_refusals_of_the_binding():
    z, ids, cuts, _ = inputs(20, 8, 2, 1, F32, 1)
    with pytest.raises(ValueError, match="topk_ids"):
        M.moe_balance_loss(z, ids.long())
    with pytest.raises(ValueError, match="token_mask"):
        M.moe_balance_loss(z, ids, token_mask=torch.ones(19, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError, match="token_mask"):
        M.moe_balance_loss(z, ids, token_mask=torch.ones(20, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_balance_loss(z.t().contiguous().t(), ids)
    with pytest.raises(KeyError):
        M.moe_balance_loss(z, ids, scores="tanh")
    with pytest.raises(ValueError, match="counts"):
        M.moe_balance_loss_backward(z, {"counts": torch.zeros((2, 8), dtype=torch.int32, device=DEV),
                                        "seq_weight": torch.zeros(1, device=DEV)})
