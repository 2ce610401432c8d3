"""Routing of few slots whose tokens one workgroup would take in many rounds."""
import numpy as np
import pytest

import bit_gemm_token_amd as bgt

# (T, E, k), at most 1024 slots: a workgroup takes 128 tokens of 8 experts at once, 64 of
# 16 to 64, 32 of 128, 16 of 256
MANY_ROUNDS = [(1024, 256, 1), (512, 256, 2), (64, 256, 16), (256, 256, 1), (1024, 64, 1), (512, 64, 2),
               (128, 128, 8), (1024, 8, 1), (81, 200, 1)]
FEW_ROUNDS = [(1, 8, 2), (128, 8, 8), (256, 8, 2), (64, 64, 16), (32, 128, 8), (16, 256, 16), (32, 256, 8)]


@pytest.mark.parametrize("T,E,k", MANY_ROUNDS)
def test_many_rounds_go_to_several_workgroups(T, E, k):
    # the workspace is the workgroups' counts: there is none where one workgroup does it all
    assert bgt.lib().bgt_moe_sort_workspace_bytes(T, E, k) >= 2 * 4 * E


@pytest.mark.parametrize("T,E,k", FEW_ROUNDS)
def test_few_rounds_are_one_launch(T, E, k):
    assert bgt.lib().bgt_moe_sort_workspace_bytes(T, E, k) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", MANY_ROUNDS + FEW_ROUNDS)
@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_route_and_sort(T, E, k, norm):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"route T={T} E={E} k={k} {norm}", flush=True)
    g = np.random.default_rng(T + E + k)
    v = np.round(g.standard_normal((T, E)) * 8).astype(np.float32) / 8         # ties
    v[g.random((T, E)) < 0.1] = -np.inf
    v[T // 2] = -np.inf
    w, ids, offs, tok, pos = [t.cpu().numpy() for t in bgt.moe_route(torch.from_numpy(v).cuda(), k, norm=norm)]
    order = np.argsort(-v, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(v, order, 1).astype(np.float64)
    want = np.where(top > -np.inf, order, -1)
    np.testing.assert_array_equal(ids, want)
    flat, slot = want.reshape(-1), np.arange(T * k)
    n = int((flat >= 0).sum())
    by = np.argsort(np.where(flat >= 0, flat, E), kind="stable")
    np.testing.assert_array_equal(offs, np.searchsorted(flat[by[:n]], np.arange(E + 1)))
    np.testing.assert_array_equal(tok, np.where(slot < n, by // k, -1))
    where = np.full(T * k, -1)
    where[by[:n]] = slot[:n]
    np.testing.assert_array_equal(pos.reshape(-1), where)
    base = top if norm == "chosen" else v.astype(np.float64)
    m = np.where(top[:, :1] > -np.inf, top[:, :1], 0.0)
    total = np.exp(base - m).sum(1, keepdims=True)
    p = np.divide(np.exp(top - m), total, out=np.zeros_like(top), where=total > 0)
    # a difference rounded once, an exponential, a tree of sums of depth at most 12, a division
    far = np.abs(np.where(want >= 0, top, m) - m)
    assert (np.abs(w - p) <= p * (far + 48) * 2 * 2.0 ** -24 + 1e-37).all()
    for a, b in zip(bgt.moe_sort(torch.from_numpy(ids).cuda(), E), (offs, tok, pos)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
