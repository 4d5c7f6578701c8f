"""Prompt attention and the weight of prompt tokens on the GPU against float64.

Tolerances, from the arithmetic: u = eps / 2 of the cache dtype, A = sum_j p |v|, S = max_j
sum_d |q k| / sqrt(D).
- A score's products are exact in float32 and its D additions lose at most D 2^-24 S (twice that for
  truncating adders); the exponent's argument is rounded to 2^-24 of its size, at most about 2 S.
  So a weight is off by at most e_p = 2 D 2^-24 S + 4 S 2^-24 + 2^-20 relative (the last term: ex2,
  reciprocal, the sum of weights).
- out: u |o| for the final rounding, u A for the weights' rounding, 2 e_p A.
- lse: e_p + 2^-22 |lse| absolute. mass: the weights' e_p, relative, with the float32 lse given.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import prompt_int4_oracle as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def _draw(seed, T, Hq, Hkv, D, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g)
    x[:, Hq:, 3] *= 8.0
    return (x * gain).to(DT[dtype])


def _cu(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32)


def _check(lens, Hq, Hkv, D, dtype, x, out, lse, mass, first=0):
    f = lambda t: t.double().cpu().numpy()
    q, k, v = f(x[:, :Hq]), f(x[:, Hq:Hq + Hkv]), f(x[:, Hq + Hkv:])
    out, lse32, mass = f(out), lse.cpu().numpy(), f(mass)
    a = first
    for n in lens:
        s = slice(a, a + n)
        if n:
            o, ls, A, S = P.prompt_attend(q[s], k[s], v[s])
            ep = ((2 * D + 4) * S + 16) * 2.0 ** -24
            assert (np.abs(out[s] - o) <= U[dtype] * (np.abs(o) + A) + 2 * ep[..., None] * A + 1e-30).all()
            assert (np.abs(lse32[s] - ls) <= ep + 2.0 ** -22 * np.abs(ls)).all()
            m = P.prompt_mass(q[s], k[s], lse32[s].astype(np.float64))
            assert (np.abs(mass[s] - m) <= ep.max() * m + 1e-30).all()
        a += n


def _run(lens, Hq, Hkv, D, dtype, seed=0, gain=1.0):
    from kv_cache_eviction_gqa_b200 import binding as B
    x = _draw(seed, sum(lens), Hq, Hkv, D, dtype, gain).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = _cu(lens).cuda()
    out, lse, status = B.prompt_attend(q, k, v, cu)
    mass, status2 = B.prompt_mass(q, k, lse, cu)
    assert status.tolist() == [0, 0] and status2.tolist() == [0, 0]
    _check(lens, Hq, Hkv, D, dtype, x, out, lse, mass)


# one kv head's tile holds floor(128 / G) positions: lengths around one and two tiles and around the
# 128-key tiles, for every group size, both types and head dims
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_lengths_around_tiles(G, D, dtype):
    pt = 128 // G
    lens = [1, pt - 1, pt, pt + 1, 2 * pt, 2 * pt + 1, 127, 128, 129, 0, 257]
    _run(lens, 2 * G, 2, D, dtype, seed=G)


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype", [
    ([1], 1, 1, 64, "bf16"),
    ([1], 8, 1, 128, "fp16"),
    ([0, 0, 3, 0], 4, 2, 128, "bf16"),
    ([700, 1, 1300], 32, 8, 128, "bf16"),
    ([2049], 5, 1, 128, "fp16"),
    ([511, 900], 12, 4, 64, "bf16"),
    ([3] * 70, 4, 1, 64, "fp16"),          # more sequences than a warp has lanes
    ([1000], 40, 8, 64, "fp16"),
])
def test_prompts_match_float64(lens, Hq, Hkv, D, dtype):
    _run(lens, Hq, Hkv, D, dtype, seed=len(lens))


def test_steep_softmax():
    """Scores of several hundred: the running maximum rises often and far."""
    _run([600], 4, 1, 128, "bf16", seed=3, gain=4.0)


def test_rising_scores():
    """Each key beats all before it, so the maximum moves in every tile, by more and by less than 2^8."""
    from kv_cache_eviction_gqa_b200 import binding as B
    n, D = 1100, 64
    for step in (0.02, 0.5):
        x = _draw(5, n, 2, 1, D, "fp16", 0.25)
        x[:, :2, 0] = 8.0
        x[:, 2, 0] = (torch.arange(n) * step).to(x.dtype)
        x = x.cuda()
        out, lse, _ = B.prompt_attend(x[:, :2], x[:, 2:3], x[:, 3:], _cu([n]).cuda())
        mass, _ = B.prompt_mass(x[:, :2], x[:, 2:3], lse, _cu([n]).cuda())
        _check([n], 2, 1, D, "fp16", x, out, lse, mass)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 64)])
def test_foreign_rows_do_not_reach_a_sequence(Hq, Hkv, D):
    """Rows before the first and behind the last sequence hold NaN and infinities, and so do the rows of
    a neighbour: what they touch stays as it was, the others' results are finite and right."""
    from kv_cache_eviction_gqa_b200 import binding as B
    lens, first, T = [70, 200, 5], 9, 9 + 275 + 30
    x = _draw(11, T, Hq, Hkv, D, "bf16")
    x[:first] = float("nan")
    x[first + 275:] = float("inf")
    x[first + 70:first + 270] = float("nan")                       # the whole second sequence
    x = x.cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    mass = torch.full((T, Hkv), 7.0, device="cuda")
    cu = _cu(lens, first).cuda()
    B.prompt_attend(q, k, v, cu, out=out, lse=lse)
    B.prompt_mass(q, k, lse, cu, mass=mass)
    for t in (out, lse, mass):
        assert (t[:first] == 7).all() and (t[first + 275:] == 7).all()
    for s, n in ((first, 70), (first + 270, 5)):
        r = slice(s, s + n)
        _check([n], Hq, Hkv, D, "bf16", x[r], out[r], lse[r], mass[r])


def test_strided_and_separate_tensors_agree():
    from kv_cache_eviction_gqa_b200 import binding as B
    x = _draw(4, 300, 8, 2, 64, "bf16").cuda()
    wide = torch.zeros((300, 20, 64), dtype=x.dtype, device="cuda")
    wide[:, 3:15] = x
    cu = _cu([100, 200]).cuda()
    a = B.prompt_attend(x[:, :8].contiguous(), x[:, 8:10].contiguous(), x[:, 10:].contiguous(), cu)
    b = B.prompt_attend(wide[:, 3:11], wide[:, 11:13], wide[:, 13:15], cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    m = B.prompt_mass(x[:, :8].contiguous(), x[:, 8:10].contiguous(), a[1], cu)[0]
    assert torch.equal(m, B.prompt_mass(wide[:, 3:11], wide[:, 11:13], a[1], cu)[0])


@pytest.mark.parametrize("bounds,bad", [([0, 10, 5, 20], 1), ([0, 10, 31], 1), ([-1, 10, 20], 0)])
def test_bad_bounds_are_recorded(bounds, bad):
    from kv_cache_eviction_gqa_b200 import binding as B
    x = _draw(4, 30, 4, 1, 64, "bf16").cuda()
    out = torch.full((30, 4, 64), 7.0, dtype=x.dtype, device="cuda")
    mass = torch.full((30, 1), 7.0, device="cuda")
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    _, lse, status = B.prompt_attend(x[:, :4], x[:, 4:5], x[:, 5:], cu, out=out)
    _, s2 = B.prompt_mass(x[:, :4], x[:, 4:5], torch.zeros_like(lse), cu, mass=mass)
    assert status.tolist() == [-1, bad] and s2.tolist() == [-1, bad]
    assert (out == 7).all() and (mass == 7).all()


def test_captured_and_on_a_side_stream():
    from kv_cache_eviction_gqa_b200 import binding as B
    x = _draw(8, 400, 8, 2, 128, "bf16").cuda()
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    cu, status = _cu([150, 250]).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    want, lse0, _ = B.prompt_attend(q, k, v, cu, status=status)
    out, lse, mass = torch.empty_like(want), torch.empty_like(lse0), torch.empty((400, 2), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.prompt_attend(q, k, v, cu, out=out, lse=lse, status=status)
        B.prompt_mass(q, k, lse, cu, mass=mass, status=status)
    x.mul_(0.5)                              # a replay reads what the tensors hold then
    cu.copy_(_cu([399, 1]))
    g.replay()
    torch.cuda.synchronize()
    _check([399, 1], 8, 2, 128, "bf16", x, out, lse, mass)


def test_binding_refusals():
    from kv_cache_eviction_gqa_b200 import binding as B
    x = torch.zeros((16, 6, 64), dtype=torch.bfloat16, device="cuda")
    cu = _cu([16]).cuda()
    q, k, v = x[:, :4], x[:, 4:5], x[:, 5:]
    with pytest.raises(ValueError):
        B.prompt_attend(q, k.float(), v, cu)
    with pytest.raises(ValueError):
        B.prompt_attend(q, k[:8], v, cu)
    with pytest.raises(ValueError):
        B.prompt_attend(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, cu)
    with pytest.raises(ValueError):
        B.prompt_attend(q, k, v, cu.long())
    with pytest.raises(ValueError):
        B.prompt_attend(q, k, v, cu.cpu())
    with pytest.raises(ValueError):
        B.prompt_mass(q, k, torch.zeros((16, 5), device="cuda"), cu)
    with pytest.raises(RuntimeError, match="invalid"):
        B.prompt_attend(x[:, :3], x[:, 3:5], x[:, 3:5], cu)             # 3 query heads over 2


@pytest.mark.slow
def test_long_prompt_sampled_rows():
    """A 20 000-token sequence: sampled rows of the output and lse, and all of one key's weight."""
    from kv_cache_eviction_gqa_b200 import binding as B
    n, D = 20000, 128
    x = _draw(21, n, 4, 1, D, "bf16").cuda()
    q, k, v = x[:, :4], x[:, 4:5], x[:, 5:]
    cu = _cu([n]).cuda()
    out, lse, _ = B.prompt_attend(q, k, v, cu)
    mass, _ = B.prompt_mass(q, k, lse, cu)
    kd, vd = k[:, 0].double(), v[:, 0].double()
    for i in (0, 127, 128, 9999, 19871, 19999):
        s = q[i].double() @ kd[:i + 1].T / D ** 0.5
        p = torch.softmax(s, -1)
        o, A = p @ vd[:i + 1], p @ vd[:i + 1].abs()
        ep = ((2 * D + 4) * (q[i].double().abs() @ kd[:i + 1].abs().T / D ** 0.5).max().item() + 16) * 2.0 ** -24
        assert ((out[i].double() - o).abs() <= U["bf16"] * (o.abs() + A) + 2 * ep * A).all()
        assert ((lse[i].double() - torch.logsumexp(s, -1)).abs() <= ep + 2.0 ** -22 * 20).all()
        w = torch.exp(q[i:].double().flatten(0, 1) @ kd[i] / D ** 0.5 - lse[i:].double().flatten()).sum()
        assert abs(mass[i, 0].item() - w.item()) <= (ep + 2.0 ** -18) * w.item()
    assert abs(mass.double().sum().item() - 4 * n) <= 4 * n * 2.0 ** -12


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_shows_in_every_weight_it_gives(bad):
    """Sixteen sequences, each with one query row that is not finite, at every place of a run of 16 columns:
    its output and the weights of all keys it sees are NaN, nothing else is."""
    from kv_cache_eviction_gqa_b200 import binding as B
    n, Hq, Hkv, D = 600, 4, 2, 64
    x = _draw(17, 16 * n, Hq, Hkv, D, "bf16")
    rows = [b * n + 484 + b for b in range(16)]
    x[rows, 1] = bad                                     # of kv head 0
    x = x.cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = _cu([n] * 16).cuda()
    out, lse, status = B.prompt_attend(q, k, v, cu)
    mass, _ = B.prompt_mass(q, k, lse, cu)
    assert status.tolist() == [0, 0]
    hit = torch.zeros((16 * n, Hq), dtype=torch.bool)
    hit[rows, 1] = True
    assert torch.equal(out.isnan().all(-1).cpu(), hit) and torch.equal(out.isnan().any(-1).cpu(), hit)
    want = torch.zeros((16 * n, Hkv), dtype=torch.bool)
    for b, i in enumerate(rows):
        want[b * n:i + 1, 0] = True
    assert torch.equal(mass.isnan().cpu(), want)
