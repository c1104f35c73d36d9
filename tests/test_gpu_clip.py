"""Gradient norm, clipping and the clipped Adam step through the C ABI against
the fp64 oracle.

Tolerances: the norm and the factor are computed in double and rounded once
to fp32 (2^-24 relative; 2^-23 allows for the double sum); a clipped value is
one fp32 product of it (2^-23 more) rounded to its type (2^-24, 2^-11, 2^-8,
or half the smallest subnormal)."""
import math

import numpy as np
import pytest
import torch

from oracle import train as T
from implicit_attribute_decode_amd import ia, scenes as S
from implicit_attribute_decode_amd.pipeline import Adam, Decoder, GradClip, clip_grad_norm

from gpu_util import cuda, host, say

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TYPES = list(UNIT)


def _tensors(rng, sizes, dtypes, scale=1e-2):
    return [torch.as_tensor((rng.normal(0, scale, n) * np.exp(rng.normal(0, 1, n))).astype(np.float32),
                            device="cuda").to(dt) for n, dt in zip(sizes, dtypes)]


def _f64(t):
    return t.double().cpu().numpy()


def _check_clip(before, after, stats, max_norm):
    norm, factor = T.clip_factor(before, max_norm)
    s = host(stats).astype(np.float64)
    assert abs(s[0] - norm) <= 2.0 ** -23 * norm and abs(s[1] - factor) <= 2.0 ** -23 * factor and s[2] == 1.0
    for b, a in zip(before, after):
        tol = (UNIT[a.dtype] + 2.0 ** -22) * np.abs(b * factor) + TINY[a.dtype]
        assert np.all(np.abs(_f64(a) - b * factor) <= tol)


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [4096], [4095, 4097, 3], [257 * 1021, 1, 17], [3] * 200,
                                   [1 + (k * 977) % 9000 for k in range(170)]])
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
def test_clip_in_place_and_into_outputs(sizes, max_norm):
    rng = np.random.default_rng(len(sizes))
    g = _tensors(rng, sizes, [TYPES[k % 3] for k in range(len(sizes))])
    before = [_f64(t) for t in g]
    out = [torch.full_like(t, float("nan")) for t in g]
    stats = clip_grad_norm(g, max_norm, out)
    torch.cuda.synchronize()
    _check_clip(before, out, stats, max_norm)
    assert all(np.array_equal(_f64(t), b) for t, b in zip(g, before))  # the gradients themselves stay
    only = GradClip(g).norm(max_norm)
    assert torch.equal(only, stats) and all(np.array_equal(_f64(t), b) for t, b in zip(g, before))
    again = clip_grad_norm(g, max_norm)
    assert torch.equal(again, stats) and all(torch.equal(a, o) for a, o in zip(g, out))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [1, 3, 7])
def test_views_of_a_bucket_at_odd_offsets(dtype, shift):
    """Tensors that start at any element, ends included: nothing beside them is written."""
    rng = np.random.default_rng(shift)
    sizes = [1, 5000, 8, 4096, 33, 12289]
    flat = _tensors(rng, [shift + sum(sizes) + 9], [dtype])[0]
    keep = flat.clone()
    out = torch.full_like(flat, 7.0)
    view = lambda b: list(b[shift:shift + sum(sizes)].split(sizes))  # noqa: E731
    stats = clip_grad_norm(view(flat), 0.5, view(out[1:]) if shift == 3 else view(out))
    o = shift + 1 if shift == 3 else shift
    before = [_f64(t) for t in view(keep)]
    _check_clip(before, view(out[1:]) if shift == 3 else view(out), stats, 0.5)
    assert (out[:o] == 7.0).all() and (out[o + sum(sizes):] == 7.0).all() and torch.equal(flat, keep)
    clip_grad_norm(view(flat), 0.5)
    assert torch.equal(flat[:shift], keep[:shift]) and torch.equal(flat[shift + sum(sizes):], keep[shift + sum(sizes):])


def test_rows_of_a_wider_array():
    rng = np.random.default_rng(3)
    wide = cuda(rng.normal(0, 1, (3001, 4)).astype(np.float32))
    keep = wide.clone()
    out = torch.full((3001, 5), 9.0, device="cuda")
    stats = clip_grad_norm([wide[:, :3], wide[:, 3:]], 2.0, [out[:, 1:4], out[:, 4:]])
    _check_clip([_f64(keep[:, :3]), _f64(keep[:, 3:])], [out[:, 1:4], out[:, 4:]], stats, 2.0)
    assert (out[:, 0] == 9.0).all()
    clip_grad_norm([wide[:, :3]], 1.0)
    assert torch.equal(wide[:, 3], keep[:, 3]) and not torch.equal(wide[:, :3], keep[:, :3])
    empty = GradClip([torch.empty((0, 4), device="cuda")[:, :3], torch.empty((5, 4), device="cuda")[:, :0]])
    assert host(empty.norm(1.0)).tolist() == [0.0, 1.0, 1.0]


def test_many_dense_and_strided_tensors_of_every_type():
    """Several launches of either kind, more block sums than one pass adds by itself."""
    rng = np.random.default_rng(31)
    g, out, hold = [], [], []
    for k in range(640):
        dt = TYPES[k % 3]
        if k % 7 == 0:
            wide = _tensors(rng, [5 * (50 + k % 13)], [dt])[0].view(-1, 5)
            hold.append(wide)
            g.append(wide[:, 1:4])
            out.append(torch.empty((wide.shape[0], 3), dtype=dt, device="cuda"))
        else:
            g.append(_tensors(rng, [17_000 + 61 * (k % 97)], [dt])[0])
            out.append(torch.empty_like(g[-1]))
    before = [_f64(t) for t in g]
    stats = clip_grad_norm(g, 0.25, out)
    _check_clip(before, out, stats, 0.25)
    clip_grad_norm(g, 0.25)
    assert all(torch.equal(a, o) for a, o in zip(g, out))


def test_large_and_small_magnitudes_do_not_overflow():
    """Squares beyond fp32's range, and below it."""
    a = torch.full((5000,), 1e30, device="cuda")
    b = torch.full((5000,), 1e-30, device="cuda")
    s = host(GradClip([a, b]).norm(1.0)).astype(np.float64)
    want = float(np.float32(1e30)) * math.sqrt(5000)
    assert abs(s[0] / want - 1) <= 2.0 ** -23 and abs(s[1] * want - 1) <= 2.0 ** -23 and s[2] == 1.0
    s = host(GradClip([b]).norm(1e-30)).astype(np.float64)
    want = float(np.float32(1e-30)) * math.sqrt(5000)
    assert abs(s[0] / want - 1) <= 2.0 ** -23 and s[2] == 1.0


def test_infinities_and_nan():
    g = [torch.tensor([1.0, float("inf"), 2.0], device="cuda"), torch.ones(5000, device="cuda")]
    stats = host(clip_grad_norm(g, 1.0))
    assert np.isinf(stats[0]) and stats[1] == 0.0 and stats[2] == 0.0
    assert host(g[0])[0] == 0.0 and np.isnan(host(g[0])[1]) and (g[1] == 0).all()
    for at in (0, 4999):
        g = torch.ones(5000, device="cuda", dtype=torch.float16)
        g[at] = float("nan")
        stats = host(clip_grad_norm([g], 1.0))
        assert np.isnan(stats[0]) and np.isnan(stats[1]) and stats[2] == 0.0 and torch.isnan(g).all()
    z = torch.zeros(100, device="cuda")
    assert host(clip_grad_norm([z], 0.0)).tolist() == [0.0, 1.0, 1.0]
    one = torch.ones(4, device="cuda")
    assert host(clip_grad_norm([one], 0.0)).tolist() == [2.0, 0.0, 1.0] and (one == 0).all()
    assert host(clip_grad_norm([torch.ones(4, device="cuda")], math.inf)).tolist() == [2.0, 1.0, 1.0]
    assert host(clip_grad_norm([], 1.0)).tolist() == [0.0, 1.0, 1.0]


def test_norm_is_the_same_on_every_run_and_stream():
    g = _tensors(np.random.default_rng(8), [3_000_001, 77, 500_000], TYPES)
    clip = GradClip(g)
    first = clip.norm(0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        runs = [clip.norm(0.5) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(r, first) for r in runs)


def _groups(rng, n=70_001):
    """Dense, mirrored, strided and tiny groups, as a decoder with positions has them."""
    xyzt = cuda(rng.normal(0, 1, (n, 4)).astype(np.float32))
    flat = cuda(rng.normal(0, 1, 4 * n + 3).astype(np.float32))
    p = {"tables": flat[3:3 + 2 * n], "positions": xyzt[:, :3], "b": flat[1:2], "w": flat[3 + 2 * n:3 + 3 * n].view(n, 1)}
    groups = {k: {"param": t, "lr": lr} for (k, t), lr in zip(p.items(), (8e-3, 1.6e-4, 1e-3, 1e-3))}
    groups["tables"]["f16"] = torch.empty(2 * n, dtype=torch.int16, device="cuda")
    return groups, xyzt


def _grads(rng, groups):
    return {k: cuda(rng.normal(0, 1e-2, tuple(g["param"].shape)).astype(np.float32)) for k, g in groups.items()}


def test_adam_without_clipping_equals_the_per_tensor_step_bit_for_bit():
    a, xa = _groups(np.random.default_rng(5))
    b, xb = _groups(np.random.default_rng(5))
    A, B = Adam(a, warmup=2, total=10), Adam(b, warmup=2, total=10)
    rng = np.random.default_rng(6)
    for _ in range(3):
        g = _grads(rng, a)
        assert A.step(g) is None
        stats = B.step(g, max_norm=1e9)
        assert host(stats)[1] == 1.0
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k]["param"], b[k]["param"]), k
        assert all(torch.equal(u, v) for u, v in zip(A.state[k], B.state[k])), k
    assert torch.equal(a["tables"]["f16"], b["tables"]["f16"]) and torch.equal(xa, xb)


def test_adam_with_clipping_matches_the_oracle():
    rng = np.random.default_rng(9)
    groups, xyzt = _groups(rng, 5003)
    keep_t = host(xyzt)[:, 3].copy()
    opt = Adam(groups, warmup=0, total=1000)
    ref = {k: [_f64(g["param"]), 0.0, 0.0] for k, g in groups.items()}
    b1, b2, eps = (float(np.float32(v)) for v in (0.9, 0.999, 1e-15))
    for t in range(1, 4):
        g = _grads(rng, groups)
        want_norm, factor = T.clip_factor([_f64(v) for v in g.values()], 0.3)
        stats = host(opt.step(g, max_norm=0.3)).astype(np.float64)
        assert factor < 1 and abs(stats[0] / want_norm - 1) <= 2.0 ** -23 and abs(stats[1] / factor - 1) <= 2.0 ** -23
        for k, (p, m, v) in ref.items():
            lr = float(np.float32(T.lr_schedule(t - 1, groups[k]["lr"], 0, 1000)))
            ref[k] = list(T.adam_step(p, _f64(g[k]) * factor, m, v, lr, b1, b2, eps, t))
    torch.cuda.synchronize()
    for k, (p, m, v) in ref.items():
        got = _f64(groups[k]["param"])
        ulps = 3 * np.spacing(np.abs(p).astype(np.float32)).astype(np.float64)
        assert np.all(np.abs(got - p) <= 1e-5 * 3 * groups[k]["lr"] + ulps), k
        assert np.allclose(_f64(opt.state[k][0]), m, rtol=1e-5, atol=1e-6 * np.abs(m).max()), k
        assert np.allclose(_f64(opt.state[k][1]), v, rtol=1e-5, atol=1e-6 * np.abs(v).max()), k
    tab = groups["tables"]
    assert torch.equal(tab["f16"].view(torch.float16), tab["param"].half())
    assert np.array_equal(host(xyzt)[:, 3], keep_t)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_adam_step_on_gradients_that_are_not_finite_changes_nothing(bad):
    rng = np.random.default_rng(10)
    groups, xyzt = _groups(rng, 3000)
    opt = Adam(groups, warmup=0, total=1000)
    opt.step(_grads(rng, groups), max_norm=1.0)
    tensors = [g["param"] for g in groups.values()] + [t for s in opt.state.values() for t in s] + [
        groups["tables"]["f16"], xyzt]
    before = [t.clone() for t in tensors]
    g = _grads(rng, groups)
    g["positions"][2999, 2] = bad
    stats = host(opt.step(g, max_norm=1.0))
    assert stats[2] == 0.0 and all(torch.equal(a, b) for a, b in zip(before, tensors))
    opt.step(_grads(rng, groups), max_norm=1.0)
    assert not torch.equal(before[0], tensors[0])


def test_adam_with_some_groups_left_out_and_none():
    rng = np.random.default_rng(12)
    groups, _ = _groups(rng, 300)
    opt = Adam(groups, warmup=0, total=1000)
    w = groups["w"]["param"].clone()
    g = _grads(rng, groups)
    del g["w"]
    stats = host(opt.step(g, max_norm=0.1)).astype(np.float64)
    assert abs(stats[0] / T.clip_factor([_f64(v) for v in g.values()], 0.1)[0] - 1) <= 2.0 ** -23
    assert torch.equal(groups["w"]["param"], w)
    assert host(opt.step({}, max_norm=0.1)).tolist() == [0.0, 1.0, 1.0]


def test_many_groups_take_several_launches():
    rng = np.random.default_rng(14)
    P = {f"p{k}": {"param": cuda(rng.normal(0, 1, 1 + 37 * k).astype(np.float32)), "lr": 1e-3} for k in range(120)}
    Q = {k: {"param": g["param"].clone(), "lr": 1e-3} for k, g in P.items()}
    A, B = Adam(P, warmup=0, total=10), Adam(Q, warmup=0, total=10)
    g = _grads(rng, P)
    A.step(g)
    B.step(g, max_norm=1e9)
    assert all(torch.equal(P[k]["param"], Q[k]["param"]) for k in P)


def test_refusals():
    g = torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        GradClip([g, g.double()])
    with pytest.raises(ValueError):
        GradClip([torch.ones((4, 4), device="cuda").t()[:2]])
    with pytest.raises(ValueError):
        GradClip([g], [g.half()])
    with pytest.raises(ValueError):
        GradClip([g], [])
    for bad in (-1.0, float("nan")):
        with pytest.raises(ia.IAError) as e:
            clip_grad_norm([g], bad)
        assert e.value.status == ia.IA_ERR_INVALID_ARG
    buf = torch.ones(12, device="cuda")
    with pytest.raises(ia.IAError) as e:
        clip_grad_norm([buf[:8]], 1.0, [buf[4:]])  # overlapping
    assert e.value.status == ia.IA_ERR_INVALID_ARG
    clip = GradClip([g])
    ws = torch.empty(clip._ws_bytes, dtype=torch.uint8, device="cuda")
    with pytest.raises(ia.IAError) as e:
        ia.ia_clip_grad_norm(clip._arr, 1.0, ws[: ws.numel() - 256], torch.empty(3, device="cuda"))
    assert e.value.status == ia.IA_ERR_WORKSPACE_TOO_SMALL
    groups = {"a": {"param": torch.ones((4, 4), device="cuda").t()[1:], "lr": 1e-3}}
    with pytest.raises(ValueError):
        Adam(groups, warmup=0, total=1).step({"a": torch.ones((3, 4), device="cuda")}, max_norm=1.0)
    assert (g == 1).all()


RATES = {"encoder": 8e-3, "color": 1e-3, "scale": 3e-4, "rotation": 3e-5, "opacity": 8e-4}


def test_decoder_gradients_clip_and_update():
    """The shared-trunk decoder's own backward, its groups' gradients clipped in the step."""
    rng = np.random.default_rng(21)
    n = 20_000
    D = Decoder(S.single_decoder())
    pos = np.concatenate([S.shell_points(rng, n, 1.0), np.full((n, 1), 0.4)], 1).astype(np.float32)
    xyzt = cuda(pos)
    attrs = D.decode_xyzt(xyzt)
    up = {k: cuda(rng.normal(0, 1, tuple(v.shape)).astype(np.float32)) for k, v in attrs.items()}
    dg = D.backward(xyzt, up)
    grads = D.group_grads(dg)
    grads["positions"] = dg["pos"]
    groups = D.param_groups(RATES)
    groups["positions"] = {"param": xyzt[:, :3], "lr": 1.6e-4}
    stats = host(Adam(groups, warmup=1, total=1000).step(grads, max_norm=1.0)).astype(np.float64)
    D.update_params()
    norm, factor = T.clip_factor([_f64(g) for g in grads.values()], 1.0)
    say(f"decoder gradient norm {norm:.4f}, factor {factor:.3e}")
    assert factor < 1 and abs(stats[0] / norm - 1) <= 2.0 ** -23 and abs(stats[1] / factor - 1) <= 2.0 ** -23
    assert all(torch.isfinite(v).all() for v in D.decode_xyzt(xyzt).values())
