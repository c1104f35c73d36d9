"""The clipped Adam step after steps that were left out because their norm was
not finite, or refused: the bias corrections are those of the steps applied.

Tolerances as for the step without any left out: a step moves a parameter by at
most its rate, which the kernel's fp32 arithmetic holds to 1e-5; three ulps of
the parameter for its own roundings."""
import numpy as np
import pytest
import torch

from oracle import train as T
from implicit_attribute_decode_amd.pipeline import Adam

from gpu_util import cuda, host

pytestmark = pytest.mark.gpu

B1, B2, EPS = (float(np.float32(v)) for v in (0.9, 0.999, 1e-15))


def _f64(t):
    return t.double().cpu().numpy()


def _run(pattern, shapes, warmup=0, spoil=float("nan")):
    """Steps on new gradients, those marked "x" with one spoilt value; checks every applied one."""
    rng = np.random.default_rng(len(pattern))
    wide = cuda(rng.normal(0, 1, (shapes[0][0], 4)).astype(np.float32))
    groups = {"rows": {"param": wide[:, :3], "lr": 3e-3}}
    groups.update({f"p{k}": {"param": cuda(rng.normal(0, 1, s).astype(np.float32)), "lr": 1e-3}
                   for k, s in enumerate(shapes[1:])})
    opt = Adam(groups, warmup=warmup, total=1000)
    ref = {k: [_f64(g["param"]), 0.0, 0.0] for k, g in groups.items()}
    applied = 0
    for t, what in enumerate(pattern):
        g = {k: cuda(rng.normal(0, 1e-2, tuple(v["param"].shape)).astype(np.float32)) for k, v in groups.items()}
        if what == "x":
            last = list(groups)[-1]
            g[last].view(-1)[-1] = spoil
            assert host(opt.step(g, max_norm=0.3))[2] == 0.0
        elif what == "r":
            with pytest.raises(ValueError):
                opt.step({k: v.double() for k, v in g.items()}, max_norm=0.3)
            continue
        else:
            factor = T.clip_factor([_f64(v) for v in g.values()], 0.3)[1]
            assert host(opt.step(g, max_norm=0.3))[2] == 1.0
            applied += 1
            for k, (p, m, v) in ref.items():
                lr = float(np.float32(T.lr_schedule(opt.t - 1, groups[k]["lr"], warmup, 1000)))
                ref[k] = list(T.adam_step(p, _f64(g[k]) * factor, m, v, lr, B1, B2, EPS, applied))
        for k, (p, m, v) in ref.items():
            ulps = 3 * np.spacing(np.abs(p).astype(np.float32)).astype(np.float64)
            assert np.all(np.abs(_f64(groups[k]["param"]) - p) <= 1e-5 * (t + 1) * groups[k]["lr"] + ulps), (t, k)
    assert opt.t == len(pattern) - pattern.count("r") and opt.skipped.tolist() == [pattern.count("x")]
    return opt


@pytest.mark.parametrize("spoil", [float("nan"), float("inf")])
@pytest.mark.parametrize("pattern", ["xo", "xxxxxo", "oxo", "ooxxoxo", "xoxoxooo"])
def test_corrections_count_the_steps_applied(pattern, spoil):
    _run(pattern, [(2001, 3), (70, 30), (5,)], spoil=spoil)


def test_a_refused_step_is_no_step():
    _run("rororro", [(300, 3), (64,)])


def test_several_launches_count_a_step_once():
    _run("xxoxo", [(50, 3)] + [(1 + 37 * k,) for k in range(119)], warmup=3)


def test_without_a_step_left_out_nothing_changes():
    """Bit for bit the unclipped steps, and the count follows a restored optimiser."""
    rng = np.random.default_rng(5)
    a, b = ({"w": {"param": cuda(rng2.normal(0, 1, 5000).astype(np.float32)), "lr": 1e-3}}
            for rng2 in (np.random.default_rng(1), np.random.default_rng(1)))
    A, B = Adam(a, warmup=0, total=100), Adam(b, warmup=0, total=100)
    for _ in range(4):
        g = {"w": cuda(rng.normal(0, 1, 5000).astype(np.float32))}
        A.step(g)
        B.step(g, max_norm=1e9)
    assert torch.equal(a["w"]["param"], b["w"]["param"]) and B.skipped.tolist() == [0]
    B.skipped = torch.tensor([3], dtype=torch.int32)  # as loaded on the host: one step had been applied
    g = {"w": cuda(rng.normal(0, 1, 5000).astype(np.float32))}
    p, m, v = (_f64(t) for t in (b["w"]["param"], *B.state["w"]))
    lr = float(np.float32(T.lr_schedule(4, 1e-3, 0, 100)))
    want = T.adam_step(p, _f64(g["w"]), m, v, lr, B1, B2, EPS, 2)[0]
    B.step(g, max_norm=1e9)
    assert np.all(np.abs(_f64(b["w"]["param"]) - want) <= 1e-5 * 1e-3 * 5 + 3 * np.spacing(np.abs(want).astype(np.float32)))
