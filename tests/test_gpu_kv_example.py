"""GPU check of examples/decode_attention.py: products, append, attend and evict together.

Every step's attention result is checked from the tensors that the step itself used: the keys
and values of all tokens so far (recorded from the qkv product) and the positions that each
head still holds say what the cache has to contain and what attention has to give, computed
here in fp64.  The tolerance is the storage's rounding: bf16 keys move a score by up to 2^-8
of the sum of its terms' magnitudes (8-bit ones by 2^-4), and a weight by that, relatively;
values and the result are rounded likewise.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import kv as okv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("decode_attention", os.path.join(ROOT, "examples", "decode_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().float().double().numpy()


@pytest.mark.parametrize("kind,unit", [("bf16", 2.0**-8), ("fp8", 2.0**-4)])
def test_decode_within_a_budget(monkeypatch, kind, unit):
    ex = example()
    rows, budget, steps = 3, 24, 60
    layer = ex.AttentionHalf(rows, budget, page=8, sink=2, recent=6, positions=steps, cache=kind, seed=3)
    attend, product, seen = ex.nbw.kv_attend, ex.nbw.qgemm, {}

    def spy_attend(cache, q, lens, **kw):
        seen.update(q=q.clone(), lens=lens.tolist(), pos=layer.pos[0].cpu().numpy().copy(), acc=layer.acc[0].clone())
        seen["out"] = attend(cache, q, lens, **kw).clone()
        seen["acc_out"] = layer.acc[0].clone()
        return seen["out"]

    def spy_product(x, w, scales, r, **kw):
        y = product(x, w, scales, r, **kw)
        if y.dtype == torch.bfloat16:
            seen["qkv"] = y.clone()
        return y

    monkeypatch.setattr(ex.nbw, "kv_attend", spy_attend)
    monkeypatch.setattr(ex.nbw, "qgemm", spy_product)
    rope, ones = f64(layer.rope), np.ones(128)
    keys, values = [], []
    x = torch.randn(rows, 4096, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    for step in range(steps):
        x = torch.nn.functional.normalize(x, dim=1) * 64
        y = layer.decode(x.to(torch.bfloat16))
        assert bool(y.isfinite().all())
        x = 0.5 * x + y
        qkv = f64(seen["qkv"]).reshape(rows, 48, 128)
        keys.append(np.stack([okv.turned(qkv[r, 32:40], step, rope, ones, 1e-6) for r in range(rows)]))
        values.append(qkv[:, 40:])
        q = f64(seen["q"])
        for r in range(rows):
            n = seen["lens"][r]
            assert n == min(step + 1, budget + 1)
            for h in range(8):
                pos = seen["pos"][r, h, :n]
                assert len(set(pos.tolist())) == n and set(range(min(2, n))) <= set(pos.tolist())
                assert set(range(max(0, step - 6), step + 1)) <= set(pos.tolist())  # the recent ones, and the new one
                k = np.stack([keys[p][r, h] for p in pos])
                v = np.stack([values[p][r, h] for p in pos])
                weight = np.zeros(n)
                for g in range(4 * h, 4 * h + 4):
                    s = (k * q[r, g]).sum(axis=1) * 128 ** -0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    weight += p
                    move = 2 * unit * (np.abs(k) * np.abs(q[r, g])).sum(axis=1).max() * 128 ** -0.5
                    bound = (np.expm1(min(move, 5.0)) + 3 * unit) * (p @ np.abs(v)) + 1e-6
                    assert np.all(np.abs(f64(seen["out"][r, g]) - p @ v) <= bound)
                got = f64(seen["acc_out"][r, h, :n]) - f64(seen["acc"][r, h, :n])
                assert abs(got.sum() - 4) < 1e-4 and np.all(got >= -1e-6)
    # what is left is what the totals say: each head kept its budget, the protected ones among it
    assert layer.lens[0].tolist() == [budget] * rows


def test_the_command_runs(capsys):
    assert example().main(["--rows", "2", "--steps", "20", "--budget", "12"]) == 0
    assert "12 kept for each head" in capsys.readouterr().out
