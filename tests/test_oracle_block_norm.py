"""The float64 oracle of the norms around the layer, pinned: the forward
against a loop over single elements, the gradients against central finite
differences of the forward."""

import math

import numpy as np
import pytest

import oracle

FLAGS = [dict(block=b, post=p, gate=g, scale=s, next=n)
         for b in (False, True) for p in (False, True) for g in (False, True) for s in (False, True)
         for n in (False, True) if (b or not (p or g or s)) and (b or n)]


def _inputs(f, R=3, D=5, seed=0):
    rng = np.random.default_rng(seed)
    return dict(r=rng.normal(size=(R, D)),
                o=rng.normal(size=(R, D)) if f["block"] else None,
                gate=2 * rng.normal(size=(R, D)) if f["gate"] else None,
                scale=rng.uniform(0.2, 1.5, D) if f["scale"] else None,
                w_post=rng.uniform(0.5, 1.5, D) if f["post"] else None,
                w_next=rng.uniform(0.5, 1.5, D) if f["next"] else None)


def _run(x, eps=1e-3):
    return oracle.block_norm(x["r"], x["w_next"], eps, o=x["o"], gate=x["gate"], scale=x["scale"],
                             w_post=x["w_post"])


@pytest.mark.parametrize("f", FLAGS, ids=str)
def test_forward_against_single_elements(f):
    x = _inputs(f)
    r_out, h, rp, rn = _run(x)
    R, D = x["r"].shape
    for i in range(R):
        row = []
        ms = sum(v * v for v in x["o"][i]) / D if f["block"] else 0.0
        for e in range(D):
            v = x["r"][i, e]
            if f["block"]:
                n = x["o"][i, e]
                if f["post"]:
                    n = n / math.sqrt(ms + 1e-3) * x["w_post"][e]
                if f["gate"]:
                    n = n / (1 + math.exp(-x["gate"][i, e]))
                if f["scale"]:
                    n = n * x["scale"][e]
                v = v + n
                assert abs(r_out[i, e] - v) < 1e-13
            row.append(v)
        if f["post"]:
            assert abs(rp[i] * math.sqrt(ms + 1e-3) - 1) < 1e-13
        if f["next"]:
            root = math.sqrt(sum(v * v for v in row) / D + 1e-3)
            assert abs(rn[i] * root - 1) < 1e-13
            for e in range(D):
                assert abs(h[i, e] - row[e] / root * x["w_next"][e]) < 1e-13
    assert (r_out is None) == (not f["block"]) and (h is None) == (not f["next"])


@pytest.mark.parametrize("f", FLAGS, ids=str)
def test_gradients_against_differences(f):
    x = _inputs(f, seed=1)
    rng = np.random.default_rng(2)
    a, b = rng.normal(size=x["r"].shape), rng.normal(size=x["r"].shape)

    def loss(x):
        r_out, h, _, _ = _run(x)
        return (np.sum(a * r_out) if r_out is not None else np.sum(a * x["r"])) + \
            (np.sum(b * h) if h is not None else 0.0)

    r_out, _, rp, rn = _run(x)
    got = oracle.block_norm_vjp(a, b if f["next"] else None, r_out if f["block"] else x["r"], rn,
                                x["w_next"], o=x["o"], gate=x["gate"], scale=x["scale"],
                                w_post=x["w_post"], rstd_post=rp)
    names = dict(r="dr", o="do", gate="dgate", scale="dscale", w_post="dw_post", w_next="dw_next")
    for name, grad in names.items():
        if x[name] is None:
            assert grad not in got
            continue
        for idx in np.ndindex(*x[name].shape):
            step = 1e-5
            hi, lo = (dict(x, **{name: x[name].copy()}) for _ in range(2))
            hi[name][idx] += step
            lo[name][idx] -= step
            num = (loss(hi) - loss(lo)) / (2 * step)
            assert abs(num - got[grad][idx]) < 1e-7 * max(1.0, abs(num)), (name, idx)
