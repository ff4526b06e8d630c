"""Sampled requests through the engine (cdb_admit_sampled).

The traced logits of every token, drawn from by the float64 restatement of the
sampler with the request's numbers, give the engine's tokens; greedy requests of
the same batch keep theirs; modes and batch sizes agree.
"""

import numpy as np
import pytest

from tests.test_gpu_sample import reference

pytestmark = pytest.mark.gpu

SETTINGS = [dict(temperature=0.9), dict(temperature=1.3, top_k=20), dict(temperature=1.0, top_p=0.8), None,
            dict(temperature=0.7, min_p=0.1), dict(temperature=1.5, top_k=50, top_p=0.9, min_p=0.01),
            dict(temperature=0.0), None]


def requests():
    from synth import make_requests, make_weights, model_shape, workload
    shape, wl = model_shape("tiny"), workload("tiny")
    return shape, make_weights(shape), make_requests(wl, shape.vocab)[:8], wl


def run(mode="refill", W=4, settings=SETTINGS, force=None, order=None):
    from continuous_depth_batching_gb300 import binding
    shape, wts, reqs, wl = requests()
    eng = binding.Engine(shape, binding.device_weights(shape, wts), mode=mode, W=W, M=wl.M, K=wl.K, max_ctx=64,
                         max_new_cap=16, trace_tokens=16)
    us = {}
    for i in order if order is not None else range(len(reqs)):
        r = reqs[i]
        us[r["seq_id"]] = np.random.default_rng(100 + i).random(r["gen_len"]).astype(np.float32)
        ft = None
        if force is not None:
            ft = np.full(r["gen_len"], -1, dtype=np.int32)
            ft[force] = 7
        s = settings[i]
        eng.admit(r["seq_id"], r["prompt"], r["gen_len"], None, ft, **({} if s is None else dict(sampling=s, u=us[r["seq_id"]])))
    eng.run()
    out = {o["seq_id"]: o for o in eng.drain()}
    eng.close()
    return reqs, us, out


def test_tokens_follow_their_logits():
    reqs, us, out = run()
    for i, r in enumerate(reqs):
        s, o = SETTINGS[i], out[r["seq_id"]]
        for t in range(r["gen_len"]):
            x = o["logits"][t]
            if s is None:
                assert o["tokens"][t] == int(np.argmax(x))
            else:
                want, _ = reference(x, us[r["seq_id"]][t], np.float32(s["temperature"]), s.get("top_k"),
                                    np.float32(s.get("top_p", 1.0)), np.float32(s.get("min_p", 0.0)))
                assert o["tokens"][t] == want, (i, t)


def test_modes_and_batches_agree():
    _, _, a = run()
    for kw in (dict(mode="no_refill"), dict(W=1), dict(W=8), dict(order=[7, 3, 5, 1, 0, 2, 6, 4])):
        _, _, b = run(**kw)
        for k in a:
            assert list(a[k]["tokens"]) == list(b[k]["tokens"]) and list(a[k]["exit_depths"]) == list(b[k]["exit_depths"])


def test_greedy_requests_keep_their_tokens():
    _, _, mixed = run()
    reqs, _, greedy = run(settings=[None] * 8)
    for i, r in enumerate(reqs):
        if SETTINGS[i] is None or SETTINGS[i]["temperature"] == 0.0:
            assert list(mixed[r["seq_id"]]["tokens"]) == list(greedy[r["seq_id"]]["tokens"])
    assert any(list(mixed[r["seq_id"]]["tokens"]) != list(greedy[r["seq_id"]]["tokens"]) for r in reqs)


def test_forced_tokens_take_precedence():
    reqs, _, out = run(force=[0, 5])
    for r in reqs:
        assert out[r["seq_id"]]["tokens"][0] == 7 and out[r["seq_id"]]["tokens"][5] == 7


def test_refusals():
    from continuous_depth_batching_gb300 import binding
    shape, wts, reqs, wl = requests()
    eng = binding.Engine(shape, binding.device_weights(shape, wts), W=4, M=wl.M, K=wl.K, max_ctx=64, max_new_cap=16)
    r = reqs[0]
    u = np.full(r["gen_len"], 0.5, dtype=np.float32)
    for s, v in ((dict(temperature=float("nan")), u), (dict(top_p=float("nan")), u), (dict(min_p=float("nan")), u),
                 (dict(), u + 0.5), (dict(), u - 1.0), (dict(), u * np.float32("nan"))):
        with pytest.raises(binding.CdbError):
            eng.admit(0, r["prompt"], r["gen_len"], sampling=s, u=v)
    with pytest.raises(ValueError):
        eng.admit(0, r["prompt"], r["gen_len"], sampling=dict(), u=u[:-1])
    eng.admit(0, r["prompt"], r["gen_len"], sampling=dict(), u=u)  # still usable
    eng.run()
    assert len(eng.drain()) == 1
    eng.close()
