"""The training step that README shows with its activations kept in 8 bits: run as
it stands there, with the block's tokens freed between forward and backward, so
that nothing but what was kept can be read; its router's gradients against fp64 at
the kept tokens (bounds: test_gpu_router_grad.py)."""
import os
import re

import pytest
import torch

from tests._ckpt_ref import keep
from tests._train_ref import bf16, check, f32
from tests.test_gpu_router_grad import reference

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    import moe_layer_04_amd as m
    m.load_library()
    return m


def step():
    """(forward, backward) of README's block"""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    parts = next(b for b in blocks if "# backward\n" in b).split("# backward\n")
    assert len(parts) == 2
    return parts


@pytest.mark.parametrize("T,K,N,E,topk", [(40, 136, 72, 5, 3), (300, 256, 192, 8, 2)])
def test_step_without_the_tokens(moe, T, K, N, E, topk):
    print(f"[gpu-test] README's step T={T} K={K} E={E}", flush=True)
    v = dict(moe=moe, T=T, topk=topk, u=bf16((T, K), 1), w_router=bf16((E, K), 2, K ** -0.5), bias=f32((E,), 3, 0.3),
             w1=bf16((E, 2 * N, K), 4, K ** -0.5), w2=bf16((E, K, N), 5, N ** -0.5), do=bf16((T, K), 6, 0.1),
             coefficient=f32((1,), 7, 0.1, 5.0), mask=f32((T,), 8) < 1)
    v["ids"] = moe.moe_topk(v["u"], v["w_router"], v["bias"], topk)[0]
    v["slots"], _, v["offsets"], _ = moe.moe_align(v["ids"], E, 1)
    v["g"] = moe.moe_grouped_gemm(v["u"], v["w1"], v["offsets"], sorted_ids=v["slots"], topk=topk, gather=True)
    u = v["u"]
    forward, backward = step()
    exec(forward, v)
    for name in ("u", "g", "a"):                 # what the step is meant to save
        del v[name]
    rows = {}

    class Calls:
        """moe, whose topk_bwd's joined rows are looked at"""
        def __getattr__(self, name):
            f = getattr(moe, name)
            if name != "moe_topk_bwd":
                return f

            def call(*args, **kw):
                rows.update(dx=kw["dx_rows"], dw=args[4])
                return f(*args, **kw)
            return call

    v["moe"] = Calls()
    exec(backward, v)
    back = moe.moe_ckpt_restore(*v["kept_u"])
    assert torch.equal(back.double(), keep(u)[2])
    want, bound = reference(dict(x=back, w_router=v["w_router"], topk_ids=v["ids"], topk_weights=v["weights"],
                                 dtopk_weights=rows["dw"], dlogits=v["dlogits"], dx_rows=rows["dx"]))
    for got, w, b, name in zip((v["du"], v["dw_router"], v["dbias"]), want, bound, ("du", "dw_router", "dbias")):
        check(got, w, b, name)
    for name in ("dw1", "dw2"):
        assert v[name].shape == v["w" + name[2]].shape and torch.isfinite(v[name]).all()
