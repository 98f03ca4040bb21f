"""The attention layer's binding takes the tensors of a call from one device (CPU: tensors that say
they lie on a GPU, and the call itself left out)."""
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import attention as A

bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32


class On:
    """A host tensor that says it lies on GPU `at`."""
    is_cuda = True

    def __init__(self, t, at):
        self.t, self.at = t, at

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.at


def rope(m):
    x = dict(q=torch.zeros(2, 4, 3, 64, dtype=bf), k=torch.zeros(2, 2, 3, 64, dtype=bf),
             cos=torch.zeros(8, 32), sin=torch.zeros(8, 32), pos=torch.zeros(2, 3, dtype=i32),
             qo=torch.zeros(2, 4, 3, 64, dtype=bf), ko=torch.zeros(2, 2, 3, 64, dtype=bf))
    x = {n: m(n, t) for n, t in x.items()}
    return list(x), lambda: gdn.gdn_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"],
                                         out=(x["qo"], x["ko"]))


def cache(m, **more):
    x = dict(pages=torch.zeros(5, 2, 16 * 72, dtype=torch.uint8), table=torch.zeros(2, 3, dtype=i32),
             length=torch.zeros(2, dtype=i32), cu=torch.zeros(3, dtype=i32), scale=torch.zeros(2, 2),
             **more)
    return {n: m(n, t) for n, t in x.items()}


def append(m):
    x = cache(m, k=torch.zeros(4, 2, 64, dtype=bf), v=torch.zeros(4, 2, 64, dtype=bf),
              q=torch.zeros(4, 4, 64, dtype=bf), out=torch.zeros(4, 4, 64, dtype=bf),
              cos=torch.zeros(8, 32), sin=torch.zeros(8, 32), pos=torch.zeros(4, dtype=i32))
    return list(x), lambda: gdn.gdn_kv_append(
        x["pages"], x["k"], x["v"], x["table"], x["length"], q=x["q"], cu_seqlens=x["cu"],
        kv_scale=x["scale"], cos=x["cos"], sin=x["sin"], pos=x["pos"], out=x["out"])


def read(m):
    x = cache(m, k=torch.zeros(4, 2, 64, dtype=bf), v=torch.zeros(4, 2, 64, dtype=bf))
    return list(x), lambda: gdn.gdn_kv_read(x["pages"], x["table"], x["length"], 4, 64,
                                            cu_seqlens=x["cu"], kv_scale=x["scale"],
                                            out=(x["k"], x["v"]))


def attn(m):
    x = cache(m, q=torch.zeros(4, 4, 64, dtype=bf), out=torch.zeros(4, 4, 64, dtype=bf))
    return list(x), lambda: gdn.gdn_kv_attn(x["q"], x["pages"], x["table"], x["length"],
                                            cu_seqlens=x["cu"], kv_scale=x["scale"], out=x["out"])


@pytest.mark.parametrize("make", [rope, append, read, attn])
def test_tensors_of_a_call_share_a_device(make, monkeypatch):
    calls = []
    monkeypatch.setattr(A, "_call", lambda *a: calls.append(a))
    names, call = make(lambda n, t: On(t, 3))
    call()
    assert len(calls) == 1
    for other in names:
        for at in (0, -1):
            _, call = make(lambda n, t: On(t, at if n == other else 3))
            with pytest.raises(ValueError):
                call()
    _, call = make(lambda n, t: On(t, -1))      # all of them on the host
    with pytest.raises(ValueError):
        call()
    assert len(calls) == 1
