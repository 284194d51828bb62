"""W4A4Linear refuses a call before anything of it runs: the residual stream, which
forward_normed updates (in place, where the caller asks for it), must not be changed
by a call that is then refused.  And the whole call runs on its input's device.
On the CPU: the library's calls are replaced by recorders."""
import contextlib

import pytest
import torch

from w4a4_bit_gemm_hq_b200 import build_lib

F16, F32, I32 = torch.float16, torch.float32, torch.int32
M, K, N, n, r = 4, 256, 64, 3, 8


@pytest.fixture()
def hq(monkeypatch):
    build_lib.build()
    from w4a4_bit_gemm_hq_b200 import hq as module
    return module


class OnDevice:
    """A tensor as the checks see it, on a CUDA device of that number."""

    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def layer_of(hq, offq=False, out=F16, dev=0):
    weights = OnDevice(torch.zeros(1), dev)
    return hq.W4A4Linear(128, 128, None, weights, weights, weights, None, None, None, K, N, out, 4, offq)


@pytest.fixture()
def calls(hq, monkeypatch):
    """(name, device at the time) of every library call that the layer makes."""
    log, current = [], [0]

    def record(name, result):
        def call(*a, **kw):
            log.append((name, current[0]))
            return result() if callable(result) else result
        monkeypatch.setattr(hq, name, call)

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    x = lambda: OnDevice(torch.zeros(M, K, dtype=F16), current[0])                     # noqa: E731
    codes = lambda: OnDevice(torch.zeros(M, K // 2, dtype=torch.uint8), current[0])    # noqa: E731
    y = lambda: OnDevice(torch.zeros(M, N, dtype=F16), current[0])                     # noqa: E731
    record("hq_norm_rotate_quant", lambda: (codes(), None, x(), x()))
    record("hq_residual_norm", lambda: (x(), x()))
    record("hq_rotate_quant", lambda: (codes(), None))
    record("hq_rotate_quant_asym", lambda: (codes(), None, None))
    record("w4a4_linear", y)
    record("w4a4_linear_asym", y)
    record("_launch", None)
    monkeypatch.setattr(hq.torch, "empty", lambda shape, dtype=None, device=None: torch.zeros(shape, dtype=dtype))
    record("hq_linear_workspace_size", 0)
    monkeypatch.setattr(hq.torch.cuda, "device", device)
    monkeypatch.setattr(hq.torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    return log


def launches(log):
    return [c for c in log if c[0] != "hq_linear_workspace_size"]


def plan_of(hq, m=M, adapters=n, dev=0):
    return (OnDevice(torch.zeros(m, dtype=I32), dev),
            OnDevice(torch.zeros(hq.hq_lora_max_tiles(m, adapters), 3, dtype=I32), dev))


def adapters(dt=F16, dev=0, rank=r):
    return OnDevice(torch.zeros(n, rank, K, dtype=dt), dev), OnDevice(torch.zeros(n, N, rank, dtype=dt), dev)


@pytest.mark.parametrize("kind", ["fused", "post", "offq"])
def test_refused_before_the_stream_is_touched(hq, calls, kind):
    layer = layer_of(hq, kind == "offq")
    H, w = OnDevice(torch.zeros(M, K, dtype=F16)), OnDevice(torch.zeros(K, dtype=F16))
    kw = {"block": H, "H_out": H, "w_post": w if kind == "post" else None}

    def refused(X=H, **more):
        with pytest.raises((ValueError, TypeError)):
            layer.forward_normed(X, w, 1e-5, **{**kw, **more})
        assert not calls

    refused(plan=plan_of(hq))                                        # no adapters
    layer.set_adapters(*adapters(torch.bfloat16))
    refused(plan=plan_of(hq))                                        # adapters of another type
    layer.set_adapters(*adapters(dev=1))
    refused(plan=plan_of(hq))                                        # on another device
    layer.set_adapters(*adapters())
    refused(plan=plan_of(hq, m=M + 1))                               # the plan of another batch
    refused(plan=plan_of(hq, adapters=1))                            # of other adapters
    refused(plan=plan_of(hq, dev=1))
    refused(plan=(plan_of(hq)[0],))
    refused(OnDevice(torch.zeros(M, K + 128, dtype=F16)))            # rows of another width
    refused(OnDevice(torch.zeros(K, dtype=F16)))
    refused(Y=OnDevice(torch.zeros(M - 1, N, dtype=F16)))            # results of another shape
    refused(Y=OnDevice(torch.zeros(M, 2 * N, dtype=F16)[:, ::2]))
    refused(Y=OnDevice(torch.zeros(M, N, dtype=F16), 1))
    refused(OnDevice(torch.zeros(M, K, dtype=F16), 1))               # the layer is on another device
    refused(torch.zeros(M, K, dtype=F16))                            # on none
    refused(OnDevice(torch.zeros(M, K)))                             # a stream of a type that the layer does not take
    refused(Y=OnDevice(torch.zeros(M * N + 1, dtype=F16)[1:].view(M, N)))    # results between 16-byte boundaries
    refused(Y=OnDevice(torch.zeros(M, N, dtype=torch.float64)))
    layer.forward_normed(H, w, 1e-5, plan=plan_of(hq), **kw)
    assert launches(calls)[-1][0] == "_launch"


def test_forward_refuses_rows_and_plans(hq, calls):
    layer = layer_of(hq)
    X = OnDevice(torch.zeros(M, K, dtype=F16))
    for bad in (OnDevice(torch.zeros(M, K - 128, dtype=F16)), OnDevice(torch.zeros(M, K + 128, dtype=F16)),
                OnDevice(torch.zeros(M, 2, K, dtype=F16))):
        with pytest.raises(ValueError):
            layer(bad)
    with pytest.raises(ValueError):
        layer(X, plan=plan_of(hq))
    layer.set_adapters(*adapters())
    with pytest.raises(ValueError):
        layer(X, plan=plan_of(hq, m=M + 64))
    assert not calls
    layer(X)
    layer(X, plan=plan_of(hq))
    assert [c[0] for c in launches(calls)] == ["hq_rotate_quant", "w4a4_linear"] * 2 + ["_launch"]


def test_adapters_that_no_call_could_use_are_refused(hq):
    layer = layer_of(hq)
    A, B = torch.zeros(n, r, K, dtype=F16), torch.zeros(n, N, r, dtype=F16)
    ranks, scales = torch.zeros(n, dtype=I32), torch.ones(n)
    layer.set_adapters(A, B, ranks, scales)
    kept = layer.adapters
    for bad in ((A, B[:, :56]), (A[:, :, :128], B), (A[0], B), (A.float(), B.float()), (A, B.bfloat16()),
                (torch.zeros(n, 12, K, dtype=F16), torch.zeros(n, N, 12, dtype=F16)),
                (torch.zeros(n, 264, K, dtype=F16), torch.zeros(n, N, 264, dtype=F16)),
                (torch.zeros(1023, r, K, dtype=F16), torch.zeros(1023, N, r, dtype=F16)),
                (torch.zeros(n, K, r, dtype=F16).transpose(1, 2), B), (A, torch.zeros(n, r, N, dtype=F16).transpose(1, 2)),
                (A, B, ranks.long()), (A, B, ranks[:2]), (A, B, None, scales.double()), (A, B, None, scales[:2]),
                (OnDevice(A, 0), OnDevice(B, 1))):
        with pytest.raises(ValueError):
            layer.set_adapters(*bad)
        assert layer.adapters is kept
    layer.set_adapters(None, None)
    assert layer.adapters is None


@pytest.mark.gpu
@pytest.mark.parametrize("post", [False, True])
def test_a_refused_call_leaves_the_stream(hq, post):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")    # noqa: E731
    layer = hq.W4A4Linear.prepare(rand(N, K) * 0.05, 128, 128, 0)
    H, Y, w = rand(M, K).half(), rand(M, K).half(), rand(K).half()
    kept = H.clone()
    kw = {"block": Y, "w_post": w if post else None, "H_out": H}
    plan = hq.hq_lora_plan(torch.zeros(M, dtype=I32, device="cuda"), n)
    with pytest.raises(ValueError):
        layer.forward_normed(H, w, 1e-5, plan=plan, **kw)
    layer.set_adapters(rand(n, r, K).bfloat16(), rand(n, N, r).bfloat16())
    with pytest.raises(ValueError):
        layer.forward_normed(H, w, 1e-5, plan=plan, **kw)
    layer.set_adapters(rand(n, r, K).half(), rand(n, N, r).half())
    with pytest.raises(ValueError):
        layer.forward_normed(H, w, 1e-5, plan=hq.hq_lora_plan(torch.zeros(M, dtype=I32, device="cuda"), n - 1), **kw)
    with pytest.raises(ValueError):
        layer.forward_normed(H, w, 1e-5, Y=torch.empty(M, N + 8, dtype=F16, device="cuda"), **kw)
    torch.cuda.synchronize()
    assert torch.equal(H, kept)
    out, h = layer.forward_normed(H, w, 1e-5, plan=plan, **kw)
    assert h is H and not torch.equal(H, kept) and out.isfinite().all()


@pytest.mark.parametrize("kind", ["fused", "post", "offq"])
def test_every_launch_is_on_the_device_of_the_rows(hq, calls, kind):
    layer = layer_of(hq, kind == "offq", dev=1)
    layer.set_adapters(*adapters(dev=1))
    H, w = OnDevice(torch.zeros(M, K, dtype=F16), 1), OnDevice(torch.zeros(K, dtype=F16), 1)
    layer.forward_normed(H, w, 1e-5, block=H, w_post=w if kind == "post" else None, plan=plan_of(hq, dev=1))
    layer.forward(H, plan=plan_of(hq, dev=1))
    assert len(launches(calls)) >= 6 and all(d == 1 for _, d in launches(calls))
    assert hq.torch._C._cuda_getDevice() == 0
