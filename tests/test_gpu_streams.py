"""Calls that name a stream other than the current one and leave workspace and outputs to the call.

What a call allocates must belong to the stream it runs on: its workspace is zeroed in order with
its kernels, and freed memory is not handed to other work while they run.  So with the current
stream held up, the call finishes on its own stream with the right result; and memory that the
current stream writes afterwards is not the call's.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import kda_workloads as W
from test_gpu_attention import BF16, D, SCALE, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


# Each maker returns what makes a call's own state (caches to append to) and the call.
def norm():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(300, 4096, generator=g, device="cuda").to(BF16) for _ in range(2))
    w = torch.ones(4096, device="cuda")
    return list, lambda own, **kw: kda.add_rms_norm(x, r, w, want="both", **kw)


def append():
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = torch.randn(700, 16, D, generator=g, device="cuda").to(BF16).split((8, 4, 4), 1)
    rope = kda.rope_table(700, D)
    table = torch.arange(11, dtype=torch.int32, device="cuda").view(1, -1)
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([700], [0, 700]))

    def pools():
        return [torch.zeros(11, 4, 64, D, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
            [torch.zeros(11, 4, device="cuda") for _ in range(2)]
    return pools, lambda own, **kw: (kda.rope_append(q, k, v, rope, *own, table, lens, cu, **kw), *own)


def attend(q_lens, kv_lens):
    d = make(q_lens, kv_lens, 16, 4, 64, seed=41)
    a = [d[x].cuda() for x in ("q", "k", "v", "ks", "vs", "table", "kv", "cu")]
    return list, lambda own, **kw: kda.cached_attention(*a, SCALE, max(q_lens), lse=True, **kw)


def kda_layer(lengths, call, **more):
    inp = W.make_inputs(W.custom(lengths, 4, seed=43))
    a = [x.cuda() if isinstance(x, torch.Tensor) else x
         for x in (inp[n] for n in ("q", "k", "v", "g", "beta", "A_log", "dt_bias", "lower_bound",
                                    "scale", "initial_state", "cu_seqlens"))]
    return list, lambda own, **kw: call(*a, **more, **kw)


def proj():
    g = torch.Generator(device="cuda").manual_seed(3)
    x, ab, b = (torch.randn(*s, generator=g, device="cuda").to(BF16) for s in ((6, 1024), (256, 1024), (512, 128)))
    return list, lambda own, **kw: kda.skinny_proj(x, ab, b, **kw)


CALLS = dict(
    norm=norm, append=append, proj=proj,
    decode=lambda: attend([1, 1], [9000, 700]), mixed=lambda: attend([150, 2, 70], [2000, 900, 70]),
    prefill=lambda: kda_layer([900, 64], kda.chunk_prefill_fwd),
    recurrent=lambda: kda_layer([2, 1, 3], kda.recurrent_fwd, token_states=True))


@pytest.mark.parametrize("name", CALLS)
def test_a_named_stream_owns_what_the_call_allocates(name):
    fresh, call = CALLS[name]()
    want = call(fresh())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(fresh(), stream=side)       # (the stream's own memory is there from now on)
    torch.cuda.synchronize()
    for _ in range(2):
        own, held = fresh(), torch.cuda.Event()
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)               # some 0.2 s of the current stream
        held.record()
        got = call(own, stream=side)
        junk = [torch.full((1 << n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (8, 12, 20, 24, 25)]
        side.synchronize()
        assert not held.query()                      # nothing waited for the current stream
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            if a is None or b is None:
                assert a is None and b is None
            else:
                assert a.shape == b.shape and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        del junk


def test_a_given_stream_that_is_current_changes_nothing():
    _, call = attend([1, 5], [700, 300])
    a, b = call([]), call([], stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_other_stream_objects():
    """Any object with a cuda_stream handle names a stream."""
    class Handle:
        pass
    _, call = attend([1, 5], [700, 300])
    a = call([])
    torch.cuda.synchronize()
    side, h = torch.cuda.Stream(), Handle()
    h.cuda_stream = side.cuda_stream
    b = call([], stream=h)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name", CALLS)
def test_a_call_runs_on_its_tensors_device(name, monkeypatch):
    """With another device current (here: said to be), the call is made again with the tensors' one."""
    fresh, call = CALLS[name]()
    want = call(fresh())
    now, entered = [1], []

    class Device(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            now.append(self.idx)
            return super().__enter__()

        def __exit__(self, *a):
            now.pop()
            return super().__exit__(*a)

    class NoNative:          # (the C++ marshalling asks the runtime itself, and leaves such calls alone)
        add_rms_norm = rope_append = cached_attention = staticmethod(lambda *a: None)

    monkeypatch.setattr(kda.layer, "_native", NoNative)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    got = call(fresh())
    monkeypatch.undo()
    assert 0 in entered and now == [1]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)))
