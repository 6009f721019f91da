"""Tensors that a call with ``stream=`` allocates: their memory is the caller's alone from the
call on, whatever the current stream still does with what was there before, and until
both streams are done with them."""
import pytest

pytestmark = pytest.mark.gpu

SLEEP = 40_000_000      # cycles of a busy stream: about 20 ms


@pytest.fixture(scope="module")
def fa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_tiled_attention_forward_gb300 as fa
    from exact_tiled_attention_forward_gb300 import build
    build.build()
    fa.lib()
    return fa


def _calls(fa):
    """name -> (call(**kw) -> tuple of outputs) on one set of inputs."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v, do = r(2, 8, 512, 128), r(2, 2, 512, 128), r(2, 2, 512, 128), r(2, 8, 512, 128)
    codes = [torch.randint(0x20, 0x60, t.shape, dtype=torch.uint8, device="cuda") for t in (q, k, v)]
    o, lse = fa.fa_forward(q, k, v, causal=True)
    ow, lsew = fa.fa_forward_window(q, k, v, 100, 2)
    pages = [r(8, 2, 128, 128) for _ in range(2)]
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.full((2,), 512, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda")
    rows, one = r(600, 8, 128), q[:, :, :1].contiguous()
    half = [t.half() for t in (q, k, v)]
    torch.cuda.synchronize()
    return {
        "fa_forward": lambda **kw: fa.fa_forward(q, k, v, **kw),
        "fa_forward_fp16": lambda **kw: fa.fa_forward_fp16(*half, **kw),
        "fa_forward_fp8": lambda **kw: fa.fa_forward_fp8(*codes, (1.0, 1.0, 1.0), **kw),
        "fa_forward_noalloc": lambda **kw: fa.fa_forward_noalloc(q, k, v, **kw),
        "fa_naive_forward": lambda **kw: fa.fa_naive_forward(q, k, v, **kw),
        "fa_backward": lambda **kw: fa.fa_backward(q, k, v, o, lse, do, causal=True, **kw),
        "fa_forward_window": lambda **kw: fa.fa_forward_window(q, k, v, 100, 2, **kw),
        "fa_backward_window": lambda **kw: fa.fa_backward_window(q, k, v, ow, lsew, do, 100, 2, **kw),
        "fa_decode_paged": lambda **kw: fa.fa_decode_paged(one, *pages, table, lens, **kw),
        "fa_extend_paged": lambda **kw: fa.fa_extend_paged(rows, *pages, table, cu, lens, 300, **kw),
        "fa_cache_read": lambda **kw: fa.fa_cache_read(*pages, table, cu, lens, 600, **kw),
    }


NAMES = ["fa_forward", "fa_forward_fp16", "fa_forward_fp8", "fa_forward_noalloc", "fa_naive_forward", "fa_backward",
         "fa_forward_window", "fa_backward_window", "fa_decode_paged", "fa_extend_paged", "fa_cache_read"]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_before_the_call_has_run(fa, name, handle):
    import torch
    call = _calls(fa)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    out = call(stream=side.cuda_stream if handle else side)
    shapes = [(t.shape, t.dtype) for t in out]
    del out
    later = [torch.full(s, -7.0, dtype=dt, device="cuda") for s, dt in shapes]    # takes any block that is free
    torch.cuda.synchronize()
    for t in later:
        assert bool(torch.all(t == -7.0))
    side.wait_stream(torch.cuda.current_stream())
    out = call(stream=side)
    side.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_where_the_current_stream_still_reads(fa, name):
    import torch
    call = _calls(fa)[name]
    shapes = [(t.shape, t.dtype) for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = [torch.full(s, -7.0, dtype=dt, device="cuda") for s, dt in shapes]
    copies = [torch.zeros_like(t) for t in before]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for c, t in zip(copies, before):
        c.copy_(t)
    del t, before            # free for this stream, which has yet to read them
    out = call(stream=side)
    torch.cuda.synchronize()
    for c in copies:
        assert bool(torch.all(c == -7.0))
    assert len(out) == len(shapes)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_while_the_current_stream_reads(fa, name):
    # made on another stream, waited for, read and dropped here: the next call there must not take them
    import torch
    call = _calls(fa)[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(stream=side)
    want = []
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in out]
    torch.cuda._sleep(SLEEP)
    got = [t.clone() for t in out]
    del out
    with torch.cuda.stream(side):
        later = [torch.full(t.shape, -7.0, dtype=t.dtype, device="cuda") for t in want]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert len(later) == len(got)
