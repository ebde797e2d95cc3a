"""Memory that the binding allocates for a call on another stream than the current one: it belongs to that
stream, so that a result that is dropped early is not handed out under the running call, and a result that
the current stream still reads is not handed to the next call."""
import pytest
import torch

from causal_attention_attn_b200 import attn, build
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
D = 128
B, HQ, HKV, S, PAGE = 2, 8, 2, 64, 16
DELAY = 20_000_000  # cycles: about 10 ms of another stream's time, far more than the calls take on the host


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.get_device_capability(0) != (10, 0):
        pytest.skip("needs an sm_100 device")
    build.build()
    attn.load_library()
    yield
    torch.cuda.synchronize()
    assert attn.device_status() == 0


def calls(seed=0):
    """Every call that allocates results, as name -> f(stream) -> tuple of tensors."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, q1, k, v, dout = draw(B, HQ, S, D), draw(B, HQ, 1, D), draw(B, HKV, S, D), draw(B, HKV, S, D), draw(B, HQ, S, D)
    per = S // PAGE
    kp, vp = draw(B * per + 4, HKV, PAGE, D), draw(B * per + 4, HKV, PAGE, D)
    table = torch.arange(B * per, dtype=torch.int32).view(B, per).cuda()
    ptab = torch.arange(B * per, B * per + 4, dtype=torch.int32).cuda()
    plen = torch.tensor([50], dtype=torch.int32).cuda()
    lens = torch.full((B,), S, dtype=torch.int32).cuda()
    codes = lambda *shape: torch.randint(0, 120, shape, generator=g).to(torch.uint8).cuda()  # noqa: E731
    k8, v8, kp8, vp8 = codes(B, HKV, S, D), codes(B, HKV, S, D), codes(*kp.shape), codes(*kp.shape)
    coef = torch.full((HKV, D), 2.0 ** -7).cuda()
    w = torch.ones((D,), dtype=torch.bfloat16).cuda()
    cos, sin = (t.cuda() for t in ref.angle_tables(S, D))
    o, lse = attn.attn_fwd(q, k, v)
    # What a call reads or updates is the caller's to keep until the call is done: nothing of it is made per call.
    q_rows, kp_new, vp_new = q.transpose(1, 2).contiguous().transpose(1, 2), kp.clone(), vp.clone()
    torch.cuda.synchronize()
    return {
        "fwd": lambda s: attn.attn_fwd(q, k, v, stream=s),
        "fwd strided": lambda s: attn.attn_fwd(q_rows, k, v, stream=s),
        "noalloc": lambda s: attn.attn_decode_noalloc(q1, k, v, stream=s),
        "decode paged": lambda s: attn.attn_decode_paged(q1, kp, vp, table, lens, S, stream=s),
        "prefill paged": lambda s: attn.attn_prefill_paged(q, kp, vp, table, lens, S, stream=s),
        "decode fp8": lambda s: attn.attn_decode_fp8(q1, k8, v8, coef, coef, stream=s),
        "prefill fp8": lambda s: attn.attn_prefill_fp8(q, k8, v8, coef, coef, stream=s),
        "decode paged fp8": lambda s: attn.attn_decode_paged_fp8(q1, kp8, vp8, coef, coef, table, lens, S, stream=s),
        "bwd": lambda s: attn.attn_bwd(q, k, v, o, lse, dout, stream=s),
        "norm rope": lambda s: attn.attn_qk_norm_rope(q, k, cos, sin, q_weight=w, k_weight=w, stream=s),
        "norm rope bwd": lambda s: attn.attn_qk_norm_rope_bwd(q, k, cos, sin, dout, k, q_weight=w, k_weight=w, stream=s),
        "append": lambda s: (attn.attn_append_paged(k, v, cos, sin, kp_new, vp_new, table, lens, q=q, stream=s),),
        "prefix": lambda s: attn.attn_decode_prefix(q1, kp, vp, ptab, plen, table, lens, 50, S, stream=s),
    }


NAMES = ("fwd", "fwd strided", "noalloc", "decode paged", "prefill paged", "decode fp8", "prefill fp8", "decode paged fp8",
         "bwd", "norm rope", "norm rope bwd", "append", "prefix")


def owner(t):
    """The stream (its handle) that the caching allocator orders a tensor's memory by."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("the tensor is in no segment")


@pytest.mark.parametrize("name", NAMES)
def test_results_belong_to_the_calls_stream(name):
    fn = calls()[name]
    side = torch.cuda.Stream()
    want = fn(None)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, torch.cuda.ExternalStream(side.cuda_stream)):
        got = fn(stream)
        torch.cuda.synchronize()
        assert all(owner(t) == side.cuda_stream for t in got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(owner(t) == torch.cuda.current_stream().cuda_stream for t in want)
    with torch.cuda.stream(side):
        for stream in (0, torch.cuda.default_stream()):  # named while another one is current
            got = fn(stream)
            torch.cuda.synchronize()
            assert all(owner(t) == 0 for t in got) and all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(owner(t) == side.cuda_stream for t in fn(side))
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_dropped_results_are_not_handed_out_under_the_call(name):
    fn = calls()[name]
    side = torch.cuda.Stream()
    shapes = [(t.shape, t.dtype) for t in fn(side)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    fn(side)  # nothing of it is kept; it runs behind the delay
    mine = [torch.full(shape, 7, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert all(torch.all(t == 7) for t in mine)


@pytest.mark.parametrize("name", NAMES)
def test_results_that_the_current_stream_reads_are_not_handed_to_the_next_call(name):
    first, second = calls(0)[name], calls(1)[name]
    want = [t.clone() for t in first(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = first(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(DELAY)
    kept = [t.clone() for t in got]  # read behind the delay
    del got
    again = second(side)             # not ordered behind the reads
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)) and len(again) == len(want)


def test_host_buffers_through_another_stream():
    """attn_fwd_host's staging memory, when it is not given, belongs to the call's stream as well."""
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn((1, h, 96, D), generator=g).to(torch.bfloat16).pin_memory() for h in (HQ, HKV, HKV))
    want = attn.attn_fwd_host(q, k, v)
    side = torch.cuda.Stream()
    torch.cuda._sleep(DELAY)
    for stream in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        got = attn.attn_fwd_host(q, k, v, stream=stream)
        mine = [torch.full((1, h, 96, D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV, HQ)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.all(t == 7) for t in mine)


@pytest.mark.parametrize("name", NAMES)
def test_a_captured_fork(name):
    """A capture that forks to another stream, where the call runs and its first results are dropped: the graph's
    replays give the call's results, and what the capture's own stream makes meanwhile is not written over."""
    fn = calls()[name]
    want = [t.clone() for t in fn(None)]
    side = torch.cuda.Stream()
    fn(side)  # workspaces are in place before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000)
        fn(side)
        mine = [torch.full_like(t, 7) for t in want for _ in range(3)]
        got = fn(side)
        main.wait_stream(side)
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.all(t == 7) for t in mine)
