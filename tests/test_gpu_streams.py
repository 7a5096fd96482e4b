"""Calls with stream=: what they allocate belongs to that stream, whatever the current one still does or does next."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import online_hadamard_b200 as m
    m.load_library()
    m.macaq_device_status(clear=True)
    return m


def calls(mq):
    """name -> (call(stream), bytes of its workspace)"""
    g = torch.Generator().manual_seed(60)
    Hq, Hk, D, page, T, K, N = 8, 2, 128, 32, 96, 1024, 512
    x = torch.randn(T, (Hq + 2 * Hk) * D, generator=g).to(torch.bfloat16).cuda()
    h = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn(N, K, generator=g) * 0.05).cuda()
    s = torch.ones(K).cuda()
    Wq, Ws, am = mq.macaq_fold_weights(W, s)
    Aq, As = mq.macaq_act_transform_quant(h, am)
    cache = torch.zeros(4, Hk, mq.kv4_page_bytes(page, D), dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, device="cuda")
    q = mq.macaq_kv4_append(x, Hq, Hk, D, cache, page, slots)
    tab = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    counts = torch.tensor([T // 3, T - T // 3], device="cuda")
    pair = (torch.stack((am, am)), torch.cat((Wq, Wq)), torch.cat((Ws, Ws)), (N, N))
    two = (torch.stack((am, am)), torch.stack((Wq, Wq)), torch.cat((Ws, Ws)), N)
    return {
        "norm_rope": (lambda st: mq.macaq_qk_norm_rope(x, Hq, Hk, D, stream=st), 0),
        "append": (lambda st: mq.macaq_kv4_append(x, Hq, Hk, D, cache, page, slots, stream=st), 0),
        "gather": (lambda st: mq.macaq_kv4_gather(cache, D, page, slots, stream=st), 0),
        "attention": (lambda st: mq.macaq_kv4_attention(q, cache, page, tab, lens, cu, max_q=T, stream=st),
                      mq.kv4_attention_workspace_bytes(T, 1, Hq, Hk, D, T)),
        "linear": (lambda st: mq.macaq_w4a4_linear(h, am, Wq, Ws, N, stream=st), mq.linear_workspace_bytes(T, N, K)),
        "plain linear": (lambda st: mq.macaq_mxfp4_linear(h, Wq, Ws, N, stream=st), mq.linear_workspace_bytes(T, N, K)),
        "noalloc": (lambda st: mq.macaq_w4a4_linear_noalloc(h, am, Wq, Ws, N, stream=st), 0),
        "stacked": (lambda st: mq.macaq_w4a4_linear_multi(h, *pair, stream=st), mq.linear_multi_workspace_bytes(T, 2, K)),
        "grouped": (lambda st: mq.macaq_w4a4_grouped_linear(h, [T // 3, T - T // 3], *two, stream=st),
                    mq.grouped_workspace_bytes([T // 3, T - T // 3], N, K)),
        "grouped device": (lambda st: mq.macaq_w4a4_grouped_linear_device(h, counts, *two, stream=st),
                           mq.grouped_device_workspace_bytes(T, 2, N, K)),
        "gemm": (lambda st: mq.macaq_mxfp4_gemm(Aq, As, Wq, Ws, T, N, K, stream=st), mq.gemm_workspace_bytes(T, N, K)),
        "fold": (lambda st: mq.macaq_fold_weights(W, s, stream=st), 0),
        "quantise": (lambda st: mq.macaq_act_transform_quant(h, am, stream=st), 0),
        "quantise plain": (lambda st: mq.macaq_act_quant_plain(h, stream=st), 0),
        "calibrate": (lambda st: mq.macaq_calibrate_scale(h, W, stream=st), 0),
        "hessian": (lambda st: mq.macaq_calib_hessian(h, am, stream=st), 0),
        "row-major scales": (lambda st: mq.macaq_scales_to_rowmajor(As, T, K, stream=st), 0),
    }


NAMES = ["norm_rope", "append", "gather", "attention", "linear", "plain linear", "noalloc", "stacked", "grouped", "grouped device",
         "gemm", "fold", "quantise", "quantise plain", "calibrate", "hessian", "row-major scales"]


@pytest.mark.parametrize("name", NAMES)
def test_results_are_not_where_the_current_stream_still_writes(mq, name):
    """The current stream is late: what it does with memory that it has given back comes after the call's result."""
    call, _ = calls(mq)[name]
    want = call(None)
    want = want if isinstance(want, tuple) else (want,)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    warm = call(side)
    torch.cuda.synchronize()
    del warm
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    late = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda").fill_(0x5A) for t in want for _ in range(3)]
    del late
    got = call(side)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    if name in ("fold", "quantise", "quantise plain"):  # the scales' padding is unspecified
        keep = [0] + ([2] if name == "fold" else [])
        want, got = [want[i] for i in keep], [got[i] for i in keep]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["attention", "linear", "plain linear", "stacked", "grouped", "grouped device"])
def test_workspaces_are_the_streams_own(mq, name):
    """Dropped when the call returns, they are not handed to the current stream while the kernels still run."""
    call, need = calls(mq)[name]
    assert need > 0
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    out = call(side)
    sizes = [b["size"] for seg in torch.cuda.memory_snapshot() if seg["stream"] == side.cuda_stream for b in seg["blocks"]]
    torch.cuda.synchronize()
    del out
    assert max(sizes, default=0) >= need


def test_results_live_until_the_current_stream_is_done_with_them(mq):
    """A result that is read on the current stream and dropped is not used again by the next call before that."""
    call, _ = calls(mq)["linear"]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    y = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copy = y.clone()
    del y
    with torch.cuda.stream(side):
        for _ in range(8):
            torch.empty_like(want).fill_(3.0)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_a_stream_of_its_own_inside_a_graph(mq):
    """A call on a forked stream while the current one captures."""
    call, _ = calls(mq)["attention"]
    want = call(None)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_the_gather_of_a_split_linear_follows_it_on_its_stream(mq, monkeypatch):
    from online_hadamard_b200 import tensor_parallel as tp
    g = torch.Generator().manual_seed(61)
    x = torch.randn(40, 512, generator=g).to(torch.bfloat16).cuda()
    Wq, Ws, am = mq.macaq_fold_weights((torch.randn(256, 512, generator=g) * 0.05).cuda(), torch.ones(512).cuda())
    want = mq.macaq_w4a4_linear(x, am, Wq, Ws, 256)
    at = []
    monkeypatch.setattr(tp, "gather_columns", lambda y, N, group=None: at.append(torch.cuda.current_stream()) or y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = tp.tp_w4a4_linear(x, am, Wq, Ws, 256, stream=side)
    side.synchronize()
    assert at == [side] and torch.equal(y, want)
