"""The token mixers as a serving program uses them: captured into graphs, on other streams, two calls at
once, a layer stack from prompt to tokens, and rows that lie far apart.  Every comparison here is of a
call with the same call made eagerly, alone or on contiguous rows, bit for bit: no sum depends on how
a call is issued or on where its rows lie.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _r(seed, dtype, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype]).cuda()


def _neg(seed, H):
    return -torch.rand(H, generator=torch.Generator().manual_seed(seed)).cuda() * 8 - 1


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _conv_prefill(kda, dtype):
    x, w, bias = _r(1, dtype, 2, 70, 136), _r(2, dtype, 136, 4), _r(3, dtype, 136)
    state, y, lens = _r(4, dtype, 2, 3, 136), _r(5, dtype, 2, 70, 136), _i32(70, 41)
    return [state, y], lambda: kda.conv_prefill(x, w, bias, state, lens=lens, y=y, state_out=state)


def _conv_step(kda, dtype):
    x, w, state, y = _r(1, dtype, 7, 136), _r(2, dtype, 136, 3), _r(3, dtype, 7, 2, 136), _r(4, dtype, 7, 136)
    return [state, y], lambda: kda.conv_step(x, w, state, y=y)


def _ssm(kda, dtype, n, p, seg, workspace):
    B, T, H, G = 2, 333, 4, 2
    x, z, dt = _r(1, dtype, B, T, H, p), _r(2, dtype, B, T, H, p), _r(3, dtype, B, T, H)
    Bm, Cm, S, y = _r(4, dtype, B, T, G, n), _r(5, dtype, B, T, G, n), _r(6, "f32", B, H, n, p), _r(7, dtype, B, T, H, p)
    A, D, lens = _neg(8, H), _r(9, "f32", H), _i32(333, 150)
    ws = None
    if workspace:
        need = kda.ssm_workspace_bytes(B, T, H, G, n, p, DT[dtype], seg)
        assert need > 0
        ws = torch.full((need // 4,), float("nan"), device="cuda")
    return [S, y], lambda: kda.ssm_prefill(x, dt, A, Bm, Cm, S, D=D, z=z, lens=lens, seg_len=seg, y=y, S_T=S, workspace=ws)


def _ssm_step(kda, dtype):
    N, H, G, n, p = 3, 6, 3, 64, 128
    x, z, dt = _r(1, dtype, N, H, p), _r(2, dtype, N, H, p), _r(3, dtype, N, H)
    Bm, Cm, S, y = _r(4, dtype, N, G, n), _r(5, dtype, N, G, n), _r(6, "f32", N, H, n, p), _r(7, dtype, N, H, p)
    A, D = _neg(8, H), _r(9, "f32", H)
    return [S, y], lambda: kda.ssm_step(x, dt, A, Bm, Cm, S, D=D, z=z, y=y)


def _window_prefill(kda, dtype):
    B, T, H, Hkv, d, win, sinks = 2, 130, 6, 2, 64, 50, 3
    q, k, v, o = _r(1, dtype, B, T, H, d), _r(2, dtype, B, T, Hkv, d), _r(3, dtype, B, T, Hkv, d), _r(4, dtype, B, T, H, d)
    kc, vc = _r(5, dtype, B, win + sinks, Hkv, d), _r(6, dtype, B, win + sinks, Hkv, d)
    start, lens = _i32(77, 1000), _i32(130, 33)
    return [o, kc, vc], lambda: kda.window_prefill(q, k, v, win, sinks, k_cache=kc, v_cache=vc, start=start, lens=lens, o=o)


def _window_split(kda, dtype, workspace):
    B, T, H, Hkv, d, win, sinks = 2, 20, 4, 2, 128, 900, 4
    q, k, v, o = _r(1, dtype, B, T, H, d), _r(2, dtype, B, T, Hkv, d), _r(3, dtype, B, T, Hkv, d), _r(4, dtype, B, T, H, d)
    kc, vc = _r(5, dtype, B, win + sinks, Hkv, d), _r(6, dtype, B, win + sinks, Hkv, d)
    start, lens = _i32(77, 5000), _i32(20, 13)
    need = kda.window_prefill_workspace_bytes(B, T, H, Hkv, d, win, sinks, DT[dtype], continued=True)
    assert need > 0
    ws = torch.full((need // 4,), float("nan"), device="cuda") if workspace else None
    return [o, kc, vc], lambda: kda.window_prefill(q, k, v, win, sinks, k_cache=kc, v_cache=vc, start=start, lens=lens, o=o,
                                                   workspace=ws)


def _window_step(kda, dtype, workspace):
    N, H, Hkv, d, win, sinks = 2, 6, 2, 128, 1500, 4
    q, k, v, o = _r(1, dtype, N, H, d), _r(2, dtype, N, Hkv, d), _r(3, dtype, N, Hkv, d), _r(4, dtype, N, H, d)
    kc, vc = _r(5, dtype, N, win + sinks, Hkv, d), _r(6, dtype, N, win + sinks, Hkv, d)
    pos = _i32(9000, 800)
    need = kda.window_step_workspace_bytes(N, H, Hkv, d, win, sinks, DT[dtype])
    assert need > 0
    ws = torch.full((need // 4,), float("nan"), device="cuda") if workspace else None
    return [o, kc, vc], lambda: kda.window_step(q, k, v, kc, vc, pos, win, sinks, o=o, workspace=ws)


CALLS = {
    "conv_prefill-bf16": lambda k: _conv_prefill(k, "bf16"),
    "conv_prefill-f32": lambda k: _conv_prefill(k, "f32"),
    "conv_step-bf16": lambda k: _conv_step(k, "bf16"),
    "ssm_prefill-one_pass": lambda k: _ssm(k, "bf16", 128, 64, 512, False),
    "ssm_prefill-split": lambda k: _ssm(k, "bf16", 128, 64, 64, True),
    "ssm_prefill-split-own_workspace": lambda k: _ssm(k, "bf16", 64, 128, 128, False),
    "ssm_prefill-split-f32": lambda k: _ssm(k, "f32", 64, 64, 64, True),
    "ssm_step-bf16": lambda k: _ssm_step(k, "bf16"),
    "window_prefill-bf16": lambda k: _window_prefill(k, "bf16"),
    "window_prefill-f32": lambda k: _window_prefill(k, "f32"),
    "window_prefill-split": lambda k: _window_split(k, "bf16", True),
    "window_prefill-split-f32-own_workspace": lambda k: _window_split(k, "f32", False),
    "window_step-bf16": lambda k: _window_step(k, "bf16", True),
    "window_step-f32-own_workspace": lambda k: _window_step(k, "f32", False),
}


def _eager(call, outs):
    """The results of one call from the buffers' present contents, which are put back."""
    before = [t.clone() for t in outs]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t, b in zip(outs, before):
        t.copy_(b)
    torch.cuda.synchronize()
    return before, want


@pytest.mark.parametrize("name", CALLS)
def test_calls_replay_in_a_graph(name):
    kda = _kda()
    print("graph", name, flush=True)
    outs, call = CALLS[name](kda)
    before, want = _eager(call, outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        for t, b in zip(outs, before):
            t.copy_(b)
        torch.full((1 << 16,), float("nan"), device="cuda").add_(1)   # memory of other calls, between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip(outs, want):
            assert torch.equal(t, u), f"replay {i}"


@pytest.mark.parametrize("name", CALLS)
def test_calls_run_on_the_current_stream(name):
    """Inputs that a side stream is still about to write: a call on any other stream would miss them."""
    kda = _kda()
    print("stream", name, flush=True)
    outs, call = CALLS[name](kda)
    before, want = _eager(call, outs)
    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    m = torch.zeros(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            m = m @ m
        for t, b in zip(outs, before):
            t.copy_(b)
        call()
    side.synchronize()
    for t, u in zip(outs, want):
        assert torch.equal(t, u)


@pytest.mark.parametrize("name", CALLS)
def test_two_calls_at_once_keep_apart(name):
    """Two streams, a set of buffers and a workspace each (the caller's or the call's own)."""
    kda = _kda()
    print("two at once", name, flush=True)
    pairs = [CALLS[name](kda), CALLS[name](kda)]
    before, want = _eager(pairs[0][1], pairs[0][0])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for outs, _ in pairs:
            for t, b in zip(outs, before):
                t.copy_(b)
        torch.cuda.synchronize()
        for s, (_, call) in zip(streams, pairs):
            with torch.cuda.stream(s):
                call()
        torch.cuda.synchronize()
        for outs, _ in pairs:
            for t, u in zip(outs, want):
                assert torch.equal(t, u)


def test_host_threads_call_side_by_side():
    """Four host threads, a stream and a set of buffers each; every call's results are those of a lone call."""
    import threading
    kda = _kda()
    names = ["conv_prefill-bf16", "ssm_prefill-split-own_workspace", "window_prefill-split-f32-own_workspace",
             "window_step-f32-own_workspace"]
    print("threads", names, flush=True)
    jobs, wrong = [], []
    for name in names:
        outs, call = CALLS[name](kda)
        jobs.append((name, outs, call, *_eager(call, outs)))

    def work(name, outs, call, before, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(20):
                for t, b in zip(outs, before):
                    t.copy_(b)
                call()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(t, u) for t, u in zip(outs, want)):
                    wrong.append((name, i))

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_a_captured_layer_stack_answers_token_by_token_like_eager_calls():
    """Projection rows -> convolution -> scan, and window attention beside it, for a prompt; then tokens
    from one captured graph that also moves the positions on, against the same tokens made eagerly."""
    kda = _kda()
    N, T, more, H, G, n, p, W = 3, 150, 5, 4, 1, 128, 64, 4
    Ha, Hkv, d, win, sinks = 4, 2, 64, 60, 2
    width = H * p + 2 * G * n
    rows = _r(1, "bf16", N, T + more, width + H * p + H + 4)
    qkv = _r(2, "bf16", N, T + more, (Ha + 2 * Hkv) * d)
    w, bias, A, D, dtb = _r(3, "bf16", width, W) * 0.5, _r(4, "bf16", width), _neg(5, H), _r(6, "f32", H), _r(7, "f32", H) - 3

    def scan_args(u, part):
        return (u[..., :H * p].unflatten(-1, (H, p)), part[..., width + H * p:width + H * p + H], A,
                u[..., H * p:H * p + G * n].unflatten(-1, (G, n)), u[..., H * p + G * n:].unflatten(-1, (G, n)))

    def heads(part):
        return (part[..., :Ha * d].unflatten(-1, (Ha, d)), part[..., Ha * d:(Ha + Hkv) * d].unflatten(-1, (Hkv, d)),
                part[..., (Ha + Hkv) * d:].unflatten(-1, (Hkv, d)))

    hist = torch.empty(N, W - 1, width, dtype=torch.bfloat16, device="cuda")
    S = torch.zeros(N, H, n, p, device="cuda")
    kc = torch.full((N, win + sinks, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc, pos = kc.clone(), torch.full((N,), T, dtype=torch.int32, device="cuda")
    prompt, attn = rows[:, :T].contiguous(), qkv[:, :T].contiguous()
    u, _ = kda.conv_prefill(prompt[..., :width], w, bias, state_out=hist)
    kda.ssm_prefill(*scan_args(u, prompt), S, D=D, z=prompt[..., width:width + H * p].unflatten(-1, (H, p)), dt_bias=dtb, S_T=S)
    kda.window_prefill(*heads(attn), win, sinks, k_cache=kc, v_cache=vc)
    state = [hist, S, kc, vc, pos]
    start = [t.clone() for t in state]

    row, att = torch.empty_like(rows[:, 0]), torch.empty_like(qkv[:, 0])
    y, o = torch.empty(N, H, p, dtype=torch.bfloat16, device="cuda"), torch.empty(N, Ha, d, dtype=torch.bfloat16, device="cuda")

    def token():
        c = kda.conv_step(row[:, :width], w, hist, bias)
        kda.ssm_step(*scan_args(c, row), S, D=D, z=row[:, width:width + H * p].unflatten(-1, (H, p)), dt_bias=dtb, y=y)
        kda.window_step(*heads(att), kc, vc, pos, win, sinks, o=o)
        pos.add_(1)

    def run(step):
        for t, b in zip(state, start):
            t.copy_(b)
        got = []
        for t in range(T, T + more):
            row.copy_(rows[:, t])
            att.copy_(qkv[:, t])
            step()
            got += [y.clone(), o.clone()]
        torch.cuda.synchronize()
        return got + [t.clone() for t in state]

    want = run(token)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    for _ in range(2):
        for g, e in zip(run(graph.replay), want):
            assert torch.equal(g, e)
    assert all(torch.isfinite(t.float()).all() for t in want[:2 * more])


def _spread(t, stride):
    """The same rows with `stride` elements between them (rows = all axes but the last ones of a token)."""
    width = t[0, 0].numel()
    rows = t.shape[0] * t.shape[1]
    far = torch.empty((rows - 1) * stride + width, dtype=t.dtype, device=t.device)
    view = far.as_strided((*t.shape[:2], width), (t.shape[1] * stride, stride, 1))
    view.copy_(t.reshape(*t.shape[:2], width))
    return view.unflatten(-1, t.shape[2:]) if t.dim() > 3 else view


@pytest.mark.parametrize("op", ["conv", "ssm", "window"])
def test_rows_far_apart_pass_32_bits(op):
    """Rows of one input lie so far apart that the last ones begin past 2^32 bytes and 2^31 elements."""
    kda = _kda()
    print("far rows", op, flush=True)
    B, T = 1, 700
    far = (1 << 31) // (T - 100) // 8 * 8   # the last rows begin past 2^31 elements
    assert far <= 1 << 22 and far * (T - 1) > 1 << 31
    if op == "conv":
        x, w = _r(1, "bf16", B, T, 64), _r(2, "bf16", 64, 4)
        a, b = kda.conv_prefill(x, w), kda.conv_prefill(_spread(x, far), w)
    elif op == "ssm":
        x, dt, Bm, Cm = _r(1, "bf16", B, T, 1, 64), _r(2, "bf16", B, T, 1), _r(3, "bf16", B, T, 1, 64), _r(4, "bf16", B, T, 1, 64)
        a = kda.ssm_prefill(x, dt, _neg(5, 1), Bm, Cm, seg_len=128)
        b = kda.ssm_prefill(_spread(x, far), _spread(dt, far), _neg(5, 1), _spread(Bm, far), Cm, seg_len=128)
    else:
        q, k, v = _r(1, "bf16", B, T, 2, 64), _r(2, "bf16", B, T, 1, 64), _r(3, "bf16", B, T, 1, 64)
        a = [kda.window_prefill(q, k, v, 90, 3)]
        b = [kda.window_prefill(_spread(q, far), _spread(k, far), _spread(v, far), 90, 3)]
    torch.cuda.synchronize()
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_window_cache_past_32_bits():
    """The caches of later sequences begin past 2^31 elements, and one sequence's rows span 2^31 bytes; keys
    of zero weigh every row equally, so the output is the mean of the values."""
    kda = _kda()
    N, Hkv, d, win = 4, 64, 128, 1 << 17
    shape = (N, win, Hkv, d)
    assert N * win * Hkv * d > 1 << 31
    kc, vc = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))   # 8 GiB each
    kc[N - 1].zero_()
    vc[N - 1].zero_()
    vc[N - 1, 100000:100512] = 1.0
    pos = _i32(0, 0, 0, 5 * win)
    q = _r(1, "bf16", N, Hkv, d)
    k = torch.zeros(N, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 2.0)
    o = kda.window_step(q, k, v, kc, vc, pos, win)
    torch.cuda.synchronize()
    want = (512.0 + 2.0) / win
    # weights are 1 exactly and the sums of 1s and 2s exact; the division and the rounding to bf16 are left
    assert float((o[N - 1].double() - want).abs().max()) <= want * (2.0 ** -8 + 2.0 ** -22)
    assert bool((o[:N - 1] == 2.0).all())
    assert bool((vc[N - 1, 0] == 2.0).all()) and bool((vc[N - 1, 1] == 0.0).all())


def test_binding_refuses_rows_it_cannot_describe():
    """Row strides that the library's one stride cannot say, wrong types, shapes and workspaces: all refused on
    the host, before any launch, and with the argument's name."""
    kda = _kda()
    w = torch.zeros(16, 4, device="cuda")
    base = torch.zeros(4, 6, 48, device="cuda")
    for bad in (base[..., :32:2], base[..., 8:24].transpose(-1, -2).contiguous().transpose(-1, -2)):
        with pytest.raises(ValueError, match="x: the elements of a token must be contiguous"):
            kda.conv_prefill(bad, w)
    part = base[..., 8:24]
    for bad in (part[:, :5], part.transpose(0, 1), part[:, :1].expand(4, 6, 16), part[:1].expand(4, 6, 16)):
        with pytest.raises(ValueError, match="x: sequence b must start at row b"):
            kda.conv_prefill(bad, w)
    for good in (part, part[:1, :5], part[:, :1], part[:, :0], part[:0]):
        y, state = kda.conv_prefill(good, w)
        assert y.shape == good.shape and state.shape == (good.shape[0], 3, 16)
    with pytest.raises(TypeError, match="w must be torch.float32, got torch.bfloat16"):
        kda.conv_prefill(part, w.bfloat16())
    with pytest.raises(ValueError, match=r"w must have shape \(16, 4\), got \(8, 4\)"):
        kda.conv_prefill(part, w[:8])
    with pytest.raises(ValueError, match="state must be on"):
        kda.conv_step(part[:, 0], w, torch.zeros(4, 3, 16))
    with pytest.raises(ValueError, match="y must be contiguous"):
        kda.conv_step(part[:, 0], w, torch.zeros(4, 3, 16, device="cuda"), y=part[:, 0])
    with pytest.raises(TypeError, match="inputs must be bfloat16 or float32"):
        kda.conv_step(part[:, 0].half(), w, torch.zeros(4, 3, 16, device="cuda"))
    with pytest.raises(TypeError, match="bias must be a tensor"):
        kda.conv_step(part[:, 0], w, torch.zeros(4, 3, 16, device="cuda"), 1.0)

    x = torch.zeros(2, 70, 4, 64, device="cuda")
    dt, A, Bm = torch.zeros(2, 70, 4, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(2, 70, 2, 64, device="cuda")
    with pytest.raises(ValueError, match=r"Cm must have shape \(2, 70, 2, 64\)"):
        kda.ssm_prefill(x, dt, A, Bm, Bm[..., :1, :])
    with pytest.raises(ValueError, match="x: the elements"):
        kda.ssm_prefill(x.transpose(2, 3).contiguous().transpose(2, 3), dt, A, Bm, Bm)
    with pytest.raises(ValueError, match="workspace must be on"):
        kda.ssm_prefill(x, dt, A, Bm, Bm, seg_len=64, workspace=torch.zeros(1 << 20))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        kda.ssm_prefill(x, dt, A, Bm, Bm, seg_len=64, workspace=torch.zeros(1 << 10, 1 << 10, device="cuda").t())
    with pytest.raises(ValueError, match="32 bits"):
        kda.ssm_prefill(x, dt, A, Bm, Bm, seg_len=2 ** 32 + 64)
    with pytest.raises(TypeError):
        kda.ssm_prefill(x, dt, A, Bm, Bm, seg_len=64.0)
    with pytest.raises(RuntimeError, match="ssm_prefill") as e:
        kda.ssm_prefill(x, dt, A, Bm, Bm, seg_len=100)
    assert isinstance(e.value, kda.KDAError) and e.value.status == 1

    q = torch.zeros(2, 70, 4, 64, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        kda.window_prefill(q, q, q, 2 ** 32 + 5)
    with pytest.raises(ValueError, match="come together"):
        kda.window_prefill(q, q, q, 5, k_cache=torch.zeros(2, 5, 4, 64, device="cuda"))
    with pytest.raises(ValueError, match=r"k_cache must have shape \(2, 7, 4, 64\)"):
        c = torch.zeros(2, 5, 4, 64, device="cuda")
        kda.window_prefill(q, q, q, 5, 2, k_cache=c, v_cache=c)
    with pytest.raises(TypeError, match="k_cache must be a tensor"):
        kda.window_step(q[:, 0], q[:, 0], q[:, 0], None, None, _i32(0, 0), 5)
    with pytest.raises(TypeError, match="pos must be torch.int32"):
        c = torch.zeros(2, 5, 4, 64, device="cuda")
        kda.window_step(q[:, 0], q[:, 0], q[:, 0], c, c.clone(), _i32(0, 0).long(), 5)
    with pytest.raises(kda.KDAError):
        kda.window_prefill(q, q, q, 5, scale=float("nan"))
