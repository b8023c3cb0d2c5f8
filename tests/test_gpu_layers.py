"""Full-attention layers over the 4-bit cache and gated delta layers as a serving program uses them: captured into
graphs, on other streams, two calls at once, a hybrid stack from prompts to tokens, rows that lie far apart, results that go
past the caches.  Every comparison here is of a call with the same call made eagerly, alone, in pieces or on contiguous
rows, bit for bit, but for the one that names its bound.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as lref
from tests import mixers_reference as ref
from tests.test_gpu_mixers import DT, _eager, _i32, _kda, _r, _spread

pytestmark = pytest.mark.gpu


def _u8(seed, *shape):
    """Bytes that stand for numbers as elements and as sizes (2^-97 to 2^-7)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(30, 121, shape, generator=g, dtype=torch.uint8).cuda()


def _room(need):
    assert need > 0
    return torch.full((need // 4,), float("nan"), device="cuda")


def _attn(kda, dtype):
    H, Hkv, d, cu = 6, 2, 64, _i32(0, 90, 90, 260)
    q, k, v, o = _r(1, dtype, 262, H, d), _r(2, dtype, 262, Hkv, d), _r(3, dtype, 262, Hkv, d), _r(4, dtype, 262, H, d)
    return [o], lambda: kda.attn_prefill(q, k, v, cu, o=o)


def _attn_split(kda, dtype, workspace):
    H, Hkv, d, Nk = 4, 2, 128, 5000
    q, k, v, o = _r(1, dtype, 20, H, d), _r(2, dtype, Nk, Hkv, d), _r(3, dtype, Nk, Hkv, d), _r(4, dtype, 20, H, d)
    cu, cu_k = _i32(0, 8, 20), _i32(0, 3000, Nk)
    ws = _room(kda.attn_prefill_workspace_bytes(2, 20, Nk, H, Hkv, d, DT[dtype]))
    return [o], lambda: kda.attn_prefill(q, k, v, cu, cu_k, o=o, workspace=ws if workspace else None)


def _cache(kda, dtype):
    Hkv, d, page = 3, 128, 16
    k, v = _r(1, dtype, 70, Hkv, d), _r(2, dtype, 70, Hkv, d)
    kc, vc = (_u8(s, 12, Hkv, kda.cache_page_bytes(d, page)) for s in (3, 4))
    pages, cu, start, all_cu = _i32([5, 0, 9, -1], [1, 7, 3, 11]), _i32(0, 30, 70), _i32(3, 11), _i32(0, 33, 84)
    rk, rv = _r(5, dtype, 84, Hkv, d), _r(6, dtype, 84, Hkv, d)

    def call():
        kda.cache_write(k, v, kc, vc, pages, cu, start)
        kda.cache_read(kc, vc, pages, all_cu, 84, d, dtype=DT[dtype], k=rk, v=rv)
    return [kc, vc, rk, rv], call


def _attn_step(kda, dtype, m, workspace):
    N, H, Hkv, d, page = 3, 8, 2, 128, 64
    n_pages = 120
    kc, vc = (_u8(s, n_pages, Hkv, kda.cache_page_bytes(d, page)) for s in (3, 4))
    pages = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).int().view(N, -1).cuda()
    q, o, lens = _r(1, dtype, N, m, H, d), _r(2, dtype, N, m, H, d), _i32(2500, 1, 777)
    ws = _room(kda.attn_step_workspace_bytes(N, m, H, Hkv, d, pages.shape[1], page, DT[dtype]))
    return [o], lambda: kda.attn_step(q, kc, vc, pages, lens, o=o, workspace=ws if workspace else None)


def _delta(kda, dtype, dk, dv, seg, workspace):
    B, T, H, Hk = 2, 333, 4, 2
    q, k, v = _r(1, dtype, B, T, Hk, dk) * dk ** -0.5, _r(2, dtype, B, T, Hk, dk) * dk ** -0.5, _r(3, dtype, B, T, H, dv)
    g, beta = -_r(4, "f32", B, T, H).abs() * 0.2, torch.sigmoid(_r(5, "f32", B, T, H))
    S, o, lens = _r(6, "f32", B, H, dk, dv), _r(7, dtype, B, T, H, dv), _i32(333, 150)
    ws = _room(kda.delta_workspace_bytes(B, T, H, Hk, dk, dv, DT[dtype], seg)) if workspace else None
    return [S, o], lambda: kda.delta_prefill(q, k, v, g, beta, S, lens=lens, seg_len=seg, o=o, S_T=S, workspace=ws)


def _delta_step(kda, dtype):
    N, H, Hk, dk, dv = 5, 6, 3, 128, 64
    q, k, v = _r(1, dtype, N, Hk, dk) * dk ** -0.5, _r(2, dtype, N, Hk, dk) * dk ** -0.5, _r(3, dtype, N, H, dv)
    g, beta, S, o = -_r(4, "f32", N, H).abs(), torch.sigmoid(_r(5, "f32", N, H)), _r(6, "f32", N, H, dk, dv), _r(7, dtype, N, H, dv)
    return [S, o], lambda: kda.delta_step(q, k, v, g, beta, S, o=o)


CALLS = {
    "attn_prefill-bf16": lambda k: _attn(k, "bf16"),
    "attn_prefill-f32": lambda k: _attn(k, "f32"),
    "attn_prefill-split": lambda k: _attn_split(k, "bf16", True),
    "attn_prefill-split-f32-own_workspace": lambda k: _attn_split(k, "f32", False),
    "cache-bf16": lambda k: _cache(k, "bf16"),
    "cache-f32": lambda k: _cache(k, "f32"),
    "attn_step-bf16": lambda k: _attn_step(k, "bf16", 1, True),
    "attn_step-three-f32-own_workspace": lambda k: _attn_step(k, "f32", 3, False),
    "delta_prefill-bf16": lambda k: _delta(k, "bf16", 128, 128, 384, False),
    "delta_prefill-split": lambda k: _delta(k, "bf16", 128, 64, 64, True),
    "delta_prefill-split-f32-own_workspace": lambda k: _delta(k, "f32", 64, 64, 128, False),
    "delta_step-bf16": lambda k: _delta_step(k, "bf16"),
}


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
    names = ["attn_prefill-split-f32-own_workspace", "cache-bf16", "attn_step-three-f32-own_workspace",
             "delta_prefill-split-f32-own_workspace"]
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


def test_a_captured_hybrid_stack_answers_token_by_token_like_eager_calls():
    """Projection rows -> convolution -> gated delta rule, and full attention with its 4-bit cache beside it, for packed
    prompts of one length; then tokens from one captured graph that also moves the lengths on, against the same tokens made
    eagerly."""
    kda = _kda()
    N, T, more, H, Hk, dk, dv, W = 3, 150, 5, 4, 2, 128, 128, 4
    Ha, Hkv, d, page = 4, 2, 64, 16
    width = 2 * Hk * dk + H * dv
    rows = _r(1, "bf16", N, T + more, width + 2 * H)
    qkv = _r(2, "bf16", N, T + more, (Ha + 2 * Hkv) * d)
    w, bias = _r(3, "bf16", width, W) * 0.5, _r(4, "bf16", width)

    def delta_args(u, part):
        q, k = (u[..., i * Hk * dk:(i + 1) * Hk * dk].unflatten(-1, (Hk, dk)) for i in (0, 1))
        k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
        gate = part[..., width:].float()
        return (q * dk ** -0.5, k, u[..., 2 * Hk * dk:].unflatten(-1, (H, dv)), -torch.nn.functional.softplus(gate[..., :H]),
                torch.sigmoid(gate[..., H:]).contiguous())

    def heads(part):
        return (part[..., :Ha * d].unflatten(-1, (Ha, d)), part[..., Ha * d:(Ha + Hkv) * d].unflatten(-1, (Hkv, d)),
                part[..., (Ha + Hkv) * d:].unflatten(-1, (Hkv, d)))

    hist = torch.empty(N, W - 1, width, dtype=torch.bfloat16, device="cuda")
    S = torch.zeros(N, H, dk, dv, device="cuda")
    n_pages = N * -(-(T + more) // page)
    pages = torch.randperm(n_pages, generator=torch.Generator().manual_seed(2)).int().view(N, -1).cuda()
    kc, vc = (torch.full((n_pages, Hkv, kda.cache_page_bytes(d, page)), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    lens = torch.full((N,), T, dtype=torch.int32, device="cuda")
    cu = _i32(*range(0, N * T + 1, T))
    prompt, attn = rows[:, :T].contiguous(), qkv[:, :T].reshape(N * T, -1)
    u, _ = kda.conv_prefill(prompt[..., :width], w, bias, state_out=hist)
    kda.delta_prefill(*delta_args(u, prompt), S, S_T=S)
    q, k, v = heads(attn)
    kda.cache_write(k, v, kc, vc, pages, cu)
    kda.attn_prefill(q, k, v, cu)
    state = [hist, S, kc, vc, lens]
    start = [t.clone() for t in state]

    row, att = torch.empty_like(rows[:, 0]), torch.empty_like(qkv[:, 0])
    y, o = torch.empty(N, H, dv, dtype=torch.bfloat16, device="cuda"), torch.empty(N, Ha, d, dtype=torch.bfloat16, device="cuda")

    def token():
        c = kda.conv_step(row[:, :width], w, hist, bias)
        kda.delta_step(*delta_args(c, row), S, o=y)
        q, k, v = heads(att)
        kda.cache_write(k, v, kc, vc, pages, None, lens)
        lens.add_(1)
        kda.attn_step(q, kc, vc, pages, lens, o=o)

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


@pytest.mark.parametrize("op", ["attn_prefill", "cache_write", "attn_step", "delta_prefill", "delta_step"])
def test_rows_far_apart_pass_32_bits(op):
    """Rows of the inputs lie so far apart that the last ones begin past 2^32 bytes and 2^31 elements."""
    kda = _kda()
    print("far rows", op, flush=True)
    T = 700
    far = (1 << 31) // (T - 100) // 8 * 8   # the last rows begin past 2^31 elements
    assert far <= 1 << 22 and far * (T - 1) > 1 << 31

    def spread(t):
        return _spread(t[None], far)[0]

    if op == "attn_prefill":
        q, k, v, cu = _r(1, "bf16", T, 2, 64), _r(2, "bf16", T, 1, 64), _r(3, "bf16", T, 1, 64), _i32(0, 20, T)
        a, b = [kda.attn_prefill(q, k, v, cu)], [kda.attn_prefill(spread(q), spread(k), spread(v), cu)]
        q, k, v = q.float(), k.float(), v.float()
        a.append(kda.attn_prefill(q, k, v, cu))
        b.append(kda.attn_prefill(spread(q), spread(k), spread(v), cu))
    elif op in ("cache_write", "attn_step"):
        k, v, q = _r(1, "bf16", T, 1, 64), _r(2, "bf16", T, 1, 64), _r(3, "bf16", T, 2, 64)
        pages = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
        pools = [[torch.zeros(T, 1, kda.cache_page_bytes(64, 16), dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
        kda.cache_write(k, v, *pools[0], pages)
        kda.cache_write(spread(k), spread(v), *pools[1], pages)
        a, b = pools
        if op == "attn_step":
            lens = torch.ones(T, dtype=torch.int32, device="cuda")
            a, b = [kda.attn_step(q, *a, pages, lens)], [kda.attn_step(spread(q), *a, pages, lens)]
    else:
        q, k, v = _r(1, "bf16", T, 1, 64) * 0.1, _r(2, "bf16", T, 1, 64) * 0.1, _r(3, "bf16", T, 2, 64)
        g, beta = -_r(4, "f32", T, 2).abs(), torch.sigmoid(_r(5, "f32", T, 2))
        if op == "delta_prefill":
            a, b = (kda.delta_prefill(*(x[None] for x in (*rows, g, beta)), seg_len=128)
                    for rows in ((q, k, v), (spread(q), spread(k), spread(v))))
        else:
            S = [torch.ones(T, 2, 64, 64, device="cuda") for _ in range(2)]
            a = [kda.delta_step(q, k, v, g, beta, S[0]), S[0]]
            b = [kda.delta_step(spread(q), spread(k), spread(v), g, beta, S[1]), S[1]]
    torch.cuda.synchronize()
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("dtype,Hkv,d", [("bf16", 8, 128), ("f32", 5, 64)])
def test_cache_rows_that_go_past_the_caches(dtype, Hkv, d):
    """Results of 128 MiB and more are stored past the caches: the same rows as in pieces."""
    kda = _kda()
    page, esz = 64, 2 if dtype == "bf16" else 4
    tokens = (128 << 20) // (2 * Hkv * d * esz) + 3
    n_pages = -(-tokens // page)
    kc, vc = (_u8(s, n_pages, Hkv, kda.cache_page_bytes(d, page)) for s in (1, 2))
    pages = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).int()[None].cuda()
    assert 2 * tokens * Hkv * d * esz >= 128 << 20
    k, v = kda.cache_read(kc, vc, pages, _i32(0, tokens), tokens, d, dtype=DT[dtype])
    for at in range(0, tokens, 10007):
        n = min(10007, tokens - at)
        a, b = kda.cache_read(kc, vc, pages, _i32(0, n), n, d, start=_i32(at), dtype=DT[dtype])
        assert torch.equal(k[at:at + n], a) and torch.equal(v[at:at + n], b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_updates_that_expand_run_without_a_split(dtype):
    """beta |k|^2 = 3 along one direction beside decays of a half: every token takes that part of the state to minus
    itself, however long the prompt.  The signs alternate exactly, so that v = 0 leaves +-S0 there and nothing elsewhere."""
    kda = _kda()
    T, d = 700, 64
    k = torch.zeros(1, T, 1, d, dtype=DT[dtype])
    k[..., 0] = 1.0
    q, v = k.clone(), torch.zeros(1, T, 1, d, dtype=DT[dtype])
    g, beta = torch.full((1, T, 1), float(np.log(0.5))), torch.full((1, T, 1), 3.0)
    S0 = torch.ones(1, 1, d, d)
    o, S = kda.delta_prefill(q.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), S0.cuda(), seg_len=T + 4)
    torch.cuda.synchronize()
    # log(0.5) in fp32 is off by 2^-25 of it: (1 + 2^-25)^700 of decays, and a block's own roundings, T 90 u in all
    tol = T * 90 * ref.U32
    sign = 1.0 if T % 2 == 0 else -1.0
    assert float((S[0, 0, 0] - sign).abs().max()) <= tol and float(S[0, 0, 1:].abs().max()) <= tol
    want = torch.tensor([-1.0, 1.0]).repeat(T // 2)[None, :, None, None]
    assert float((o.float().cpu() - want).abs().max()) <= tol + ref.half_step(DT[dtype]) * 2


def test_attention_in_fp32_over_the_range():
    """Values from 1e-20 to 1e30 with scores of order one: three bf16 parts hold 24 bits of each."""
    kda = _kda()
    n, H, d = 200, 2, 64
    q, k, v = _r(1, "f32", n, H, d).cpu(), _r(2, "f32", n, 1, d).cpu(), _r(3, "f32", n, 1, d).cpu()
    v = v * torch.exp2(torch.linspace(-66, 99, d).round())
    q, k = q * 2.0 ** 40, k * 2.0 ** -43
    want, mag, a = lref.attn_prefill(q, k, v, [0, n], [0, n], 1.0)
    o = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), _i32(0, n), scale=1.0)
    torch.cuda.synchronize()
    e = ref.U32 * ((2 * d + 32) * a[..., None] + 40)
    assert (np.abs(ref.f64(o) - want) <= (2 * e + 4 * n * ref.U32) * mag).all()


def test_binding_refuses_rows_it_cannot_describe():
    """Wrong strides, types, shapes and pools: refused on the host, before any launch, with the argument's name."""
    kda = _kda()
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    cu = _i32(0, 10)
    q, k = f(10, 4, 64), f(10, 2, 64)
    pool, pages = torch.zeros(3, 2, kda.cache_page_bytes(64, 16), dtype=torch.uint8, device="cuda"), _i32([0, 1, 2])
    for call, err, text in (
            (lambda: kda.attn_prefill(f(10, 4, 128)[..., ::2], k, k, cu), ValueError, "q: the elements of a token must be contiguous"),
            (lambda: kda.attn_prefill(q, k.bfloat16(), k, cu), TypeError, "k must be torch.float32, got torch.bfloat16"),
            (lambda: kda.attn_prefill(q, k, k[:9], cu), ValueError, "v must have shape"),
            (lambda: kda.attn_prefill(q, k, k, cu.long()), TypeError, "cu_q must be torch.int32"),
            (lambda: kda.attn_prefill(q, k.cpu(), k, cu), ValueError, "k must be on"),
            (lambda: kda.cache_write(k, k, pool[..., :-2], pool, pages, cu), ValueError, "k_cache"),
            (lambda: kda.cache_write(k, k, pool, pool.float(), pages, cu), TypeError, "v_cache must be torch.uint8"),
            (lambda: kda.cache_write(k[:, :1], k[:, :1], pool, pool.clone(), pages, cu), ValueError, "k must have shape"),
            (lambda: kda.cache_read(pool, pool.clone(), pages, cu, 10, 64, dtype=torch.float16), TypeError, "bfloat16 or"),
            (lambda: kda.attn_step(f(2, 4, 64), pool, pool.clone(), pages, _i32(3)), ValueError, "pages must have a row"),
            (lambda: kda.delta_prefill(q[None], q[None], q[None], f(1, 10, 4), f(1, 10, 3)), ValueError, "beta must have shape"),
            (lambda: kda.delta_prefill(q[None], q[None], q[None], f(1, 10, 4).bfloat16(), f(1, 10, 4)), TypeError, "g must be torch.float32"),
            (lambda: kda.delta_step(q, q, q, f(10, 4), f(10, 4), f(10, 4, 64, 64).transpose(2, 3)), ValueError, "S must be contiguous"),
    ):
        with pytest.raises(err, match=text):
            call()
