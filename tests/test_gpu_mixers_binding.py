"""The token mixers' binding on the device: every argument of every call in turn as a batch of torch.vmap,
which has no memory that a kernel could use.  All are refused by name, on the host, before any launch.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _f(*shape):
    return torch.zeros(*shape, device="cuda")


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


def _room():
    return torch.zeros(1 << 20, device="cuda")


B, T, D, W, H, n, p, d, win = 2, 70, 16, 4, 2, 64, 64, 64, 7
CALLS = {
    "conv_prefill": lambda: dict(x=_f(B, T, D), w=_f(D, W), bias=_f(D), state=_f(B, W - 1, D), lens=_i(B), y=_f(B, T, D),
                                 state_out=_f(B, W - 1, D)),
    "conv_step": lambda: dict(x=_f(B, D), w=_f(D, W), state=_f(B, W - 1, D), bias=_f(D), y=_f(B, D)),
    "ssm_prefill": lambda: dict(x=_f(B, T, H, p), dt=_f(B, T, H), A=_f(H), Bm=_f(B, T, 1, n), Cm=_f(B, T, 1, n),
                                S0=_f(B, H, n, p), D=_f(H), z=_f(B, T, H, p), dt_bias=_f(H), lens=_i(B), y=_f(B, T, H, p),
                                S_T=_f(B, H, n, p), workspace=_room()),
    "ssm_step": lambda: dict(x=_f(B, H, p), dt=_f(B, H), A=_f(H), Bm=_f(B, 1, n), Cm=_f(B, 1, n), S=_f(B, H, n, p), D=_f(H),
                             z=_f(B, H, p), dt_bias=_f(H), y=_f(B, H, p)),
    "window_prefill": lambda: dict(q=_f(B, T, H, d), k=_f(B, T, H, d), v=_f(B, T, H, d), k_cache=_f(B, win, H, d),
                                   v_cache=_f(B, win, H, d), start=_i(B), lens=_i(B), o=_f(B, T, H, d), workspace=_room()),
    "window_step": lambda: dict(q=_f(B, H, d), k=_f(B, H, d), v=_f(B, H, d), k_cache=_f(B, win, H, d),
                                v_cache=_f(B, win, H, d), pos=_i(B), o=_f(B, H, d), workspace=_room()),
}


def _more(op):
    return {"window": win} if op.startswith("window") else {}


@pytest.mark.parametrize("op", CALLS)
def test_every_argument_of_a_batched_call_is_refused_by_name(op):
    kda = _kda()
    args = CALLS[op]()
    call = getattr(kda, op)
    call(**args, **_more(op))            # as it stands, it runs
    for name, t in args.items():
        rest = {k: v for k, v in args.items() if k != name}
        with pytest.raises(ValueError, match=f"{name} has no memory"):
            torch.vmap(lambda a: call(**{name: a}, **rest, **_more(op)))(t[None].expand(3, *t.shape))
    call(**args, **_more(op))            # and still does
    torch.cuda.synchronize()


@pytest.mark.parametrize("op", CALLS)
def test_calls_inside_a_gradient_transform_are_refused(op):
    """Inputs are wrappers there, and so are the outputs that a call makes for itself."""
    kda = _kda()
    args = CALLS[op]()
    call = getattr(kda, op)
    first = next(iter(args))
    rest = {k: v for k, v in args.items() if k != first}

    def of_input(a):
        call(**{first: a}, **rest, **_more(op))
        return a.sum()

    def of_nothing(a):
        call(**{k: v for k, v in args.items() if k not in ("y", "o", "state_out", "S_T")}, **_more(op))
        return a.sum()

    with pytest.raises(ValueError, match=f"{first} has no memory"):
        torch.func.grad(of_input)(args[first])
    try:    # an output made here is a wrapper or a plain tensor, as torch has it; the first is refused
        torch.func.grad(of_nothing)(torch.ones(3, device="cuda"))
    except RuntimeError as e:
        assert "storage" in str(e)
    torch.cuda.synchronize()
