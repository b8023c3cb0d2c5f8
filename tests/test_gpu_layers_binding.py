"""The binding of full-attention and gated delta layers on the device: every argument of every call in turn as a batch
of torch.vmap, which has no memory that a kernel could use.  All are refused by name, on the host, before any launch.
"""
import pytest
import torch

from tests.test_gpu_mixers_binding import _f, _i, _kda, _room

pytestmark = pytest.mark.gpu

B, T, H, d = 2, 40, 2, 64


def _pool():
    return torch.zeros(6, H, 16 * 34, dtype=torch.uint8, device="cuda")


def _cu():
    return torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")


def _pages():
    return torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)


CALLS = {
    "attn_prefill": lambda: dict(q=_f(2 * T, H, d), k=_f(2 * T, H, d), v=_f(2 * T, H, d), cu_q=_cu(), cu_k=_cu(), o=_f(2 * T, H, d),
                                 workspace=_room()),
    "cache_write": lambda: dict(k=_f(2 * T, H, d), v=_f(2 * T, H, d), k_cache=_pool(), v_cache=_pool(), pages=_pages(), cu=_cu(),
                                start=_i(B)),
    "cache_read": lambda: dict(k_cache=_pool(), v_cache=_pool(), pages=_pages(), cu=_cu(), start=_i(B), k=_f(2 * T, H, d),
                               v=_f(2 * T, H, d)),
    "attn_step": lambda: dict(q=_f(B, H, d), k_cache=_pool(), v_cache=_pool(), pages=_pages(), lens=_i(B), o=_f(B, H, d),
                              workspace=_room()),
    "delta_prefill": lambda: dict(q=_f(B, T, H, d), k=_f(B, T, H, d), v=_f(B, T, H, d), g=_f(B, T, H), beta=_f(B, T, H),
                                  S0=_f(B, H, d, d), lens=_i(B), o=_f(B, T, H, d), S_T=_f(B, H, d, d), workspace=_room()),
    "delta_step": lambda: dict(q=_f(B, H, d), k=_f(B, H, d), v=_f(B, H, d), g=_f(B, H), beta=_f(B, H), S=_f(B, H, d, d), o=_f(B, H, d)),
}
MORE = {"cache_read": dict(tokens=2 * T, d=d, dtype=torch.float32)}


@pytest.mark.parametrize("op", CALLS)
def test_every_argument_of_a_batched_call_is_refused_by_name(op):
    kda = _kda()
    args, more = CALLS[op](), MORE.get(op, {})
    call = getattr(kda, op)
    call(**args, **more)            # as it stands, it runs
    for name, t in args.items():
        rest = {k: v for k, v in args.items() if k != name}
        with pytest.raises(ValueError, match=f"{name} has no memory"):
            torch.vmap(lambda a: call(**{name: a}, **rest, **more))(t[None].expand(3, *t.shape))
    call(**args, **more)            # and still does
    torch.cuda.synchronize()


@pytest.mark.parametrize("op", ["attn_prefill", "cache_write", "attn_step", "delta_prefill", "delta_step"])
def test_calls_inside_a_gradient_transform_are_refused(op):
    """Inputs are wrappers there: no gradient of these calls is formed, and none is answered with zeros."""
    kda = _kda()
    args = CALLS[op]()
    call = getattr(kda, op)
    first = next(iter(args))
    rest = {k: v for k, v in args.items() if k != first}

    def of_input(a):
        call(**{first: a}, **rest)
        return a.sum()

    with pytest.raises(ValueError, match=f"{first} has no memory"):
        torch.func.grad(of_input)(args[first])
    torch.cuda.synchronize()
