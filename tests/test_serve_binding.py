"""Refusals of the attention-layer operators' compiled binding (no GPU needed: the tensors have a device, a
type and a shape, but no memory, and every call is refused before anything is launched)."""
import pytest
import torch

from gated_deltanet_rule_gb300 import build as gbuild
from gated_deltanet_rule_gb300 import gdr

BF16, F32, F64, I32, I64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64, torch.uint8


class Shell(torch.Tensor):
    """A tensor without memory."""

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


def T(shape, dtype=I32, device="cuda:0", strides=None):
    return torch.Tensor._make_wrapper_subclass(Shell, shape, strides=strides, dtype=dtype, device=device)


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def _attn(**kw):
    a = dict(q=T((2, 3, 4, 128), BF16), k_pages=T((9, 16, 2, 128), BF16), v_pages=T((9, 16, 2, 128), BF16), table=T((2, 4)), ctx=T((2,)),
             lengths=T((2,)), mask=T((2, 3, 1), I64), o=T((2, 3, 4, 128), BF16), lse=T((2, 3, 4), F32), ws=T((1 << 28,), U8))
    return gdr.gdr_tree_attn, {**a, **kw}


def _rope(**kw):
    a = dict(q=T((2, 3, 4, 128), BF16), k=T((2, 3, 2, 128), BF16), q_w=T((128,), F32), k_w=T((128,), F32), inv_freq=T((32,), F64), pos=T((2, 3)),
             q_out=T((2, 3, 4, 128), BF16), k_out=T((2, 3, 2, 128), BF16))
    return gdr.gdr_qk_norm_rope, {**a, **kw}


def _append(**kw):
    a = _rope()[1]
    del a["k_out"]
    a.update(v=T((2, 3, 2, 128), BF16), k_pages=T((9, 16, 2, 128), BF16), v_pages=T((9, 16, 2, 128), BF16), table=T((2, 4)), ctx=T((2,)),
             lengths=T((2,)))
    return gdr.gdr_qk_norm_rope_append, {**a, **kw}


def _back(**kw):
    a = _rope()[1]
    a.update(dq_out=a.pop("q_out"), dk_out=a.pop("k_out"), ws=T((1 << 26,), U8))
    return gdr.gdr_qk_norm_rope_backward, {**a, **kw}


def _verify(**kw):
    a = dict(tokens=T((2, 3)), parents=T((2, 3)), lengths=T((2,)), p=T((2, 3, 50), F32), q=T((2, 3, 50), F32), u=T((2, 3), F32),
             u_next=T((2,), F32), path=T((2, 3)), n_path=T((2,)), next_token=T((2,)))
    return gdr.gdr_verify_draft, {**a, **kw}


def _rows(**kw):
    return {**dict(table=T((6, 4)), ctx=T((6,)), refs=T((9,)), rows=T((2,))), **kw}


def _reserve(**kw):
    return gdr.gdr_cache_reserve, {**_rows(), **dict(extra=3, page=16, ws=T((1 << 20,), U8)), **kw}


def _free(**kw):
    return gdr.gdr_cache_free, _rows(**kw)


def _fork(**kw):
    a = _rows()
    a.update(k_cache=T((2, 9, 16, 2, 64), BF16), v_cache=T((2, 9, 16, 2, 64), BF16), src=T((2,)), dst=a.pop("rows"), ws=T((1 << 20,), U8))
    return gdr.gdr_cache_fork, {**a, **kw}


def _compact(**kw):
    a = dict(k_cache=T((2, 9, 16, 2, 64), BF16), v_cache=T((2, 9, 16, 2, 64), BF16), table=T((6, 4)), ctx=T((6,)), path=T((6, 5)), n_path=T((6,)),
             new_ctx=T((6,)))
    return gdr.gdr_cache_compact, {**a, **kw}


CALLS = [_attn, _rope, _append, _back, _verify, _reserve, _free, _fork, _compact]


def _refused(make, match, error=ValueError, **kw):
    fn, a = make(**kw)
    with pytest.raises(error, match=match):
        fn(**a)


@pytest.mark.parametrize("make", CALLS)
def test_tensors_of_two_devices(make):
    """Any one tensor on another device than the rest."""
    for name, t in make()[1].items():
        if isinstance(t, torch.Tensor):
            _refused(make, "device of the other tensors", **{name: T(tuple(t.shape), t.dtype, "cuda:1")})


BIG = 2 ** 32


@pytest.mark.parametrize("make,kw", [
    (_reserve, dict(extra=BIG)), (_reserve, dict(extra=-BIG - 3)), (_reserve, dict(page=BIG + 16)), (_reserve, dict(refs=T((BIG + 9,)))),
    (_reserve, dict(rows=T((BIG + 2,)))), (_free, dict(table=T((6, BIG + 4)))), (_free, dict(refs=T((BIG + 9,)))),
    (_fork, dict(k_cache=T((BIG + 2, 9, 16, 2, 64), BF16), v_cache=T((BIG + 2, 9, 16, 2, 64), BF16))),
    (_compact, dict(path=T((6, BIG + 5)))), (_compact, dict(table=T((6, BIG + 4)))),
    (_verify, dict(p=T((2, 3, BIG + 50), F32), q=None)), (_attn, dict(table=T((2, BIG + 4)))),
    (_attn, dict(k_pages=T((BIG + 9, 16, 2, 128), BF16), v_pages=T((BIG + 9, 16, 2, 128), BF16))),
    (_rope, dict(inv_freq=T((2 ** 31 + 32,), F64))),
])
def test_what_does_not_fit_in_32_bits(make, kw):
    _refused(make, "32 bits", **kw)


class Odd:
    def __bool__(self):
        raise ArithmeticError("neither true nor false")


@pytest.mark.parametrize("make,kw", [(_rope, dict(interleaved=Odd())), (_append, dict(interleaved=Odd())), (_back, dict(interleaved=Odd())),
                                     (_attn, dict(want_lse=Odd(), lse=None))])
def test_a_truth_value_that_raises(make, kw):
    _refused(make, "neither true nor false", ArithmeticError, **kw)


class OddStream:
    cuda_stream = "seven"


@pytest.mark.parametrize("make", [_attn, _reserve])
def test_a_stream_handle_that_is_no_number(make):
    _refused(make, None, TypeError, stream=OddStream(), ws=None)


@pytest.mark.parametrize("make", [_attn, _back, _reserve, _fork])
@pytest.mark.parametrize("strides", [(0,), (2,)])
def test_a_workspace_with_less_or_other_memory_than_elements(make, strides):
    """One byte seen many times would pass for as many bytes."""
    _refused(make, "ws must be contiguous", ws=T((1 << 28,), U8, strides=strides))
