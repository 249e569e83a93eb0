"""CPU tests of the kv_* binding's type checks: a tensor of another type than the
call takes is refused, however many bytes its elements have."""
import pytest
import torch

import affine_group_quantized_b200 as agq

A = 0x10000  # a fake device address; never dereferenced
B, T, H, HQ, D, W, STATE = 2, 4, 2, 4, 128, 4, 64


def _cache(bits=4):
    return agq.KVCache(A, A, A, A, A, A, 8, H, 16, D, bits, 64)


def _t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


ROWS, QS = (T, H, D), (B, HQ, D)
STATES = (B, H, STATE)
# argument: (kind, shape)
CALLS = {
    "kv_append": dict(k=("bf16", ROWS), v=("bf16", ROWS), block_table=("int", (B, W)),
                      lens=("int", (B,)), token_starts=("int", (B + 1,)), batch=B, num_tokens=T,
                      table_width=W, seen=("int", (B,)), positions=("int", STATES),
                      weights=("float", STATES), state_width=STATE, d_status=("int", (1,))),
    "kv_read": dict(k=("bf16", ROWS), v=("bf16", ROWS), block_table=("int", (B, W)),
                    lens=("int", (B,)), token_starts=("int", (B + 1,)), batch=B, num_tokens=T,
                    table_width=W, d_status=("int", (1,))),
    "kv_attention": dict(q=("bf16", QS), block_table=("int", (B, W)), lens=("int", (B,)),
                         out=("bf16", QS), batch=B, num_q_heads=HQ, table_width=W, scale=0.1,
                         workspace=("any", (16,)), weights=("float", STATES), state_width=STATE,
                         d_status=("int", (1,))),
    "kv_evict": dict(block_table=("int", (B, W)), lens=("int", (B,)), seen=("int", (B,)),
                     weights=("float", STATES), positions=("int", STATES), new_lens=("int", (B,)),
                     new_weights=("float", STATES), new_positions=("int", STATES), batch=B,
                     table_width=W, state_width=STATE, budget=32, d_status=("int", (1,))),
}
WRONG = {"bf16": (torch.float16, torch.float32, torch.uint8), "int": (torch.float32, torch.int64),
         "float": (torch.int32, torch.float64, torch.bfloat16)}
MESSAGE = {"bf16": "must hold bf16", "int": "must hold 4-byte integers", "float": "must hold 4-byte floats"}
CASES = [(c, n, t) for c, args in CALLS.items() for n, a in args.items() if isinstance(a, tuple)
         for t in WRONG.get(a[0], ())]


@pytest.mark.parametrize("call, name, dtype", CASES)
def test_another_type_is_refused(call, name, dtype):
    args = {n: A if isinstance(a, tuple) else a for n, a in CALLS[call].items()}
    if "workspace" in args:
        args["workspace"] = _t(torch.uint8, 16)
    kind, shape = CALLS[call][name]
    # (twice the shape: an element of fewer bytes must not be refused for its size)
    args[name] = _t(dtype, *shape) if dtype.itemsize >= (2 if kind == "bf16" else 4) else \
        _t(dtype, *(4 * s for s in shape))
    with pytest.raises(ValueError, match=f"{name}: {MESSAGE[kind]}"):
        getattr(agq, call)(_cache(), stream=0, **args)


@pytest.mark.parametrize("bits", [4, 16])
def test_another_types_cache_is_refused(bits):
    n = 8 * H * 16
    some = [A] * 6
    for i, name in enumerate(("k", "v")):
        for t in (torch.float16, torch.float32) + ((torch.bfloat16,) if bits == 4 else (torch.uint8,)):
            bufs = list(some)
            bufs[i] = _t(t, n, 4 * D)
            with pytest.raises(ValueError, match=f"{name}: must hold"):
                agq.KVCache(*bufs, 8, H, 16, D, bits, 64)
    for i, name in enumerate(("k_scales", "k_biases", "v_scales", "v_biases"), 2):
        bufs = list(some)
        bufs[i] = _t(torch.float16, n, 2)
        if bits == 4:
            with pytest.raises(ValueError, match=f"{name}: must hold"):
                agq.KVCache(*bufs, 8, H, 16, D, bits, 64)


def test_bit_patterns_pass():
    # 2-byte integers hold bf16 bit patterns: refused further on, for their device
    for t in (torch.bfloat16, torch.int16, torch.uint16):
        with pytest.raises(ValueError, match="CUDA"):
            agq.KVCache(_t(t, 8 * H * 16, D), A, None, None, None, None, 8, H, 16, D, 16, 0)
    for t in (torch.int32, torch.uint32, torch.uint8):
        with pytest.raises(ValueError, match="CUDA"):
            agq.KVCache(_t(t, 8 * H * 16, D), A, A, A, A, A, 8, H, 16, D, 4, 64)
