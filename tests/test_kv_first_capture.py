"""GPU test: the very first call of each operator in a process may be a captured
one."""
import os
import subprocess
import sys

import pytest

from affine_group_quantized_b200 import build

STEP = r"""
import math, torch
import affine_group_quantized_b200 as agq

B, H, HQ, D, page, W, bits, gs = 2, 2, 8, 128, 16, 4, BITS, 64
room = W * page
bufs = [torch.zeros((B * W, H, page, D * bits // 32), dtype=torch.int32, device="cuda") for _ in "kv"]
bufs = [b.view(torch.bfloat16) for b in bufs] + [None] * 4 if bits == 16 else \
    bufs + [torch.zeros((B * W, H, page, D // gs), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
cache = agq.KVCache(*bufs, B * W, H, page, D, bits, gs)
table = torch.arange(B * W, dtype=torch.int32, device="cuda").view(B, W)
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
lens, starts, seen, new_lens = i32(0, 0), i32(0, 40, 60), i32(0, 0), i32(0, 0)
full = i32(40, 20)
qkv = torch.randn((60, HQ + 2 * H, D), device="cuda").bfloat16()
pos, w = torch.full((B, H, room), -1, dtype=torch.int32, device="cuda"), torch.zeros((B, H, room), device="cuda")
k, v = (torch.zeros((60, H, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
q = qkv[:B, :HQ].contiguous()
out = torch.zeros_like(q)
ws = torch.empty(agq.kv_attention_workspace(cache, B, HQ, W, True), dtype=torch.uint8, device="cuda")


def step():
    agq.kv_append(cache, qkv[:, HQ:HQ + H], qkv[:, HQ + H:], table, lens, starts, B, 60, W, seen=seen,
                  positions=pos, weights=w, state_width=room)
    agq.kv_read(cache, k, v, table, lens, starts, B, 60, W)
    agq.kv_attention(cache, q, table, full, out, B, HQ, W, 0.1, ws, weights=w, state_width=room)
    agq.kv_evict(cache, table, full, full, w, pos, new_lens, w, pos, B, W, room, 24, 8, 2)


g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    step()
assert (out == 0).all() and (pos == -1).all()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (out, w, pos, new_lens, k, v)]
assert first[3].tolist() == [24, 20]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (out, w, pos, new_lens, k, v)))
kd, vd = (t.float().repeat_interleave(HQ // H, 1) for t in (k, v))
for b, (t0, t1) in enumerate(((0, 40), (40, 60))):
    p = torch.softmax(0.1 * torch.einsum("hd,nhd->hn", q[b].float(), kd[t0:t1]), -1)
    ref = torch.einsum("hn,nhd->hd", p, vd[t0:t1])
    # k and v are the stored values rounded to bf16 (2^-8): two scores' errors, the
    # value's, the probability's (2^-11) and the output's
    size = 0.1 * torch.einsum("hd,nhd->hn", q[b].float().abs(), kd[t0:t1].abs()).amax(-1)
    tol = (2.0 ** -7 * size + 2.0 ** -7).unsqueeze(1) * torch.einsum("hn,nhd->hd", p, vd[t0:t1].abs())
    assert ((out[b].float() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all()
print("ok")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8, 16])
def test_first_calls_are_captured(bits):
    root = os.path.dirname(os.path.dirname(build.LIB))
    r = subprocess.run([sys.executable, "-c", STEP.replace("BITS", str(bits))], cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
