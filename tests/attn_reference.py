"""Softmax attention in 64 bits and how far the kernels' outputs may be from it, for the attention tests.

Bounds, for u the 16-bit type's half step (bf16 2^-8, f16 2^-11) and e = 2^-24:
 - a score is an f32 sum of D products: off by 2 D e sum_d |q k| scale (every addition rounded or cut), and by 4 e of
   itself and of the maximum, where scale and maximum go in; exp2 and its argument add 8 e. So a weight is relatively off by
   w = 2 D e A + 8 e S + 8 e with A, S the largest sum of products and score of the row.
 - weights are rounded to the type: u. (f16 below 2^-14: 2^-25 of the row's largest, whatever the weight.)
 - n weighted values are summed in f32, their weights too: 2 n e each, and once more where partial sums are joined; running
   sums are scaled a few times: 64 e.
 - the result is rounded: u of it (f16 below 2^-14: 2^-25).
All of them are relative to sum_j p_j |v_j|, the last to |o|.
"""
import math

import torch

E = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attention64(q, k, v, sees, scale):
    """q [T][Hq][D], k, v [n][Hkv][D], sees [T][n] bool: (out, lse, room of out, room of lse) in 64 bits."""
    T, Hq, D = q.shape
    n, Hkv = k.shape[:2]
    dtype = q.dtype
    u = half_step(dtype)
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    room, room_l = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or T == 0:
        return out, lse, room, room_l
    for h in range(Hq):
        qh, kh, vh = q[:, h].double(), k[:, h // (Hq // Hkv)].double(), v[:, h // (Hq // Hkv)].double()
        s = (qh @ kh.T) * scale
        s = torch.where(sees, s, -math.inf)
        most = s.amax(1, keepdim=True)
        p = torch.exp(s - torch.where(most == -math.inf, 0.0, most))
        p = torch.where(sees, p, 0.0)
        total = p.sum(1, keepdim=True)
        some = total[:, 0] > 0
        weight = p / total.clamp_min(1e-300)
        # values of keys that no query sees do not count, whatever they are
        vh = torch.where(sees.any(0)[:, None], vh, 0.0)
        out[:, h] = weight @ vh
        lse[:, h] = torch.where(some, most[:, 0] + total[:, 0].clamp_min(1e-300).log(), -math.inf)
        products = torch.where(sees, (qh.abs() @ kh.abs().T) * scale, 0.0).amax(1, keepdim=True)
        largest = torch.where(sees, s.abs(), 0.0).amax(1, keepdim=True)
        w = 2 * D * E * products + 8 * E * largest + 8 * E
        size = weight @ vh.abs()
        room[:, h] = size * (u + 2 * w + 6 * n * E + 64 * E) + u * out[:, h].abs()
        if dtype == torch.float16:
            room[:, h] += 2.0 ** -25 * (torch.where(sees, 1.0, 0.0).to(torch.float64) @ vh.abs()) + 2.0 ** -25
        room_l[:, h] = torch.where(some, (w + 4 * n * E)[:, 0] + 4 * E * lse[:, h].abs(), 0.0)
    return out, lse, room, room_l


def near(got, want, room):
    got = got.double()
    bad = ~((got - want).abs() <= room)
    bad &= ~((got == want) & torch.isinf(want))
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()} within {room[bad][0].item()}")


def causal(T, n, device):
    """Query i of T sees the keys up to n - T + i."""
    return torch.arange(n, device=device)[None] <= torch.arange(T, device=device)[:, None] + n - T
