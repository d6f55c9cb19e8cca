"""Run one case of the library a fixed number of times, for profiler captures.

    python -m long_context_02_b200.profile_run CASE [--heads H] [--seq-len N]
           [--segment-tokens S] [--launches K]

CASE is one of
  prefill   la_prefill, bf16 Q/K/V, bf16 O, fp32 final state
  backward  la_backward (three launches each: dQ forward, dK and dV reversed)
  state     la_prefill_state (final state only)
  scan, scan_backward, conv, conv_backward, norm, norm_backward
            the state space layer over N tokens of H * 128 channels, 16 states each
on seeded synthetic inputs of B=1, H heads, N tokens, d=128 (Q, K = SiLU(z)/sqrt(d),
V = N(0,1)). --segment-tokens sets the scan segment length (0 = automatic; a
value above N gives one segment per (head, value half)). Every call goes
through the C ABI; the device status is checked after the last one.
"""
from __future__ import annotations

import argparse

import torch

from . import binding as L
from . import inputs


LAYER = ["scan", "scan_backward", "conv", "conv_backward", "norm", "norm_backward"]


def layer_step(case, N, D):
    """A call of one of the state space layer's operators on seeded bf16 inputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    low = lambda *shape: rnd(*shape).to(torch.bfloat16)
    x, dy, n = low(1, N, D), low(1, N, D), 16
    if case.startswith("scan"):
        A = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32).repeat(D, 1)
        a = (x, low(1, N, D), A, low(1, N, 1, n), low(1, N, 1, n), rnd(D), low(1, N, D), rnd(D) - 4)
        if case == "scan":
            return lambda: L.selective_scan(*a)
        return lambda: L.selective_scan_backward(dy, *a)
    w, b = rnd(D, 4), rnd(D)
    if case == "conv":
        return lambda: L.short_conv(x, w, b)
    if case == "conv_backward":
        return lambda: L.short_conv_backward(dy, x, w, b)
    _, mean, rstd = L.layer_norm(x, b, b)
    if case == "norm":
        return lambda: L.layer_norm(x, b, b)
    return lambda: L.layer_norm_backward(dy, x, b, mean, rstd)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["prefill", "backward", "state"] + LAYER)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--seq-len", type=int, default=8192)
    ap.add_argument("--segment-tokens", type=int, default=0)
    ap.add_argument("--launches", type=int, default=3)
    a = ap.parse_args(argv)
    B, H, N, d = 1, a.heads, a.seq_len, 128
    if a.case in LAYER:
        step = layer_step(a.case, N, H * d)
        for _ in range(a.launches):
            step()
        torch.cuda.synchronize()
        print(f"{a.case}: {a.launches} calls of {N} tokens, {H * d} channels done")
        return
    L.la_set_tuning(0, a.segment_tokens)
    q, k, v, s = inputs.prefill_inputs(B, H, N, d, torch.bfloat16, "cuda", seed=5)
    op = L.LA_OP_BACKWARD if a.case == "backward" else L.LA_OP_PREFILL
    ws = L.workspace(op, B, H, N, d)
    st = torch.empty((B, H, d, d), dtype=torch.float32, device="cuda")
    if a.case == "prefill":
        o = torch.empty_like(q)
        step = lambda: L.la_prefill(q, k, v, s, o, st, ws)
    elif a.case == "state":
        step = lambda: L.la_prefill_state(k, v, s, None, st, ws)
    else:
        do = inputs.grad_output(q.shape, torch.bfloat16, "cuda", seed=6)
        dq, dk, dv = (torch.empty_like(q) for _ in range(3))
        step = lambda: L.la_backward(do, q, k, v, s, dq, dk, dv, ws)
    for _ in range(a.launches):
        step()
    torch.cuda.synchronize()
    status = L.la_read_device_status(ws)
    if status != L.LA_OK:
        raise SystemExit(f"device status {L.la_status_string(status)}")
    print(f"{a.case}: {a.launches} calls of B=1 H={H} N={N} d=128 done")


if __name__ == "__main__":
    main()
