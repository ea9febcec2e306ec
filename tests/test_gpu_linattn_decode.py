"""The single-token step of linear attention as a serving loop runs it:
captured and replayed, on a stream of its own, with a state past 4 GiB."""

import pytest
import torch

import gated_delta_rule_79_amd as gdn

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def rows(N, H, Hq, dk, dv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    return r(N, Hq, dk), r(N, Hq, dk), r(N, H, dv)


def decays(H):
    return torch.log1p(-torch.exp2(-torch.linspace(1, 9, H))).cuda()


def test_captured_and_replayed(gpu_lib):
    N, H, Hq, dk, dv = 3, 4, 2, 64, 80
    la, x = decays(H), rows(N, H, Hq, dk, dv, 1)
    state = torch.randn(N, H, dk, dv, device="cuda")
    eager = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.linear_attn_decode_step(*x, la, state.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.linear_attn_decode_step(*x, la, state)
    for t in range(5):
        for a, b in zip(x, rows(N, H, Hq, dk, dv, 10 + t)):
            a.copy_(b)
        want = gdn.linear_attn_decode_step(*x, la, eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(state, eager), t


def test_two_streams_at_once(gpu_lib):
    jobs = [(rows(5, 8, 8, 128, 128, s), decays(8), torch.zeros(5, 8, 128, 128, device="cuda"))
            for s in (1, 2)]
    want = []
    for x, la, s in jobs:
        s = s.clone()
        want.append(([gdn.linear_attn_decode_step(*x, la, s) for _ in range(4)], s))
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        for i, (x, la, s) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(gdn.linear_attn_decode_step(*x, la, s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i][0]))
        assert torch.equal(jobs[i][2], want[i][1])


def test_states_past_four_gigabytes(gpu_lib):
    # the last sequences' states lie behind 2^32 bytes (and 2^31 elements)
    N, H, d = 4400, 32, 128
    x, la = rows(N, H, H, d, d, 3), decays(H)
    state = torch.zeros(N, H, d, d, device="cuda")
    tail = torch.randn(2, H, d, d, device="cuda")
    state[-2:] = tail
    o = gdn.linear_attn_decode_step(*x, la, state)
    o1 = gdn.linear_attn_decode_step(*(t[-2:].contiguous() for t in x), la, tail)
    torch.cuda.synchronize()
    assert torch.equal(o[-2:], o1) and torch.equal(state[-2:], tail)
