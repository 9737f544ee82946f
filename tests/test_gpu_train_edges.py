"""The calls on the GPU where they are easiest to get wrong: scratch memory of
captured calls, steps counted per tensor, weight decay far below a rounding,
batches at the edges of a kernel's loops and grids, and the forms that
RouterTrainer can be built in.

Bounds count roundings as those of test_gpu_train.py do; U is half a step of
fp32."""
import copy
import ctypes
import weakref

import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
import synth
from grouped_top_routing_amd import _lib
from oracle import train
from parity_util import say
from test_gpu_train import (BF, DEV, F, HP, NAMES, U, _adam_bounds, _opt, _route_bounds,
                            _router_case, n64, rows, u_of, weights, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# scratch memory of captured calls
def _route_inputs(T, seed):
    d = synth.make_inputs(synth.workload("tiny", T=T), seed, device=DEV)
    return d["x"], d["w_router"]


def test_captured_calls_leave_the_default_workspace_alone():
    """A graph captured on a stream whose default workspace exists must not
    hold that workspace: it may grow (and be given back to the allocator) while
    the graph lives, and another graph captured on the stream would share it."""
    say("[workspace] captured route and the stream's default workspace")
    x, W = _route_inputs(300, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = gtr.route(x, W, return_logits=True)
    torch.cuda.synchronize()
    buf = _lib._default_ws[(x.device, stream.cuda_stream)]._buf
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = gtr.route(x, W, return_logits=True)
    for _ in range(3):
        buf.fill_(0x5A)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((buf == 0x5A).all())


def test_two_graphs_captured_on_one_stream_replay_at_once():
    say("[workspace] two graphs of the forward stages, captured on one stream")
    cases = [_route_inputs(900, s) for s in (1, 2)]
    d = synth.make_inputs("tiny", 0, device=DEV)
    gu, dn = d["w_gate_up"], d["w_down"]

    def chain(x, W):
        ids, w, z = gtr.route(x, W, return_logits=True)
        _, off, src, dst = gtr.permute(ids)
        return ids, w, z, gtr.combine(gtr.expert_ffn(x, src, off, gu, dn), dst, w)

    want = [chain(*c) for c in cases]
    torch.cuda.synchronize()
    graphs, got, stream = [], [], torch.cuda.Stream()
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            got.append(chain(*c))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for outs in got:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for outs, ref in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_a_captured_workspace_outlives_its_growth():
    say("[workspace] the buffer a graph holds is kept when the workspace grows")
    x, W = _route_inputs(200, 3)
    big, _ = _route_inputs(6000, 4)
    ws = gtr.Workspace()
    want = gtr.route(x, W, workspace=ws)
    want_big = gtr.route(big, W)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gtr.route(x, W, workspace=ws)
    held = weakref.ref(ws._buf)
    got_big = gtr.route(big, W, workspace=ws)
    assert ws._buf is not held() and held() is not None
    for _ in range(3):
        got[0].zero_(), got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(gtr.route(big, W, workspace=ws), want_big))
    assert all(torch.equal(a, b) for a, b in zip(got_big, want_big))
