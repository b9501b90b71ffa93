"""GPU: the experts' layer where its kernels change their way: rows longer than what LDS
holds of their scales, more columns than a workgroup takes at once, several groups of
rows in one workgroup, a last portion of few tokens; and what a batch's company, other
streams and shared workspaces must not change."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from gpu_util import DEV, say
from test_gpu_moe import FORMATS, check_experts, check_route, choice, make, router, to

pytestmark = pytest.mark.gpu


def check(rng, fmt, tokens, experts, top, hidden, inter, ids=None):
    parts = S.layer(rng, fmt, experts, hidden, inter)
    x = S.bf16(rng, tokens, hidden)
    some, weights = choice(rng, tokens, max(experts, top), top)
    ids = some if ids is None else np.broadcast_to(np.asarray(ids, np.int32), (tokens, top)).copy()
    got = qbn.moe_experts(make(parts, fmt), x.to(DEV), to(ids), to(weights))
    check_experts(got, x, ids, weights, parts, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,hidden,inter", [
    (1, 2048, 32), (3, 2080, 64), (2, 4096, 32), (1, 4128, 4128), (7, 4160, 96), (2, 8224, 32),
    (8, 16416, 32),  # LDS holds three of the tokens at a time
    (1, 32, 16416), (8, 64, 8224),  # h does not fit LDS
    (1, 65024, 32), (1, 32, 16128),  # as much as fits
    (2, 65536, 32),  # nor one token
    (9, 4128, 160), (20, 2080, 4128)])
def test_long_rows(fmt, tokens, hidden, inter):
    say("long rows", fmt, tokens, hidden, inter)
    check(np.random.default_rng(hidden + tokens), fmt, tokens, 3, 2, hidden, inter)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,hidden,inter", [(64, 288, 2080), (70, 4128, 160), (66, 4128, 32), (90, 32, 2112)])
def test_several_groups_of_rows(fmt, tokens, hidden, inter):
    """So many rows that a workgroup takes more than one group of them, the last one partly beyond the end."""
    say("groups", fmt, tokens, hidden, inter)
    check(np.random.default_rng(hidden), fmt, tokens, 64, 8, hidden, inter)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,top", [(8, 8), (2, 32), (5, 9), (17, 3), (64, 1), (65, 1), (129, 2), (256, 3)])
def test_all_of_one_expert(fmt, tokens, top):
    """Every assignment, also of one token, to the same expert."""
    say("one expert", fmt, tokens, top)
    check(np.random.default_rng(tokens), fmt, tokens, 3, top, 160, 96, ids=1)


@pytest.mark.parametrize("tokens", [256, 257, 263, 270, 515])
def test_portions(tokens):
    """A last portion of one token, of a few, of more."""
    say("portions", tokens)
    check(np.random.default_rng(tokens), "mxfp4", tokens, 6, 3, 96, 64)


@pytest.mark.parametrize("tokens,experts,top", [(1, 1024, 32), (2, 300, 32), (7, 257, 9), (40, 1024, 8)])
def test_many_experts(tokens, experts, top):
    rng = np.random.default_rng(experts)
    parts = S.layer(rng, "mxfp4", experts, 64, 32)
    x, w = S.bf16(rng, tokens, 64), S.bf16(rng, experts, 64, gain=0.25)
    layer = make(parts, "mxfp4", router(w, top))
    say("many experts", tokens, experts, top)
    out, ids, weights = qbn.moe(layer, x.to(DEV))
    check_route((ids, weights), x, w, None, top, True)
    check_experts(out, x, ids.cpu().numpy(), weights.cpu().numpy(), parts, "mxfp4")


@pytest.mark.parametrize("tokens,experts,hidden", [(5, 16, 4128), (16, 64, 2080), (65, 30, 8192), (4100, 17, 512)])
def test_route_split_over_the_hidden_size(tokens, experts, hidden):
    rng = np.random.default_rng(hidden)
    x, w = S.bf16(rng, tokens, hidden), S.bf16(rng, experts, hidden, gain=2 * hidden ** -0.5)
    say("split", tokens, experts, hidden)
    first = qbn.moe_route(router(w, 4), x.to(DEV))
    check_route(first, x, w, None, 4, True)
    again = qbn.moe_route(router(w, 4), x.to(DEV))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [6, 50, 200])
def test_company_changes_no_bit(fmt, tokens):
    """The tokens in another order: the same rows, bit by bit, also where they share experts."""
    rng = np.random.default_rng(tokens)
    layer = make(S.layer(rng, fmt, 5, 544, 288), fmt)
    x = S.bf16(rng, tokens, 544).to(DEV)
    ids, weights = (to(a) for a in choice(rng, tokens, 5, 3))
    order = torch.from_numpy(rng.permutation(tokens)).to(DEV)
    say("company", fmt, tokens)
    out = qbn.moe_experts(layer, x, ids, weights)
    assert torch.equal(qbn.moe_experts(layer, x[order], ids[order], weights[order]), out[order])


@pytest.mark.parametrize("tokens", [3, 40])
def test_two_graphs_share_a_workspace(tokens):
    rng = np.random.default_rng(tokens)
    layers = [make(S.layer(rng, "mxfp4", 8, 128, 64), "mxfp4", router(S.bf16(rng, 8, 128, gain=0.2), 2)) for _ in range(2)]
    xs = [S.bf16(rng, tokens, 128).to(DEV) for _ in range(2)]
    ws = torch.empty(qbn.moe_nbytes(layers[0].router, layers[0], tokens, 2), dtype=torch.uint8, device=DEV)
    outs, graphs = [qbn.moe(l, x) for l, x in zip(layers, xs)], []
    say("two graphs", tokens)
    for l, x, (out, ids, weights) in zip(layers, xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qbn.moe(l, x, out=out, ids=ids, weights=weights, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for x in xs:
            x.copy_(S.bf16(rng, tokens, 128))
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for l, x, o in zip(layers, xs, outs):
            for a, b in zip(o, qbn.moe(l, x)):
                assert torch.equal(a, b)


def test_two_streams():
    """Calls at once, each with its own workspace."""
    rng = np.random.default_rng(3)
    layer = make(S.layer(rng, "nvfp4", 8, 256, 128), "nvfp4", router(S.bf16(rng, 8, 256, gain=0.2), 2))
    xs = [S.bf16(rng, t, 256).to(DEV) for t in (1, 30)]
    want = [qbn.moe(layer, x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[] for _ in xs]
    say("two streams")
    for _ in range(5):
        for s, x, g in zip(streams, xs, got):
            with torch.cuda.stream(s):
                g.append(qbn.moe(layer, x))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            for a, b in zip(r, w):
                assert torch.equal(a, b)
