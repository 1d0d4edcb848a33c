"""The block, the stack and the other calls of ``api`` on a stream that is not the
current one, nothing ordering the two: each against the same call on the current one."""

import numpy as np
import pytest
import torch

import generative_recommendation_ranking_b200 as mt
import synth
from _util import TOL_BF16_GRAD_PEAK, TOL_BF16_GRAD_RMS, grad_errors

pytestmark = pytest.mark.gpu


def calls():
    """Each call that allocates, on fixed inputs: its outputs on a stream."""
    w = synth.make_workload(2, B=4)
    lens = w["lens"]
    layers = [mt.BlockWeights(p, w["H"]) for p in (w["layers"] * 2)[:2]]
    x = torch.from_numpy(np.asarray(w["x"], np.float32)).cuda()
    batch = mt.PackedBatch(lens, w["ts"])
    y, saved = mt.hstu_block_forward_train(layers[0], batch, x)
    dy = torch.randn_like(x)
    t = layers[0].t
    a, b = torch.randn(2048, 512, device="cuda").bfloat16(), torch.randn(1024, 512, device="cuda").bfloat16()
    cache = mt.BatchContextCache(layers, lens, w["ts"], x)
    cand = torch.randn(cache.k_total, 512, device="cuda")
    torch.cuda.synchronize()

    def back(st):
        dx, grads = mt.hstu_block_backward(layers[0], batch, x, saved, dy, stream=st)
        return (dx, *grads.values())

    def packed(st):
        p = mt.PackedBatch(lens, w["ts"], stream=st)
        return p.seg_off, p.user_off, p.group_id, p.counts, p.d_lens, p.d_ts, p.status

    return {
        "block": lambda st: (mt.hstu_block_forward(layers[0], batch, x, stream=st),),
        "block, train": lambda st: mt.hstu_block_forward_train(layers[0], batch, x, stream=st)[:1],
        "block, backward": back,
        "stack": lambda st: (mt.hstu_stack_forward(layers, batch, x, stream=st),),
        "group norm": lambda st: (mt.group_layernorm(x, batch.group_id[:batch.T], t["gln1_gamma"], t["gln1_beta"], stream=st),),
        "gemm": lambda st: (mt.gemm(a, b, stream=st),),
        "gemm, weights": lambda st: (mt.gemm_wgrad(a, a, stream=st),),
        "batch": packed,
        "score": lambda st: (cache.score(w["ts"], cand, stream=st),),
        "context": lambda st: (mt.BatchContextCache(layers, lens, w["ts"], x, stream=st).out,),
    }


NAMES = ["block", "block, train", "block, backward", "stack", "group norm", "gemm", "gemm, weights", "batch", "score", "context"]


def same(name, got, want):
    """Bit for bit, but for the two calls that add fp32 sums up in no fixed order
    (reduce-adds): the weights' product within 2048 roundings of its terms' magnitudes on
    either side, the block's backward, whose sums meet bf16 steps on the way, within the bar
    that either side keeps to the oracle."""
    if name == "block, backward":
        for g, w in zip(got, want):
            peak, rms, _ = grad_errors(g.cpu(), w.cpu())
            assert peak <= 2 * TOL_BF16_GRAD_PEAK and rms <= 2 * TOL_BF16_GRAD_RMS, (peak, rms)
    elif name == "gemm, weights":  # a^T a of standard normal a [2048, 512]: |a|^T |a| is at most the largest norm squared
        bound = want[0].diagonal().max() * 2 * 2048 * 2.0 ** -24
        assert ((got[0] - want[0]).abs() <= bound).all()
    else:
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def fill(sizes, copies):
    return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(copies)]


@pytest.mark.parametrize("name", NAMES)
def test_buffers_are_no_dropped_ones(name):
    # the current stream is still to write buffers that were dropped
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = fill([t.numel() * t.element_size() for t in want], 3) + fill([n << 20 for n in (1, 2, 4, 8, 16, 32)], 2)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for t in junk:
        t.fill_(0x55)
    del junk, t
    got = call(side)
    torch.cuda.synchronize()
    same(name, got, want)


@pytest.mark.parametrize("name", NAMES)
def test_dropped_workspaces_are_not_handed_out(name):
    # the call waits on its stream; what it dropped is not the current stream's to write
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = call(side)
    junk = fill([n << 20 for n in (1, 2, 4, 8, 16, 32, 64)], 3) + fill([512], 64)
    for t in junk:
        t.fill_(0x55)
    torch.cuda.synchronize()
    same(name, got, want)
